"""Products of expert layers and the orthogonalisation of their updates on
torch tensors (row-major): the calls of :mod:`.ozgemm` with their shapes, strides and types taken from the tensors.

Nothing here is recorded by autograd: the gradients are calls of their own, and
tensors that require a gradient or carry a tangent are refused.
Work goes on the current stream of the tensors' device.
"""
from __future__ import annotations

import contextlib

import torch
from torch.autograd import forward_ad

from . import ozgemm as L

_TYPES = {torch.float64: L.OZGEMM_F64, torch.float32: L.OZGEMM_F32, torch.bfloat16: L.OZGEMM_BF16,
          torch.float16: L.OZGEMM_F16}


def _type_of(t, what: str, allowed=(torch.float32, torch.bfloat16, torch.float16)) -> int:
    if t.dtype not in allowed:
        raise TypeError(f"{what}: {t.dtype} is not supported (one of {', '.join(map(str, allowed))})")
    return _TYPES[t.dtype]


def _no_grad(what: str, *tensors, instead: str = "") -> None:
    """Refuses tensors whose derivatives would get lost: those that autograd
    records (unless it is switched off), and those with a tangent of its forward
    mode (which torch.no_grad() does not switch off)."""
    for t in tensors:
        if t is None:
            continue
        if t.requires_grad and torch.is_grad_enabled():
            raise RuntimeError(f"{what} is not recorded by autograd: call it under torch.no_grad(){instead}")
        if forward_ad.unpack_dual(t).tangent is not None:
            raise RuntimeError(f"{what} has no forward-mode derivative: call it on the primal of a dual tensor")


_INSTEAD = " and take the gradients from grouped_linear_grads"


def _written(*tensors) -> None:
    """Tells autograd that these tensors of the caller's hold other values now: a
    graph that had saved one refuses its backward pass, as after torch's own
    in-place operations."""
    for t in tensors:
        if t is not None:
            torch.autograd.graph.increment_version(t)


_HERE = contextlib.nullcontext()


def _on_device(device):
    """A context in which `device`, a GPU, is the current one."""
    if device.type != "cuda":
        raise ValueError(f"the tensors are on {device}: these products run on the GPU only")
    return _HERE if device.index == torch.cuda.current_device() else torch.cuda.device(device)


def _fits(*sizes) -> None:
    if max(sizes) > L.OZGEMM_MAX_ROWS:
        raise ValueError(f"sizes go up to {L.OZGEMM_MAX_ROWS}, got {max(sizes)}")


_LD_MAX = 2 ** 31 - 1  # leading dimensions are C ints


def _rows(t, what: str):
    """A 2-d tensor with its rows' entries next to each other, and their distance."""
    if t.dim() != 2:
        raise ValueError(f"{what} must have two dimensions, got {tuple(t.shape)}")
    n, q = t.shape
    t = t.resolve_neg()
    if (q > 1 and t.stride(1) != 1) or (n > 1 and not max(1, q) <= t.stride(0) <= _LD_MAX):
        t = t.contiguous()
    return t, max(1, q, t.stride(0) if n > 1 else 0)


def _weights(W):
    """(tensor, transa, lda, stridea) of weights [g, m, q] as op(A_e) = W[e]:
    in place when either q or m runs contiguously, otherwise from a copy."""
    if W.dim() != 3:
        raise ValueError(f"the weights must have three dimensions [groups, out, in], got {tuple(W.shape)}")
    g, m, q = W.shape
    W = W.resolve_neg()
    s0, s1, s2 = W.stride()
    s0 = s0 if g > 1 else 0
    if (q <= 1 or s2 == 1) and (m <= 1 or max(1, q) <= s1 <= _LD_MAX):
        return W, 1, max(1, q, s1 if m > 1 else 0), s0
    if (m <= 1 or s1 == 1) and (q <= 1 or max(1, m) <= s2 <= _LD_MAX):
        return W, 0, max(1, m, s2 if q > 1 else 0), s0
    W = W.contiguous()
    return W, 1, max(1, q), m * q


def _offsets(offsets, groups: int, device):
    if offsets.dtype != torch.int32 or offsets.dim() != 1 or offsets.shape[0] != groups + 1:
        raise ValueError(f"offsets must be {groups + 1} int32 values, got {offsets.dtype} {tuple(offsets.shape)}")
    if offsets.device != device:
        raise ValueError(f"offsets are on {offsets.device}, the operands on {device}")
    return offsets.contiguous()


def _same(a, b, what: str) -> None:
    if a.dtype != b.dtype or a.device != b.device:
        raise ValueError(f"{what} are {a.dtype} on {a.device} and {b.dtype} on {b.device}")


def _target(out, shape, dtypes, like, what: str):
    """The tensor a result goes to: `out`, checked, or a new one."""
    if out is None:
        return like.new_empty(shape, dtype=dtypes[0])
    if out.is_neg():
        raise ValueError(f"{what} must not be a negated view")
    if tuple(out.shape) != tuple(shape) or out.dtype not in dtypes or out.device != like.device:
        raise ValueError(f"{what} must be {tuple(shape)} of {dtypes[0]} on {like.device}, got {tuple(out.shape)} of "
                         f"{out.dtype} on {out.device}")
    s = out.stride()
    if (out.shape[-1] > 1 and s[-1] != 1) or (out.shape[-2] > 1 and not max(1, out.shape[-1]) <= s[-2] <= _LD_MAX) or (
            out.dim() == 3 and out.shape[0] > 1 and s[0] < max(1, out.shape[1]) * max(s[1], out.shape[2])):
        raise ValueError(f"{what} must have its rows' entries next to each other and its rows apart, strides {s}")
    return out


def _overlap(a, b) -> bool:
    """Whether two tensors share memory between their first and last entries."""
    def end(t):
        return t.data_ptr() + (sum((n - 1) * s for n, s in zip(t.shape, t.stride())) + 1) * t.element_size()

    return a.numel() > 0 and b.numel() > 0 and a.data_ptr() < end(b) and b.data_ptr() < end(a)


def _ld(t) -> int:
    return max(1, t.shape[-1], t.stride(-2) if t.shape[-2] > 1 else 0)


def grouped_linear(X, W, offsets, out=None, out_dtype=None):
    """``Y[j] = W[e] @ X[j]`` for the rows j of every group e:
    ``offsets[e] <= j < offsets[e + 1]``.

    X is [n, q], W [g, m, q] (either inner dimension contiguous), offsets
    int32 [g + 1] on the device, Y [n, m] in X's type or float32
    (``out_dtype``).  Rows of no group are left as they were in ``out``;
    without ``out`` they are not written.  ``out`` must not overlap X, W or the
    offsets, each taken from its first entry to its last.

    bfloat16 and float16 sums are float32, rounded once.  float32 products of few
    rows and small ones are formed in float32; larger ones of two half-precision
    slices per entry, which hold it to 2^-23 of itself or 2^-39 of the largest
    entry of its row of X or W, and where a row with Inf or NaN gives NaN.  The
    sizes and the alignment alone decide which.
    """
    _same(X, W, "X and W")
    _no_grad("grouped_linear", X, W, out, instead=_INSTEAD)
    t = _type_of(X, "grouped_linear")
    if X.dim() != 2 or W.dim() != 3 or X.shape[1] != W.shape[2]:
        raise ValueError(f"X {tuple(X.shape)} and W {tuple(W.shape)} do not go together")
    g, m, q = W.shape
    n = X.shape[0]
    _fits(n, m, q)
    offsets = _offsets(offsets, g, X.device)
    Y = _target(out, (n, m), (X.dtype, torch.float32) if out is not None else (out_dtype or X.dtype,), X, "out")
    if Y.dtype not in (X.dtype, torch.float32):
        raise TypeError(f"grouped_linear: results are {X.dtype} or float32, not {Y.dtype}")
    with _on_device(X.device):
        X, ldb = _rows(X, "X")
        W, transa, lda, stridea = _weights(W)
        _written(out)
        L.ozgemm_grouped_gemm(t, _TYPES[Y.dtype], g, m, n, q, transa, W, lda, stridea, X, ldb, offsets, Y, _ld(Y))
    return Y


def grouped_linear_grads(dY, X, W, offsets, dX=None, dW=None, dw_dtype=None):
    """The gradients of :func:`grouped_linear`: ``dX[j] = W[e]^T @ dY[j]`` and
    ``dW[e] = sum over j of dY[j] X[j]^T``; returns (dX, dW).

    dX is [n, q] in X's type (rows of no group as in ``out`` there), dW
    [g, m, q] in X's type or float32 (``dw_dtype``), zeros for a group
    without rows.  Sums and float32 operands as in :func:`grouped_linear` (for dW
    a "row" is a column of X or dY within a group).  Neither may overlap dY, X, the offsets or the other, nor
    dX the weights.
    """
    _same(X, W, "X and W")
    _same(dY, X, "dY and X")
    t = _type_of(X, "grouped_linear_grads")
    _no_grad("grouped_linear_grads", dY, X, W, dX, dW)
    if X.dim() != 2 or W.dim() != 3 or dY.dim() != 2 or X.shape[1] != W.shape[2] or (
            dY.shape != (X.shape[0], W.shape[1])):
        raise ValueError(f"dY {tuple(dY.shape)}, X {tuple(X.shape)} and W {tuple(W.shape)} do not go together")
    g, m, q = W.shape
    n = X.shape[0]
    _fits(n, m, q)
    offsets = _offsets(offsets, g, X.device)
    given = dX, dW
    dX = _target(dX, (n, q), (X.dtype,), X, "dX")
    dW = _target(dW, (g, m, q), (X.dtype, torch.float32) if dW is not None else (dw_dtype or X.dtype,), X, "dW")
    if dW.dtype not in (X.dtype, torch.float32):
        raise TypeError(f"grouped_linear_grads: dW is {X.dtype} or float32, not {dW.dtype}")
    with _on_device(X.device):
        X, ldx = _rows(X, "X")
        dY, ldy = _rows(dY, "dY")
        W, transa, lda, stridea = _weights(W)
        # dX is written before X is read for dW; the calls themselves refuse the other overlaps
        if given[0] is not None and (_overlap(dX, X) or _overlap(dX, dW)):
            raise ValueError("dX must not overlap X or dW")
        _written(*given)
        L.ozgemm_grouped_gemm(t, t, g, q, n, m, 1 - transa, W, lda, stridea, dY, ldy, offsets, dX, _ld(dX))
        L.ozgemm_grouped_outer(t, _TYPES[dW.dtype], g, q, m, n, X, ldx, dY, ldy, offsets, dW, _ld(dW),
                               max(dW.stride(0) if g > 1 else 0, _ld(dW) * m))
    return dX, dW


#: Muon's quintic, for every step
QUINTIC = (3.4445, -4.7750, 2.0315)


def orthogonalize(G, steps: int = 5, coeffs=QUINTIC, eps: float = 1e-7, out=None, s: int = 14):
    """``steps`` Newton-Schulz steps on every matrix of G [..., rows, cols]:
    ``X = G / (norm + eps)``, then ``X = a X + (b P + c P P) X`` with
    ``P = X X^T`` (of the smaller side).

    G is float64, float32, bfloat16 or float16 and the result of its type, rounded
    once (between the steps X is held to 22 bits, float64 to 53);
    ``coeffs`` is one triple (a, b, c) or one for each step.  ``out`` may be G
    itself.  ``s`` is the number of moduli of the float64 products.
    """
    t = _type_of(G, "orthogonalize", tuple(_TYPES))
    if G.dim() < 2:
        raise ValueError(f"orthogonalize needs matrices, got {tuple(G.shape)}")
    if steps < 0:
        raise ValueError("steps must not be negative")
    co = list(coeffs)
    if len(co) == 3 and not any(hasattr(c, "__len__") for c in co):
        co = [co] * steps
    elif not all(hasattr(c, "__len__") for c in co):
        co = []
    if len(co) != steps or any(len(c) != 3 for c in co):
        raise ValueError(f"coeffs must be one triple or {steps} of them")
    _no_grad("orthogonalize", G, out)
    r, c = G.shape[-2:]
    _fits(r, c)
    given = out
    if out is None:
        out = torch.empty(G.shape, dtype=G.dtype, device=G.device)
    elif out.is_neg():
        raise ValueError("out must not be a negated view")
    elif out.shape != G.shape or out.dtype != G.dtype or out.device != G.device:
        raise ValueError(f"out must be {tuple(G.shape)} of {G.dtype} on {G.device}, got {tuple(out.shape)} of "
                         f"{out.dtype} on {out.device}")
    if G.numel() == 0:
        return out
    with _on_device(G.device):
        G = G.resolve_neg()
        g = _matrices(G)
        o = _matrices(out)
        if o is None:
            raise ValueError(f"out must be matrices of contiguous rows evenly apart, strides {out.stride()}")
        if g is None:
            g = _matrices(G.contiguous())
        _written(given)
        L.ozgemm_orthogonalize(t, g[1], c, r, g[0], g[2], g[3], steps, [v for x in co for v in x], eps, s, o[0], o[2],
                               o[3])
    return out


def _matrices(t):
    """(tensor, batch, row distance, matrix distance) of a batch of matrices
    with contiguous rows, all evenly apart; None if it is none."""
    r, c = t.shape[-2:]
    ld = max(1, c, t.stride(-2) if r > 1 else 0)
    if (c > 1 and t.stride(-1) != 1) or (r > 1 and not c <= t.stride(-2) <= _LD_MAX):
        return None
    batch, step = 1, 0
    for size, stride in zip(reversed(t.shape[:-2]), reversed(t.stride()[:-2])):
        if size == 1:
            continue
        if batch > 1 and stride != step * batch:
            return None
        if batch == 1:
            step = stride
        batch *= size
    return t, batch, ld, step
