"""A layer in 8 bits on torch tensors (row-major): the root-mean-square norm in
front of it, blocks of 128 in 8-bit floating point, and their products: the
calls of :mod:`.ozgemm` with their shapes, strides and types taken from the
tensors.

A matrix in blocks is a pair of tensors: values of ``torch.float8_e4m3fn`` or
``torch.float8_e5m2``, and float32 scales, one for every 128 entries of a row
([rows, ceil(columns / 128)]) or for every 128 x 128 tile
([ceil(rows / 128), ceil(columns / 128)]).

As in :mod:`.layers` nothing here is recorded by autograd: the gradients are
calls of their own, and tensors that require a gradient or carry a tangent are
refused.  Work goes on the current stream of the tensors' device.
"""
from __future__ import annotations

import torch

from . import ozgemm as L
from .layers import _LD_MAX, _TYPES, _fits, _ld, _no_grad, _on_device, _overlap, _rows, _target, _type_of, _written

BLOCK = 128
_EIGHT = {torch.float8_e4m3fn: L.OZGEMM_E4M3, torch.float8_e5m2: L.OZGEMM_E5M2}
_OUT = (torch.bfloat16, torch.float16, torch.float32)


def _eight(dtype, what: str) -> int:
    if dtype not in _EIGHT:
        raise TypeError(f"{what}: {dtype} is not supported (one of {', '.join(map(str, _EIGHT))})")
    return _EIGHT[dtype]


def _new_blocks(n: int, q: int, rows: int, dtype, like):
    """(values, scales) to be written: values whose rows begin on 16-byte
    boundaries, as the products read them in place; scales of a row each with
    those of one block next to one another, as they load them."""
    blocks = -(-q // BLOCK)
    v = like.new_empty_strided((n, q), (-(-q // 16) * 16, 1), dtype=dtype)
    if rows == 1:
        return v, like.new_empty_strided((n, blocks), (1, n), dtype=torch.float32)
    return v, like.new_empty((-(-n // rows), blocks), dtype=torch.float32)


def quantize_blocks(X, rows: int = 1, both: bool = False, dtype=torch.float8_e4m3fn):
    """(values, scales) of X [n, q] in blocks of ``rows`` (1 or 128) x 128; with
    ``both`` (values, scales, values of X^T [q, n], scales of X^T) from one
    reading of X: blocks of the transpose are ``rows`` x 128 of *its* entries.

    X is bfloat16, float16 or float32, either dimension contiguous.  A block's
    scale is the least power of two that keeps its finite entries within the
    type's range, and an entry is rounded once; Inf and NaN become NaN.
    """
    _type_of(X, "quantize_blocks")
    _eight(dtype, "quantize_blocks")
    if rows not in (1, BLOCK):
        raise ValueError(f"blocks have 1 or {BLOCK} rows, not {rows}")
    if X.dim() != 2:
        raise ValueError(f"X must have two dimensions, got {tuple(X.shape)}")
    _no_grad("quantize_blocks", X)
    _fits(*X.shape)
    with _on_device(X.device):
        return _quantize(X, rows, both, dtype)


def _quantize(X, rows: int, both: bool, dtype):
    n, q = X.shape
    V, S = _new_blocks(n, q, rows, dtype, X)
    Vt, St = _new_blocks(q, n, rows, dtype, X) if both else (None, None)
    plain, turned, t = (V, S), (Vt, St), _TYPES[X.dtype]
    if n > 1 and q > 1 and X.stride(0) == 1 and X.stride(1) >= n:  # the transpose lies row by row
        X, (n, q), plain, turned = X.t(), (q, n), turned, plain
    X, ldx = _rows(X, "X")
    L.ozgemm_quantize_blocks(t, _EIGHT[dtype], rows, n, q, X, ldx, *_block_args(*plain), *_block_args(*turned))
    return (V, S, Vt, St) if both else (V, S)


def _block_args(V, S):
    """(values, leading dimension, scales, their strides) as the calls take them."""
    if V is None:
        return None, 0, None, 0, 0
    return V, _ld(V), S, S.stride(0), S.stride(1)


def _values(V, what: str):
    """8-bit rows with their entries next to each other, and their distance."""
    n, q = V.shape
    if V.is_contiguous():
        return V, max(1, q)
    if (q > 1 and V.stride(1) != 1) or (n > 1 and not max(1, q) <= V.stride(0) <= _LD_MAX):
        copy = torch.empty((n, -(-q // 16) * 16), dtype=V.dtype, device=V.device)[:, :q]
        V = copy.copy_(V)
    return V, _ld(V)


def _scales(S, rows: int, cols: int, what: str, like, shared: bool):
    """(scales, rows that share one)"""
    blocks = -(-cols // BLOCK)
    if S.dtype != torch.float32 or S.dim() != 2:
        raise ValueError(f"{what} must be a matrix of float32, got {S.dtype} {tuple(S.shape)}")
    if S.device != like.device:
        raise ValueError(f"{what} are on {S.device}, the values on {like.device}")
    if S.is_neg():
        S = S.resolve_neg()
    if tuple(S.shape) == (rows, blocks):
        return S, 1
    if shared and tuple(S.shape) == (-(-rows // BLOCK), blocks):
        return S, BLOCK
    raise ValueError(f"{what} of {rows} x {cols} values must be {(rows, blocks)}"
                     f"{f' or {(-(-rows // BLOCK), blocks)}' if shared else ''}, got {tuple(S.shape)}")


def scaled_linear(X, xs, W, ws, out=None, out_dtype=None):
    """``Y = (X xs) (W ws)^T`` for matrices in blocks: X [n, q] with a scale for
    every row and 128 columns, W [m, q] with those or one for every 128 x 128 tile,
    Y [n, m] in bfloat16 (``out_dtype``: float16 or float32).

    Values are either 8-bit type; scales are any float32, and so must be the product of a
    row's of X and one of W, which is taken first (1e20 and 1e20 make NaN of a block of zeros).
    Rows on 16-byte boundaries are read in place, others from a copy.  ``out`` must not overlap the operands.

    float32 results, and those of up to 16 rows of X, are summed in float32.  Of others a
    block's 128 products are summed by the 8-bit matrix cores, which drop what lies below
    2^-13 of the largest product next to it, and blocks in float32.  Over all results that
    is 1.5e-5 of their norm for gaussian entries and 4.6e-5 where one column of X in a
    hundred is 21 times larger (float16 rounds to 2.1e-4, bfloat16 to 1.7e-3); it is not bounded relative
    to a single result whose products cancel, for which ``out_dtype=torch.float32`` is there.
    A row's last bits depend on how many rows come with it: of those two ways, and
    by the order of sums, which follows the sizes.
    """
    _eight(X.dtype, "scaled_linear")
    _eight(W.dtype, "scaled_linear")
    _no_grad("scaled_linear", X, xs, W, ws, out, instead=" and take the gradients from scaled_linear_grads")
    if X.dim() != 2 or W.dim() != 2 or X.shape[1] != W.shape[1]:
        raise ValueError(f"X {tuple(X.shape)} and W {tuple(W.shape)} do not go together")
    if X.device != W.device:
        raise ValueError(f"X and W are on {X.device} and {W.device}")
    (n, q), m = X.shape, W.shape[0]
    _fits(n, m, q)
    xs, _ = _scales(xs, n, q, "xs", X, False)
    ws, wrows = _scales(ws, m, q, "ws", W, True)
    if out is None:
        out_dtype = out_dtype or torch.bfloat16
        if out_dtype not in _OUT:
            raise TypeError(f"scaled_linear: results are bfloat16, float16 or float32, not {out_dtype}")
        Y, ldy = X.new_empty((n, m), dtype=out_dtype), max(1, m)
    else:
        Y = _target(out, (n, m), _OUT, X, "out")
        ldy = _ld(Y)
    with _on_device(X.device):
        if out is not None:
            _written(out)
        _product(X, xs, W, ws, wrows, Y, ldy)
    return Y


def _product(X, xs, W, ws, wrows: int, Y, ldy: int) -> None:
    (n, q), m = X.shape, W.shape[0]
    tx, tw = _EIGHT[X.dtype], _EIGHT[W.dtype]
    X, ldx = _values(X, "X")
    W, ldw = _values(W, "W")
    L.ozgemm_scaled_gemm(tw, tx, _TYPES[Y.dtype], m, n, q, W, ldw, ws, wrows, *ws.stride(), X, ldx, xs, *xs.stride(), Y, ldy)


def scaled_linear_grads(dY, Xt, xts, Wt, wts, dX=None, dW=None, dx_dtype=None, dw_dtype=None, dtype=torch.float8_e4m3fn):
    """The gradients of :func:`scaled_linear` as a layer in 8 bits takes them;
    returns (dX, dW).

    dY [n, m] (bfloat16, float16 or float32) is put in blocks of ``dtype`` along
    both of its dimensions, from one reading; then ``dX = dY W`` [n, q] with
    Wt [q, m], the weights turned over, in blocks, and ``dW = dY^T X`` [m, q] with
    Xt [q, n], the activations turned over, in blocks of 1 x 128 along their rows
    (``quantize_blocks(..., both=True)`` gives both).  dX is of dY's type
    (``dx_dtype``), dW too (``dw_dtype``); sums as in :func:`scaled_linear`.
    """
    _type_of(dY, "scaled_linear_grads")
    _eight(dtype, "scaled_linear_grads")
    _eight(Xt.dtype, "scaled_linear_grads")
    _eight(Wt.dtype, "scaled_linear_grads")
    _no_grad("scaled_linear_grads", dY, Xt, xts, Wt, wts, dX, dW)
    if dY.dim() != 2 or Xt.dim() != 2 or Wt.dim() != 2 or Xt.shape != (Wt.shape[0], dY.shape[0]) or (
            Wt.shape[1] != dY.shape[1]):
        raise ValueError(f"dY {tuple(dY.shape)}, Xt {tuple(Xt.shape)} and Wt {tuple(Wt.shape)} do not go together")
    if not dY.device == Xt.device == Wt.device:
        raise ValueError(f"dY, Xt and Wt are on {dY.device}, {Xt.device} and {Wt.device}")
    (n, m), q = dY.shape, Xt.shape[0]
    _fits(n, m, q)
    xts, xrows = _scales(xts, q, n, "xts", Xt, True)
    wts, wrows = _scales(wts, q, m, "wts", Wt, True)
    given = dX, dW
    for t, want in ((dX, dx_dtype), (dW, dw_dtype)):
        if t is None and (want or dY.dtype) not in _OUT:
            raise TypeError(f"scaled_linear_grads: results are bfloat16, float16 or float32, not {want}")
    dX = _target(dX, (n, q), _OUT if dX is not None else (dx_dtype or dY.dtype,), dY, "dX")
    dW = _target(dW, (m, q), _OUT if dW is not None else (dw_dtype or dY.dtype,), dY, "dW")
    # dX is written before Xt is read for dW (new tensors overlap nothing)
    held = (Xt, xts, Wt, wts) if given[1] is None else (Xt, xts, Wt, wts, dW)
    if (given[0] is not None and any(_overlap(dX, t) for t in held)) or (
            given[1] is not None and any(_overlap(dW, t) for t in held[:4])):
        raise ValueError("dX and dW must not overlap the operands or each other")
    with _on_device(dY.device):
        V, S, Vt, St = _quantize(dY, 1, True, dtype)
        _written(*given)
        _product(V, S, Wt, wts, wrows, dX, _ld(dX))
        _product(Vt, St, Xt, xts, xrows, dW, _ld(dW))
    return dX, dW


def _norm_rows(t, what: str, like):
    if t.shape != like.shape or t.dtype != like.dtype or t.device != like.device:
        raise ValueError(f"{what} must be {tuple(like.shape)} of {like.dtype} on {like.device}, got {tuple(t.shape)} of "
                         f"{t.dtype} on {t.device}")
    return _rows(t, what)


def _norm_weight(weight, X):
    if weight.dtype not in (X.dtype, torch.float32):
        raise TypeError(f"the weight must be {X.dtype} or float32, not {weight.dtype}")
    if weight.shape != (X.shape[1],) or weight.device != X.device:
        raise ValueError(f"the weight must be {X.shape[1]} entries on {X.device}, got {tuple(weight.shape)} on "
                         f"{weight.device}")
    return weight.resolve_neg().contiguous()


def _rms_norm(what: str, X, weight, residual, eps, out, H, dtype):
    t = _type_of(X, what)
    _no_grad(what, X, weight, residual, out, H, instead=" and take the gradients from rms_norm_grads")
    if X.dim() != 2:
        raise ValueError(f"X must have two dimensions, got {tuple(X.shape)}")
    if not eps >= 0:
        raise ValueError(f"eps must not be negative, got {eps}")
    n, q = X.shape
    _fits(n, q)
    weight = _norm_weight(weight, X)
    if residual is None and H is not None:
        raise ValueError("H is the sum with a residual: without one it is X itself")
    given = out, H
    if dtype is None:
        out = _target(out, (n, q), (X.dtype,), X, "out")
    if residual is not None:
        H = _target(H, (n, q), (X.dtype,), X, "H")
    with _on_device(X.device):
        S = None
        if dtype is not None:
            out, S = _new_blocks(n, q, 1, dtype, X)
        kept = X if residual is None else H
        X, ldx = _rows(X, "X")
        R, ldr = (None, 0) if residual is None else _norm_rows(residual, "the residual", kept)
        _written(*given)
        L.ozgemm_rms_norm(t, t if dtype is None else _EIGHT[dtype], _TYPES[weight.dtype], n, q, X, ldx, R, ldr, weight,
                          eps, H, _ld(H) if H is not None else 0, out, _ld(out), S, *(S.stride() if S is not None else (0, 0)))
    return out, S, kept


def rms_norm(X, weight, residual=None, eps: float = 1e-6, out=None, H=None):
    """(Y, H): the root-mean-square norm of the rows of ``H = X + residual``,
    ``Y = H weight / sqrt(mean(H^2) + eps)``.

    X is [n, q] of bfloat16, float16 or float32, the residual and H of its shape
    and type (the sum is rounded to it, as X + residual is; without a residual H is
    X itself), the weight [q] of its type or float32.  Y is formed in
    float64 and rounded once.  ``H`` may be X or the residual itself, and so may ``out``
    (but not both the same).
    """
    Y, _, H = _rms_norm("rms_norm", X, weight, residual, eps, out, H, None)
    return Y, H


def rms_norm_quantized(X, weight, residual=None, eps: float = 1e-6, H=None, dtype=torch.float8_e4m3fn):
    """(values, scales, H): :func:`rms_norm` with Y in blocks of 1 x 128, as
    :func:`scaled_linear` takes them, rounded once from the exact norm."""
    _eight(dtype, "rms_norm_quantized")
    return _rms_norm("rms_norm_quantized", X, weight, residual, eps, None, H, dtype)


def rms_norm_grads(dY, H, weight, dH=None, eps: float = 1e-6, dX=None):
    """The gradients of :func:`rms_norm`: returns (dX, dweight), where dX is the
    residual's gradient too.

    H is what rms_norm returned (X without a residual), dH the gradient that
    reaches H from elsewhere.  ``dX`` may be dY, H or dH itself.  dweight is of the
    weight's type; its sums over the rows are float32 and float64.
    """
    t = _type_of(dY, "rms_norm_grads")
    _no_grad("rms_norm_grads", dY, H, weight, dH, dX)
    if dY.dim() != 2:
        raise ValueError(f"dY must have two dimensions, got {tuple(dY.shape)}")
    if not eps >= 0:
        raise ValueError(f"eps must not be negative, got {eps}")
    n, q = dY.shape
    _fits(n, q)
    weight = _norm_weight(weight, dY)
    given = dX
    dX = _target(dX, (n, q), (dY.dtype,), dY, "dX")
    with _on_device(dY.device):
        like = dY
        dY, lddy = _rows(dY, "dY")
        H, ldh = _norm_rows(H, "H", like)
        dH, lddh = (None, 0) if dH is None else _norm_rows(dH, "dH", like)
        dw = torch.empty_like(weight)
        _written(given)
        L.ozgemm_rms_norm_grads(t, _TYPES[weight.dtype], n, q, dY, lddy, H, ldh, weight, dH, lddh, eps, dX, _ld(dX), dw)
    return dX, dw
