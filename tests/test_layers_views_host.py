"""Which memory the tensor calls hand to the library, for views whose memory
does not hold their values.  The library is a stand-in: no GPU."""
import contextlib
import ctypes

import pytest
import torch

from fp64_gemm_emulation_ozii_amd import layers


def values(t, shape, ld):
    """What lies at rows of `shape`, `ld` entries apart, from t's first entry on."""
    n = (shape[0] - 1) * ld + shape[1]
    return torch.frombuffer((ctypes.c_char * (n * 4)).from_address(t.data_ptr()), dtype=torch.float32).as_strided(
        shape, (ld, 1)).clone()


@pytest.fixture
def seen(monkeypatch):
    got = {}
    monkeypatch.setattr(layers, "_on_device", lambda device: contextlib.nullcontext())

    def gemm(type, ctype, groups, m, n, q, transa, A, lda, stridea, B, ldb, *rest):
        a = values(A, (m, q) if transa else (q, m), lda)
        got["gemm"] = a if transa else a.T, values(B, (n, q), ldb)

    def outer(type, ctype, groups, m, q, n, A, lda, B, ldb, *rest):
        got["outer"] = values(A, (n, m), lda), values(B, (n, q), ldb)

    def ortho(type, batch, m, n, G, ldg, *rest):
        got["ortho"] = values(G, (n, m), ldg)

    monkeypatch.setattr(layers.L, "ozgemm_grouped_gemm", gemm)
    monkeypatch.setattr(layers.L, "ozgemm_grouped_outer", outer)
    monkeypatch.setattr(layers.L, "ozgemm_orthogonalize", ortho)
    return got


def negated(*shape):
    """The imaginary part of a conjugate: a view of memory that holds the negated values."""
    t = torch.complex(torch.randn(*shape, 1), torch.randn(*shape, 1)).conj().imag[..., 0]
    # one column of it lies as a row-major array of one column does
    return t


@pytest.mark.parametrize("n, q", [(5, 1), (1, 1), (4, 3)])
def test_negated_views_are_read_as_their_values(seen, n, q):
    X, W, dY = negated(n, q), negated(1, 2, q), negated(n, 2)
    assert X.is_neg() and W.is_neg() and dY.is_neg()
    off = torch.tensor([0, n], dtype=torch.int32)
    layers.grouped_linear(X, W, off)
    assert torch.equal(seen["gemm"][0], W[0].resolve_neg()) and torch.equal(seen["gemm"][1], X.resolve_neg())
    layers.grouped_linear_grads(dY, X, W, off)
    assert torch.equal(seen["gemm"][0], W[0].resolve_neg().T) and torch.equal(seen["gemm"][1], dY.resolve_neg())
    assert torch.equal(seen["outer"][0], X.resolve_neg()) and torch.equal(seen["outer"][1], dY.resolve_neg())
    layers.orthogonalize(X)
    assert torch.equal(seen["ortho"], X.resolve_neg())


def test_results_do_not_go_to_negated_views(seen):
    off = torch.tensor([0, 5], dtype=torch.int32)
    X, W, dY = torch.zeros(5, 1), torch.zeros(1, 1, 1), torch.zeros(5, 1)
    with pytest.raises(ValueError, match="negated"):
        layers.grouped_linear(X, W, off, out=negated(5, 1))
    with pytest.raises(ValueError, match="negated"):
        layers.grouped_linear_grads(dY, X, W, off, dX=negated(5, 1))
    with pytest.raises(ValueError, match="negated"):
        layers.grouped_linear_grads(dY, X, W, off, dW=negated(1, 1, 1))
    with pytest.raises(ValueError, match="negated"):
        layers.orthogonalize(X, out=negated(5, 1))
    assert not seen


def test_gradients_that_would_overwrite_what_is_still_read(seen):
    off = torch.tensor([0, 2, 6], dtype=torch.int32)
    X, W, dY = torch.randn(6, 3), torch.randn(2, 4, 3), torch.randn(6, 4)
    both = torch.zeros(6 * 3 + 2 * 4 * 3)
    for bad in (dict(dX=X), dict(dX=both[:18].view(6, 3), dW=both[17:41].view(2, 4, 3)),
                dict(dX=both[20:38].view(6, 3), dW=both[:24].view(2, 4, 3))):
        with pytest.raises(ValueError, match="overlap"):
            layers.grouped_linear_grads(dY, X, W, off, **bad)
        assert not seen
    # next to each other, and over an X that is read from a copy
    layers.grouped_linear_grads(dY, X, W, off, dX=both[:18].view(6, 3), dW=both[18:42].view(2, 4, 3))
    wide = torch.zeros(3, 6)
    layers.grouped_linear_grads(dY, wide.t(), W, off, dX=wide.view(6, 3))
