"""Argument checks of the grouped products: they run before anything is
enqueued, so they need no GPU."""
import pytest
import torch

import fp64_gemm_emulation_ozii_amd as oz
from fp64_gemm_emulation_ozii_amd import ozgemm as L

P = 1 << 40  # never read: every call below is refused, or has nothing to do
A, B, C, O, WS = P, P + (1 << 34), P + (2 << 34), P + (3 << 34), P + (4 << 34)


def gemm(type=L.OZGEMM_BF16, ctype=None, groups=4, m=64, n=100, q=128, transa=1, A=A, lda=128, stridea=64 * 128, B=B,
         ldb=128, off=O, C=C, ldc=64, ws=None, nbytes=0):
    return L.lib().ozgemm_grouped_gemm(type, type if ctype is None else ctype, groups, m, n, q, transa, A, lda,
                                       stridea, B, ldb, off, C, ldc, ws, nbytes, None)


def outer(type=L.OZGEMM_BF16, ctype=None, groups=4, m=64, q=128, n=100, A=A, lda=64, B=B, ldb=128, off=O, C=C, ldc=64,
          stridec=64 * 128, ws=None, nbytes=0):
    return L.lib().ozgemm_grouped_outer(type, type if ctype is None else ctype, groups, m, q, n, A, lda, B, ldb, off,
                                        C, ldc, stridec, ws, nbytes, None)


@pytest.mark.parametrize("change, status", [
    (dict(type=L.OZGEMM_F64), -1), (dict(type=7), -1), (dict(ctype=L.OZGEMM_F16), -2), (dict(groups=-1), -3),
    (dict(m=-1), -4), (dict(n=-1), -5), (dict(q=-1), -6), (dict(transa=2), -7), (dict(A=None), -8),
    (dict(lda=127), -9), (dict(transa=0, lda=63), -9), (dict(stridea=-1), -10), (dict(B=None), -11),
    (dict(ldb=127), -12), (dict(off=None), -13), (dict(C=None), -14), (dict(ldc=63), -15),
    (dict(C=A + 64), -14), (dict(C=B), -14), (dict(C=O), -14), (dict(A=C - 2), -14),
    (dict(m=L.OZGEMM_MAX_ROWS + 1, ldc=1 << 22), L.OZGEMM_RANGE), (dict(n=L.OZGEMM_MAX_ROWS + 1), L.OZGEMM_RANGE),
    (dict(q=L.OZGEMM_MAX_ROWS + 1, lda=1 << 22, ldb=1 << 22), L.OZGEMM_RANGE),
    (dict(groups=L.OZGEMM_GROUPS_MAX + 1), L.OZGEMM_RANGE),
    (dict(type=L.OZGEMM_F32, n=100000), -16), (dict(type=L.OZGEMM_F32, n=100000, ws=WS + 16, nbytes=1 << 30), -16),
    (dict(type=L.OZGEMM_F32, n=100000, ws=WS, nbytes=1000), L.OZGEMM_WORKSPACE_TOO_SMALL),
    (dict(type=L.OZGEMM_F32, A=A + 4, n=100000), -16), (dict(type=L.OZGEMM_F32, transa=0, n=100000), -16),
    (dict(type=L.OZGEMM_F32, ldb=129, n=100000), -16), (dict(q=126, n=100000), -16),
    (dict(ldb=129, n=100000), -16), (dict(A=A + 2, n=100000), -16), (dict(B=B + 8, n=100000), -16),
    (dict(m=0), 0), (dict(n=0), 0), (dict(groups=0), 0), (dict(m=0, A=None, B=None, off=None, C=None), 0),
])
def test_grouped_gemm_refusals(change, status):
    assert gemm(**change) == status


# too many entries for the kernel that reads any operands as they lie
WIDE = dict(q=20000, n=10000, ldb=20000, stridec=64 * 20000)


@pytest.mark.parametrize("change, status", [
    (dict(type=L.OZGEMM_F64), -1), (dict(ctype=L.OZGEMM_F16), -2), (dict(groups=-1), -3), (dict(m=-1), -4),
    (dict(q=-1), -5), (dict(n=-1), -6), (dict(A=None), -7), (dict(lda=63), -8), (dict(B=None), -9),
    (dict(ldb=127), -10), (dict(off=None), -11), (dict(C=None), -12), (dict(ldc=63), -13),
    (dict(stridec=64 * 128 - 1), -14), (dict(stridec=-1, groups=1), -14), (dict(C=A), -12), (dict(C=B), -12),
    (dict(C=O + 4), -12), (dict(n=L.OZGEMM_MAX_ROWS + 1), L.OZGEMM_RANGE),
    (dict(type=L.OZGEMM_F32, **WIDE), -15),
    (dict(type=L.OZGEMM_F32, ws=WS, nbytes=1000, **WIDE), L.OZGEMM_WORKSPACE_TOO_SMALL),
    (dict(WIDE, A=A + 2), -15), (dict(WIDE, ldb=20001), -15),
    # 2^21 columns, each group's rounded up to 64: the rows of the slices would pass 32-bit offsets
    (dict(type=L.OZGEMM_F32, n=2090000, groups=1000, C=P + (40 << 34)), L.OZGEMM_RANGE),
    (dict(m=0), 0), (dict(q=0), 0), (dict(groups=0), 0),
])
def test_grouped_outer_refusals(change, status):
    assert outer(**change) == status


def test_workspace_bytes():
    w = L.ozgemm_grouped_gemm_workspace_bytes
    assert w(L.OZGEMM_BF16, 4, 64, 100, 128, 1, A, 128, 64 * 128, B, 128) == 0  # read in place
    assert w(L.OZGEMM_BF16, 4, 64, 100, 128, 1, A + 2, 128, 64 * 128, B, 128) == 0  # so are few columns wherever they lie
    assert w(L.OZGEMM_BF16, 4, 64, 100000, 128, 1, A + 2, 128, 64 * 128, B, 128) >= 4 * 64 * 128 * 2
    assert w(L.OZGEMM_BF16, 4, 64, 100000, 129, 1, A, 136, 64 * 136, B, 136) >= (4 * 64 + 100000) * 192 * 2
    assert w(L.OZGEMM_F32, 4, 64, 100000, 128, 1, A, 128, 64 * 128, B, 128) >= (4 * 64 + 100000) * (128 * 4 + 4)
    assert w(L.OZGEMM_F32, 4, 64, 100, 128, 1, A, 128, 64 * 128, B, 128) == 0
    assert w(L.OZGEMM_F32, 4, 64, 100, 128, 0, A, 64, 64 * 128, B, 128) == 0
    assert w(L.OZGEMM_F64, 4, 64, 100, 128, 1, A, 128, 64 * 128, B, 128) == 0
    assert w(L.OZGEMM_F32, 4, 64, 0, 128, 1, A, 128, 64 * 128, B, 128) == 0
    # sizes past 32 bits
    assert w(L.OZGEMM_F32, 64, 1 << 15, 1 << 15, 1 << 15, 1, A, 1 << 15, 1 << 30, B, 1 << 15) >= 1 << 38
    o = L.ozgemm_grouped_outer_workspace_bytes
    assert o(L.OZGEMM_F16, 4, 64, 128, 100, A, 64, B, 128) == 0
    assert o(L.OZGEMM_F16, 4, 60, 128, 100, A, 64, B, 128) == 0
    assert o(L.OZGEMM_F16, 4, 60, 20000, 10000, A, 64, B, 20000) >= (60 + 20000) * 10000 * 2
    assert o(L.OZGEMM_F32, 4, 64, 20000, 10000, A, 64, B, 20000) >= (64 + 20000) * 10000 * 4


def _args(**change):
    a = dict(X=torch.zeros(10, 8), W=torch.zeros(3, 4, 8), offsets=torch.zeros(4, dtype=torch.int32))
    a.update(change)
    return a


@pytest.mark.parametrize("change, error", [
    (dict(X=torch.zeros(10, 8, dtype=torch.float64), W=torch.zeros(3, 4, 8, dtype=torch.float64)), TypeError),
    (dict(X=torch.zeros(10, 8, dtype=torch.bfloat16)), ValueError),
    (dict(X=torch.zeros(10, 7)), ValueError), (dict(X=torch.zeros(10)), ValueError),
    (dict(W=torch.zeros(4, 8)), ValueError), (dict(offsets=torch.zeros(4)), ValueError),
    (dict(offsets=torch.zeros(3, dtype=torch.int32)), ValueError),
    (dict(out=torch.zeros(10, 5)), ValueError), (dict(out=torch.zeros(10, 4, dtype=torch.float16)), ValueError),
    (dict(out=torch.zeros(4, 10).t()), ValueError), (dict(out=torch.zeros(1, 4).expand(10, 4)), ValueError),
    (dict(out_dtype=torch.float64), TypeError),
    (dict(W=torch.zeros(3, 4, 8, requires_grad=True)), RuntimeError),
])
def test_grouped_linear_refusals(change, error):
    with pytest.raises(error):
        oz.grouped_linear(**_args(**change))


@pytest.mark.parametrize("change, error", [
    (dict(dY=torch.zeros(10, 5)), ValueError), (dict(dY=torch.zeros(9, 4)), ValueError),
    (dict(dY=torch.zeros(10, 4, dtype=torch.float16)), ValueError), (dict(dW=torch.zeros(3, 4, 7)), ValueError),
    (dict(dX=torch.zeros(10, 8, dtype=torch.bfloat16)), ValueError), (dict(dw_dtype=torch.float16), TypeError),
    (dict(dW=torch.zeros(1, 4, 8).expand(3, 4, 8)), ValueError),
])
def test_grouped_linear_grads_refusals(change, error):
    with pytest.raises(error):
        oz.grouped_linear_grads(**_args(**{"dY": torch.zeros(10, 4), **change}))


def ortho(type=L.OZGEMM_F32, batch=2, m=64, n=32, G=A, ldg=64, strideg=64 * 32, steps=5, co=(3.4445, -4.775, 2.0315),
          eps=1e-7, s=14, O=C, ldo=64, strideo=64 * 32, ws=WS, nbytes=1 << 33):
    import ctypes
    c = None if co is None else (ctypes.c_double * max(1, 3 * steps))(*(list(co) * steps))
    return L.lib().ozgemm_orthogonalize(type, batch, m, n, G, ldg, strideg, steps, c, eps, s, O, ldo, strideo, ws,
                                        nbytes, None)


@pytest.mark.parametrize("change, status", [
    (dict(type=4), -1), (dict(type=-1), -1), (dict(batch=-1), -2), (dict(m=-1), -3), (dict(n=-1), -4),
    (dict(G=None), -5), (dict(ldg=63), -6), (dict(strideg=-1), -7), (dict(steps=-1, co=None), -8),
    (dict(steps=L.OZGEMM_ORTHO_STEPS_MAX + 1), -8), (dict(co=None), -9), (dict(co=(1e6, 0, 0)), -9),
    (dict(co=(float("nan"), 0, 0)), -9), (dict(eps=-1.0), -10), (dict(eps=float("nan")), -10),
    (dict(eps=float("inf")), -10), (dict(type=L.OZGEMM_F64, s=0), -11), (dict(type=L.OZGEMM_F64, s=21), -11),
    (dict(O=None), -12), (dict(ldo=63), -13), (dict(strideo=64 * 32 - 1), -14), (dict(O=A + 4), -12),
    (dict(O=A, ldo=65, strideo=65 * 32), -12), (dict(O=A + 64 * 32 * 4), -12), (dict(ws=None), -15),
    (dict(ws=WS + 16), -15), (dict(nbytes=1000), L.OZGEMM_WORKSPACE_TOO_SMALL),
    (dict(m=L.OZGEMM_ORTHO_MAX + 1, ldg=1 << 20, ldo=1 << 20, strideo=1 << 40), L.OZGEMM_RANGE),
    (dict(batch=65536), L.OZGEMM_RANGE), (dict(co=(1e5, 0, 0)), L.OZGEMM_RANGE),
    (dict(type=L.OZGEMM_F64, s=1), L.OZGEMM_RANGE),
    (dict(batch=0), 0), (dict(m=0), 0), (dict(n=0, G=None, O=None), 0),
])
def test_orthogonalize_refusals(change, status):
    assert ortho(**change) == status


def test_orthogonalize_workspace_bytes():
    w = L.ozgemm_orthogonalize_workspace_bytes
    assert w(L.OZGEMM_F32, 2, 100, 50, 0) == w(L.OZGEMM_F32, 2, 50, 100, 0) >= 2 * 12 * 100 * 50
    assert w(L.OZGEMM_BF16, 1, 16384, 16384, 0) > 1 << 32
    assert w(L.OZGEMM_F64, 1, 2048, 2048, 14) >= 5 * 2048 ** 2 * 8 + L.ozgemm_workspace_bytes(2048, 2048, 2048, 14)
    assert w(L.OZGEMM_F64, 3, 96, 200, 14) >= 3 * (2 * 96 * 200 + 2 * 96 * 96) * 8
    for bad in ((4, 1, 8, 8, 14), (L.OZGEMM_F32, 0, 8, 8, 14), (L.OZGEMM_F64, 1, 8, 8, 0), (L.OZGEMM_F64, 1, 8, 8, 21)):
        assert w(*bad) == 0


@pytest.mark.parametrize("how, error", [
    (dict(G=torch.zeros(4)), ValueError), (dict(G=torch.zeros(4, 4, dtype=torch.int32)), TypeError),
    (dict(steps=-1), ValueError), (dict(coeffs=(1.0, 2.0)), ValueError),
    (dict(coeffs=[(1.0, 2.0, 3.0)] * 4), ValueError), (dict(out=torch.zeros(4, 5)), ValueError),
    (dict(out=torch.zeros(8, 8, dtype=torch.float64)), ValueError),
    (dict(G=torch.zeros(8, 8, requires_grad=True)), RuntimeError),
])
def test_orthogonalize_python_refusals(how, error):
    with pytest.raises(error):
        oz.orthogonalize(**{"G": torch.zeros(8, 8), **how})


def test_tensors_off_the_gpu_are_refused():
    with pytest.raises(ValueError, match="GPU"):
        oz.grouped_linear(**_args())
    with pytest.raises(ValueError, match="GPU"):
        oz.grouped_linear_grads(**_args(dY=torch.zeros(10, 4)))
    with pytest.raises(ValueError, match="GPU"):
        oz.orthogonalize(torch.zeros(8, 8))


def test_sizes_past_the_limits_are_refused():
    wide = torch.zeros(1).expand(1, L.OZGEMM_MAX_ROWS + 1)
    with pytest.raises(ValueError, match="sizes"):
        oz.grouped_linear(wide, torch.zeros(1).expand(1, 4, L.OZGEMM_MAX_ROWS + 1), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="sizes"):
        oz.orthogonalize(wide)
