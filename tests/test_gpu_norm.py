"""The root-mean-square norm, its values in 8 bits and its gradients against 64 bits.

Tolerances.  Y is the exact value rounded once: half a step, and 1e-12 of it for
the sums in FP64.  Values in 8 bits and their scales come out equal.  An entry of
dX is formed in FP32 from two products and up to two additions: 6 roundings of
2^-24 of the sum of its terms' magnitudes, then half a step.  dw: n + 2
roundings of 2^-24 of the sum of the magnitudes, then half a step."""
import pytest
import torch

import fp64_gemm_emulation_ozii_amd as oz
from blocks_util import EIGHT, blocks, same
from fp64_gemm_emulation_ozii_amd import ozgemm as L

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6
# every shape of threads, whole and ragged, and rows too long for them
SIZES = [(1, 1), (3, 7), (5, 128), (1, 512), (9, 513), (300, 1000), (2, 1025), (77, 2048), (4, 2049), (10, 4096),
         (3, 5003), (6, 8192), (3, 8193), (5, 20000), (5000, 130), (2, 70001)]


def draw(n, q, t, wt, seed, residual=True):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*s):
        return torch.randn(*s, generator=g, device="cuda")

    X = (normal(n, q) * torch.exp(normal(n, 1))).to(t)
    R = (normal(n, q) * 3).to(t) if residual else None
    return X, R, (1 + 0.3 * normal(q)).to(wt), (normal(n, q) * 0.1).to(t), normal(n, q).to(t)


def norm(H, w, eps=EPS):
    h = H.double()
    return h / torch.sqrt(h.square().mean(1, keepdim=True) + eps) * w.double()


def half_step(want, t):
    f = torch.finfo(t)
    return f.eps / 2 * want.abs() + f.smallest_normal * f.eps / 2


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("n, q", SIZES)
def test_norm(n, q, t):
    for wt, residual in ((TYPES[t], True), (torch.float32, False)):
        X, R, w, _, _ = draw(n, q, TYPES[t], wt, n + q, residual)
        Y, H = oz.rms_norm(X, w, R, EPS)
        if residual:
            assert torch.equal(H, X + R)
        else:
            assert H is X
        want = norm(H, w)
        assert Y.dtype == X.dtype
        assert ((Y.double() - want).abs() <= half_step(want, Y.dtype) + 1e-12 * want.abs()).all()


@pytest.mark.parametrize("dtype", list(EIGHT), ids=str)
@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("n, q", SIZES)
def test_norm_in_8_bits(n, q, t, dtype):
    for wt, residual in ((TYPES[t], True), (torch.float32, False)):
        X, R, w, _, _ = draw(n, q, TYPES[t], wt, n + q + 1, residual)
        V, S, H = oz.rms_norm_quantized(X, w, R, EPS, dtype=dtype)
        v, s = blocks(norm(X + R if residual else X, w), 1, dtype)
        assert same(S, s) and same(V, v)
        assert torch.equal(H, X + R if residual else X)


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("n, q", SIZES + [(0, 40)])
def test_gradients(n, q, t):
    for wt, residual in ((TYPES[t], True), (torch.float32, False)):
        X, R, w, dY, dH = draw(n, q, TYPES[t], wt, n + q + 2, residual)
        H = X + R if residual else X
        dX, dw = oz.rms_norm_grads(dY, H, w, dH if residual else None, EPS)
        assert dX.dtype == X.dtype and dw.dtype == wt and dw.shape == (q,)
        h, g = H.double(), dY.double() * w.double()
        r = 1 / torch.sqrt(h.square().mean(1, keepdim=True) + EPS)
        a, b = r * g, h * r ** 3 * (g * h).mean(1, keepdim=True)
        c = dH.double() if residual else torch.zeros_like(a)
        want = a - b + c
        tol = 6 * 2.0 ** -24 * (a.abs() + b.abs() + c.abs())
        assert ((dX.double() - want).abs() <= tol * 1.01 + half_step(want, dX.dtype)).all()
        terms = dY.double() * h * r
        want = terms.sum(0)
        tol = (n + 2) * 2.0 ** -24 * terms.abs().sum(0)
        assert ((dw.double() - want).abs() <= tol * 1.01 + half_step(want, wt)).all()


def test_gradients_against_differences():
    X, R, w, dY, dH = draw(7, 300, torch.float32, torch.float32, 4)
    H = X + R
    dX, dw = oz.rms_norm_grads(dY, H, w, dH, EPS)
    g = torch.Generator(device="cuda").manual_seed(8)
    for which in range(2):
        D = torch.randn((7, 300) if which == 0 else (300,), generator=g, device="cuda", dtype=torch.float64)

        def loss(step):
            h, v = H.double(), w.double()
            h, v = (h + step * D, v) if which == 0 else (h, v + step * D)
            return (norm(h, v) * dY.double()).sum() + (h * dH.double()).sum()

        # the third derivative's part of a central difference: step^2 / 6 of terms of order 1
        slope = (loss(1e-5) - loss(-1e-5)) / 2e-5
        size = (dX if which == 0 else dw).double().norm() * D.norm()
        assert abs(((dX if which == 0 else dw).double() * D).sum() - slope) <= 1e-6 * size


@pytest.mark.parametrize("q", [100, 3000, 9000])
def test_in_place_and_in_views(q):
    X, R, w, dY, dH = draw(12, q, torch.bfloat16, torch.bfloat16, q)
    Y, H = oz.rms_norm(X, w, R)
    for kept, out in (("R", "X"), ("X", "R"), ("R", None), (None, "X")):
        a = {"X": X.clone(), "R": R.clone()}
        y, h = oz.rms_norm(a["X"], w, a["R"], H=a.get(kept), out=a.get(out))
        assert torch.equal(y, Y) and torch.equal(h, H)
        assert kept is None or h is a[kept]
    assert torch.equal(oz.rms_norm(H, w, out=(c := H.clone()))[0], Y) and torch.equal(c, Y)
    want = oz.rms_norm_grads(dY, H, w, dH)
    for k in range(3):
        args = [dY.clone(), H.clone(), dH.clone()]
        dX, dw = oz.rms_norm_grads(args[0], args[1], w, args[2], dX=args[k])
        assert torch.equal(dX, want[0]) and torch.equal(dw, want[1]) and dX is args[k]
    # rows of a wider array, a dimension apart, a broadcast residual and weight
    wide = torch.full((2, 12, q + 3), 5.0, device="cuda", dtype=torch.bfloat16)
    wide[0, :, 1:q + 1] = X
    y, h = oz.rms_norm(wide[0, :, 1:q + 1], w, R, H=wide[1, :, 2:q + 2])
    assert torch.equal(y, Y) and torch.equal(wide[1, :, 2:q + 2], H)
    assert (wide[0, :, 0] == 5).all() and (wide[1, :, :2] == 5).all() and (wide[1, :, -1] == 5).all()
    wide = torch.zeros((12, 2 * q), device="cuda", dtype=torch.bfloat16)  # rows that interleave overlap
    with pytest.raises(L.OzgemmError):
        oz.rms_norm(wide[:, :q], w, R, H=wide[:, q:])
    y, _ = oz.rms_norm(X.t().contiguous().t(), w, R)
    assert torch.equal(y, Y)
    y, _ = oz.rms_norm(X, w[:1].expand(q), R[:1].expand(12, q))
    assert torch.equal(y, oz.rms_norm(X, w[:1].expand(q).clone(), R[:1].expand(12, q).clone())[0])


@pytest.mark.parametrize("q", [130, 9000])
def test_rows_without_a_norm(q):
    # zeros, infinities and NaN stay in their rows; eps = 0 divides zeros by zero
    X, _, w, dY, _ = draw(6, q, torch.float16, torch.float16, 3, False)
    X[1] = 0
    X[2, 5] = float("inf")
    X[3, q - 1] = float("nan")
    Y, _ = oz.rms_norm(X, w)
    assert same(Y[[0, 4, 5]], oz.rms_norm(X[[0, 4, 5]], w)[0]) and (Y[1] == 0).all()
    assert Y[2, 5].isnan() and (Y[2, :5] == 0).all() and Y[3].isnan().all()
    V, S, _ = oz.rms_norm_quantized(X, w)
    assert (S[1:4] == 1).all() and (V[1].float() == 0).all() and V[3].float().isnan().all()
    v, s = blocks(norm(X, w), 1, torch.float8_e4m3fn)
    assert same(V, v) and same(S, s)
    assert oz.rms_norm(X, w, eps=0.0)[0][1].isnan().all()
    dX, dw = oz.rms_norm_grads(dY, X, w)
    assert same(dX[[0, 4, 5]], oz.rms_norm_grads(dY[[0, 4, 5]], X[[0, 4, 5]], w)[0])
    assert dX[1].isfinite().all() and dX[2].isnan().any() and dX[3].isnan().all() and dw.isnan().any()


@pytest.mark.parametrize("q", [300, 9000])
@pytest.mark.parametrize("size", [1e-30, 1e-19, 1e15])
def test_gradients_of_small_and_large_rows(q, size):
    g = torch.Generator(device="cuda").manual_seed(q)
    H, dY = (torch.randn(5, q, generator=g, device="cuda") * f for f in (size, 1e-3))
    w = torch.ones(q, device="cuda")
    dX, dw = oz.rms_norm_grads(dY, H, w, eps=0.0)
    h, d = H.double(), dY.double()
    r = 1 / h.square().mean(1, keepdim=True).sqrt()
    a, b = r * d, h * r ** 3 * (d * h).mean(1, keepdim=True)
    assert ((dX.double() - (a - b)).abs() <= 6.06 * 2.0 ** -24 * (a.abs() + b.abs()) + half_step(a - b, H.dtype)).all()
    terms = d * h * r
    assert ((dw.double() - terms.sum(0)).abs() <= 7.07 * 2.0 ** -24 * terms.abs().sum(0) + half_step(terms.sum(0), H.dtype)).all()


def test_no_rows():
    for q in (40, 9000):
        w = torch.ones(q, device="cuda")
        Y, H = oz.rms_norm(torch.empty(0, q, device="cuda"), w)
        V, S, _ = oz.rms_norm_quantized(torch.empty(0, q, device="cuda"), w, torch.empty(0, q, device="cuda"))
        assert Y.shape == (0, q) and V.shape == (0, q) and S.shape == (0, -(-q // 128))
    assert oz.rms_norm(torch.empty(5, 0, device="cuda"), torch.empty(0, device="cuda"))[0].shape == (5, 0)
