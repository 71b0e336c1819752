"""Newton-Schulz orthogonalisation against the iteration in 64 bits.

The iteration grows an error of one step by at most max(|p'|, |p(x)/x|) < 3.9
in the Frobenius norm (p the step's polynomial on [0, 1.2]), so per step it is
a matter of what the step itself adds.  Tolerances, relative in the Frobenius
norm:
  bf16, f16  the result's one rounding, u = eps/2, and as much again for all
             that comes before it (bf16: 8 times the 2^-11 that its product
             operands are off by; f16: three slice products, as f32);
  f32        twice what the same iteration in plain FP32 is off by, and 2^-22:
             the slices hold a state to 2^-23 where FP32 holds it to 2^-24, and
             the products drop at most 2^-22 of a term where FP32 rounds each sum;
  f64        s = 14 leaves k >= 46 bits at q <= 2^12: 2^-45 for a product,
             three products and 3.9^4 growth: under 2^-30.
"""
import pytest
import torch

import fp64_gemm_emulation_ozii_amd as oz
from fp64_gemm_emulation_ozii_amd import ozgemm as L

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "f64": torch.float64}
QUINTIC = (3.4445, -4.7750, 2.0315)


def plain(G, steps=5, coeffs=QUINTIC, eps=1e-7, dtype=torch.float64):
    x = G.to(dtype)
    x = x / (x.square().sum((-2, -1), keepdim=True).sqrt() + eps)
    tall = x.shape[-2] > x.shape[-1]
    if tall:
        x = x.transpose(-2, -1).contiguous()
    for k in range(steps):
        a, b, c = coeffs[k] if isinstance(coeffs[0], tuple) else coeffs
        p = x @ x.transpose(-2, -1).contiguous()
        x = a * x + (b * p + c * (p @ p)) @ x
    return x.transpose(-2, -1) if tall else x


def rel(a, b):
    return ((a.double() - b).norm() / b.norm().clamp_min(1e-300)).item()


def tolerance(G, want, **how):
    u = torch.finfo(G.dtype).eps / 2
    if G.dtype == torch.float64:
        return 2.0 ** -30
    if G.dtype == torch.float32:
        return 2 * rel(plain(G, dtype=torch.float32, **how), want) + 2.0 ** -22
    return 2 * u


def draw(shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    *b, r, c = shape
    k = max(1, min(r, c) // 16)
    u = torch.randn(*b, r, k, generator=g, device="cuda", dtype=torch.float64)
    v = torch.randn(*b, k, c, generator=g, device="cuda", dtype=torch.float64)
    G = u @ v * (3.0 / k ** 0.5) + torch.randn(*b, r, c, generator=g, device="cuda", dtype=torch.float64)
    return (G * 1e-3).to(dtype)


SHAPES = [(1, 1), (1, 7), (7, 1), (2, 2), (16, 16), (17, 33), (64, 64), (65, 64), (64, 200), (200, 63), (129, 128),
          (3, 1000), (1000, 3), (257, 300), (333, 1003), (1003, 333), (512, 512), (3, 100, 70), (2, 3, 40, 90),
          (5, 130, 129), (1024, 640), (9, 700, 1100), (2, 2048, 1100), (1300, 4000), (40, 3000), (2900, 130),
          (4, 1700, 64), (2, 200, 1024)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_five_steps(shape, dtype):
    G = draw(shape, TYPES[dtype], sum(shape))
    keep = G.clone()
    O = oz.orthogonalize(G)
    assert O.shape == G.shape and O.dtype == G.dtype and torch.equal(G, keep)
    want = plain(G)
    assert rel(O, want) <= tolerance(G, want)
    assert torch.equal(O, oz.orthogonalize(G))


@pytest.mark.parametrize("dtype", list(TYPES))
def test_other_coefficients_and_steps(dtype):
    G = draw((2, 96, 160), TYPES[dtype], 1)
    cubic = (1.5, -0.5, 0.0)
    varied = [(8.2, -23.0, 17.0), (4.0, -2.9, 0.53), (3.3, -2.4, 0.46)]
    for steps, coeffs in ((1, QUINTIC), (2, cubic), (3, varied), (0, QUINTIC), (4, (1.0, 0.0, 0.0))):
        want = plain(G, steps, coeffs if not isinstance(coeffs, list) else coeffs)
        O = oz.orthogonalize(G, steps=steps, coeffs=coeffs)
        assert rel(O, want) <= tolerance(G, want, steps=steps, coeffs=coeffs)


def test_singular_values_and_vectors():
    # G = U diag(v) V^T: the result is U diag(p(p(...(v / |v|)))) V^T
    g = torch.Generator(device="cuda").manual_seed(3)
    U = torch.linalg.qr(torch.randn(48, 48, generator=g, device="cuda", dtype=torch.float64).cpu())[0].cuda()
    V = torch.linalg.qr(torch.randn(80, 48, generator=g, device="cuda", dtype=torch.float64).cpu())[0].cuda()
    v = torch.logspace(0, -3, 48, device="cuda", dtype=torch.float64)
    G = (U * v) @ V.T
    x = v / (v.norm() + 1e-7)
    for _ in range(5):
        x = QUINTIC[0] * x + QUINTIC[1] * x ** 3 + QUINTIC[2] * x ** 5
    want = (U * x) @ V.T
    assert rel(oz.orthogonalize(G), want) <= 2.0 ** -30
    # f32 slices: inputs rounded to 2^-24, three steps' growth of the smallest values is part of the result itself
    assert rel(oz.orthogonalize(G.float()), want) <= 2.0 ** -16


@pytest.mark.parametrize("dtype", list(TYPES))
def test_layouts_strides_and_in_place(dtype):
    G = draw((3, 70, 110), TYPES[dtype], 5)
    want = oz.orthogonalize(G)
    big = torch.full((3, 75, 123), float("nan"), device="cuda", dtype=G.dtype)
    big[:, :70, :110] = G
    out = torch.full((3, 90, 117), 2.0, device="cuda", dtype=G.dtype)
    oz.orthogonalize(big[:, :70, :110], out=out[:, :70, :110])
    assert torch.equal(out[:, :70, :110], want)
    assert (out[:, 70:] == 2).all() and (out[:, :, 110:] == 2).all()
    H = G.clone()
    assert oz.orthogonalize(H, out=H) is H and torch.equal(H, want)
    one = G[:1].expand(3, -1, -1)  # one matrix for the whole batch
    assert torch.equal(oz.orthogonalize(one)[2], want[0])
    t = oz.orthogonalize(G.transpose(1, 2))  # rows not contiguous: from a copy
    want64 = plain(G).transpose(1, 2)
    assert rel(t, want64) <= tolerance(G, plain(G))


@pytest.mark.parametrize("dtype", list(TYPES))
def test_zeros_nan_and_range(dtype):
    t = TYPES[dtype]
    G = draw((4, 40, 66), t, 6)
    want = oz.orthogonalize(G)
    G[1] = 0
    G[2, 3, 5] = float("nan")
    G[3, 30, 60] = float("inf")
    O = oz.orthogonalize(G)
    assert torch.equal(O[0], want[0]) and (O[1] == 0).all() and torch.isnan(O[2:]).all()
    # far from 1, where squares leave the type's range
    for scale in ((2.0 ** 12, 2.0 ** -6) if t == torch.float16 else (2.0 ** 100, 2.0 ** -40)):
        H = draw((1, 50, 60), t, 7) * scale
        w = plain(H, eps=0.0)
        assert rel(oz.orthogonalize(H, eps=0.0), w) <= tolerance(H.double().mul(1 / scale).to(t), plain(
            H.double().mul(1 / scale).to(t), eps=0.0), eps=0.0)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_streams_and_graphs(dtype):
    G, H = draw((2, 150, 200), TYPES[dtype], 8), draw((260, 100), TYPES[dtype], 9)
    wantG, wantH = oz.orthogonalize(G), oz.orthogonalize(H)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(a):
            x = oz.orthogonalize(G)
        with torch.cuda.stream(b):
            y = oz.orthogonalize(H)
        torch.cuda.synchronize()
        assert torch.equal(x, wantG) and torch.equal(y, wantH)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = oz.orthogonalize(G)
    for k in range(3):
        cap.zero_()
        G.copy_(draw((2, 150, 200), TYPES[dtype], 20 + k))
        graph.replay()
        eager = oz.orthogonalize(G)
        torch.cuda.synchronize()
        assert torch.equal(cap, eager)


def test_bound_setting_does_not_matter():
    G = draw((60, 90), torch.float64, 10)
    want = oz.orthogonalize(G)
    L.ozgemm_set_bound(L.OZGEMM_BOUND_FAST)
    try:
        assert torch.equal(oz.orthogonalize(G), want)
    finally:
        L.ozgemm_set_bound(L.OZGEMM_BOUND_CONSERVATIVE)


def test_a_layer_and_its_update():
    # forward, gradients and the update of a layer of experts, as they are used together
    g = torch.Generator(device="cuda").manual_seed(11)
    sizes = [40, 0, 100, 9]
    off = torch.tensor([0, 40, 40, 140, 149], dtype=torch.int32, device="cuda")
    for dtype in (torch.bfloat16, torch.float32):
        X = torch.randn(149, 96, generator=g, device="cuda").to(dtype)
        W = (torch.randn(4, 64, 96, generator=g, device="cuda") * 0.1).to(dtype)
        Y = oz.grouped_linear(X, W, off)
        dX, dW = oz.grouped_linear_grads(Y, X, W, off)  # of sum(Y^2) / 2
        O = oz.orthogonalize(dW)
        assert (O[1] == 0).all()
        for e in (0, 2, 3):
            s = slice(int(off[e]), int(off[e]) + sizes[e])
            y = X[s].double() @ W[e].double().T
            assert rel(Y[s], y) <= 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -20
            want = plain(dW[e])
            assert rel(O[e], want) <= tolerance(dW[e], want)
