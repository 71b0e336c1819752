"""Blocks of 128 in 8 bits, their products and the products' gradients, against
64 bits.

Tolerances.  Blocks are exact: a power of two and one rounding.  A product's
entry is a sum of q products in blocks of 128: 128 + 4 additions in a block,
two roundings of its scaling and one addition per block, none off by more than
2^-23 of the sum of the magnitudes so far (matrix cores may cut instead of
round).  The 8-bit matrix cores (results of 16 bits and more than 16 columns) drop what lies under 2^-13 of the largest of the
products that they add at once, so at most that per product.  A result of 16 bits
is then off by half a step."""
import pytest
import torch

import fp64_gemm_emulation_ozii_amd as oz
from blocks_util import EIGHT, blocks, same, spread, value

pytestmark = pytest.mark.gpu

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = [(1, 1), (1, 128), (3, 130), (128, 128), (129, 127), (200, 4), (64, 1000), (517, 261), (1, 4099), (1000, 16)]


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def check_blocks(got, x, rows, dtype):
    v, s = blocks(x, rows, dtype)
    assert got[0].dtype == dtype and got[1].dtype == torch.float32
    assert same(got[1], s)
    assert same(got[0], v)


@pytest.mark.parametrize("dtype", list(EIGHT), ids=str)
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("n, q", SIZES)
def test_blocks_of_a_matrix_and_its_transpose(n, q, t, rows, dtype):
    x = (normal(gen(n + q), n, q) * torch.exp(3 * normal(gen(q), n, 1))).to(TYPES[t])
    V, S, Vt, St = oz.quantize_blocks(x, rows=rows, both=True, dtype=dtype)
    check_blocks((V, S), x, rows, dtype)
    check_blocks((Vt, St), x.t(), rows, dtype)
    one = oz.quantize_blocks(x, rows=rows, dtype=dtype)
    assert same(one[0], V) and same(one[1], S)


@pytest.mark.parametrize("t", list(TYPES))
def test_blocks_of_views(t):
    base = normal(gen(3), 300, 400).to(TYPES[t])
    for x in (base[7:250, 3:301], base.t(), base.t()[5:, 1:200], base[::2], base[:, ::3], base[:1], base[:, :1].t(),
              base[5].expand(9, 400)):
        V, S, Vt, St = oz.quantize_blocks(x, both=True)
        check_blocks((V, S), x, 1, E4M3)
        check_blocks((Vt, St), x.t(), 1, E4M3)


@pytest.mark.parametrize("dtype", list(EIGHT), ids=str)
@pytest.mark.parametrize("rows", [1, 128])
def test_blocks_with_extreme_entries(rows, dtype):
    top = EIGHT[dtype][0]
    x = torch.zeros(260, 384, device="cuda")
    x[0, :3] = torch.tensor([float("inf"), 1.0, -2.0])
    x[1, 128:131] = torch.tensor([float("nan"), float("-inf"), 3e38])
    x[2, 256:258] = torch.tensor([2.0 ** -149, -(2.0 ** -149)])  # below the least scale's grid: zeros
    x[3, 0] = 2.0 ** -120
    x[140, :4] = torch.tensor([top, -top, top * 2.0 ** -9, 0.5])  # exactly the largest
    x[141, 130] = top * (1 + 2.0 ** -20)  # just above
    x[142, 300:303] = torch.tensor([torch.finfo(torch.float32).max, 1.0, -0.0])
    x[259, 380] = -1.0
    V, S, Vt, St = oz.quantize_blocks(x, rows=rows, both=True, dtype=dtype)
    check_blocks((V, S), x, rows, dtype)
    check_blocks((Vt, St), x.t(), rows, dtype)


def test_every_half_and_bfloat16_is_rounded_right():
    for t in (torch.float16, torch.bfloat16):
        x = torch.arange(-2 ** 15, 2 ** 15, dtype=torch.int32).to(torch.int16).view(t).view(512, 128).cuda()
        for dtype in EIGHT:
            for rows in (1, 128):
                check_blocks(oz.quantize_blocks(x, rows=rows, dtype=dtype), x, rows, dtype)


# ---------------------------------------------------------------- products

def aligned(v, dtype, pad=0.0):
    """The values as 8-bit rows on 16-byte boundaries, `pad` behind them."""
    n, q = v.shape
    out = torch.full((n, -(-q // 16) * 16), pad, device=v.device).to(dtype)
    out[:, :q] = v.to(dtype)
    return out[:, :q]


def tolerance(x, xs, w, ws, rows, out, wide):
    a, b = value(x, xs, 1).abs(), value(w, ws, rows).abs()
    q = x.shape[1]
    sums = a @ b.T.contiguous()
    tol = sums * (128 + 4 + 2 + -(-q // 128) + 8) * 2.0 ** -23
    if not wide:  # per block: 128 products, each off by 2^-13 of the block's largest
        for k in range(0, q, 128):
            tol += a[:, k:k + 128].amax(1)[:, None] * b[:, k:k + 128].amax(1)[None] * 128 * 2.0 ** -13
    return tol


def check_product(got, x, xs, w, ws, rows, wide):
    want = value(x, xs, 1) @ value(w, ws, rows).T.contiguous()
    tol = tolerance(x, xs, w, ws, rows, got.dtype, wide)
    half = 0.0 if got.dtype == torch.float32 else torch.finfo(got.dtype).eps / 2
    tol = tol * (1 + half) + half * want.abs() + (2.0 ** -25 if got.dtype == torch.float16 else 0.0)
    assert ((got.double() - want).abs() <= tol).all()


PRODUCTS = [(1, 128, 16), (1, 4096, 1000), (5, 130, 33), (16, 1, 1), (17, 100, 129), (33, 257, 31), (64, 2048, 512),
            (65, 128, 128), (100, 1531, 77), (128, 64, 300), (200, 8192, 130), (300, 16, 257), (512, 500, 4100),
            (1001, 1531, 2049), (3000, 260, 3000), (100, 300, 2000), (200, 1100, 4001), (1000, 1000, 1000), (4097, 700, 3333),
            (3000, 200, 1), (2000, 600, 17), (70, 1, 70), (65, 2000, 5000)]


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("tx, tw", [(E4M3, E4M3), (E5M2, E4M3), (E4M3, E5M2), (E5M2, E5M2)], ids=str)
@pytest.mark.parametrize("n, q, m", PRODUCTS)
def test_whole_numbers_come_out_exactly(n, q, m, tx, tw, rows):
    # entries of -1, 0 and 1 (one in eight not 0) under scales of 1, 2 and 4: every partial sum is a whole number below 2^24
    g = gen(n + q + m)

    def whole(a, b, t):
        k = torch.randint(0, 16, (a, b), generator=g, device="cuda")
        return aligned(((k == 0).float() - (k == 1).float()), t, float("nan"))

    def scales(a, b):
        return 2.0 ** torch.randint(0, 3, (a, b), generator=g, device="cuda").float()

    nb = -(-q // 128)
    x, w, xs, ws = whole(n, q, tx), whole(m, q, tw), scales(n, nb), scales(-(-m // rows), nb)
    want = value(x, xs, 1) @ value(w, ws, rows).T.contiguous()
    for t in TYPES.values():
        assert torch.equal(oz.scaled_linear(x, xs, w, ws, out_dtype=t), want.to(t))
    xs = xs.t().contiguous().t()
    assert torch.equal(oz.scaled_linear(x, xs, w, ws, out_dtype=torch.float32).double(), want)


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("n, q, m", PRODUCTS)
def test_products_of_any_scales(n, q, m, t, rows):
    g = gen(n * 3 + q + m)
    x, xs = oz.quantize_blocks(normal(g, n, q) * torch.exp(normal(g, n, 1)))
    w, ws = oz.quantize_blocks(normal(g, m, q), rows=rows)
    xs, ws = (s * (1 + torch.rand(s.shape, generator=g, device="cuda")) for s in (xs, ws))
    got = oz.scaled_linear(x, xs, w, ws, out_dtype=TYPES[t])
    check_product(got, x, xs, w, ws, rows, t == "f32" or n <= 16)
    # the same from rows off the 16-byte grid, bit for bit
    for a, b in ((x.clone().contiguous()[:, :], w), (x, odd_rows(w)), (odd_rows(x), odd_rows(w))):
        assert torch.equal(oz.scaled_linear(a, xs, b, ws, out_dtype=TYPES[t]), got)


def odd_rows(v):
    out = torch.zeros((v.shape[0], v.shape[1] + 3), device="cuda").to(v.dtype)[:, 1:-2]
    return out.copy_(v)


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("n, q, m", [(1, 1531, 8192), (1, 1, 40), (1, 130, 9000), (100, 1531, 1), (1, 77, 1), (3000, 517, 1)])
def test_one_row_of_any_length(n, q, m, t):
    # a row alone, its leading dimension its length: in place, NaN behind it in its last 16 bytes
    g = gen(n + q)
    x, w = (torch.randint(-8, 9, s, generator=g, device="cuda").float() for s in ((n, q), (m, q)))
    xs, ws = (torch.rand(s.shape[0], -(-q // 128), generator=g, device="cuda") + 0.5 for s in (x, w))
    rows = [aligned(v, E4M3, float("nan")) for v in (x, w)]
    alone = [v.as_strided(v.shape, (q, 1)) if v.shape[0] == 1 else v for v in rows]
    got = oz.scaled_linear(alone[0], xs, alone[1], ws, out_dtype=TYPES[t])
    check_product(got, x, xs, w, ws, 1, t == "f32" or n <= 16)
    assert torch.equal(got, oz.scaled_linear(odd_rows(x.to(E4M3)), xs, odd_rows(w.to(E4M3)), ws, out_dtype=TYPES[t]))


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("n", [3, 300])
def test_sums_of_gaussian_entries_keep_their_digits(n, t):
    # the 8-bit matrix cores are off by 1.5e-5 of the sums' norm; twice that, and the result's own rounding
    g = gen(5)
    x, xs = oz.quantize_blocks(normal(g, n, 4096))
    w, ws = oz.quantize_blocks(normal(g, 512, 4096), rows=128)
    got = oz.scaled_linear(x, xs, w, ws, out_dtype=TYPES[t]).double()
    want = value(x, xs, 1) @ value(w, ws, 128).T.contiguous()
    off = ((got - want).norm() / want.norm()).item()
    assert off <= (1e-6 if t == "f32" else 3e-5 + torch.finfo(TYPES[t]).eps / 2)


# The k of a block that one lane holds, of each of the four that share a result.
LANES = [[*range(16 * h, 16 * h + 16), *range(64 + 16 * h, 80 + 16 * h)] for h in range(4)]


def dropped(x, xs, w, ws, rows):
    """What the sums lose where every product of a lane loses what lies below 2^-13 of the lane's largest."""
    lost = torch.zeros(x.shape[0], w.shape[0], dtype=torch.float64, device=x.device)
    per = ws.double() if rows == 1 else ws.double().repeat_interleave(128, 0)[:w.shape[0]]
    for b in range(xs.shape[1]):
        for lane in LANES:
            k = torch.tensor(lane, device=x.device) + 128 * b
            k = k[k < x.shape[1]]
            p = x[:, None, k].double() * w[None, :, k].double()
            most = p.abs().amax(-1, keepdim=True)
            cut = torch.where(most == 0, 1.0, torch.exp2(torch.floor(torch.log2(most)) - 13))
            lost += (p - torch.trunc(p / cut) * cut).sum(-1) * xs[:, b, None].double() * per[None, :, b]
    return lost


def rms(t):
    return t.double().square().mean().sqrt().item()


@pytest.mark.parametrize("far", [1, 21, 301])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("n, q, m", [(3, 2048, 600), (40, 2048, 600), (130, 2100, 4096), (512, 2048, 4096), (1000, 1531, 1100), (3000, 1024, 3000)])
def test_sums_of_entries_with_far_columns_keep_their_digits(n, q, m, t, rows, far):
    # Activations as layers have them: rows of different size, one column in a hundred `far` times larger, scales that are no
    # powers of two.  The mean square of the error, over 64 x 64 results (3 x 64) spread over all, is at most that of
    #   the result's own rounding, uniform within a step: step^2 / 12 on average;
    #   what the 8-bit matrix cores drop, at most what the model above loses (the two are independent);
    #   float32 sums: 2^-23 of the magnitudes for each of the additions of a block's four parts and of the blocks, sqrt of their number at random.
    # The square of an error uniform within a step has the variance step^4 (1/80 - 1/144) = step^4 / 180 about its mean, so the mean of
    # N of them scatters by sqrt(sum of step^4 / 180) / N, more than N alike ones by as much as their steps differ: six times that.
    g = gen(n + q + far)
    X = normal(g, n, q) * torch.exp(0.3 * normal(g, n, 1)) * (1 + (far - 1) * (torch.rand(1, q, generator=g, device="cuda") < 0.01))
    x, xs = oz.quantize_blocks(X)
    w, ws = oz.quantize_blocks(normal(g, m, q) / q ** 0.5, rows=rows)
    xs, ws = (s * (1 + torch.rand(s.shape, generator=g, device="cuda")) for s in (xs, ws))
    got = oz.scaled_linear(x, xs, w, ws, out_dtype=TYPES[t])
    at, to = torch.arange(min(n, 64), device="cuda") * max(1, n // 64), torch.arange(64, device="cuda") * (m // 64)
    x, xs, w, ws = x.float()[at], xs[at], w.float()[to], ws[to] if rows == 1 else ws[to // 128].contiguous()
    got = got[at][:, to].double()
    a, b = value(x, xs, 1), value(w, ws, 1)
    want = a @ b.T.contiguous()
    bound = rms(a.abs() @ b.abs().T.contiguous()) ** 2 * (4 + -(-q // 128)) * 2.0 ** -46
    if t != "f32":
        step = torch.exp2(torch.floor(torch.log2(want.abs().clamp(min=2.0 ** -14)))) * torch.finfo(TYPES[t]).eps
        bound += rms(step) ** 2 / 12 + 6 * rms(step.square()) / (180 * step.numel()) ** 0.5
        if n > 16:
            bound += rms(dropped(x, xs, w, ws, 1)) ** 2
    off = rms(got - want) ** 2
    assert off <= bound


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("tx, tw", [(E4M3, E4M3), (E5M2, E4M3), (E4M3, E5M2), (E5M2, E5M2)], ids=str)
@pytest.mark.parametrize("n, q, m", [(1, 300, 70), (9, 4096, 130), (40, 300, 200), (200, 700, 3000), (1000, 513, 1100), (2500, 300, 2500)])
def test_subnormal_entries_count(n, q, m, tx, tw, rows):
    # whole multiples of the least subnormal value, up to the second binade of normal ones: products are whole numbers up to 225
    # of the least product, none of them under 2^-13 of another, and sums stay below 2^24: exact in every way
    g = gen(n + q + m + 1)

    def least(a, b, t):
        most, unit = (15, 2.0 ** -9) if t == E4M3 else (7, 2.0 ** -16)
        k = torch.randint(-most, most + 1, (a, b), generator=g, device="cuda").float()
        held = aligned(k * unit, t, float("nan"))
        assert torch.equal(held.float(), k * unit)
        return held, unit

    (x, ux), (w, uw) = least(n, q, tx), least(m, q, tw)
    xs, ws = torch.full((n, -(-q // 128)), 1 / ux, device="cuda"), torch.full((-(-m // rows), -(-q // 128)), 1 / uw, device="cuda")
    want = value(x, xs, 1) @ value(w, ws, rows).T.contiguous()
    assert want.abs().amax() > 0
    for t in TYPES.values():
        assert torch.equal(oz.scaled_linear(x, xs, w, ws, out_dtype=t), want.to(t))


@pytest.mark.parametrize("n, m", [(3, 40), (300, 200), (1000, 9000)])
@pytest.mark.parametrize("t", list(TYPES))
def test_nan_and_infinities_stay_in_their_rows(n, m, t):
    q = 200
    g = gen(7)
    x, xs = oz.quantize_blocks(normal(g, n, q), dtype=E5M2)
    w, ws = oz.quantize_blocks(normal(g, m, q), dtype=E5M2)
    x, w = x.float(), w.float()
    w[m - 1, 199] = float("nan")
    x[n - 1, 3] = float("inf")
    w[0, 3] = 0.0
    got = oz.scaled_linear(aligned(x, E5M2), xs, aligned(w, E5M2), ws, out_dtype=TYPES[t])
    want = value(x, xs, 1) @ value(w, ws, 1).T.contiguous()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.isfinite(), want.isfinite())
    assert got[:, m - 1].isnan().all() and got[n - 1, 0].isnan() and got[0, 0].isfinite()


def test_results_go_where_they_are_asked_to():
    g = gen(9)
    for n, m in ((7, 50), (300, 270)):
        x, xs = oz.quantize_blocks(normal(g, n, 300))
        w, ws = oz.quantize_blocks(normal(g, m, 300), rows=128)
        want = oz.scaled_linear(x, xs, w, ws)
        frame = torch.full((n + 2, m + 5), 7.0, device="cuda", dtype=torch.bfloat16)
        out = frame[1:-1, 3:-2]
        assert oz.scaled_linear(x, xs, w, ws, out=out) is out
        assert torch.equal(out, want)
        frame[1:-1, 3:-2] = 7.0
        assert (frame == 7.0).all()


def test_no_entries():
    e = torch.empty(0, 0, device="cuda")
    for n, q, m in ((0, 5, 3), (4, 0, 3), (100, 0, 3), (4, 5, 0)):
        x, xs = oz.quantize_blocks(torch.ones(n, q, device="cuda"))
        w, ws = oz.quantize_blocks(torch.ones(m, q, device="cuda"))
        assert x.shape == (n, q) and xs.shape == (n, -(-q // 128))
        got = oz.scaled_linear(x, xs, w, ws)
        assert got.shape == (n, m) and (got == 0).all()
    assert oz.quantize_blocks(e, both=True)[2].shape == (0, 0)


@pytest.mark.parametrize("n, q, m", [(40, 300, 200), (1000, 513, 129), (129, 1000, 2000)])
@pytest.mark.parametrize("t", list(TYPES))
def test_gradients(n, q, m, t):
    g = gen(n)
    X, W = normal(g, n, q).to(TYPES[t]), normal(g, m, q).to(TYPES[t])
    dY = (normal(g, n, m) * torch.exp(normal(g, n, 1))).to(TYPES[t])
    _, _, Xt, xts = oz.quantize_blocks(X, both=True)
    _, _, Wt, wts = oz.quantize_blocks(W, rows=128, both=True)
    for dtype in EIGHT:
        dX, dW = oz.scaled_linear_grads(dY, Xt, xts, Wt, wts, dw_dtype=torch.float32, dtype=dtype)
        assert dX.dtype == dY.dtype and dX.shape == (n, q) and dW.shape == (m, q)
        v, s = blocks(dY, 1, dtype)
        check_product(dX, v, s, Wt, wts, 128, t == "f32" or n <= 16)
        v, s = blocks(dY.t(), 1, dtype)
        check_product(dW, v, s, Xt, xts, 1, True)


def test_gradients_of_a_layer_against_differences():
    # Y = X W^T is linear in both: a step along D changes sum(Y dY) by sum(dX D); whole numbers, exact in 8 bits
    g = gen(21)
    X, W, dY, D = (torch.randint(-2, 3, s, generator=g, device="cuda").float() for s in
                   ((150, 200), (90, 200), (150, 90), (150, 200)))
    w, ws, Wt, wts = oz.quantize_blocks(W, rows=128, both=True)
    _, _, Xt, xts = oz.quantize_blocks(X, both=True)

    def loss(X):
        return (oz.scaled_linear(*oz.quantize_blocks(X), w, ws, out_dtype=torch.float32).double() * dY.double()).sum()

    dX, dW = oz.scaled_linear_grads(dY, Xt, xts, Wt, wts)
    assert (dX.double() * D).sum() == (loss(X + D) - loss(X - D)) / 2
    assert torch.equal(dW.double(), dY.double().T.contiguous() @ X.double())
    assert torch.equal(dX.double(), dY.double() @ W.double())


def test_the_spread_of_scales_matches_the_products():
    s = torch.arange(6.0).view(2, 3)
    assert spread(s, 130, 300, 128)[129, 299] == 5 and spread(s, 130, 300, 128)[127, 128] == 1
