"""Products over ragged groups against plain products in 64 bits.

Tolerances, per entry, with u = eps(type)/2 for the one rounding of a result
and P = (|A||B|) the product of the absolute values:
  16-bit operands: products of two entries are exact in FP32; q additions, each
    off by at most one step (2^-23) of a partial sum <= P, whatever order and
    rounding the matrix cores use:           u |C| + q 2^-23 P
  FP32 operands: each entry is two half slices.  Half's step in [2^E, 2^(E+1))
    is 2^(E-10), so hi is off by <= 2^(E-11), and lo, below 2^(E-11), by
    <= 2^(E-23): 2^-23 relative for each operand, or 2^-40 of the row's largest
    entry (half of half's smallest step under a grid maximum of 2^15).  The
    dropped lo lo is <= 2^-22 of a term.  Together 2^-23 + 2^-23 + 2^-22 = 8 2^-24
    of P; 3 q additions of terms whose absolute sum is <= P (1 + 2^-10), 2^-23 each:
                      2^-24 |C| + (8 + 6.01 q) 2^-24 P + 4 q 2^-40 max max
  plus the type's smallest step for results below its normal range.
Whole numbers whose sums stay below 2^24 have to come out exactly.
"""
import numpy as np
import pytest
import torch

import fp64_gemm_emulation_ozii_amd as oz
from fp64_gemm_emulation_ozii_amd import ozgemm as L

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}


def bound(C, P, q, operand, result, big=0.0):
    u = torch.finfo(result).eps / 2
    if operand == torch.float32:
        return u * C.abs() + (8 + 6.01 * q) * 2.0 ** -24 * P + 4 * q * 2.0 ** -40 * big + TINY[result]
    return u * C.abs() + q * 2.0 ** -23 * P + TINY[result]


def draw(sizes, m, q, dtype, seed, before=0, behind=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = before + sum(sizes) + behind
    off = torch.tensor(np.concatenate([[0], np.cumsum(sizes)]) + before, dtype=torch.int32, device="cuda")

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    X = (normal(n, q) * torch.exp(0.5 * normal(n, 1))).to(dtype)
    W = (normal(len(sizes), m, q) * torch.exp(0.5 * normal(len(sizes), m, 1))).to(dtype)
    dY = (normal(n, m) * torch.exp(0.5 * normal(n, 1))).to(dtype)
    return X, W, dY, off


def check(got, want, tol):
    d = (got.double() - want).abs()
    worst = (d - tol).max().item() if d.numel() else -1.0
    assert worst <= 0, f"an entry is {worst:.3g} past its tolerance (largest error {d.max().item():.3g})"


def check_all(X, W, dY, off, Y, dX, dW):
    o = off.tolist()
    n, q = X.shape
    m = W.shape[1]
    Xd, Wd, Gd = X.double(), W.double(), dY.double()
    for e in range(W.shape[0]):
        s = slice(o[e], o[e + 1])
        x, w, g = Xd[s], Wd[e], Gd[s]
        top = lambda v, d: v.abs().amax(d) if v.numel() else torch.zeros(v.shape[1 - d], device=v.device, dtype=v.dtype)  # noqa: E731
        C, P = x @ w.T, x.abs() @ w.abs().T
        check(Y[s], C, bound(C, P, q, X.dtype, Y.dtype, top(x, 1)[:, None] * top(w, 1)[None]))
        if dX is not None:
            C, P = g @ w, g.abs() @ w.abs()
            check(dX[s], C, bound(C, P, m, X.dtype, dX.dtype, top(g, 1)[:, None] * top(w, 0)[None]))
            C, P = g.T @ x, g.T.abs() @ x.abs()
            check(dW[e], C, bound(C, P, len(x), X.dtype, dW.dtype, top(g, 0)[:, None] * top(x, 0)[None]))


SHAPES = [
    # sizes, m, q
    ([1], 1, 1),
    ([1], 64, 128),
    ([0, 3, 0, 1, 0], 72, 64),
    ([5, 0, 7], 33, 17),                       # rows on no 16-byte boundary
    ([16, 17, 15, 1], 256, 192),
    ([100, 30, 0, 300], 264, 520),
    ([257, 255, 256], 512, 64),
    ([700, 1, 2, 640], 300, 1000),
    ([63, 65, 64, 129], 1024, 2048),
    ([3] * 70 + [0] * 60 + [5] * 5, 40, 72),   # more groups than a wavefront has lanes
    ([513], 777, 131),
    ([40, 1000, 8], 2, 3),
    # past what the kernels for few columns and small outer products take
    ([9000, 0, 1, 8001, 77], 777, 515),
    ([97, 0, 130] * 40, 648, 712),
    ([301, 2, 240] * 30, 649, 713),
]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("case", range(len(SHAPES)))
@pytest.mark.parametrize("layout", ["mq", "qm"])
def test_product_and_gradients(case, dtype, layout):
    sizes, m, q = SHAPES[case]
    X, W, dY, off = draw(sizes, m, q, TYPES[dtype], case)
    if layout == "qm":
        W = W.transpose(1, 2).contiguous().transpose(1, 2)
    Y = oz.grouped_linear(X, W, off)
    dX, dW = oz.grouped_linear_grads(dY, X, W, off)
    assert Y.dtype == dX.dtype == dW.dtype == X.dtype
    check_all(X, W, dY, off, Y, dX, dW)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_results_in_single_precision(dtype):
    X, W, dY, off = draw([100, 0, 41, 300], 136, 264, TYPES[dtype], 3)
    Y = oz.grouped_linear(X, W, off, out_dtype=torch.float32)
    dX, dW = oz.grouped_linear_grads(dY, X, W, off, dw_dtype=torch.float32)
    assert Y.dtype == dW.dtype == torch.float32
    check_all(X, W, dY, off, Y, dX, dW)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("sizes, m, q", [([70, 0, 333, 13], 200, 600), ([500, 0, 700, 313], 1100, 601)])
def test_whole_numbers_are_exact(sizes, m, q, dtype):
    # f32 entries of 13 bits need both slices; |sums| <= 1100 x 4097 x 2 < 2^24
    g = torch.Generator(device="cuda").manual_seed(1)
    n = sum(sizes)
    off = torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device="cuda")
    sign = torch.randint(0, 2, (n, q), generator=g, device="cuda") * 2 - 1
    X = (sign * (4097 if dtype == "f32" else 7)).to(TYPES[dtype])
    W = torch.randint(-2, 3, (4, m, q), generator=g, device="cuda").to(TYPES[dtype])
    dY = torch.randint(-2, 3, (n, m), generator=g, device="cuda").to(TYPES[dtype])
    Y = oz.grouped_linear(X, W, off, out_dtype=torch.float32)
    dX, dW = oz.grouped_linear_grads(dY, X, W, off, dw_dtype=torch.float32)
    o = off.tolist()
    for e in range(4):
        s = slice(o[e], o[e + 1])
        assert torch.equal(Y[s].double(), X[s].double() @ W[e].double().T)
        assert torch.equal(dX[s].double(), (dY[s].double() @ W[e].double()).to(dX.dtype).double())
        assert torch.equal(dW[e].double(), dY[s].double().T @ X[s].double())


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("sizes, m, q", [([20, 0, 45], 96, 80), ([4001, 0, 13050], 1037, 579)])
def test_rows_of_no_group_are_left_alone(sizes, m, q, dtype):
    X, W, dY, off = draw(sizes, m, q, TYPES[dtype], 5, before=7, behind=30)
    Y = torch.full((X.shape[0], m), 7.5, device="cuda", dtype=X.dtype)
    dX = torch.full(X.shape, 7.5, device="cuda", dtype=X.dtype)
    oz.grouped_linear(X, W, off, out=Y)
    _, dW = oz.grouped_linear_grads(dY, X, W, off, dX=dX)
    for t in (Y, dX):
        assert (t[:7] == 7.5).all() and (t[-30:] == 7.5).all()
    check_all(X, W, dY, off, Y, dX, dW)


@pytest.mark.parametrize("sizes, m, q", [([20, 1, 45], 96, 80), ([20, 1, 45], 95, 79), ([4001, 1, 13050], 1037, 579)])
def test_rows_of_no_group_are_not_read_into_results(sizes, m, q):
    # what lies around the groups is NaN: no result may see it
    for dtype in TYPES.values():
        X, W, dY, off = draw(sizes, m, q, dtype, 6, before=9, behind=31)
        for t in (X, dY):
            t[:9] = float("nan")
            t[-31:] = float("nan")
        Y = oz.grouped_linear(X, W, off)
        dX, dW = oz.grouped_linear_grads(dY, X, W, off)
        check_all(X, W, dY, off, Y, dX, dW)


def test_neighbouring_rows_and_groups_do_not_meet():
    # group 1's rows and weights are NaN and Inf; inner dimensions end inside a slice
    for dtype in TYPES.values():
        X, W, dY, off = draw([70, 50, 33], 104, 72, dtype, 7)
        X[70:120] = float("nan")
        dY[70:120] = float("inf")
        W[1] = float("nan")
        Y = oz.grouped_linear(X, W, off)
        dX, dW = oz.grouped_linear_grads(dY, X, W, off)
        assert torch.isnan(Y[70:120]).all() and torch.isnan(dX[70:120]).all() and torch.isnan(dW[1]).all()
        keep = torch.tensor([0, 2], device="cuda")
        rows = torch.cat([torch.arange(70), torch.arange(120, 153)]).cuda()
        off2 = torch.tensor([0, 70, 103], dtype=torch.int32, device="cuda")
        check_all(X[rows], W[keep], dY[rows], off2, Y[rows], dX[rows], dW[keep])


def test_infinities():
    # the usual rules, but for f32 in slices (many rows): there a row with an infinity makes its results NaN
    for n, q in ((4, 64), (300, 64), (4, 65), (200000, 128), (200000, 67)):
        X = torch.ones(n, q, device="cuda")
        W = torch.ones(1, 8, q, device="cuda")
        X[1, 3] = float("inf")
        off = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        for dtype in (torch.bfloat16, torch.float16, torch.float32):
            Y = oz.grouped_linear(X.to(dtype), W.to(dtype), off)
            if dtype == torch.float32 and n > 100000:
                assert torch.isnan(Y[1]).all()
            else:
                assert torch.isinf(Y[1]).all()
            assert (Y[2:] == q).all() and (Y[0] == q).all()


def test_f32_range():
    # rows far apart in size, subnormal rows and the largest; as they lie, and in slices (whose grids follow each row)
    for n, q in ((6, 96), (300, 96), (6, 97), (200000, 96), (200000, 97)):
        g = torch.Generator(device="cuda").manual_seed(2)
        X = torch.randn(n, q, generator=g, device="cuda")
        X[:6] *= torch.tensor([1e-40, 1e-30, 1.0, 1e30, 3e37, 0.0], device="cuda")[:, None]
        W = torch.randn(1, 24, q, generator=g, device="cuda") * 0.1
        W[0, 0] *= 1e-25
        off = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        Y = oz.grouped_linear(X, W, off)
        C, P = X.double() @ W[0].double().T, X.double().abs() @ W[0].double().abs().T
        big = X.double().abs().amax(1)[:, None] * W[0].double().abs().amax(1)[None]
        # in FP32, q products and q sums each round by at most half the smallest number, 2^-150
        check(Y, C, bound(C, P, q, torch.float32, torch.float32, big) + q * 2.0 ** -149)


def test_strides():
    # padded rows (in place and, off the 16-byte grid, through the workspace), shared weights, a strided result
    for dtype in TYPES.values():
        for pad in (8, 3):
            X, W, dY, off = draw([40, 9, 130], 88, 136, dtype, 11)
            Xp = torch.full((X.shape[0], 136 + pad), float("nan"), device="cuda", dtype=dtype)
            Wp = torch.full((3, 88, 136 + pad), float("nan"), device="cuda", dtype=dtype)
            Gp = torch.full((X.shape[0], 88 + pad), float("nan"), device="cuda", dtype=dtype)
            Xp[:, :136], Wp[:, :, :136], Gp[:, :88] = X, W, dY
            out = torch.full((X.shape[0], 88 + pad), 3.0, device="cuda", dtype=dtype)
            oz.grouped_linear(Xp[:, :136], Wp[:, :, :136], off, out=out[:, :88])
            dWp = torch.full((3, 88, 136 + pad), 3.0, device="cuda", dtype=dtype)
            dX, dW = oz.grouped_linear_grads(Gp[:, :88], Xp[:, :136], Wp[:, :, :136], off, dW=dWp[:, :, :136])
            check_all(X, W, dY, off, out[:, :88], dX, dW)
            assert (out[:, 88:] == 3).all() and (dWp[:, :, 136:] == 3).all()
        one = W[:1].expand(3, -1, -1)
        Y = oz.grouped_linear(X, one, off)
        check_all(X, one, dY, off, Y, None, None)


def test_wild_offsets_stay_inside():
    # out of order and out of range: read as the nearest ordered ones
    X, W, dY, _ = draw([50, 50, 50, 50], 64, 64, torch.bfloat16, 12)
    wild = torch.tensor([-5, 120, 60, 10 ** 9, 130], dtype=torch.int32, device="cuda")
    tame = torch.tensor([0, 120, 120, 200, 200], dtype=torch.int32, device="cuda")
    Y = oz.grouped_linear(X, W, wild)
    dX, dW = oz.grouped_linear_grads(dY, X, W, wild)
    check_all(X, W, dY, tame, Y, dX, dW)


def test_repeats_agree_bit_for_bit():
    for dtype in TYPES.values():
        X, W, dY, off = draw([300, 7, 0, 200], 520, 1032, dtype, 13)
        first = (oz.grouped_linear(X, W, off), *oz.grouped_linear_grads(dY, X, W, off))
        for _ in range(3):
            again = (oz.grouped_linear(X, W, off), *oz.grouped_linear_grads(dY, X, W, off))
            assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_empty_calls():
    W = torch.randn(2, 16, 8, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    X, dY = torch.empty(0, 8, device="cuda"), torch.empty(0, 16, device="cuda")
    assert oz.grouped_linear(X, W, off).shape == (0, 16)
    dX, dW = oz.grouped_linear_grads(dY, X, W, off)
    assert dX.shape == (0, 8) and (dW == 0).all()
    # no inner dimension: zeros in the rows of groups
    out = torch.full((5, 16), 2.0, device="cuda")
    oz.grouped_linear(torch.empty(5, 0, device="cuda"), torch.empty(2, 16, 0, device="cuda"),
                      torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda"), out=out)
    assert (out[:4] == 0).all() and (out[4] == 2).all()


def test_two_streams_and_a_captured_graph():
    for dtype in TYPES.values():
        X, W, dY, off = draw([90, 0, 160, 31], 200, 256, dtype, 14)
        X2, W2, dY2, off2 = draw([60, 100], 129, 77, dtype, 15)
        want = (oz.grouped_linear(X, W, off), *oz.grouped_linear_grads(dY, X, W, off))
        want2 = (oz.grouped_linear(X2, W2, off2), *oz.grouped_linear_grads(dY2, X2, W2, off2))
        torch.cuda.synchronize()
        a, b = torch.cuda.Stream(), torch.cuda.Stream()
        for _ in range(3):
            with torch.cuda.stream(a):
                got = (oz.grouped_linear(X, W, off), *oz.grouped_linear_grads(dY, X, W, off))
            with torch.cuda.stream(b):
                got2 = (oz.grouped_linear(X2, W2, off2), *oz.grouped_linear_grads(dY2, X2, W2, off2))
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(want, got))
            assert all(torch.equal(x, y) for x, y in zip(want2, got2))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            cap = (oz.grouped_linear(X, W, off), *oz.grouped_linear_grads(dY, X, W, off))
        for k in range(3):
            for t in cap:
                t.zero_()
            # new sizes in the same offsets, as a router would write them between replays
            off.copy_(torch.tensor([0, 10 * k, 100, 260 + k, 281], dtype=torch.int32))
            graph.replay()
            eager = (oz.grouped_linear(X, W, off), *oz.grouped_linear_grads(dY, X, W, off))
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(cap, eager))


def test_gradients_against_differences():
    # the layer is linear in each argument: (Y(X + h) - Y(X)) . dY is dX . h, exactly so in whole numbers
    g = torch.Generator(device="cuda").manual_seed(4)

    def whole(*shape):
        return torch.randint(-3, 4, shape, generator=g, device="cuda").float()

    off = torch.tensor([0, 12, 12, 45], dtype=torch.int32, device="cuda")
    X, W, dY, hX, hW = whole(45, 30), whole(3, 20, 30), whole(45, 20), whole(45, 30), whole(3, 20, 30)
    dX, dW = oz.grouped_linear_grads(dY, X, W, off)
    Y = oz.grouped_linear(X, W, off)
    assert ((oz.grouped_linear(X + hX, W, off) - Y) * dY).double().sum() == (dX * hX).double().sum()
    assert ((oz.grouped_linear(X, W + hW, off) - Y) * dY).double().sum() == (dW * hW).double().sum()


def test_a_given_workspace():
    X, W, _, off = draw([33, 100000], 50, 70, torch.float32, 16)
    sizes = (2, 50, 100033, 70, 1, W, 70, 3500, X, 70)
    need = L.ozgemm_grouped_gemm_workspace_bytes(L.OZGEMM_F32, *sizes)
    assert need > 0
    ws = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    Y = torch.empty(100033, 50, device="cuda")
    L.ozgemm_grouped_gemm(L.OZGEMM_F32, L.OZGEMM_F32, *sizes, off, Y, 50, workspace=ws[:need])
    assert torch.equal(Y, oz.grouped_linear(X, W, off))
    assert (ws[need:] == 0x5A).all()
    with pytest.raises(L.OzgemmError) as e:
        L.ozgemm_grouped_gemm(L.OZGEMM_F32, L.OZGEMM_F32, *sizes, off, Y, 50, workspace=ws[:need - 1])
    assert e.value.status == L.OZGEMM_WORKSPACE_TOO_SMALL


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("layout", ["mq", "qm"])
@pytest.mark.parametrize("sizes, m, q", [([9, 0, 30], 37, 45), ([1], 8, 1025), ([70, 3], 130, 7), ([5, 40], 3, 66),
                                         ([33, 1], 515, 264), ([600], 129, 131)])
def test_rows_off_the_16_byte_grid(sizes, m, q, layout, dtype):
    # every operand begins one entry into rows of its own length + 3; what lies between them is NaN
    def inside(t):
        wide = torch.full((*t.shape[:-1], t.shape[-1] + 3), float("nan"), device="cuda", dtype=t.dtype)
        wide[..., 1:-2] = t
        return wide[..., 1:-2]

    X, W, dY, off = draw(sizes, m, q, TYPES[dtype], m + 2 * q)
    if layout == "qm":
        W = inside(W.transpose(1, 2)).transpose(1, 2)
    else:
        W = inside(W)
    X, dY = inside(X), inside(dY)
    Y, dX, dW = inside(dY.new_zeros(X.shape[0], m)), inside(torch.zeros_like(X)), torch.empty_like(W)
    oz.grouped_linear(X, W, off, out=Y)
    oz.grouped_linear_grads(dY, X, W, off, dX=dX)
    _, dW = oz.grouped_linear_grads(dY, X, W, off)
    check_all(X, W, dY, off, Y, dX, dW)


@pytest.mark.parametrize("layout", ["mq", "qm"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("sizes, m, q", [
    ([1], 8, 8), ([2, 0, 1], 136, 1024), ([16] * 9, 264, 2056), ([17, 0, 31, 33, 1], 520, 264), ([100, 20, 3], 72, 520),
    ([24] * 40, 128, 96), ([1] * 130, 40, 48), ([65, 2], 1032, 4104), ([5], 2048, 1008)])
def test_few_rows(sizes, m, q, dtype, layout):
    # single tokens and small batches: the weights are streamed, K shared by the wavefronts of a block
    X, W, dY, off = draw(sizes, m, q, TYPES[dtype], m + q, before=3, behind=2)
    X[:3], X[-2:] = float("nan"), float("inf")
    if layout == "qm":
        W = W.transpose(1, 2).contiguous().transpose(1, 2)
    for out_dtype in (None, torch.float32):
        out = torch.full((X.shape[0], m), 5.0, device="cuda", dtype=out_dtype or X.dtype)
        Y = oz.grouped_linear(X, W, off, out=out)
        check_all(X, W, dY, off, Y, None, None)
        assert (out[:3] == 5).all() and (out[-2:] == 5).all()
    dX = torch.full(X.shape, 5.0, device="cuda", dtype=X.dtype)
    _, dW = oz.grouped_linear_grads(dY, X, W, off, dX=dX)
    check_all(X, W, dY, off, Y, dX, dW)


# tiles of 256 x 256 (f32: 128 x 128) in whole rounds of 256 compute units and every kind of rest: none, a
# few tiles and half a round (cut into quarters), more than half a round
@pytest.mark.parametrize("dtype, sizes, m", [
    ("bf16", [256] * 32, 4096), ("bf16", [256] * 33, 4096), ("bf16", [200, 256, 300] * 13, 4096),
    ("f16", [128] * 70, 2304), ("f16", [300] * 25, 6400), ("bf16", [1024, 0, 7000, 30, 5000], 2560),
    ("f32", [128] * 32, 2048), ("f32", [128] * 37, 2304), ("f32", [60, 300] * 12, 2432)])
@pytest.mark.parametrize("layout", ["mq", "qm"])
def test_every_tile_is_written(dtype, sizes, m, layout):
    X, W, dY, off = draw(sizes, m, 72, TYPES[dtype], len(sizes) + m)
    if layout == "qm":
        W = W.transpose(1, 2).contiguous().transpose(1, 2)
    Y = torch.full(dY.shape, float("nan"), device="cuda", dtype=X.dtype)
    oz.grouped_linear(X, W, off, out=Y)
    check_all(X, W, dY, off, Y, None, None)
    # the gradients of a layer with the sides exchanged: many tiles for them too
    Wt = W.transpose(1, 2)
    dX = torch.full(dY.shape, float("nan"), device="cuda", dtype=X.dtype)
    dW = torch.full(Wt.shape, float("nan"), device="cuda", dtype=X.dtype)
    oz.grouped_linear_grads(X, dY, Wt, off, dX=dX, dW=dW)
    assert torch.equal(dX, Y)
    o = off.tolist()
    for e in range(len(sizes)):
        s = slice(o[e], o[e + 1])
        C, P = X[s].double().T @ dY[s].double(), X[s].double().abs().T @ dY[s].double().abs()
        big = (X[s].double().abs().amax(0)[:, None] * dY[s].double().abs().amax(0)[None]) if sizes[e] else 0.0
        check(dW[e], C, bound(C, P, sizes[e], X.dtype, dW.dtype, big))


@pytest.mark.parametrize("dtype, groups, m, q", [("bf16", 9, 2048, 2048), ("f16", 3, 2560, 4096), ("f32", 5, 1024, 1152),
                                                 ("bf16", 70, 520, 264), ("f32", 70, 264, 392)])
def test_every_tile_of_the_weights_gradient_is_written(dtype, groups, m, q):
    sizes = [(37 * e) % 101 for e in range(groups)]
    X, W, dY, off = draw(sizes, m, q, TYPES[dtype], groups)
    dW = torch.full(W.shape, float("nan"), device="cuda", dtype=X.dtype)
    oz.grouped_linear_grads(dY, X, W, off, dW=dW)
    o = off.tolist()
    for e in range(groups):
        s = slice(o[e], o[e + 1])
        C, P = dY[s].double().T @ X[s].double(), dY[s].double().abs().T @ X[s].double().abs()
        big = (dY[s].double().abs().amax(0)[:, None] * X[s].double().abs().amax(0)[None]) if sizes[e] else 0.0
        check(dW[e], C, bound(C, P, sizes[e], X.dtype, dW.dtype, big))


@pytest.mark.parametrize("dtype, sizes, m, q", [("bf16", [3000], 64, 96), ("f16", [1500, 0, 2600, 40], 40, 136),
                                                ("f32", [5000, 3], 72, 130), ("bf16", [9000], 33, 257),
                                                ("f32", [70, 2000, 0, 1100], 128, 64),
                                                ("bf16", [30000, 0, 9000], 512, 264), ("f32", [40000], 500, 260),
                                                ("f16", [33000], 511, 257), ("bf16", [33000], 1536, 2048),
                                                ("f32", [20, 33000], 1024, 1032)])
def test_weights_gradient_summed_in_parts(dtype, sizes, m, q):
    X, W, dY, off = draw(sizes, m, q, TYPES[dtype], m * q, before=5, behind=7)
    X[:5], dY[-7:] = float("nan"), float("nan")
    for dw_dtype in (None, torch.float32):
        Y = oz.grouped_linear(X, W, off)
        dX, dW = oz.grouped_linear_grads(dY, X, W, off, dw_dtype=dw_dtype)
        check_all(X, W, dY, off, Y, dX, dW)
        assert torch.equal(dW, oz.grouped_linear_grads(dY, X, W, off, dw_dtype=dw_dtype)[1])


@pytest.mark.parametrize("layout", ["mq", "qm"])
@pytest.mark.parametrize("dtype, sizes, m, q", [("bf16", [300, 0, 200], 96, 4096), ("f16", [700], 33, 1601),
                                                ("f32", [100, 40], 72, 2000), ("f32", [1], 24, 4096),
                                                ("f32", [0, 130, 61], 200, 1090), ("bf16", [999], 264, 2056),
                                                ("bf16", [256], 2048, 32768), ("f16", [300, 212], 1030, 8190)])
def test_products_summed_in_parts(dtype, sizes, m, q, layout):
    X, W, dY, off = draw(sizes, m, q, TYPES[dtype], m * q + 1, before=6, behind=4)
    X[:6], X[-4:] = float("nan"), float("inf")
    if layout == "qm":
        W = W.transpose(1, 2).contiguous().transpose(1, 2)
    for out_dtype in (X.dtype, torch.float32):
        out = torch.full((X.shape[0], m), 5.0, device="cuda", dtype=out_dtype)
        Y = oz.grouped_linear(X, W, off, out=out)
        check_all(X, W, dY, off, Y, None, None)
        assert (out[:6] == 5).all() and (out[-4:] == 5).all()
        assert torch.equal(out, oz.grouped_linear(X, W, off, out=out.clone()))


@pytest.mark.parametrize("layout", ["mq", "qm"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("sizes, m, q", [([5, 0, 17], 40, 12288), ([1], 24, 32768), ([130, 66], 72, 8200),
                                         ([0, 0, 200], 130, 8232), ([3], 1000, 16388)])
def test_few_columns_summed_in_parts(dtype, sizes, m, q, layout):
    X, W, dY, off = draw(sizes, m, q, TYPES[dtype], m * q + 2, before=3, behind=2)
    X[:3], X[-2:] = float("nan"), float("inf")
    if layout == "qm":
        W = W.transpose(1, 2).contiguous().transpose(1, 2)
    for out_dtype in (X.dtype, torch.float32):
        out = torch.full((X.shape[0], m), 5.0, device="cuda", dtype=out_dtype)
        Y = oz.grouped_linear(X, W, off, out=out)
        check_all(X, W, dY, off, Y, None, None)
        assert (out[:3] == 5).all() and (out[-2:] == 5).all()
        assert torch.equal(out, oz.grouped_linear(X, W, off, out=out.clone()))


@pytest.mark.parametrize("dtype, sizes, m, q", [("f32", [5, 3], 40, 12288), ("bf16", [300, 212], 1030, 8190),
                                                ("f32", [20000, 19000], 500, 260), ("f16", [33000, 8], 512, 257)])
def test_parts_in_a_captured_graph(dtype, sizes, m, q):
    X, W, dY, off = draw(sizes, m, q, TYPES[dtype], m + q + 3)
    run = lambda: (oz.grouped_linear(X, W, off), *oz.grouped_linear_grads(dY, X, W, off))  # noqa: E731
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = run()
    for k in range(3):
        X.mul_(-1.25)
        off[1] -= k
        graph.replay()
        eager = run()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(cap, eager))
        check_all(X, W, dY, off, *cap)
