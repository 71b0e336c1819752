"""A layer of experts, its gradients and its update as they are used together,
every value against 64 bits; whole numbers that need both slices on either side;
calls from several host threads.  Tolerances: test_gpu_grouped.py and
test_gpu_ortho.py."""
import threading

import pytest
import torch

import fp64_gemm_emulation_ozii_amd as oz
from fp64_gemm_emulation_ozii_amd import ozgemm as L
from test_gpu_grouped import TYPES, check_all, draw
from test_gpu_ortho import plain, rel, tolerance

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("sizes, m, q", [([40, 0, 100, 9], 64, 96), ([700, 0, 900, 1300], 320, 513)])
def test_a_layer_its_gradients_and_its_update(sizes, m, q, dtype):
    X, W, _, off = draw(sizes, m, q, TYPES[dtype], 11)
    X, W = X / 8, W / 8
    Y = oz.grouped_linear(X, W, off)
    dX, dW = oz.grouped_linear_grads(Y, X, W, off)  # of sum(Y^2) / 2
    check_all(X, W, Y, off, Y, dX, dW)
    O = oz.orthogonalize(dW)
    assert (O[1] == 0).all()
    for e in (0, 2, 3):
        want = plain(dW[e])
        assert rel(O[e], want) <= tolerance(dW[e], want)


@pytest.mark.parametrize("wide", ["X", "W", "dY"])
def test_whole_numbers_that_need_the_low_slices_of_any_operand(wide):
    # 4097 has 13 bits, a slice 11; every other operand is -1, 0 or 1, and |sums| <= 3700 x 4097 < 2^24
    sizes, m, q = [2500, 0, 3700, 1313], 1100, 601
    n, g = sum(sizes), torch.Generator(device="cuda").manual_seed(7)
    off = torch.tensor([0, 2500, 2500, 6200, n], dtype=torch.int32, device="cuda")

    def whole(name, *shape):
        if name == wide:
            return (torch.randint(0, 2, shape, generator=g, device="cuda") * 2 - 1).float() * 4097
        return torch.randint(-1, 2, shape, generator=g, device="cuda").float()

    X, W, dY = whole("X", n, q), whole("W", 4, m, q), whole("dY", n, m)
    # every product of the three goes by slices: it needs room for them
    f32 = L.OZGEMM_F32
    assert L.ozgemm_grouped_gemm_workspace_bytes(f32, 4, m, n, q, 1, W, q, m * q, X, q) > 4 * (4 * m + n) * q
    assert L.ozgemm_grouped_gemm_workspace_bytes(f32, 4, q, n, m, 0, W, q, m * q, dY, m) > 4 * (4 * q + n) * m
    assert L.ozgemm_grouped_outer_workspace_bytes(f32, 4, q, m, n, X, q, dY, m) > 4 * (m + q) * n
    Y = oz.grouped_linear(X, W, off)
    dX, dW = oz.grouped_linear_grads(dY, X, W, off)
    o = off.tolist()
    for e in range(4):
        s = slice(o[e], o[e + 1])
        assert torch.equal(Y[s].double(), X[s].double() @ W[e].double().T)
        assert torch.equal(dX[s].double(), dY[s].double() @ W[e].double())
        assert torch.equal(dW[e].double(), dY[s].double().T @ X[s].double())


@pytest.mark.parametrize("layout", ["mq", "qm"])
@pytest.mark.parametrize("dtype, sizes, m, q", [
    ("bf16", [300, 0, 200], 96, 4096), ("f16", [700], 33, 1601), ("f32", [100, 40], 72, 2000),
    ("bf16", [256], 2048, 32768), ("f16", [300, 212], 1030, 8190), ("f32", [5, 0, 17], 40, 12288),
    ("f32", [3], 1000, 16388), ("bf16", [3], 1000, 16389), ("f32", [9000, 0, 777], 520, 1031),
    ("bf16", [30000, 0, 9000], 512, 264), ("f32", [40000], 500, 260), ("f16", [33000], 511, 257),
    ("f32", [20, 33000], 1024, 1032), ("bf16", [33000], 1536, 2048), ("f16", [70, 0, 5000, 300] * 8, 264, 520)])
def test_whole_numbers_over_long_sums(dtype, sizes, m, q, layout):
    # no entry may be lost where the tolerances of long sums would let one pass: what is exact in FP32 comes out exactly
    t, g = TYPES[dtype], torch.Generator(device="cuda").manual_seed(m + q)
    n = sum(sizes)
    off = torch.tensor([0, *torch.tensor(sizes).cumsum(0).tolist()], dtype=torch.int32, device="cuda")

    def sparse(*shape):  # -1, 0 or 1, one in sixteen not 0
        k = torch.randint(0, 32, shape, generator=g, device="cuda", dtype=torch.int8)
        return (k == 0).to(t) - (k == 1).to(t)

    X = (torch.randint(0, 2, (n, q), generator=g, device="cuda") * 2 - 1).to(t) * (4097 if dtype == "f32" else 7)
    W, dY = sparse(len(sizes), m, q), sparse(n, m)
    if layout == "qm":
        W = W.transpose(1, 2).contiguous().transpose(1, 2)
    Y = oz.grouped_linear(X, W, off, out_dtype=torch.float32)
    dX, dW = oz.grouped_linear_grads(dY, X, W, off, dw_dtype=torch.float32)
    o = off.tolist()
    for e in range(len(sizes)):
        s = slice(o[e], o[e + 1])
        x, w, y = X[s].double(), W[e].double().contiguous(), dY[s].double()
        for got, a, b in ((Y[s], x, w.T.contiguous()), (dX[s], y, w), (dW[e], y.T.contiguous(), x)):
            assert not a.numel() or (a.abs() @ b.abs()).max() < 2 ** 24  # of ones: every partial sum is exact
            assert torch.equal(got, (a @ b).to(got.dtype))


def test_calls_from_several_host_threads():
    jobs = []
    for k, dtype in enumerate((torch.bfloat16, torch.float32, torch.float16, torch.float32)):
        X, W, dY, off = draw([300 + k, 0, 4100], 200 + 8 * k, 264, dtype, 30 + k)
        G = X[:150 + k].clone()
        jobs.append((X, W, dY, off, G, torch.cuda.Stream()))

    def run(X, W, dY, off, G):
        return (oz.grouped_linear(X, W, off), *oz.grouped_linear_grads(dY, X, W, off), oz.orthogonalize(G),
                oz.orthogonalize(G.double()))

    wants = [run(*job[:5]) for job in jobs]
    torch.cuda.synchronize()
    gots, errors = [[] for _ in jobs], []

    def work(k):
        try:
            with torch.cuda.stream(jobs[k][5]):
                for _ in range(5):
                    gots[k].append(run(*jobs[k][:5]))
        except Exception as e:  # (shown by the main thread)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for want, got in zip(wants, gots):
        assert len(got) == 5
        assert all(torch.equal(a, b) for g in got for a, b in zip(want, g))

