"""The norm over many tensors and the clipping of gradients against 64 bits.

Tolerances.  The norm: FP64 sums of N squares in a few hundred partial sums, (1 +
log2 N + chunk / 2048 ...) roundings; 1e-13 of it covers a thousand.  An entry:
the factor's rounding to FP32 and the product's, 2 x 2^-24 of it, then half a
step (FP64: 3 roundings of 2^-53 and the norm's)."""
import math

import pytest
import torch

import fp64_gemm_emulation_ozii_amd as oz
from fp64_gemm_emulation_ozii_amd import ozgemm as L

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32, torch.float64]
SETS = {"one": [(1,)], "few": [(5,), (3, 7), (), (2, 3, 4)], "empty among": [(0,), (9,), (4, 0), (70000,), (0,)],
        "chunks": [(16384,), (16385,), (8191,), (32768 * 3 + 1,), (65536,), (8193,)], "many": [(k % 37 + 1,) for k in range(300)],
        "large": [(3000, 1000), (1 << 22,), (17,)]}


def draw(shapes, types, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(s, generator=g, device="cuda").mul(0.1).to(types[k % len(types)]) for k, s in enumerate(shapes)]


def norm_of(grads):
    return math.sqrt(math.fsum(g.double().square().sum().item() for g in grads))


def check(got, grads, factor):
    for o, g in zip(got, grads):
        want = g.double() * factor
        f = torch.finfo(g.dtype)
        tol = 1e-13 * want.abs() if g.dtype == torch.float64 else (
            (f.eps / 2 * (g.dtype != torch.float32) + 2.01 * 2.0 ** -24) * want.abs() + f.smallest_normal * f.eps)
        assert o.dtype == g.dtype and ((o.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("types", [[t] for t in TYPES] + [TYPES], ids=str)
@pytest.mark.parametrize("name", list(SETS))
def test_norm_and_clipping(name, types):
    grads = draw(SETS[name], types, len(name))
    want = norm_of(grads)
    norm = oz.gradient_norm(grads)
    assert norm.dtype == torch.float64 and norm.shape == () and abs(norm.item() - want) <= 1e-13 * want
    for bound in (want / 3, want * 2):
        factor = min(1.0, bound / (want + 1e-6))
        out = [torch.full_like(g, 9.0) for g in grads]
        assert torch.equal(oz.clip_gradients(grads, bound, out=out), norm)
        check(out, grads, factor)
        again = [g.clone() for g in grads]
        assert torch.equal(oz.clip_gradients(again, bound), norm)
        assert all(torch.equal(a, b) for a, b in zip(again, out))
        if factor == 1.0:
            assert all(torch.equal(a, g) for a, g in zip(again, grads))


def test_views():
    base = draw([(50, 60), (8, 9, 10), (40, 40)], [torch.bfloat16], 5)
    grads = [base[0][:, 3:20], base[1].permute(2, 0, 1), base[2].t()[::2]]
    want, copies = norm_of(grads), [g.clone() for g in grads]
    rest = base[0][:, 20:].clone()
    assert abs(oz.gradient_norm(grads).item() - want) <= 1e-13 * want
    oz.clip_gradients(grads, 1.0)
    check(grads, copies, min(1.0, 1.0 / (want + 1e-6)))
    assert torch.equal(base[0][:, 20:], rest)
    # out of another layout
    out = [torch.zeros(g.shape[::-1], dtype=g.dtype, device="cuda").permute(*reversed(range(g.dim()))) for g in copies]
    oz.clip_gradients(copies, 0.5, out=out)
    check(out, copies, 0.5 / (norm_of(copies) + 1e-6))
    # at any byte of 16
    flat = torch.randn(1000, device="cuda").bfloat16()
    parts, copies = [flat[1:300], flat[303:1000]], [flat[1:300].clone(), flat[303:1000].clone()]
    oz.clip_gradients(parts, 0.25)
    check(parts, copies, 0.25 / (norm_of(copies) + 1e-6))
    # expanded: every entry counts
    assert abs(oz.gradient_norm(torch.full((1,), 2.0, device="cuda").expand(9)).item() - 6.0) < 1e-12


def test_norms_brought_together():
    a, b = draw([(100,), (200,)], [torch.float32], 1), draw([(300,)], [torch.bfloat16], 2)
    whole = torch.sqrt(oz.gradient_norm(a).square() + oz.gradient_norm(b).square())
    copies = [t.clone() for t in a + b]
    assert oz.clip_gradients(a, 0.5, norm=whole) is whole
    oz.clip_gradients(b, 0.5, norm=whole)
    check(a + b, copies, 0.5 / (whole.item() + 1e-6))


def test_norms_that_are_none():
    inf, nan = float("inf"), float("nan")
    g = [torch.tensor([1.0, inf, -2.0], device="cuda"), torch.ones(5, device="cuda", dtype=torch.bfloat16)]
    assert oz.clip_gradients(g, 1.0).item() == inf
    assert g[0][1].isnan() and g[0][0] == 0 and (g[1] == 0).all()
    g = [torch.tensor([1.0, nan], device="cuda"), torch.ones(5, device="cuda", dtype=torch.float16)]
    assert math.isnan(oz.clip_gradients(g, 1e9).item()) and g[0].isnan().all() and g[1].isnan().all()
    big = [torch.full((4,), 3e38, device="cuda"), torch.full((3,), 60000.0, device="cuda", dtype=torch.float16)]
    assert abs(oz.gradient_norm(big).item() - 6e38) < 1e32  # beyond float32
    zero = [torch.zeros(4, device="cuda")]
    assert oz.clip_gradients(zero, 0.0).item() == 0 and (zero[0] == 0).all()
    assert oz.gradient_norm([]).item() == 0 and oz.clip_gradients([], 1.0).item() == 0


def test_shared_memory_is_refused():
    t = torch.ones(100, device="cuda")
    for grads, out in (([t, t], None), ([t[:60], t[50:]], None), ([t[:50], t[50:]], [t[50:], t[:50]]),
                       ([t[:50], t[50:]], [torch.ones(50, device="cuda"), t[:50]])):
        with pytest.raises(L.OzgemmError):
            oz.clip_gradients(grads, 0.1, out=out)
        assert (t == 1).all()
    assert abs(oz.gradient_norm([t, t]).item() - math.sqrt(200)) < 1e-12
    # only read twice
    out = [torch.zeros(100, device="cuda"), torch.zeros(100, device="cuda")]
    oz.clip_gradients([t, t], 1.0, out=out)
    assert torch.equal(out[0], out[1]) and out[0][0] > 0


def test_writing_counts_as_a_change():
    t, o = torch.ones(4, device="cuda"), torch.ones(4, device="cuda")
    for k in range(2):
        was = t._version, o._version
        oz.clip_gradients([t], 0.5, out=None if k else [o])
        assert (t._version > was[0]) == (k == 1) and (o._version > was[1]) == (k == 0)


def test_interleaved_tensors_are_not_shared_memory():
    t, o = torch.ones(64, 100, device="cuda"), torch.zeros(64, 100, device="cuda")
    parts = [t[:, ::2], t[:, 1::2]]
    want = 1.0 / (80.0 + 1e-6)
    oz.clip_gradients(parts, 1.0, out=[o[:, 1::2], o[:, ::2]])
    check([o], [torch.ones_like(t)], want)
    assert (t == 1).all()
    for out in ([o[:, ::2], o[:, ::2]], [o[:, ::2], o.as_strided((64, 50), (98, 2), 4)], [o[:, ::2], o.view(-1)[:3200].view(64, 50)]):
        before = o.clone()
        with pytest.raises(ValueError, match="share memory"):
            oz.clip_gradients(parts, 1.0, out=out)
        assert torch.equal(o, before)
    with pytest.raises(ValueError, match="share memory"):
        oz.clip_gradients([t[:, ::2], t[:, :2]], 1.0)
    assert (t == 1).all()
    oz.clip_gradients(parts, 1.0)
    check([t], [torch.ones_like(t)], want)


@pytest.mark.parametrize("bound", [1e30, 1.0, 1e-3, 1e-20])
@pytest.mark.parametrize("types", [[t] for t in TYPES] + [TYPES], ids=str)
def test_factors_below_the_range_of_float32(types, bound):
    # entries up to 3e38 (float64: 1e100) under a small bound: the factor underflows float32, the products do not have to
    g = torch.Generator(device="cuda").manual_seed(8)
    grads = []
    for k, size in enumerate((40, 70000, 9)):
        t = types[k % len(types)]
        top = {torch.float64: 1e100, torch.float16: 6e4}.get(t, 3e38)
        grads.append((torch.rand(size, generator=g, device="cuda", dtype=torch.float64) * top * 10.0 ** -torch.randint(0, 4, (size,), generator=g, device="cuda")).to(t))
    want = norm_of(grads)
    out = [torch.full_like(x, 9.0) for x in grads]
    norm = oz.clip_gradients(grads, bound, out=out)
    assert abs(norm.item() - want) <= 1e-13 * want
    check(out, grads, min(1.0, bound / (norm.item() + 1e-6)))
    if any(t is torch.float32 for t in types) and torch.float64 not in types:
        assert bound < 1e-3 or any(o.abs().amax() > 0 for o in out)
