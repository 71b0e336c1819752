"""Newton-Schulz steps on matrices whose norm is far below eps, and with
schedules that shrink their iterates: the states' grids have to follow each
matrix.  Tolerances are those of test_gpu_ortho.py (a step is
scale-free in what it adds: every state is rounded relative to its own bound)."""
import pytest
import torch

import fp64_gemm_emulation_ozii_amd as oz
from test_gpu_ortho import QUINTIC, TYPES, draw, plain, rel, tolerance

pytestmark = pytest.mark.gpu

SHAPES = [(40, 66), (300, 200), (64, 1500), (600, 1100)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("norm", [1e-8, 1e-10, 1e-12, 1e-14, 1e-20, 1e-26])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_norms_below_eps(shape, norm, dtype):
    G = draw(shape, torch.float64, sum(shape))
    G = (G * (norm / G.norm())).to(TYPES[dtype])
    want = plain(G)
    assert rel(oz.orthogonalize(G), want) <= tolerance(G, want)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_matrices_of_one_batch_have_grids_of_their_own(dtype):
    sizes = (1.0, 1e-2, 1e-3) if dtype == "f16" else (1.0, 1e-9, 1e-18, 1e-30, 1e5, 0.0)
    G = draw((len(sizes), 70, 90), torch.float64, 3)
    G = G / G.flatten(1).norm(dim=1)[:, None, None]
    G = (G * torch.tensor(sizes, device="cuda", dtype=torch.float64)[:, None, None]).to(TYPES[dtype])
    eps = 1e-1 if dtype == "f16" else 1e-7
    O = oz.orthogonalize(G, eps=eps)
    for k, size in enumerate(sizes):
        want = plain(G[k], eps=eps)
        if size == 0:
            assert (O[k] == 0).all()
        else:
            assert rel(O[k], want) <= tolerance(G[k], want, eps=eps)


def below_the_grids(shape, coeffs):
    """What the low ends of the grids add, in the Frobenius norm.  A state whose singular values are at most t lies on a
    grid where t is 2^13 or more and the smallest step of a low slice 2^-24: an entry is off by half of that, 2^-38 t, even
    where the state itself is far below its bound (as x^9 of singular values of 1/4 is).  X, of r c entries, with t; P, of
    r^2, with t^2, through b X and (twice) c P X; Q with |b| t^2 + |c| t^4, through X.  A later step grows what is there by
    its largest slope, |a| + 3 |b| t^2 + 5 |c| t^4."""
    r, c = sorted(shape)
    t, off = 1.0, 0.0
    for a, b, e in coeffs:
        a, b, e = abs(a), abs(b), abs(e)
        here = r * (b + 2 * e * t * t) * t ** 3 + r * (b * t * t + e * t ** 4) * t
        off = (off + (r * c) ** 0.5 * t * 2.0 ** -38) * (a + 3 * b * t * t + 5 * e * t ** 4) + here * 2.0 ** -38
        t = a * t + b * t ** 3 + e * t ** 5
    return off


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("coeffs", [
    [(0.1, -0.05, 0.01)] * 3, [(1e-2, 0.0, 0.0)] * 2, [(1e-3, 0.0, 0.0)] * 3 + [(1e3, 0.0, 0.0)] * 3,
    [(0.01, -0.02, 0.01)] * 4 + [QUINTIC] * 8, [(0.0, 0.03, 0.0)] * 2 + [(300.0, 0.0, 0.0)] * 2], ids=range(5))
def test_schedules_that_shrink(coeffs, dtype):
    for shape in ((96, 160), (300, 280)):
        G = draw(shape, TYPES[dtype], 9)
        want = plain(G, len(coeffs), coeffs)
        O = oz.orthogonalize(G, steps=len(coeffs), coeffs=coeffs)
        if dtype == "f16" and want.abs().max() < 2.0 ** -10:
            continue  # most of the result lies below half's normal range
        low = 0.0 if dtype == "f64" else below_the_grids(shape, coeffs) / want.norm().item()
        assert rel(O, want) <= tolerance(G, want, steps=len(coeffs), coeffs=coeffs) + low


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_growth_over_many_steps(dtype):
    # the iterate climbs from 1e-12 of eps to where the polynomial bends
    coeffs = [(4.0, -3.0, 0.6)] * 20 + [(1.5, -0.5, 0.0)] * 4
    G = draw((80, 120), torch.float64, 12)
    G = (G * (1e-19 / G.norm())).to(TYPES[dtype])
    want = plain(G, len(coeffs), coeffs)
    assert rel(oz.orthogonalize(G, steps=len(coeffs), coeffs=coeffs), want) <= tolerance(
        G, want, steps=len(coeffs), coeffs=coeffs)


def test_results_near_the_end_of_single_precision():
    # 1e-36: the last step's factors are below single precision's normal range, its results are not
    G = draw((50, 60), torch.float64, 13)
    G = (G * (1e-25 / G.norm())).float()
    want = plain(G, eps=1e10)
    assert want.abs().max() < 1e-32
    assert rel(oz.orthogonalize(G, eps=1e10), want) <= tolerance(G, want, eps=1e10)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("c", [1e-16, -1e-18, 1e-30])
def test_a_quintic_that_is_next_to_a_cubic(c, dtype):
    # a first step to singular values up to 3 ** 0.5, where the cubic's p is 0: its peak lies before
    coeffs = [(3 ** 0.5, 0.0, 0.0), (1.5, -0.5, c), (1.0, 0.0, 0.0)]
    G = draw((70, 90), TYPES[dtype], 14)
    want = plain(G, 3, coeffs)
    assert rel(oz.orthogonalize(G, steps=3, coeffs=coeffs), want) <= tolerance(G, want, steps=3, coeffs=coeffs)
