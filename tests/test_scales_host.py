"""The grids of the Newton-Schulz states (csrc/scales.h) against bounds found by
looking: on grids of points, for schedules and first bounds of every size."""
import math
import os
import random
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
QUINTIC = (3.4445, -4.7750, 2.0315)


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("scales") / "scales_driver")
    subprocess.run(["g++", "-O2", "-std=c++17", os.path.join(HERE, "scales_driver.cpp"), "-o", exe], check=True)

    def run(rows, *args):
        text = "\n".join(" ".join(repr(float(v)) for v in row) for row in rows)
        out = subprocess.run([exe, *args], input=text, capture_output=True, text=True, check=True).stdout
        return [[float(v) for v in line.split()] for line in out.splitlines()]

    return run


def steps(seed, count):
    r = random.Random(seed)
    for _ in range(count):
        kind = r.randrange(4)
        a, b, c = QUINTIC if kind == 0 else (
            [r.choice((-1, 1)) * 10 ** r.uniform(-5, 4) for _ in range(3)] if kind == 1 else
            (r.uniform(1, 9), r.uniform(-25, 0), r.uniform(0, 20)) if kind == 2 else
            [r.choice((0.0, r.uniform(-3, 3))) for _ in range(3)])
        yield a, b, c, 10 ** r.choice((r.uniform(-3, 1), r.uniform(-110, 0), 0.0))


def test_bounds_hold_and_are_no_wider_than_they_need(driver):
    rows = list(steps(1, 400))
    x = np.linspace(0, 1, 20001)
    for (a, b, c, t), (X, P, Q, nxt, *_rest) in zip(rows, driver(rows)):
        assert X == t and P == t * t
        y = t * x
        p = np.abs(y * (a + y * y * (b + y * y * c))).max()
        # 20001 points find a peak to (5 / 20000)^2 of it and better
        assert p <= nxt * (1 + 1e-12) and nxt <= p * (1 + 1.0 / 1024) * (1 + 1e-6) + 1e-300
        y = t * t * x
        q = np.abs(y * (b + c * y)).max()
        assert q <= Q * (1 + 1e-12) and Q <= q * (1 + 1e-6) + 1e-300


def test_grids_and_factors(driver):
    rows = list(steps(2, 400))
    for (a, b, c, t), (X, P, Q, nxt, ex, ep, eq, en, f0, f1, g1, f2, g2, _ok) in zip(rows, driver(rows)):
        for bound, e in ((X, ex), (P, ep), (Q, eq), (nxt, en)):
            if bound > 2.0 ** -1000:
                assert 2.0 ** 13 <= math.ldexp(bound, int(e)) < 2.0 ** 14
        # P = f0 X X^T and so on, in units of the grids; single precision's rounding of a, b and c apart
        assert f0 == math.ldexp(1.0, int(ep - 2 * ex))
        for got, coefficient, e in ((f1, c, eq - 2 * ep), (g1, b, eq - ep), (f2, 1.0, en - eq - ex), (g2, a, en - ex)):
            want = math.ldexp(coefficient, int(e))
            assert math.isfinite(got) and abs(got - want) <= 2.0 ** -24 * abs(want) + 2.0 ** -126
        # the terms that carry a state on are in single precision's normal range: next to them what underflows is nothing
        if a and nxt > 2.0 ** -1000:
            assert abs(g2) > 2.0 ** -126 * abs(a) / max(abs(a), 1) or abs(a) * t < 2.0 ** -100 * nxt


def test_schedules_are_followed_from_any_first_bound(driver):
    # an iterate with one singular value at its bound stays inside the bounds, and five steps of the
    # quintic grow a tiny one by a^5 and no more
    for t0 in (1.0, 0.99999, 1e-3, 1e-12, 1e-40, 2.0 ** -400):
        t, x = t0, t0
        for _ in range(5):
            (X, P, Q, nxt, *_rest), = driver([(*QUINTIC, t)])
            x = abs(x * (QUINTIC[0] + QUINTIC[1] * x * x + QUINTIC[2] * x ** 4))
            assert x <= nxt
            t = nxt
        if t0 < 1e-6:
            assert t == pytest.approx(t0 * QUINTIC[0] ** 5 * (1 + 1 / 1024) ** 5, rel=1e-6)


def test_first_bound(driver):
    inf, nan = math.inf, math.nan
    rows = [(1.0, 0.0), (1e-3, 1e-7), (1e-20, 1e-7), (0.0, 1e-7), (0.0, 0.0), (inf, 1e-7), (nan, 1e-7), (1e-45, 1e290), (5.0, 1e-300)]
    got = [v for v, in driver(rows, "first")]
    assert got[:3] == [1.0, 1e-3 / (1e-3 + 1e-7), 1e-20 / (1e-20 + 1e-7)]
    assert got[3:7] == [1.0] * 4 and got[7] == 2.0 ** -400 and got[8] == 1.0


@pytest.mark.parametrize("c", [1e-9, -1e-9, 1e-14, 1e-16, -1e-16, 1e-18, -1e-30, 1e-300, 0.0])
@pytest.mark.parametrize("a, b, t", [(1.5, -0.5, 3 ** 0.5), (1.5, -0.5, 1.5), (3.0, -1.0, 1.2), (0.0, -1.0, 1.0), (-2.0, 2.0, 1.0)])
def test_peaks_next_to_a_cubic(driver, a, b, c, t):
    # the quintic's term is next to nothing: its stationary points are the cubic's (and one far away)
    (X, P, Q, nxt, *_rest), = driver([(a, b, c, t)])
    x = np.linspace(0, t, 20001)
    p = np.abs(x * (a + x * x * (b + x * x * c))).max()
    assert p <= nxt * (1 + 1e-12) and nxt <= p * (1 + 1.0 / 1024) * (1 + 1e-6)
