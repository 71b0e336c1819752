"""Results in 16 bits are off by their one rounding and what the same iteration
in FP32 is off by, whatever the matrix and the schedule.

With d the error before the rounding, a result either rounds as the exact value
does, or a tie lies between the two: then the exact value is within |d| of half a
step and the result within |d| past it.  So it is off by at most 2 |d| more than
the exact value's rounding; d is held to the FP32 bound of test_gpu_ortho.py."""
import pytest
import torch

import fp64_gemm_emulation_ozii_amd as oz
from test_gpu_ortho import QUINTIC, plain, rel

pytestmark = pytest.mark.gpu

# a schedule that bends hard: small singular values grow eightfold in its first step
STEEP = [(8.2, -23.0, 17.0), (4.0, -2.9, 0.53), (3.3, -2.4, 0.46)]
SCHEDULES = {"quintic": [QUINTIC] * 5, "eight": [QUINTIC] * 8, "steep": STEEP}


def matrix(kind, r, c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float64)

    if kind == "noise":
        return normal(r, c)
    if kind == "low rank":
        return normal(r, 8) @ normal(8, c)
    if kind == "flat":  # all singular values alike
        return torch.linalg.qr(normal(c, r).cpu())[0].cuda().mT.contiguous()
    return normal(r, c) * torch.exp(2 * normal(1, c))  # "columns": of very different sizes


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("schedule", list(SCHEDULES))
@pytest.mark.parametrize("kind", ["noise", "low rank", "flat", "columns"])
@pytest.mark.parametrize("r, c", [(200, 300), (256, 256), (256, 1000), (512, 512), (1024, 1536)])
def test_one_rounding(r, c, kind, schedule, dtype):
    co = SCHEDULES[schedule]
    G = matrix(kind, r, c, r + c)
    G = (G / G.norm()).to(dtype)
    want = plain(G, len(co), co)
    single = 2 * rel(plain(G, len(co), co, dtype=torch.float32), want) + 2.0 ** -22
    O = oz.orthogonalize(G, steps=len(co), coeffs=co)
    assert rel(O, want) <= rel(want.to(dtype), want) + 2 * single
