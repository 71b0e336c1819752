"""Calls whose passes need more threads than one launch may have (2^32)."""
import pytest
import torch

import fp64_gemm_emulation_ozii_amd as oz

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype, q", [(torch.bfloat16, 17), (torch.float32, 16)])
def test_weights_of_2_to_the_26_rows(dtype, q):
    # weights that pass through the workspace, a wavefront for each of their rows
    groups, m, each = 4096, 16384, 49
    g = torch.Generator(device="cuda").manual_seed(q)
    W = torch.randn(groups, m, q, generator=g, device="cuda", dtype=dtype)
    X = torch.randn(groups * each, q, generator=g, device="cuda", dtype=dtype)
    off = torch.arange(0, groups * each + 1, each, dtype=torch.int32, device="cuda")
    Y = oz.grouped_linear(X, W, off)
    for e in (0, 1, 2047, 2048, 3071, 3072, 4094, 4095):
        s = slice(e * each, (e + 1) * each)
        x, w = X[s].double(), W[e].double()
        C, P = x @ w.T, x.abs() @ w.abs().T
        # the bounds of test_gpu_grouped.py: one rounding; q sums in FP32, three times as many of slices, which
        # are off by 8 2^-24 of a term and by 2^-40 of the rows' largest entries
        tol = torch.finfo(dtype).eps / 2 * C.abs() + q * 2.0 ** -23 * P
        if dtype == torch.float32:
            big = x.abs().amax(1)[:, None] * w.abs().amax(1)[None]
            tol += (8 + 4.01 * q) * 2.0 ** -24 * P + 4 * q * 2.0 ** -40 * big
        assert ((Y[s].double() - C).abs() <= tol + 2.0 ** -133).all()


def test_a_matrix_of_2_to_the_32_entries_is_normalised():
    n = 65536
    G = torch.empty(n, n, device="cuda", dtype=torch.bfloat16)
    g = torch.Generator(device="cuda").manual_seed(5)
    total = 0.0
    for i in range(0, n, 4096):
        G[i:i + 4096] = torch.randn(4096, n, generator=g, device="cuda")
        total += G[i:i + 4096].double().square().sum().item()
    scale = 1.0 / (total ** 0.5 + 1e-7)
    out = torch.full_like(G, float("nan"))
    oz.orthogonalize(G, steps=0, out=out)
    for i in range(0, n, 4096):
        want = G[i:i + 4096].double() * scale
        # a rounding to bf16 is off by 2^-8 at most, the norm's sums in 64 bits by far less
        assert ((out[i:i + 4096].double() - want).abs() <= 2.0 ** -8 * (1 + 2.0 ** -20) * want.abs()).all()
