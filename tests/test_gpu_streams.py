"""The grouped products and the orthogonalisation on a stream that is not torch's current one."""
import pytest
import torch

import fp64_gemm_emulation_ozii_amd as oz
from fp64_gemm_emulation_ozii_amd import ozgemm as L

pytestmark = pytest.mark.gpu


def gemm():
    g = torch.Generator(device="cuda").manual_seed(1)
    n, m, q = 100000, 50, 70
    X, W = torch.randn(n, q, generator=g, device="cuda"), torch.randn(2, m, q, generator=g, device="cuda")
    off = torch.tensor([0, 33, n], dtype=torch.int32, device="cuda")
    sizes = (L.OZGEMM_F32, 2, m, n, q, 1, W, q, m * q, X, q)
    need = L.ozgemm_grouped_gemm_workspace_bytes(*sizes)

    def call(out, stream):
        L.ozgemm_grouped_gemm(L.OZGEMM_F32, L.OZGEMM_F32, *sizes[1:], off, out, m, stream=stream)

    return call, need, oz.grouped_linear(X, W, off)


def outer():
    g = torch.Generator(device="cuda").manual_seed(2)
    n, m, q = 20000, 500, 520
    X, dY = torch.randn(n, q, generator=g, device="cuda"), torch.randn(n, m, generator=g, device="cuda")
    off = torch.tensor([0, 9000, n], dtype=torch.int32, device="cuda")
    sizes = (L.OZGEMM_F32, 2, q, m, n, X, q, dY, m)
    need = L.ozgemm_grouped_outer_workspace_bytes(*sizes)

    def call(out, stream):
        L.ozgemm_grouped_outer(L.OZGEMM_F32, L.OZGEMM_F32, *sizes[1:], off, out, q, m * q, stream=stream)

    return call, need, oz.grouped_linear_grads(dY, X, torch.zeros(2, m, q, device="cuda"), off)[1]


def ortho():
    g = torch.Generator(device="cuda").manual_seed(3)
    G = torch.randn(2, 300, 700, generator=g, device="cuda")
    need = L.ozgemm_orthogonalize_workspace_bytes(L.OZGEMM_F32, 2, 700, 300, 14)
    co = [3.4445, -4.7750, 2.0315] * 5

    def call(out, stream):
        L.ozgemm_orthogonalize(L.OZGEMM_F32, 2, 700, 300, G, 700, 700 * 300, 5, co, 1e-7, 14, out, 700, 700 * 300,
                               stream=stream)

    return call, need, oz.orthogonalize(G)


@pytest.mark.parametrize("what", [gemm, outer, ortho])
def test_work_on_another_stream_keeps_its_workspace(what):
    call, need, want = what()
    assert need > 0
    busy = torch.randn(4096, 4096, device="cuda")
    other = torch.cuda.Stream()
    for stream, current in ((other, torch.cuda.current_stream()), (other.cuda_stream, torch.cuda.current_stream()),
                            (torch.cuda.default_stream(), other), (0, other)):
        runs_on = other if current != other else torch.cuda.default_stream()
        out = torch.full_like(want, float("nan"))
        torch.cuda.synchronize()
        with torch.cuda.stream(runs_on):
            for _ in range(8):  # the call waits for these, some ms
                busy @ busy
        with torch.cuda.stream(current):
            # blocks that were used on the current stream before, and that it uses again as soon as the call returns
            for _ in range(3):
                torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
            call(out, stream)
            taken = [torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(3)]
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert all((t == 0xFF).all() for t in taken)
