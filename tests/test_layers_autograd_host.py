"""What the tensor calls do about derivatives, which they do not record.  The
checks come before the tensors' device is looked at, so they need no GPU."""
import pytest
import torch
from torch.autograd import forward_ad

import fp64_gemm_emulation_ozii_amd as oz


def linear(**change):
    a = dict(X=torch.zeros(10, 8), W=torch.zeros(3, 4, 8), offsets=torch.zeros(4, dtype=torch.int32), out=torch.zeros(10, 4))
    a.update(change)
    return oz.grouped_linear(**a)


def grads(**change):
    a = dict(dY=torch.zeros(10, 4), X=torch.zeros(10, 8), W=torch.zeros(3, 4, 8),
             offsets=torch.zeros(4, dtype=torch.int32), dX=torch.zeros(10, 8), dW=torch.zeros(3, 4, 8))
    a.update(change)
    return oz.grouped_linear_grads(**a)


def ortho(**change):
    return oz.orthogonalize(**{"G": torch.zeros(6, 8), "out": torch.zeros(6, 8), **change})


ARGUMENTS = [(linear, "X", (10, 8)), (linear, "W", (3, 4, 8)), (linear, "out", (10, 4)),
             (grads, "dY", (10, 4)), (grads, "X", (10, 8)), (grads, "W", (3, 4, 8)), (grads, "dX", (10, 8)),
             (grads, "dW", (3, 4, 8)), (ortho, "G", (6, 8)), (ortho, "out", (6, 8))]


@pytest.mark.parametrize("call, name, shape", ARGUMENTS)
def test_a_tangent_is_refused(call, name, shape):
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(torch.zeros(shape), torch.ones(shape))
        assert not dual.requires_grad
        for mode in (torch.enable_grad(), torch.no_grad()):
            with mode, pytest.raises(RuntimeError, match="forward-mode"):
                call(**{name: dual})
            with mode, pytest.raises(ValueError, match="GPU"):  # the next check: the primal passes
                call(**{name: forward_ad.unpack_dual(dual).primal})


@pytest.mark.parametrize("call, name, shape", ARGUMENTS)
def test_a_tensor_that_requires_a_gradient_is_refused(call, name, shape):
    t = torch.zeros(shape, requires_grad=True)
    with pytest.raises(RuntimeError, match="no_grad"):
        call(**{name: t})
    with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
        call(**{name: t})


@pytest.fixture
def no_library(monkeypatch):
    # the calls as far as the library's, which stand-ins take: tensors on the CPU get there
    import contextlib

    from fp64_gemm_emulation_ozii_amd import layers
    called = []
    monkeypatch.setattr(layers, "_on_device", lambda device: contextlib.nullcontext())
    for name in ("ozgemm_grouped_gemm", "ozgemm_grouped_outer", "ozgemm_orthogonalize"):
        monkeypatch.setattr(layers.L, name, lambda *a, name=name: called.append(name))
    return called


@pytest.mark.parametrize("call, name, shape", [a for a in ARGUMENTS if a[1] in ("out", "dX", "dW")])
def test_a_graph_that_saved_a_result_learns_that_it_was_written(no_library, call, name, shape):
    w = torch.ones(shape, requires_grad=True)
    result = torch.ones(shape)
    y = (w * result).sum()  # saves `result` for w's gradient
    call(**{name: result})
    assert no_library
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_in_place_and_in_inference_mode(no_library):
    G = torch.zeros(6, 8)
    before = G._version
    assert ortho(G=G, out=G) is G and G._version > before
    with torch.inference_mode():
        linear()
        grads()
        ortho()
    assert len(no_library) == 5
