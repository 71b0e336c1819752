"""Where the bindings of the grouped products and the orthogonalisation take a
workspace that the caller did not give: from torch's allocator, on the stream
that the call runs on.  The library and torch's streams are stand-ins here, so
this needs no GPU."""
import contextlib

import pytest
import torch

from fp64_gemm_emulation_ozii_amd import ozgemm as L

CURRENT, OTHER, NEED = 0x7000, 0x9000, 4096


class Stream:
    def __init__(self, handle, device=None):
        self.cuda_stream = handle


class Library:
    """Answers like the library: a call without a workspace is refused, one with it runs."""

    def __init__(self):
        self.calls = []  # (stream, workspace) of the calls that ran

    def ozgemm_grouped_gemm_workspace_bytes(self, *a):
        return NEED

    ozgemm_grouped_outer_workspace_bytes = ozgemm_orthogonalize_workspace_bytes = ozgemm_grouped_gemm_workspace_bytes

    def _run(self, refusal, args):
        workspace, nbytes, stream = args[-3:]
        if workspace is None:
            return refusal
        assert nbytes == NEED
        self.calls.append((stream, workspace))
        return 0

    def ozgemm_grouped_gemm(self, *a):
        return self._run(-16, a)

    def ozgemm_grouped_outer(self, *a):
        return self._run(-15, a)

    def ozgemm_orthogonalize(self, *a):
        return self._run(-15, a)


@pytest.fixture
def world(monkeypatch):
    now, taken, lib = [CURRENT], {}, Library()

    @contextlib.contextmanager
    def use(stream):
        now.append(stream.cuda_stream)
        yield
        now.pop()

    empty = torch.empty

    def tell(*a, **k):
        k.pop("device", None)
        t = empty(*a, **k)
        taken[t.data_ptr()] = now[-1]  # the stream whose pool the block came from
        return t

    monkeypatch.setattr(L, "lib", lambda: lib)
    monkeypatch.setattr(L, "_current_stream", lambda: now[-1])
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream(0))
    monkeypatch.setattr(torch, "empty", tell)
    return taken, lib


def gemm(**how):
    return L.ozgemm_grouped_gemm(L.OZGEMM_F32, L.OZGEMM_F32, 1, 4, 4, 4, 1, 1 << 40, 4, 16, 1 << 41, 4, 1 << 42, 1 << 43,
                                 4, **how)


def outer(**how):
    return L.ozgemm_grouped_outer(L.OZGEMM_F32, L.OZGEMM_F32, 1, 4, 4, 4, 1 << 40, 4, 1 << 41, 4, 1 << 42, 1 << 43, 4, 16,
                                  **how)


def ortho(**how):
    return L.ozgemm_orthogonalize(L.OZGEMM_F32, 1, 4, 4, 1 << 40, 4, 16, 1, [1.0, 0.0, 0.0], 0.0, 14, 1 << 41, 4, 16, **how)


CALLS = [gemm, outer, ortho]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("stream, handle", [(None, CURRENT), (CURRENT, CURRENT), (Stream(CURRENT), CURRENT),
                                            (OTHER, OTHER), (Stream(OTHER), OTHER), (0, 0), (Stream(0), 0)])
def test_the_workspace_belongs_to_the_stream_of_the_call(world, call, stream, handle):
    taken, lib = world
    assert call(stream=stream) == 0
    (on, workspace), = lib.calls
    assert on == handle and taken[workspace] == handle


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("handle", [1, 2])  # hipStreamLegacy, hipStreamPerThread
def test_a_handle_that_is_no_stream_needs_a_workspace(world, call, handle):
    taken, lib = world
    with pytest.raises(ValueError, match="workspace"):
        call(stream=handle)
    assert not lib.calls and not taken
    given = torch.zeros(NEED, dtype=torch.uint8)
    assert call(stream=handle, workspace=given) == 0
    assert lib.calls == [(handle, given.data_ptr())]
