"""What the calls of a layer in 8 bits and of the clipping refuse, and what they
ask of a workspace: host checks, no GPU needed."""
import ctypes
import os
import time

import pytest
import torch
from torch.autograd import forward_ad

import fp64_gemm_emulation_ozii_amd as oz
from fp64_gemm_emulation_ozii_amd import ozgemm as L
from fp64_gemm_emulation_ozii_amd.layers import _dense, _lie_apart, _meet

E4M3 = torch.float8_e4m3fn


def eight(*shape):
    return torch.zeros(*shape).to(E4M3)


# ------------------------------------------------------------ tensors

def quantize(**change):
    return oz.quantize_blocks(**{"X": torch.zeros(10, 200), **change})


def linear(**change):
    a = dict(X=eight(10, 200), xs=torch.ones(10, 2), W=eight(300, 200), ws=torch.ones(3, 2),
             out=torch.zeros(10, 300, dtype=torch.bfloat16))
    return oz.scaled_linear(**{**a, **change})


def grads(**change):
    a = dict(dY=torch.zeros(10, 300), Xt=eight(200, 10), xts=torch.ones(200, 1), Wt=eight(200, 300),
             wts=torch.ones(2, 3), dX=torch.zeros(10, 200), dW=torch.zeros(300, 200))
    return oz.scaled_linear_grads(**{**a, **change})


def norm(**change):
    a = dict(X=torch.zeros(10, 200), weight=torch.ones(200), residual=torch.zeros(10, 200), out=torch.zeros(10, 200),
             H=torch.zeros(10, 200))
    return oz.rms_norm(**{**a, **change})


def norm8(**change):
    a = dict(X=torch.zeros(10, 200), weight=torch.ones(200), residual=torch.zeros(10, 200), H=torch.zeros(10, 200))
    return oz.rms_norm_quantized(**{**a, **change})


def norm_grads(**change):
    a = dict(dY=torch.zeros(10, 200), H=torch.zeros(10, 200), weight=torch.ones(200), dH=torch.zeros(10, 200),
             dX=torch.zeros(10, 200))
    return oz.rms_norm_grads(**{**a, **change})


def clip(**change):
    a = dict(grads=[torch.zeros(5), torch.zeros(2, 3)], max_norm=1.0, norm=torch.zeros((), dtype=torch.float64),
             out=[torch.zeros(5), torch.zeros(2, 3)])
    return oz.clip_gradients(**{**a, **change})


def clip_one(**change):
    return clip(**{k: [v, torch.zeros(2, 3)] if k in ("grads", "out") else v for k, v in change.items()})


ARGUMENTS = [(quantize, "X", (10, 200)), (linear, "xs", (10, 2)), (linear, "ws", (3, 2)), (grads, "dY", (10, 300)),
             (grads, "xts", (200, 1)), (grads, "wts", (2, 3)), (grads, "dX", (10, 200)), (grads, "dW", (300, 200)),
             (norm, "X", (10, 200)), (norm, "weight", (200,)), (norm, "residual", (10, 200)), (norm, "out", (10, 200)),
             (norm, "H", (10, 200)), (norm8, "X", (10, 200)), (norm8, "weight", (200,)), (norm8, "H", (10, 200)),
             (norm_grads, "dY", (10, 200)), (norm_grads, "H", (10, 200)), (norm_grads, "weight", (200,)),
             (norm_grads, "dH", (10, 200)), (norm_grads, "dX", (10, 200)), (clip_one, "grads", (5,)),
             (clip_one, "out", (5,))]


@pytest.mark.parametrize("call, name, shape", ARGUMENTS)
def test_what_carries_a_derivative_is_refused(call, name, shape):
    with pytest.raises(RuntimeError, match="no_grad"):
        call(**{name: torch.zeros(shape, requires_grad=True)})
    with torch.no_grad(), pytest.raises(ValueError, match="GPU"):  # the last check
        call(**{name: torch.zeros(shape, requires_grad=True)})
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(torch.zeros(shape), torch.ones(shape))
        with torch.no_grad(), pytest.raises(RuntimeError, match="forward-mode"):
            call(**{name: dual})


@pytest.mark.parametrize("call, change, error", [
    (quantize, {"X": torch.zeros(10, 200, dtype=torch.float64)}, TypeError),
    (quantize, {"X": torch.zeros(10)}, ValueError), (quantize, {"rows": 64}, ValueError),
    (quantize, {"dtype": torch.float16}, TypeError), (quantize, {"dtype": torch.float8_e4m3fnuz}, TypeError),
    (linear, {"X": torch.zeros(10, 200)}, TypeError), (linear, {"W": eight(300, 201)}, ValueError),
    (linear, {"xs": torch.ones(10, 3)}, ValueError), (linear, {"xs": torch.ones(1, 2)}, ValueError),
    (linear, {"ws": torch.ones(2, 2)}, ValueError), (linear, {"ws": torch.ones(3, 2, dtype=torch.float64)}, ValueError),
    (linear, {"out": torch.zeros(10, 301, dtype=torch.bfloat16)}, ValueError),
    (linear, {"out": torch.zeros(10, 300, dtype=torch.float64)}, ValueError),
    (linear, {"out": torch.zeros(300, 10, dtype=torch.bfloat16).t()}, ValueError),
    (linear, {"out": None, "out_dtype": torch.float64}, TypeError),
    (grads, {"dY": torch.zeros(10, 301)}, ValueError), (grads, {"dY": torch.zeros(10, 300, dtype=torch.float64)}, TypeError),
    (grads, {"Xt": eight(200, 11)}, ValueError), (grads, {"xts": torch.ones(2, 200)}, ValueError),
    (grads, {"Wt": eight(201, 300)}, ValueError), (grads, {"dX": None, "dx_dtype": torch.float64}, TypeError),
    (grads, {"dtype": torch.int8}, TypeError), (grads, {"dX": torch.zeros(10, 201)}, ValueError),
    (norm, {"X": torch.zeros(10, 200, dtype=torch.float64)}, TypeError), (norm, {"X": torch.zeros(200)}, ValueError),
    (norm, {"weight": torch.ones(199)}, ValueError), (norm, {"weight": torch.ones(200).half()}, TypeError),
    (norm, {"eps": -1.0}, ValueError), (norm, {"eps": float("nan")}, ValueError), (norm, {"residual": None}, ValueError),
    (norm, {"out": torch.zeros(10, 200).half()}, ValueError), (norm, {"H": torch.zeros(200, 10).t()}, ValueError),
    (norm8, {"dtype": torch.bfloat16}, TypeError),
    (norm_grads, {"eps": -1.0}, ValueError), (norm_grads, {"weight": torch.ones(10)}, ValueError),
    (clip, {"max_norm": -1.0}, ValueError), (clip, {"max_norm": float("nan")}, ValueError), (clip, {"eps": -1e-6}, ValueError),
    (clip, {"grads": [torch.zeros(5), torch.zeros(2, 3).int()]}, TypeError),
    (clip, {"grads": [torch.zeros(5), torch.zeros(2, 3).to_sparse()]}, TypeError),
    (clip, {"grads": torch.zeros(5)}, ValueError), (clip, {"out": [torch.zeros(5), torch.zeros(3, 2)]}, ValueError),
    (clip, {"out": [torch.zeros(5), torch.zeros(2, 3).half()]}, ValueError),
    (clip, {"norm": torch.zeros(())}, ValueError), (clip, {"norm": torch.zeros(2, dtype=torch.float64)}, ValueError),
    (clip, {"out": [torch.zeros(5), torch.zeros(1, 3).expand(2, 3)]}, ValueError),
    (clip, {"out": [torch._neg_view(torch.zeros(5)), torch.zeros(2, 3)]}, ValueError)])
def test_what_does_not_fit_is_refused(call, change, error):
    with pytest.raises(error) as e:
        call(**change)
    assert "GPU" not in str(e.value)


def test_overlapping_results_of_the_gradients_are_refused():
    both = torch.zeros(400, 300)
    with pytest.raises(ValueError, match="overlap"):
        grads(dX=both[:10, :200], dW=both[5:305, :200])


def test_dense_tensors():
    t = torch.zeros(4, 5, 6)
    for yes in (t, t.permute(2, 0, 1), t.transpose(0, 1), t[1], t[:, :, :6], torch.zeros(()), torch.zeros(3, 0), t[:1, :1, 2:4]):
        assert _dense(yes)
    for no in (t[:, :3], t[..., ::2], torch.zeros(1).expand(4), t[::2]):
        assert not _dense(no)


def test_no_tensors():
    for norm in (oz.gradient_norm([]), oz.clip_gradients([], 1.0)):
        assert norm.dtype == torch.float64 and norm.item() == 0


# ------------------------------------------------------------ C calls

A = 1 << 40  # addresses that no check looks behind
pytestmark = pytest.mark.skipif(not os.path.exists(L.LIB_PATH), reason="libozgemm.so not built")
no_gpu_only = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="made-up addresses, only where no kernel could run")


def at(k):
    return A + (k << 34)


def call(name, good, bad):
    """Every (argument number, value) of `bad` in the place of the good one gives that argument's error."""
    f = getattr(L.lib(), name)
    for i, value, *status in bad:
        args = list(good)
        args[i - 1] = value
        assert f(*args) == (status[0] if status else -i), (name, i, value)


@no_gpu_only
def test_quantize_arguments():
    big = L.OZGEMM_MAX_ROWS
    good = [L.OZGEMM_BF16, L.OZGEMM_E4M3, 1, 300, 200, at(0), 200, at(1), 208, at(2), 1, 300, at(3), 304, at(4), 1, 200, None]
    call("ozgemm_quantize_blocks", good, [
        (1, L.OZGEMM_F64), (1, 9), (2, L.OZGEMM_F16), (3, 0), (3, 64), (4, -1), (5, -1), (6, None), (7, 199), (9, 199),
        (10, None), (11, -1), (12, -1), (14, 299), (15, None), (16, -1), (17, -1), (4, big + 1, -14),
        (8, at(0) + 64), (10, at(0) + 64), (13, at(1) + 64), (13, at(2) + 64), (15, at(3) + 64), (10, at(1) + 64)])
    # scales of different blocks in one place
    call("ozgemm_quantize_blocks", good, [(11, 0), (11, 300), (12, 0, -11), (12, 299, -11), (16, 0), (16, 2), (17, 0, -16)])
    f = L.lib().ozgemm_quantize_blocks
    assert f(*(good[:7] + [None, 0, None, 0, 0, None, 0, None, 0, 0, None])) == -8  # neither result
    # 2^24 tiles and more
    assert f(L.OZGEMM_BF16, L.OZGEMM_E4M3, 1, big, big, at(0), big, 1 << 60, big, 1 << 50, 1, big, None, 0, None, 0, 0,
             None) == L.OZGEMM_RANGE
    assert f(L.OZGEMM_BF16, L.OZGEMM_E4M3, 1, 0, 5, None, 5, None, 0, None, 0, 0, None, 0, None, 0, 0, None) == 0


@no_gpu_only
def test_scaled_gemm_arguments():
    big = L.OZGEMM_MAX_ROWS
    good = [L.OZGEMM_E4M3, L.OZGEMM_E5M2, L.OZGEMM_BF16, 300, 20, 200, at(0), 208, at(1), 128, 2, 1, at(2), 208, at(3), 1, 20,
            at(4), 300, None, 0, None]
    call("ozgemm_scaled_gemm", good, [
        (1, L.OZGEMM_BF16), (2, 6), (3, L.OZGEMM_E4M3), (3, L.OZGEMM_F64), (4, -1), (5, -1), (6, -1), (7, None), (8, 199),
        (9, None), (10, 2), (11, -1), (12, -1), (13, None), (14, 199), (15, None), (16, -1), (17, -1), (18, None), (19, 299),
        (4, big + 1, -19), (6, big + 1, -8), (5, big + 1, L.OZGEMM_RANGE),
        (18, at(0) + 64), (18, at(1)), (18, at(2) + 64), (18, at(3) + 4),
        (8, 201, -20), (7, at(0) + 1, -20), (14, 215, -20)])  # copies need a workspace
    f, room = L.lib().ozgemm_scaled_gemm, L.ozgemm_scaled_gemm_workspace_bytes
    copies = room(300, 20, 200, at(0) + 1, 200, 128, 2, 1, at(2), 208, 1, 20)
    assert copies >= 300 * 208
    args = good[:6] + [at(0) + 1, 200] + good[8:19]
    assert f(*args, at(6), copies - 1, None) == L.OZGEMM_WORKSPACE_TOO_SMALL and f(*args, at(6) + 8, copies, None) == -20
    for empty in ([0, 20, 200], [300, 0, 200]):
        assert f(*good[:3], *empty, *good[6:]) == 0
    assert f(*good[:4], 1 << 24, *good[5:]) == L.OZGEMM_RANGE


def test_scaled_gemm_workspace():
    room = L.ozgemm_scaled_gemm_workspace_bytes
    assert room(300, 20, 200, 0, 208, 128, 2, 1, 0, 208, 1, 20) == 0  # in place
    assert room(-1, 20, 200, 0, 208, 128, 2, 1, 0, 208, 1, 20) == 0
    assert room(300, 20, 200, 0, 200, 128, 2, 1, 0, 208, 1, 20) >= 300 * 208
    assert room(300, 20, 200, 0, 208, 128, 2, 1, 8, 208, 1, 20) >= 20 * 208
    # leading dimensions past the 32-bit offsets of a tile are copied too
    assert room(300, 20, 200, 0, (1 << 22) + 16, 128, 2, 1, 0, 208, 1, 20) >= 300 * 208
    # large products turn over scales that lie row by row
    assert room(8192, 8192, 4096, 0, 4096, 128, 32, 1, 0, 4096, 32, 1) >= 8192 * 32 * 4
    assert room(8192, 8192, 4096, 0, 4096, 1, 32, 1, 0, 4096, 32, 1) >= 2 * 8192 * 32 * 4
    assert room(8192, 8192, 4096, 0, 4096, 128, 32, 1, 0, 4096, 1, 8192) == 0
    # few tiles with a long inner dimension are summed in parts
    assert room(128, 128, 1 << 20, 0, 1 << 20, 128, 1 << 13, 1, 0, 1 << 20, 1, 128) >= 2 * 128 * 128 * 4


def test_one_row_needs_no_leading_dimension():
    room = L.ozgemm_scaled_gemm_workspace_bytes
    for ld in (1531, 1540, (1 << 22) + 16, 1 << 30):  # never used
        assert room(8192, 1, 1531, 0, 1536, 128, 12, 1, 0, ld, 1, 1) == 0
        assert room(1, 1, 1531, 0, ld, 1, 12, 1, 0, 1531, 1, 1) == 0
    assert room(8192, 1, 1531, 0, 1536, 128, 12, 1, 8, 1536, 1, 1) == 1536  # off the 16-byte grid
    assert room(8192, 2, 1531, 0, 1536, 128, 12, 1, 0, 1531, 1, 2) == 2 * 1536  # two rows
    assert room(1, 0, 1531, 0, 1531, 1, 12, 1, 0, 1531, 1, 1) == 0 and room(0, 1, 1531, 0, 1531, 1, 12, 1, 0, 1531, 1, 1) == 0


ROOM = torch.zeros(4000)


def view(size, stride, at=0, dtype=torch.float32):
    return ROOM.view(dtype).as_strided(size, stride, at)


#: (two views of one storage, whether they have an entry in common)
PAIRS = [((view((10, 20), (40, 2)), view((10, 20), (40, 2))), True), ((view((10, 20), (40, 2)), view((10, 20), (40, 2), 1)), False),
         ((view((10, 20), (40, 2)), view((10, 20), (40, 2), 42)), True), ((view((10, 20), (40, 2)), view((20, 10), (2, 40), 80)), True),
         ((view((10, 5), (40, 1)), view((10, 5), (40, 1), 5)), False), ((view((10, 6), (40, 1)), view((10, 6), (40, 1), 5)), True),
         ((view((10, 5), (40, 1)), view((10, 5), (40, 1), 35)), False), ((view((10, 5), (40, 1)), view((10, 5), (40, 1), 36)), True),
         ((view((50,), (2,)), view((30,), (3,))), True), ((view((50,), (4,)), view((30,), (6,), 1)), False),
         ((view((50,), (4,)), view((30,), (6,), 2)), True), ((view((50,), (2,)), view((99,), (1,), 1)), True),
         ((view((50,), (2,)), view((1,), (1,), 97)), False), ((view((50,), (2,)), view((1,), (1,), 98)), True),
         ((view((3, 4, 5), (200, 10, 2)), view((3, 4, 5), (200, 10, 2), 40)), False),
         ((view((3, 4, 5), (200, 10, 2)), view((3, 4, 5), (200, 10, 2), 38)), True),
         ((view((50,), (2,)), view((20,), (4,), 2, torch.bfloat16)), False), ((view((50,), (2,)), view((20,), (4,), 1, torch.bfloat16)), True),
         ((view((50,), (2,)), view((10,), (1,), 3000)), False), ((view((0, 5), (2, 40)), view((10, 5), (2, 40))), False)]


@pytest.mark.parametrize("pair, shared", PAIRS)
def test_what_is_written_by_way_of_copies_must_lie_apart_too(pair, shared):
    # both orders, in place and into `out`; tensors that lie apart get as far as their device
    for a, b in (pair, pair[::-1]):
        dense = a.is_contiguous() and b.is_contiguous()
        assert not dense
        with pytest.raises(ValueError, match="share memory" if shared else "GPU only"):
            oz.clip_gradients([a, b], 1.0)
        with pytest.raises(ValueError, match="share memory" if shared else "GPU only"):
            oz.clip_gradients([torch.zeros_like(a), torch.zeros(3), torch.zeros_like(b)], 1.0, out=[a, torch.zeros(3), b])
    for a in pair:
        if a.numel() > 1 and not a.is_contiguous():
            with pytest.raises(ValueError, match="share memory"):
                oz.clip_gradients([a, a], 1.0)


def test_sharing_is_what_every_byte_says():
    def memory(t):
        at = torch.zeros((), dtype=torch.int64)
        for n, s in zip(t.shape, t.stride()):
            at = at[..., None] + torch.arange(n) * s
        at = at.reshape(-1) * t.element_size() + t.storage_offset() * t.element_size()
        return {x for k in range(t.element_size()) for x in (at + k).tolist()}

    rng = torch.Generator().manual_seed(3)

    def pick(*choices):
        return choices[int(torch.randint(len(choices), (), generator=rng))]

    met = 0
    for _ in range(600):
        pair = []
        for _ in range(2):
            dims = pick(1, 2, 2, 3)
            size, stride = [pick(1, 2, 3, 4, 7) for _ in range(dims)], [pick(1, 2, 3, 4, 6, 8, 12, 20, 40, 100) for _ in range(dims)]
            pair.append(view(size, stride, pick(0, 1, 2, 3, 7, 17, 50), pick(torch.float32, torch.bfloat16, torch.float64)))
        a, b = pair
        got = _meet(a, b)
        assert got == _meet(b, a) == bool(memory(a) & memory(b)), (a.shape, a.stride(), b.shape, b.stride())
        met += got
    assert 100 < met < 500


def test_slices_of_one_matrix_are_told_apart_quickly():
    w = torch.zeros(64, 4096)
    experts = torch.zeros(16, 512, 8)
    for parts in (list(w.chunk(2048, 1)), [experts[:, e] for e in range(512)], list(w[:, 1:].chunk(819, 1)),
                  [v for r in w.chunk(8) for v in r.chunk(256, 1)], [experts[..., k] for k in range(8)]):
        start = time.perf_counter()
        _lie_apart(parts, set(range(len(parts))))
        assert time.perf_counter() - start < 1  # (1000 of them pair by pair: 4 s)
        for twice in (parts[0], parts[len(parts) // 2], parts[-1]):
            with pytest.raises(ValueError, match="share memory"):
                _lie_apart([*parts, twice], {len(parts)})
            _lie_apart([*parts, twice], set())  # others see to it


def test_lists_of_views_are_apart_as_their_bytes_are():
    rng = torch.Generator().manual_seed(11)

    def pick(*choices):
        return choices[int(torch.randint(len(choices), (), generator=rng))]

    def memory(t):
        at = torch.zeros((), dtype=torch.int64)
        for n, s in zip(t.shape, t.stride()):
            at = at[..., None] + torch.arange(n) * s
        return set((at.reshape(-1) + t.storage_offset()).tolist())

    refused = 0
    for _ in range(400):
        step = pick(20, 40, 100)
        views = [view((pick(1, 2, 5), pick(1, 2, 3, 6)), (step if pick(0, 0, 0, 1) == 0 else pick(20, 30), pick(1, 1, 2)), pick(*range(0, 200, 3)))
                 for _ in range(pick(2, 3, 4))]
        bytes_of = [memory(v) for v in views]
        shared = any(a & b for k, a in enumerate(bytes_of) for b in bytes_of[:k])
        refused += shared
        if shared:
            with pytest.raises(ValueError, match="share memory"):
                _lie_apart(views, set(range(len(views))))
        else:
            _lie_apart(views, set(range(len(views))))
    assert 50 < refused < 350  # both among them


def test_sharing_that_takes_long_to_find_counts_as_shared():
    strides = [2 * p for p in (10007, 10009, 10037, 10039, 10061)]
    a = b = torch.empty(6000000).as_strided([60] * 5, strides)
    assert _meet(a, b)  # the same
    start = time.perf_counter()
    _meet(a, b.as_strided([60] * 5, strides, 1))
    assert time.perf_counter() - start < 5


def test_the_norm_is_not_written_over():
    norm = torch.zeros(10, dtype=torch.float64)
    out = [norm[::2]]
    for k, words in ((4, "share memory"), (5, "GPU only")):
        with pytest.raises(ValueError, match=words):
            oz.clip_gradients([torch.zeros(5, dtype=torch.float64)], 1.0, norm=norm[k], out=out)


@pytest.mark.parametrize("call", [lambda g: oz.gradient_norm(g), lambda g: oz.clip_gradients(g, 1.0),
                                  lambda g: oz.clip_gradients([torch.zeros(2)] * len(g), 1.0, out=g)])
@pytest.mark.parametrize("grads", [[None], [torch.zeros(2), None], [None, torch.zeros(2)], [1.0]])
def test_gradients_that_are_none(call, grads):
    # a parameter without a gradient has to be left out
    with pytest.raises(TypeError, match="tensor"):
        call(grads)


@no_gpu_only
def test_norm_arguments():
    big = L.OZGEMM_MAX_ROWS
    good = [L.OZGEMM_BF16, L.OZGEMM_E4M3, L.OZGEMM_F32, 30, 200, at(0), 200, at(1), 200, at(2), 1e-6, at(3), 200, at(4), 208,
            at(5), 1, 30, None]
    call("ozgemm_rms_norm", good, [
        (1, L.OZGEMM_F64), (2, L.OZGEMM_F16), (3, L.OZGEMM_F16), (4, -1), (5, -1), (6, None), (7, 199), (9, 199), (10, None),
        (11, -1.0), (11, float("nan")), (12, None), (13, 199), (14, None), (15, 199), (16, None), (17, -1), (18, -1),
        (4, big + 1, L.OZGEMM_RANGE), (12, at(0) + 8), (12, at(1) + 8), (12, at(2)), (14, at(0)), (14, at(3)), (16, at(4)),
        (16, at(0)), (12, at(0) + 2)])
    call("ozgemm_rms_norm", good, [(17, 0), (17, 30), (18, 29, -17), (18, 0, -17)])  # scales in one place
    assert L.lib().ozgemm_rms_norm(*good[:3], 0, *good[4:]) == 0
    good = [L.OZGEMM_F16, L.OZGEMM_F16, 30, 200, at(0), 200, at(1), 200, at(2), at(3), 200, 1e-6, at(4), 200, at(5), at(6),
            1 << 40, None]
    call("ozgemm_rms_norm_grads", good, [
        (1, L.OZGEMM_E4M3), (2, L.OZGEMM_BF16), (3, -1), (4, -1), (5, None), (6, 199), (7, None), (8, 199), (9, None),
        (11, 199), (12, -1.0), (13, None), (14, 199), (3, big + 1, L.OZGEMM_RANGE), (13, at(0) + 8), (13, at(2)),
        (15, at(4)), (15, at(2)), (16, None), (16, at(6) + 8), (17, 64, L.OZGEMM_WORKSPACE_TOO_SMALL)])


def test_norm_workspace():
    room = L.ozgemm_rms_norm_grads_workspace_bytes
    assert room(0, 100, 1) == 0 and room(100, 0, 1) == 0 and room(100, 100, 0) == 0
    assert room(100, 100, 1) >= 100 * 4
    assert room(100, 9000, 0) == 100 * 2 * 4  # long rows keep two numbers each
    assert room(1, 9000, 1) >= 9000 * 4 + 8


@no_gpu_only
def test_gradient_arguments():
    lib = L.lib()
    t, p, s = L._arrays([L.OZGEMM_F32, L.OZGEMM_BF16], [at(0), at(1)], [100, 50])
    need = lib.ozgemm_gradient_norm_workspace_bytes(2, t, s)
    assert need == 256
    n = lib.ozgemm_gradient_norm
    assert n(-1, t, p, s, at(5), at(6), need, None) == -1 and n(65537, t, p, s, at(5), at(6), need, None) == -1
    assert n(2, None, p, s, at(5), at(6), need, None) == -2 and n(2, t, None, s, at(5), at(6), need, None) == -3
    assert n(2, t, p, None, at(5), at(6), need, None) == -4 and n(2, t, p, s, None, at(6), need, None) == -5
    assert n(2, t, p, s, at(0) + 8, at(6), need, None) == -5 and n(2, t, p, s, at(5), None, need, None) == -6
    assert n(2, t, p, s, at(5), at(6) + 8, need, None) == -6
    assert n(2, t, p, s, at(5), at(6), need - 1, None) == L.OZGEMM_WORKSPACE_TOO_SMALL
    for types, sizes, arrays, status in (([9, 1], [1, 1], [at(0), at(1)], -2), ([1, 1], [-1, 1], [at(0), at(1)], -4),
                                         ([1, 1], [1 << 41, 1], [at(0), at(1)], -4)):
        assert n(2, *(x for x in (L._arrays(types, arrays, sizes)[k] for k in (0, 1, 2))), at(5), at(6), need, None) == status
    null = L._arrays([1, 1], [at(0), at(1)], [4, 4])
    null[1][1] = None
    assert n(2, *null, at(5), at(6), need, None) == -3
    c = lib.ozgemm_clip_gradients

    def clips(ins, outs, norm=at(5), most=1.0, eps=0.0):
        t, p, s = L._arrays([L.OZGEMM_F32] * len(ins), ins, [100] * len(ins))
        return c(len(ins), t, p, s, (ctypes.c_void_p * len(ins))(*outs) if outs else None, norm, most, eps, None)

    assert clips([at(0)], None) == -5 and clips([at(0)], [None]) == -5 and clips([at(0)], [at(1)], None) == -6
    assert clips([at(0)], [at(0)], most=-1.0) == -7 and clips([at(0)], [at(0)], most=float("nan")) == -7
    assert clips([at(0)], [at(0)], eps=-1.0) == -8
    assert clips([at(0), at(0)], [at(0), at(0)]) == -5                  # the same array twice
    assert clips([at(0), at(0) + 200], [at(0), at(0) + 200]) == -5      # halves that overlap
    assert clips([at(0), at(1)], [at(1), at(0)]) == -5                  # each other's
    assert clips([at(0), at(1)], [at(0), at(0) + 399]) == -5            # a byte of what is read
    assert clips([at(0)], [at(0) + 4]) == -5                            # its own, moved
    assert clips([at(0)], [at(5) - 396]) == -5                          # the norm


def test_gradient_workspace_counts_chunks():
    room = L.ozgemm_gradient_norm_workspace_bytes
    assert room([], []) == 256 and room([L.OZGEMM_F32], [0]) == 256
    assert room([L.OZGEMM_F32], [16384 * 100]) == 1024  # 100 sums of 8 bytes, up to a multiple of 256
    assert room([L.OZGEMM_BF16, L.OZGEMM_F64], [32768 * 31 + 1, 8192]) == 512
    assert room([7], [5]) == 0 and room([L.OZGEMM_F32], [-1]) == 0
