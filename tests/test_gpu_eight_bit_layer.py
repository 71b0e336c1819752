"""A layer in 8 bits as it is used: forward, gradients, clipping and update one
after the other against 64 bits; serving one token; captured graphs, streams
and host threads.  Tolerances: test_gpu_blocks.py, test_gpu_norm.py,
test_gpu_clip.py and test_gpu_ortho.py."""
import math
import threading

import pytest
import torch

import fp64_gemm_emulation_ozii_amd as oz
from blocks_util import blocks, same, value
from fp64_gemm_emulation_ozii_amd import ozgemm as L
from test_gpu_blocks import check_product
from test_gpu_ortho import plain, rel, tolerance

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
SIZES = [(40, 200, 136), (300, 513, 260), (1000, 1024, 640)]


class Layer:
    def __init__(self, n, q, m, seed, t=torch.bfloat16):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*s):
            return torch.randn(*s, generator=g, device="cuda")

        self.X, self.R = normal(n, q).to(t), normal(n, q).to(t)
        self.gain = (1 + 0.1 * normal(q)).to(t)
        self.W = (normal(m, q) / math.sqrt(q)).to(t)
        self.dY, self.dH = (normal(n, m) * 0.1).to(t), (normal(n, q) * 0.1).to(t)
        self.blocks = oz.quantize_blocks(self.W, rows=128, both=True)

    def step(self, clip_to=0.5):
        w, ws, wt, wts = self.blocks
        Z, H = oz.rms_norm(self.X, self.gain, self.R)
        z, zs, zt, zts = oz.quantize_blocks(Z, both=True)
        Y = oz.scaled_linear(z, zs, w, ws)
        dZ, dW = oz.scaled_linear_grads(self.dY, zt, zts, wt, wts, dw_dtype=torch.float32)
        dX, dgain = oz.rms_norm_grads(dZ, H, self.gain, self.dH)
        clipped = [torch.empty_like(dW), torch.empty_like(dgain)]
        norm = oz.clip_gradients([dW, dgain], clip_to, out=clipped)
        return {"Z": Z, "H": H, "Y": Y, "dZ": dZ, "dW": dW, "dX": dX, "dgain": dgain, "norm": norm, "dW clipped": clipped[0],
                "dgain clipped": clipped[1]}


@pytest.mark.parametrize("n, q, m", SIZES)
def test_a_training_step(n, q, m):
    layer = Layer(n, q, m, n)
    got = layer.step()
    w, ws, wt, wts = layer.blocks
    H = layer.X + layer.R
    assert torch.equal(got["H"], H)
    h = H.double()
    r = 1 / torch.sqrt(h.square().mean(1, keepdim=True) + 1e-6)
    want = h * r * layer.gain.double()
    assert ((got["Z"].double() - want).abs() <= want.abs() * (2.0 ** -8 + 1e-12)).all()
    z, zs = blocks(got["Z"], 1, E4M3)
    check_product(got["Y"], z, zs, w, ws, 128, n <= 16)
    zt, zts = blocks(got["Z"].t(), 1, E4M3)
    y, ys = blocks(layer.dY, 1, E4M3)
    check_product(got["dZ"], y, ys, wt, wts, 128, n <= 16)
    y, ys = blocks(layer.dY.t(), 1, E4M3)
    check_product(got["dW"], y, ys, zt, zts, 1, True)
    g = got["dZ"].double() * layer.gain.double()
    a, b, c = r * g, h * r ** 3 * (g * h).mean(1, keepdim=True), layer.dH.double()
    tol = 6.06 * 2.0 ** -24 * (a.abs() + b.abs() + c.abs()) + 2.0 ** -8 * (a - b + c).abs()
    assert ((got["dX"].double() - (a - b + c)).abs() <= tol).all()
    terms = got["dZ"].double() * h * r
    tol = (n + 2) * 2.0 ** -24 * 1.01 * terms.abs().sum(0) + 2.0 ** -8 * terms.sum(0).abs()
    assert ((got["dgain"].double() - terms.sum(0)).abs() <= tol).all()
    norm = math.sqrt(got["dW"].double().square().sum().item() + got["dgain"].double().square().sum().item())
    assert abs(got["norm"].item() - norm) <= 1e-13 * norm and norm > 0.5
    for name in ("dW", "dgain"):
        want = got[name].double() * (0.5 / (norm + 1e-6))
        half = torch.finfo(got[name].dtype).eps / 2 * (name == "dgain")
        assert ((got[name + " clipped"].double() - want).abs() <= want.abs() * (2.01 * 2.0 ** -24 + half)).all()
    O = oz.orthogonalize(got["dW clipped"])
    want = plain(got["dW clipped"])
    assert rel(O, want) <= tolerance(got["dW clipped"], want)


@pytest.mark.parametrize("n", [1, 3, 16, 17, 64, 100])
def test_serving(n):
    # the residual stream stays where it is; two layers one after the other
    layer, first = Layer(n, 1024, 1024, n), None
    w, ws, _, _ = layer.blocks
    stream, out = layer.R.clone(), layer.X
    for _ in range(2):
        z, zs, H = oz.rms_norm_quantized(out, layer.gain, stream, H=stream)
        assert H is stream
        if first is None:
            want = layer.X + layer.R
            assert torch.equal(stream, want)
            h = want.double()
            v, s = blocks(h / torch.sqrt(h.square().mean(1, keepdim=True) + 1e-6) * layer.gain.double(), 1, E4M3)
            assert same(z, v) and same(zs, s)
        first = out = oz.scaled_linear(z, zs, w, ws)
        check_product(out, z, zs, w, ws, 128, n <= 16)


@pytest.mark.parametrize("n, q, m", SIZES[:2])
def test_a_captured_step(n, q, m):
    layer, other = Layer(n, q, m, 1), Layer(n, q, m, 2)
    layer.step()  # what is loaded and allowed on first use is no part of the graph
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = layer.step()
    sources = [Layer(n, q, m, s) for s in (3, 4, 5)]
    for k, source in enumerate(sources + sources[:1]):
        for name in ("X", "R", "dY", "dH"):
            getattr(layer, name).copy_(getattr(source, name))
        graph.replay()
        got = {name: t.clone() for name, t in held.items()}
        if k % 2 == 0:
            other.step()  # eager work and a wait between replays
            torch.cuda.synchronize()
        want = layer.step()
        for name in want:
            assert torch.equal(got[name], want[name]), (k, name)


def test_products_in_parts_and_copies_in_a_graph():
    # what passes through a workspace: parts of the inner dimension, operands off the 16-byte grid, scales row by row
    g = torch.Generator(device="cuda").manual_seed(3)
    x, xs = oz.quantize_blocks(torch.randn(130, 8200, generator=g, device="cuda"))
    w, ws = oz.quantize_blocks(torch.randn(200, 8200, generator=g, device="cuda"), rows=128)
    x = torch.empty(130, 8203, device="cuda").to(E4M3)[:, 1:8201].copy_(x)
    xs = xs.contiguous()
    assert L.ozgemm_scaled_gemm_workspace_bytes(200, 130, 8200, w, w.stride(0), 128, 65, 1, x, x.stride(0), 65, 1) > (
        2 * 4 * 200 * 130 + 130 * 8208)
    want = oz.scaled_linear(x, xs, w, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = oz.scaled_linear(x, xs, w, ws)
    for k in range(3):
        held.zero_()
        graph.replay()
        assert torch.equal(held, want)
        xs.mul_(2)
        want = oz.scaled_linear(x, xs, w, ws)
        torch.cuda.synchronize()


def test_on_another_stream():
    layer = Layer(300, 513, 260, 7)
    want = layer.step()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    busy = torch.randn(4096, 4096, device="cuda")
    for _ in range(20):  # the default stream is busy meanwhile
        busy = busy @ busy * 1e-2
    with torch.cuda.stream(stream):
        got = layer.step()
    stream.synchronize()
    assert all(torch.equal(got[name], want[name]) for name in want)
    torch.cuda.synchronize()


def test_calls_from_several_host_threads():
    layers = [Layer(n, q, m, 20 + k) for k, (n, q, m) in enumerate(SIZES + [(17, 9000, 300)])]
    wants = [layer.step() for layer in layers]
    torch.cuda.synchronize()
    streams, gots, errors = [torch.cuda.Stream() for _ in layers], [[] for _ in layers], []

    def work(k):
        try:
            with torch.cuda.stream(streams[k]):
                for _ in range(5):
                    gots[k].append(layers[k].step())
        except Exception as e:  # (shown by the main thread)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(len(layers))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for want, got in zip(wants, gots):
        assert len(got) == 5 and all(torch.equal(g[name], want[name]) for g in got for name in want)


def test_the_same_call_gives_the_same_bits():
    layer = Layer(700, 1100, 900, 5)
    first = layer.step()
    for _ in range(3):
        again = layer.step()
        assert all(torch.equal(first[name], again[name]) for name in first)


def test_products_whose_stream_is_given_need_no_current_one():
    x, xs = oz.quantize_blocks(torch.ones(100, 300, device="cuda"))
    w, ws = oz.quantize_blocks(torch.ones(200, 300, device="cuda"), rows=128)
    out, stream = torch.zeros(100, 200, device="cuda"), torch.cuda.Stream()
    torch.cuda.synchronize()
    L.ozgemm_scaled_gemm(L.OZGEMM_E4M3, L.OZGEMM_E4M3, L.OZGEMM_F32, 200, 100, 300, w, w.stride(0), ws, 128, 3, 1, x,
                         x.stride(0), xs, *xs.stride(), out, 200, stream=stream)
    stream.synchronize()
    assert (out == 300).all() and value(x, xs, 1).sum() == 30000


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("n, q, m", [(5000, 1000, 4100), (4097, 2049, 3333), (2900, 130, 2900)])
def test_whole_numbers_over_large_tiles(n, q, m, rows):
    # several rounds of 256 x 256 tiles, ragged in every size, with scales that lie row by row; exact in float32
    g = torch.Generator(device="cuda").manual_seed(n + rows)
    k = torch.randint(0, 16, (n, q), generator=g, device="cuda")
    X = (k == 0).float() - (k == 1).float()
    W = (torch.randint(0, 2, (m, q), generator=g, device="cuda") * 2 - 1).float()
    x, xs = oz.quantize_blocks(X)
    w, ws = oz.quantize_blocks(W, rows=rows)
    want = X.double() @ W.double().T.contiguous()
    for a, b in ((xs, ws), (xs.contiguous(), ws.contiguous())):
        for t in (torch.float32, torch.bfloat16):
            assert torch.equal(oz.scaled_linear(x, a, w, b, out_dtype=t), want.to(t))


def test_offsets_past_32_bits():
    # 1024 rows over and over: every piece of a result is the first one's, bit by bit
    times, rows, q, m = 1075, 1024, 4096, 2100
    n = times * rows
    g = torch.Generator(device="cuda").manual_seed(6)
    base = torch.randn(rows, q, generator=g, device="cuda").bfloat16()
    X = base.repeat(times, 1)
    assert X.numel() > 2 ** 32

    def again(t, first, dim=0):
        t = t.view(torch.uint8) if t.dtype == E4M3 else t
        first = first.view(torch.uint8) if first.dtype == E4M3 else first
        size = first.shape[dim]
        return all(torch.equal(t.narrow(dim, k * size, size), first) for k in range(t.shape[dim] // size))

    V, S, Vt, St = oz.quantize_blocks(X, both=True)
    v, s, vt, st = oz.quantize_blocks(base, both=True)
    assert again(V, v) and again(S, s) and again(Vt, vt, 1) and again(St, st, 1)
    del Vt, St
    w, ws = oz.quantize_blocks(torch.randn(m, q, generator=g, device="cuda"), rows=128)
    Y = oz.scaled_linear(V, S, w, ws)
    assert Y.numel() * 2 > 2 ** 32
    check_product(Y[:rows], v, s, w, ws, 128, False)
    assert again(Y, Y[:rows])
    del Y
    few = oz.scaled_linear(v[:3], s[:3], V, S)  # as weights
    check_product(few[:, :rows], v[:3], s[:3], v, s, 1, True)
    assert again(few, few[:, :rows], 1)
    del V, S, few
    gain = torch.randn(q, generator=g, device="cuda")
    V, S, _ = oz.rms_norm_quantized(X, gain)
    v, s, _ = oz.rms_norm_quantized(base, gain)
    assert again(V, v) and again(S, s)
    del V, S
    dX, _ = oz.rms_norm_grads(X, X, gain)
    assert again(dX, oz.rms_norm_grads(base, base, gain)[0])
    norm = oz.clip_gradients([X], 1.0, out=[dX])
    want = math.sqrt(times * base.double().square().sum().item())
    assert abs(norm.item() - want) <= 1e-13 * want
    assert again(dX, dX[:rows])
    want = base.double() * (1 / (want + 1e-6))
    assert ((dX[:rows].double() - want).abs() <= want.abs() * (2.0 ** -8 + 2.01 * 2.0 ** -24)).all()
    del X, dX
    torch.cuda.empty_cache()


def test_operands_and_scales_that_lie_otherwise():
    g = torch.Generator(device="cuda").manual_seed(9)

    def eight(*s):
        return torch.randn(*s, generator=g, device="cuda").to(E4M3)

    def same_as_contiguous(x, xs, w, ws, **kw):
        want = oz.scaled_linear(x.contiguous(), xs.contiguous(), w.contiguous(), ws.contiguous(), **kw)
        assert torch.equal(oz.scaled_linear(x, xs, w, ws, **kw), want)

    xs, ws = (torch.rand(n, 5, generator=g, device="cuda") + 0.5 for n in (300, 4))
    x, w = eight(600, 300).t(), eight(400, 600)
    for t in (torch.float32, torch.bfloat16):
        same_as_contiguous(x, xs, w, ws, out_dtype=t)
        same_as_contiguous(x, xs, w[:1].expand(400, 600), ws, out_dtype=t)  # one row of weights for all
        same_as_contiguous(x, xs[:1, :1].expand(300, 5), w, ws, out_dtype=t)  # one scale for all
        same_as_contiguous(x, torch.rand(5, 300, generator=g, device="cuda").t(), w, ws[:, :1].expand(4, 5), out_dtype=t)
        same_as_contiguous(x[:2], xs[:2], w, xs[0].expand(400, 5), out_dtype=t)
    big, one = eight(4000, 608)[:, :600], torch.full((1, 1), 0.25, device="cuda").expand(4000, 5)
    same_as_contiguous(big, one, big, one)  # tiles whose scales are turned over first
    same_as_contiguous(big, torch.rand(4000, 10, generator=g, device="cuda")[:, ::2], big, one)


def test_serving_in_inference_mode():
    with torch.inference_mode():
        layer = Layer(5, 512, 512, 3)
        z, zs, H = oz.rms_norm_quantized(layer.X, layer.gain, layer.R, H=layer.R)
        assert H is layer.R
        check_product(oz.scaled_linear(z, zs, *layer.blocks[:2]), z, zs, *layer.blocks[:2], 128, True)
        grads = [torch.ones(100, device="cuda")]
        assert oz.clip_gradients(grads, 5.0).item() == 10 and (grads[0] - 0.5).abs().max() <= 1e-6
