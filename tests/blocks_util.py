"""Blocks of 128 in 8 bits, from their definition in 64 bits."""
import torch

#: (largest value, bits after the leading one, smallest normal value)
EIGHT = {torch.float8_e4m3fn: (448.0, 3, 2.0 ** -6), torch.float8_e5m2: (57344.0, 2, 2.0 ** -14)}


def power_below(v):
    """The largest power of two that is not above v > 0 (exact)."""
    m, e = torch.frexp(v)
    return v / (2 * m)


def blocks(x, rows, dtype):
    """(values as float64, scales as float64) of x [n, q]; Inf and NaN become NaN."""
    top, bits, least = EIGHT[dtype]
    x = x.double()
    n, q = x.shape
    finite = torch.where(torch.isfinite(x), x, 0.0)
    padded = torch.zeros(-(-n // rows) * rows, -(-q // 128) * 128, dtype=torch.float64, device=x.device)
    padded[:n, :q] = finite
    most = padded.view(-(-n // rows), rows, -1, 128).abs().amax((1, 3))
    some = torch.where(most == 0, 1.0, most)
    scale = power_below(some / top)
    scale = torch.where(scale * top < some, 2 * scale, scale)
    scale = torch.where(most == 0, 1.0, scale.clamp(min=2.0 ** -126))
    per = spread(scale, n, q, rows)
    v = finite / per
    step = power_below(v.abs().clamp(min=least)) * 2.0 ** -bits
    v = torch.round(v / step) * step
    return torch.where(torch.isfinite(x), v, torch.nan), scale


def spread(scale, n, q, rows):
    return scale.double().repeat_interleave(rows, 0)[:n].repeat_interleave(128, 1)[:, :q]


def value(v, s, rows):
    return v.double() * spread(s, *v.shape, rows)


def same(a, b):
    """Equal, NaN in the same places."""
    a, b = a.double(), b.double()
    return a.shape == b.shape and bool(((a == b) | (a.isnan() & b.isnan())).all())
