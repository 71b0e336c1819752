"""Measured cases of the products of expert layers and of the Newton-Schulz
orthogonalisation: their inputs, their plain forms in elementary torch
operations, their definitions in 64 bits, and what each cannot do without.

Where ``own`` is false ``run`` computes the plain form, where it is true it
calls this package.
"""
import math

import numpy as np
import torch

own = False

#: Muon's quintic: X <- a X + (b A + c A^2) X with A = X X^T, five times.
QUINTIC = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-7

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "f64": torch.float64}
BYTES = {"bf16": 2, "f16": 2, "f32": 4, "f64": 8}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    def grouped(name, op, dtype, rows, groups, q, m, spread, weights="mq"):
        return {"name": name, "op": op, "dtype": dtype, "rows": rows, "groups": groups, "q": q, "m": m,
                "spread": spread, "weights": weights}

    def ortho(name, dtype, batch, r, c):
        return {"name": name, "op": "orthogonalize", "dtype": dtype, "batch": batch, "r": r, "c": c}

    return [
        # serving: one token that its router sent to eight of 64 experts
        grouped("decode, one token", "product", "bf16", 8, 64, 2048, 1024, 0.5),
        # serving: 64 tokens in flight, four experts each; every expert's weights are read for a few rows
        grouped("decode, 64 tokens", "product", "bf16", 256, 32, 2048, 4096, 0.5),
        # serving: prompts of 4096 tokens, four experts each
        grouped("prompt", "product", "bf16", 16384, 32, 2048, 4096, 0.5),
        # ragged in every size, with weights that lie inner dimension first
        grouped("odd sizes", "product", "f16", 5003, 13, 1001, 1531, 0.7, "qm"),
        # a layer kept in single precision
        grouped("prompt, f32", "product", "f32", 8192, 16, 2048, 2048, 0.5),
        # training: the product of a layer and both its gradients
        grouped("training step", "step", "bf16", 32768, 16, 2048, 4096, 0.5),
        # the same in single precision, as a run that a bf16 one is checked against
        grouped("training step, f32", "step", "f32", 8192, 8, 1024, 2048, 0.5),
        # the optimiser: updates of four layers of one shape
        ortho("update, four layers", "bf16", 4, 1024, 4096),
        # the optimiser: one large matrix
        ortho("update, large", "bf16", 1, 4096, 8192),
        # updates held in single precision
        ortho("update, f32", "f32", 2, 2048, 2048),
        # many small and odd matrices, taller than wide
        ortho("update, small", "f32", 6, 517, 133),
        # the polar factor's polynomial in double precision
        ortho("update, f64", "f64", 1, 2048, 2048),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]: odd, a multiple of 8, or a multiple of 64."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    step = rng.choice((1, 8, 64))
    return int(min(hi, max(lo, step * round(v / step))))


def draw(rng):
    op = rng.choice(("product", "product", "step", "orthogonalize", "orthogonalize"))
    if op == "orthogonalize":
        dtype = rng.choice(("bf16", "bf16", "f16", "f32", "f32", "f64"))
        most = 2e11 if dtype == "f64" else 1.5e12
        while True:
            case = {"op": op, "dtype": dtype, "batch": _log(rng, 1, 16), "r": _log(rng, 16, 4096), "c": _log(rng, 16, 4096)}
            if work(case)["flops"] <= most:
                return case
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    while True:
        rows = _log(rng, 1, 32768) if op == "product" else _log(rng, 64, 32768)
        case = {"op": op, "dtype": dtype, "rows": rows, "groups": _log(rng, 1, 64), "q": _log(rng, 32, 4096),
                "m": _log(rng, 32, 4096), "spread": round(rng.uniform(0.0, 1.0), 2), "weights": rng.choice(("mq", "mq", "qm"))}
        if case["groups"] * case["q"] * case["m"] <= 1 << 28 and work(case)["flops"] <= (4e11 if dtype == "f32" else 1.2e12):
            return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _sizes(case, seed):
    """Rows of every group: a router's choices, some experts liked more than others and some by no row."""
    r = np.random.RandomState(seed % (1 << 31))
    p = np.exp(case["spread"] * r.standard_normal(case["groups"]))
    return r.multinomial(case["rows"], p / p.sum())


def prepare(case, seed):
    dev = torch.device("cuda")
    dtype = DTYPES[case["dtype"]]
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, t=torch.float32):
        return torch.randn(*shape, generator=g, device=dev, dtype=t)

    if case["op"] == "orthogonalize":
        # an update: directions that many samples agree on, in the noise of the others
        b, r, c = case["batch"], case["r"], case["c"]
        t = torch.float64 if dtype == torch.float64 else torch.float32
        k = max(1, min(r, c) // 16)
        strength = torch.logspace(0, -1, k, device=dev, dtype=t)
        G = torch.bmm(normal(b, r, k, t=t) * strength, normal(b, k, c, t=t)) * (4.0 / math.sqrt(k)) + normal(b, r, c, t=t)
        return {"case": case, "G": (G * 1e-3).to(dtype)}

    sizes = _sizes(case, seed)
    n, e, q, m = case["rows"], case["groups"], case["q"], case["m"]
    ends = np.cumsum(sizes)
    offsets = torch.from_numpy(np.concatenate([[0], ends]).astype(np.int32)).to(dev)
    X = (normal(n, q) * torch.exp(0.3 * normal(n, 1))).to(dtype)
    W = (normal(e, m, q) / math.sqrt(q)).to(dtype)
    if case["weights"] == "qm":  # stored inner dimension first, used through a transposed view
        W = W.transpose(1, 2).contiguous().transpose(1, 2)
    # which groups have rows, and the place of every row in a padded array of them
    active = np.flatnonzero(sizes)
    longest = int(sizes.max())
    rank = np.zeros(e, np.int64)
    rank[active] = np.arange(len(active))
    owner = np.repeat(np.arange(e), sizes)
    place = rank[owner] * longest + np.arange(n) - (ends - sizes)[owner]
    state = {"case": case, "X": X, "W": W, "offsets": offsets, "active": torch.from_numpy(active).to(dev),
             "longest": longest, "place": torch.from_numpy(place).to(dev)}
    if case["op"] == "step":
        state["dY"] = (normal(n, m) * 0.01 * torch.exp(0.5 * normal(n, 1))).to(dtype)
    return state


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return _own(state) if own else _plain(state)


def _own(state):
    import fp64_gemm_emulation_ozii_amd as oz
    op = state["case"]["op"]
    if op == "orthogonalize":
        return oz.orthogonalize(state["G"], steps=STEPS, coeffs=QUINTIC, eps=EPS)
    Y = oz.grouped_linear(state["X"], state["W"], state["offsets"])
    if op == "product":
        return Y
    dX, dW = oz.grouped_linear_grads(state["dY"], state["X"], state["W"], state["offsets"])
    return {"Y": Y, "dX": dX, "dW": dW}


def _plain(state):
    op = state["case"]["op"]
    if op == "orthogonalize":
        G = state["G"]
        x = G if G.dtype == torch.float64 else G.float()
        x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + EPS)
        tall = x.shape[1] > x.shape[2]
        if tall:
            x = x.transpose(1, 2).contiguous()
        a, b, c = QUINTIC
        for _ in range(STEPS):
            p = torch.bmm(x, x.transpose(1, 2))
            x = a * x + torch.bmm(b * p + c * torch.bmm(p, p), x)
        return (x.transpose(1, 2).contiguous() if tall else x).to(G.dtype)

    X, W, place, longest, active = state["X"], state["W"], state["place"], state["longest"], state["active"]
    Wa = W[active].float()

    def padded(v):
        p = torch.zeros(len(active) * longest, v.shape[1], device=v.device)
        p[place] = v.float()
        return p.view(len(active), longest, v.shape[1])

    def rows(p):
        return p.reshape(-1, p.shape[2])[place].to(X.dtype)

    Xp = padded(X)
    Y = rows(torch.bmm(Xp, Wa.transpose(1, 2)))
    if op == "product":
        return Y
    dYp = padded(state["dY"])
    dW = torch.zeros(W.shape, device=W.device, dtype=W.dtype)
    dW[active] = torch.bmm(dYp.transpose(1, 2), Xp).to(W.dtype)
    return {"Y": Y, "dX": rows(torch.bmm(dYp, Wa)), "dW": dW}


def work(case):
    size = BYTES[case["dtype"]]
    if case["op"] == "orthogonalize":
        # per step two products whose result is symmetric (half of it is enough) and one full product
        lo, hi = sorted((case["r"], case["c"]))
        flops = STEPS * (lo * lo * hi + lo * lo * lo + 2 * lo * lo * hi)
        return {"bytes": 2.0 * case["batch"] * lo * hi * size, "flops": float(case["batch"] * flops)}
    n, q, m = case["rows"], case["q"], case["m"]
    e = int(np.count_nonzero(_sizes(case, 0)))  # groups without rows need no weights
    one = 2.0 * n * q * m
    if case["op"] == "product":
        return {"bytes": float(size * (n * q + e * m * q + n * m)), "flops": one}
    # X, W and dY in; Y, dX and the whole dW out
    return {"bytes": float(size * (2 * n * q + 2 * n * m + e * m * q + case["groups"] * m * q)), "flops": 3 * one}


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "orthogonalize":
        # in the space of the smaller side: O = G p(G^T G) or p(G G^T) G, the polynomial built up as a matrix
        G = state["G"].double()
        if G.shape[1] < G.shape[2]:
            G = G.transpose(1, 2).contiguous()
        out = []
        a, b, c = QUINTIC
        for g in G:
            norm = torch.linalg.vector_norm(g) + EPS
            S = (g.T.contiguous() @ g) / (norm * norm)
            eye = torch.eye(S.shape[0], dtype=S.dtype, device=S.device)
            P = eye.clone()
            for _ in range(STEPS):
                # X = g P / norm, with P a polynomial in S: X^T X = P S P
                A = P @ S @ P
                P = P @ (a * eye + b * A + c * (A @ A))
            out.append((g @ P) / norm)
        O = torch.stack(out)
        return O if O.shape[1:] == state["G"].shape[1:] else O.transpose(1, 2).contiguous()
    off = state["offsets"].tolist()
    X, W = state["X"].double(), state["W"]
    Y = torch.zeros(case["rows"], case["m"], dtype=torch.float64, device=X.device)
    step = case["op"] == "step"
    if step:
        dY, dX = state["dY"].double(), torch.zeros_like(X)
        dW = torch.zeros(W.shape, dtype=torch.float64, device=X.device)
    for i in range(case["groups"]):
        s = slice(off[i], off[i + 1])
        w = W[i].double()
        Y[s] = X[s] @ w.T
        if step:
            dX[s] = dY[s] @ w
            dW[i] = dY[s].T @ X[s]
    return {"Y": Y, "dX": dX, "dW": dW} if step else Y
