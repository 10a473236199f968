"""Timed cases of the dense layers, of the optimizer's orthogonalised update and of the branch for a few tokens.

Each case names one operator and its sizes.  `run` computes it either through the package (`own`) or in plain torch:
elementary operations in 32 bits (the router's scores in 64: scores next to each other decide which expert is taken),
rounded once at the end.

  linear       y = act(x W^T + b) + residual, with the pre-activation kept where a backward follows
  linear_grad  its gradients with respect to x, W and b
  ortho        Newton-Schulz iteration that moves the singular values of a weight's update near 1
  few          the whole dropless branch for at most 16 tokens: latent projection, router, experts, shared experts
"""
import math

import torch

own = False

COEFFS = (3.4445, -4.7750, 2.0315)  # a s + b s^3 + c s^5 for every step
STEPS = 5
EPS = 1e-7


# ------------------------------------------------------------------ cases


def listed():
    return [
        # one token of a decoding step through an output projection, added to the block's input
        dict(name="linear_token", op="linear", M=1, N=6144, K=2048, act="none", bias=False, res=True, out="bf16",
             save=False),
        # a ragged batch through a small layer of odd sizes, fp32 out
        dict(name="linear_odd", op="linear", M=333, N=1001, K=1250, act="gelu", bias=True, res=False, out="f32",
             save=False),
        # four 4K sequences of a training step: the pre-activation is kept for the backward
        dict(name="linear_batch", op="linear", M=16384, N=6144, K=2048, act="silu", bias=True, res=True, out="bf16",
             save=True),
        # gradients of a small layer of odd sizes
        dict(name="linear_grad_odd", op="linear_grad", M=1001, N=520, K=775, act="relu", bias=True, dy="f32"),
        # gradients of a layer over two 4K sequences
        dict(name="linear_grad_batch", op="linear_grad", M=8192, N=2048, K=6144, act="silu", bias=True, dy="bf16"),
        # one down-projection for each of 64 small experts
        dict(name="ortho_experts", op="ortho", B=64, M=512, N=512, dtype="bf16"),
        # a tall matrix whose sizes end inside every tile, fp32 momentum
        dict(name="ortho_odd", op="ortho", B=3, M=1000, N=333, dtype="f32"),
        # wide experts' updates, eight at a time
        dict(name="ortho_wide", op="ortho", B=8, M=2048, N=4096, dtype="bf16"),
        # one token of a decoding step, a small layer: latency
        dict(name="few_one", op="few", T=1, D=1024, L=512, E=64, k=8, F=512, S=2, Fs=512, res=False),
        # sixteen sequences decoding together, sizes that are no powers of two
        dict(name="few_sixteen", op="few", T=16, D=1984, L=960, E=60, k=6, F=1408, S=1, Fs=1856, res=True),
        # four tokens through the layer of this repository's own benchmark
        dict(name="few_marin", op="few", T=4, D=6144, L=3072, E=384, k=8, F=3072, S=2, Fs=3072, res=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_grad", "ortho", "few", "few"])
    act = rng.choice(["none", "relu", "silu", "gelu"])
    if op == "linear":
        return dict(op=op, M=_log(rng, 1, 16384), N=_log(rng, 64, 6144), K=_log(rng, 64, 2048), act=act,
                    bias=rng.random() < 0.6, res=rng.random() < 0.5, out=rng.choice(["bf16", "bf16", "f32"]),
                    save=rng.random() < 0.4)
    if op == "linear_grad":
        return dict(op=op, M=_log(rng, 16, 8192), N=_log(rng, 64, 2048), K=_log(rng, 64, 6144), act=act,
                    bias=rng.random() < 0.6, dy=rng.choice(["bf16", "f32"]))
    if op == "ortho":
        B = _log(rng, 1, 64)
        most = 2048 if B <= 8 else 512
        return dict(op=op, B=B, M=_log(rng, 48, most), N=_log(rng, 48, most), dtype=rng.choice(["bf16", "f32"]))
    E = rng.randint(8, 128)
    return dict(op=op, T=rng.randint(1, 16), D=64 * _log(rng, 4, 48), L=64 * _log(rng, 4, 24), E=E,
                k=rng.randint(1, 8), F=64 * _log(rng, 4, 24), S=rng.randint(0, 2), Fs=64 * _log(rng, 4, 24),
                res=rng.random() < 0.5)


# ----------------------------------------------------------------- inputs


def _rand(g, shape, dev, scale=1.0, dtype=torch.float32):
    return torch.empty(shape, device=dev, dtype=dtype).normal_(0.0, scale, generator=g)


def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def prepare(case, seed):
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev).manual_seed(int(seed) * 7919 + 29)
    s = dict(case)
    op, bf = case["op"], torch.bfloat16
    if op in ("linear", "linear_grad"):
        M, N, K = case["M"], case["N"], case["K"]
        s["x"] = _rand(g, (M, K), dev, 1.0, bf)
        s["w"] = _rand(g, (N, K), dev, K ** -0.5, bf)
        s["b"] = _rand(g, (N,), dev, 0.1, bf) if case["bias"] else None
        if op == "linear":
            s["r"] = _rand(g, (M, N), dev).to(_type(case["out"])) if case["res"] else None
        else:
            s["dy"] = _rand(g, (M, N), dev).to(_type(case["dy"]))
            s["pre"] = None if case["act"] == "none" else _rand(g, (M, N), dev, 1.0, bf)  # as the forward kept it
    elif op == "ortho":
        # a gradient: a few strong directions that decay over a floor of noise
        B, M, N = case["B"], case["M"], case["N"]
        r = min(32, M, N)
        u = _rand(g, (B, M, r), dev) * torch.arange(1, r + 1, device=dev, dtype=torch.float32) ** -0.5
        G = u @ _rand(g, (B, r, N), dev) + _rand(g, (B, M, N), dev, 0.3)
        s["g"] = (1e-3 * G).to(_type(case["dtype"]))
    else:
        T, D, L, E, k, F, S, Fs = (case[n] for n in ("T", "D", "L", "E", "k", "F", "S", "Fs"))
        w = dict(w_latent=(L, D), w_router=(E, L), w_gate=(E, F, L), w_up=(E, F, L), w_down=(E, L, F), w_up_proj=(D, L))
        if S:
            w.update(ws_gate=(S, Fs, D), ws_up=(S, Fs, D), ws_down=(S, D, Fs))
        s["w"] = {n: _rand(g, shape, dev, shape[-1] ** -0.5, bf) for n, shape in w.items()}
        s["w"]["router_bias"] = _rand(g, (E,), dev, 0.01)
        s["x"] = _rand(g, (T, D), dev, 1.0, bf)
        s["r"] = _rand(g, (T, D), dev, 1.0, bf) if case["res"] else None
        if own:  # the handle that a serving program keeps: weights, workspace and outputs bound once
            import routing_capacity_dispatch_amd as rcd
            cfg = rcd.make_config(T, D, L, E, 1, k, F, S, Fs, 1)
            s["layer"] = rcd.ForwardFew(cfg, s["w"], dev, taps=True)
    return s


# -------------------------------------------------------------- plain forms


def _act(u, act):
    if act == "relu":
        return torch.clamp(u, min=0)
    if act == "silu":
        return u / (1 + torch.exp(-u))
    if act == "gelu":
        return 0.5 * u * (1 + torch.erf(u * 0.5 ** 0.5))
    return u


def _slope(u, act):
    if act == "relu":
        return (u > 0).to(u.dtype)
    if act == "silu":
        p = 1 / (1 + torch.exp(-u))
        return p * (1 + u * (1 - p))
    return 0.5 * (1 + torch.erf(u * 0.5 ** 0.5)) + u * torch.exp(-0.5 * u * u) * (2 * math.pi) ** -0.5


def _linear(s):
    u = s["x"].float() @ s["w"].float().t()
    if s["b"] is not None:
        u = u + s["b"].float()
    y = _act(u, s["act"])
    if s["r"] is not None:
        y = y + s["r"].float()
    y = y.to(_type(s["out"]))
    return (y, u.to(torch.bfloat16)) if s["save"] else y


def _linear_grad(s):
    d = s["dy"].float()
    if s["act"] != "none":
        d = d * _slope(s["pre"].float(), s["act"])
    dx = (d @ s["w"].float()).to(torch.bfloat16)
    dw = (d.t() @ s["x"].float()).to(torch.bfloat16)
    return (dx, dw, d.sum(0)) if s["b"] is not None else (dx, dw)


def _ortho(s):
    tall = s["M"] > s["N"]
    x = s["g"].float()
    x = x.transpose(1, 2) if tall else x
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + EPS)
    a, b, c = COEFFS
    for _ in range(STEPS):
        p = x @ x.transpose(1, 2)
        x = a * x + (b * p + c * (p @ p)) @ x
    return (x.transpose(1, 2) if tall else x).to(torch.bfloat16).contiguous()


def _few(s):
    w, k = s["w"], s["k"]
    x = s["x"].float()
    z = x @ w["w_latent"].float().t()
    logits = ((s["x"].double() @ w["w_latent"].double().t()) @ w["w_router"].double().t()).float()
    idx = torch.sort(logits + w["router_bias"], dim=1, descending=True, stable=True).indices[:, :k]
    gates = torch.softmax(logits.gather(1, idx), 1)
    e = idx.reshape(-1)
    u = z.repeat_interleave(k, 0)[:, :, None]
    a, v = (w[n][e].float() @ u for n in ("w_gate", "w_up"))
    o = (w["w_down"][e].float() @ (_act(a, "silu") * v))[:, :, 0]
    y = (o.view(-1, k, s["L"]) * gates[:, :, None]).sum(1) @ w["w_up_proj"].float().t()
    if s["S"]:
        h = _act(x @ w["ws_gate"].float().transpose(1, 2), "silu") * (x @ w["ws_up"].float().transpose(1, 2))
        y = y + (h @ w["ws_down"].float().transpose(1, 2)).sum(0)
    if s["r"] is not None:
        y = y + s["r"].float()
    return y.to(torch.bfloat16), logits


# ------------------------------------------------------------ the package


def _own(s):
    import routing_capacity_dispatch_amd as rcd
    op = s["op"]
    if op == "linear":
        return rcd.linear(s["x"], s["w"], s["b"], act=s["act"], residual=s["r"], out_dtype=_type(s["out"]),
                          save_pre=s["save"])
    if op == "linear_grad":
        dx, dw, db = rcd.linear_backward(s["dy"], s["x"], s["w"], pre=s["pre"], act=s["act"], bias=s["b"] is not None)
        return (dx, dw, db) if s["b"] is not None else (dx, dw)
    if op == "ortho":
        return rcd.orthogonalize(s["g"], steps=STEPS, coeffs=COEFFS, eps=EPS)
    y = s["layer"](s["x"], s["r"])
    return y, s["layer"].tap_t["logits"]


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    if op == "linear":
        return _linear(state)
    if op == "linear_grad":
        return _linear_grad(state)
    if op == "ortho":
        return _ortho(state)
    return _few(state)


# ------------------------------------------------------------------- work


def work(case):
    op = case["op"]
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        eb = 2 if case["out"] == "bf16" else 4
        return dict(bytes=2 * (M * K + N * K) + M * N * (eb * (2 if case["res"] else 1) + (2 if case["save"] else 0)),
                    flops=2 * M * N * K)
    if op == "linear_grad":
        M, N, K = case["M"], case["N"], case["K"]
        eb = (2 if case["dy"] == "bf16" else 4) + (0 if case["act"] == "none" else 2)
        return dict(bytes=4 * (M * K + N * K) + M * N * eb, flops=4 * M * N * K)
    if op == "ortho":
        B, m, n = case["B"], min(case["M"], case["N"]), max(case["M"], case["N"])
        # x x^T and p p are symmetric: half of each is enough
        return dict(bytes=B * m * n * (4 if case["dtype"] == "bf16" else 6),
                    flops=STEPS * B * (m * m * n + m * m * m + 2 * m * m * n))
    T, D, L, E, k, F, S, Fs = (case[n] for n in ("T", "D", "L", "E", "k", "F", "S", "Fs"))
    busy = E * (1 - (1 - k / E) ** T)  # experts that have rows, about
    per = 2 * D * L + E * L + 3 * S * Fs * D
    return dict(bytes=int(2 * (per + busy * 3 * L * F) + T * D * (6 if case["res"] else 4) + T * E * 4),
                flops=2 * T * (per + k * 3 * L * F))


# ------------------------------------------------------------- 64-bit values


def _act64(u, act):
    if act == "none":
        return u
    if act == "relu":
        return torch.where(u > 0, u, torch.zeros_like(u))
    if act == "silu":
        return torch.where(u < 0, u * torch.exp(u) / (1 + torch.exp(u)), u / (1 + torch.exp(-u)))
    return u - 0.5 * u * torch.special.erfc(u / math.sqrt(2))


def _swiglu64(x, gate, up):
    return _act64(x @ gate.double().t(), "silu") * (x @ up.double().t())


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        if 2.0 * case["M"] * case["N"] * case["K"] > 5e14:
            return None
        w = s["w"].double().t()
        bias = 0.0 if s["b"] is None else s["b"].double()
        ys, us = [], []
        for i in range(0, case["M"], 1024):
            u = s["x"][i:i + 1024].double() @ w + bias
            us.append(u)
            ys.append(_act64(u, case["act"]) + (0.0 if s["r"] is None else s["r"][i:i + 1024].double()))
        return (torch.cat(ys), torch.cat(us)) if case["save"] else torch.cat(ys)
    if op == "linear_grad":
        # the slope through autograd of the activation
        d = s["dy"].double()
        if case["act"] != "none":
            u = s["pre"].double().requires_grad_(True)
            with torch.enable_grad():
                d, = torch.autograd.grad(_act64(u, case["act"]), u, d)
        dx, dw = d @ s["w"].double(), (s["x"].double().t() @ d).t().contiguous()
        return (dx, dw, torch.ones(1, case["M"], dtype=d.dtype, device=d.device).matmul(d)[0]) if case["bias"] else \
            (dx, dw)
    if op == "ortho":
        # one matrix at a time, through x (b x^T x + c (x^T x)^2): the Gram matrix of the other side
        out = []
        for G in s["g"]:
            G = G.double() if case["M"] >= case["N"] else G.double().t()
            X = G / (torch.linalg.vector_norm(G) + EPS)
            for _ in range(STEPS):
                P = X.t() @ X
                XP = X @ P
                X = COEFFS[0] * X + COEFFS[1] * XP + COEFFS[2] * (XP @ P)
            out.append(X if case["M"] >= case["N"] else X.t())
        return torch.stack(out)
    w, k = s["w"], case["k"]
    x = s["x"].double()
    z = x @ w["w_latent"].double().t()
    logits = z @ w["w_router"].double().t()
    ys = []
    for t in range(case["T"]):
        score = (logits[t].float() + w["router_bias"]).tolist()
        ids = sorted(range(case["E"]), key=lambda e: (-score[e], e))[:k]
        top = logits[t, ids].exp()
        gate = top / top.sum()
        lat = torch.zeros_like(z[t:t + 1])
        for j, e in enumerate(ids):
            lat += gate[j] * (_swiglu64(z[t:t + 1], w["w_gate"][e], w["w_up"][e]) @ w["w_down"][e].double().t())
        ys.append(lat @ w["w_up_proj"].double().t())
    y = torch.cat(ys)
    for i in range(case["S"]):
        y += _swiglu64(x, w["ws_gate"][i], w["ws_up"][i]) @ w["ws_down"][i].double().t()
    if s["r"] is not None:
        y += s["r"].double()
    return y, logits
