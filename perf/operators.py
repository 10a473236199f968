"""Timed cases of the scored router and the block-scaled 8-bit products.

Each case names one operator and its sizes.  `run` computes it either through
the package (`own`) or in plain torch: elementary operations in 32 bits (the
selection in 64: scores next to each other decide which expert is taken),
rounded once at the end.

  route       scores -> bias -> groups -> top-k -> gates
  route_grad  gradient of the gates with respect to the logits
  quantize    e4m3 values with one fp32 scale for each block of 128
  gemm        C = A B^T on such values
  experts     SwiGLU experts over expert-ordered rows, weights in e4m3
"""
import math

import torch

own = False

E4M3_MAX = 448.0
TINY = 2.0 ** -100  # amax of a block is taken as at least this


# ------------------------------------------------------------------ cases


def listed():
    return [
        # one token of a decoding step through a group-limited sigmoid router
        dict(name="route_token", op="route", T=1, E=384, k=8, score="sigmoid", groups=8, top_groups=4, group_top=2,
             bias=True, renorm=True, scale=2.5),
        # four 4K sequences in one call
        dict(name="route_batch", op="route", T=16384, E=384, k=8, score="sigmoid", groups=8, top_groups=4, group_top=2,
             bias=True, renorm=True, scale=2.5),
        # a ragged batch, plain softmax scores, no groups, an expert count that is no power of two
        dict(name="route_softmax_odd", op="route", T=4095, E=60, k=6, score="softmax", groups=1, top_groups=1,
             group_top=1, bias=False, renorm=False, scale=1.0),
        # the training step's gradient for both kinds of scores
        dict(name="route_grad_batch", op="route_grad", T=16384, E=384, k=8, score="sigmoid", renorm=True, scale=2.5),
        dict(name="route_grad_softmax", op="route_grad", T=4095, E=64, k=8, score="softmax", renorm=False, scale=1.0),
        # activations of a whole batch before a projection
        dict(name="quantize_rows", op="quantize", rows=16384, cols=6144, dtype="bf16", block=1, transpose=False),
        # an fp32 master weight laid out for the input gradient, sizes that end inside a block
        dict(name="quantize_weight_t", op="quantize", rows=2056, cols=4100, dtype="f32", block=128, transpose=True),
        # one token through a projection
        dict(name="gemm_token", op="gemm", M=1, N=6144, K=2048, block=128, out="bf16"),
        # a weight gradient: K runs over tokens, one scale a row on both sides, fp32 result
        dict(name="gemm_wgrad_odd", op="gemm", M=1000, N=2056, K=4224, block=1, out="f32"),
        # a projection of a large batch
        dict(name="gemm_batch", op="gemm", M=8192, N=6144, K=4096, block=128, out="bf16"),
        # four tokens of a decoding step: 32 rows over 64 experts
        dict(name="experts_token", op="experts", T=4, k=8, E=64, L=2048, F=1024),
        # one 4K sequence over 64 experts
        dict(name="experts_batch", op="experts", T=4096, k=8, E=64, L=2048, F=1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_grad", "quantize", "gemm", "experts"])
    if op in ("route", "route_grad"):
        c = dict(op=op, T=_log(rng, 1, 16384), score=rng.choice(["sigmoid", "softmax"]), renorm=rng.random() < 0.5,
                 scale=rng.choice([1.0, 2.5]))
        groups = rng.choice([1, 1, 2, 4, 8]) if op == "route" else 1
        c["E"] = groups * rng.randint(max(4, 16 // groups), 384 // groups)
        c["k"] = rng.randint(1, 8)
        if op == "route":
            need = -(-c["k"] // (c["E"] // groups))
            c.update(groups=groups, top_groups=rng.randint(min(need, groups), groups), group_top=rng.choice([1, 2]),
                     bias=rng.random() < 0.7)
        return c
    if op == "quantize":
        rows, cols = _log(rng, 1, 16384), _log(rng, 64, 6144)
        return dict(op=op, rows=rows, cols=cols, dtype=rng.choice(["bf16", "f32"]), block=rng.choice([1, 128]),
                    transpose=rng.random() < 0.5)
    if op == "gemm":
        return dict(op=op, M=_log(rng, 1, 8192), N=_log(rng, 64, 6144), K=128 * _log(rng, 2, 32),
                    block=rng.choice([1, 128, 128]), out=rng.choice(["bf16", "f32"]))
    E = rng.choice([8, 16, 32, 64])
    return dict(op=op, T=_log(rng, 1, 4096), k=rng.randint(1, 8), E=E, L=128 * rng.randint(4, 16),
                F=128 * rng.randint(2, 8))


# ----------------------------------------------------------------- inputs


def _pad(n):
    return -(-n // 128) * 128


def _e4m3(v):
    """fp32 or fp64 values of magnitude at most 448, rounded to the nearest e4m3 value, ties to even."""
    step = torch.exp2(torch.frexp(v).exponent.clamp(min=-5).to(v.dtype) - 4)
    return torch.round(v / step) * step


def _quantize(x, block, transpose):
    """Values (float8) with zero-padded rows, and scales: [blocks along K][rows] for 1 x 128 blocks,
    [row blocks][blocks along K] for 128 x 128 blocks.  All in 32 bits."""
    x = x.float()
    if transpose:
        x = x.t()
    R, K = x.shape
    Rp, Kp = (_pad(R) if block == 128 else R), _pad(K)
    p = torch.zeros((Rp, Kp), dtype=torch.float32, device=x.device)
    p[:R, :K] = x
    p = p.view(Rp // block, block, Kp // 128, 128)
    amax = p.abs().amax(dim=(1, 3)).clamp(min=TINY)
    # 448 x / amax as 512 (7/8 x / amax): the product is exact for bf16 x and cannot overflow, so a quotient half
    # way between two e4m3 values is met as such
    v = (p * (E4M3_MAX / 512) / amax[:, None, :, None] * 512).clamp(-E4M3_MAX, E4M3_MAX)
    q = _e4m3(v).view(Rp, Kp)[:R].to(torch.float8_e4m3fn)
    s = amax / torch.full_like(amax, E4M3_MAX)
    return q, (s.t().contiguous() if block == 1 else s)


def _rand(g, shape, dev, scale=1.0):
    return torch.randn(shape, generator=g, device=dev, dtype=torch.float32) * scale


def prepare(case, seed):
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev).manual_seed(int(seed) * 7919 + 17)
    s = dict(case)
    op = case["op"]
    if op in ("route", "route_grad"):
        T, E, k = case["T"], case["E"], case["k"]
        s["logits"] = _rand(g, (T, E), dev, 1.5)
        if op == "route":
            s["b"] = _rand(g, (E,), dev, 0.05) if case["bias"] else None
        else:
            s["topk"] = torch.rand((T, E), generator=g, device=dev).argsort(1)[:, :k].to(torch.int32).contiguous()
            s["dg"] = _rand(g, (T, k), dev)
    elif op == "quantize":
        x = _rand(g, (case["rows"], case["cols"]), dev)
        x = x * torch.exp(_rand(g, (case["rows"], 1), dev, 0.5))  # rows of different size
        s["x"] = x.to(torch.bfloat16) if case["dtype"] == "bf16" else x
    elif op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        s["a"], s["sa"] = _quantize(_rand(g, (M, K), dev), 1, False)
        s["b"], s["sb"] = _quantize(_rand(g, (N, K), dev, K ** -0.5), case["block"], False)
    else:
        T, k, E, L, F = (case[n] for n in ("T", "k", "E", "L", "F"))
        pop = _rand(g, (1, E), dev, 0.3)
        e = (pop + _rand(g, (T, E), dev)).argsort(1)[:, :k].reshape(-1)
        n = torch.bincount(e, minlength=E)
        s["off"] = torch.cat([n.new_zeros(1), n.cumsum(0)]).to(torch.int32)
        s["most"] = int(n.max())
        s["xs"] = _rand(g, (T * k, L), dev).to(torch.bfloat16)
        for name, rows, cols in (("wg", F, L), ("wu", F, L), ("wd", L, F)):
            q, sc = _quantize(_rand(g, (E * rows, cols), dev, cols ** -0.5), 128, False)
            s[name] = q.view(E, rows, cols)
            s["s" + name] = sc.view(E, rows // 128, cols // 128)
    return s


# -------------------------------------------------------------- plain forms


def _scores(logits, score):
    return torch.sigmoid(logits) if score == "sigmoid" else torch.softmax(logits, 1)


def _route(s):
    T, E, k, G = s["T"], s["E"], s["k"], s["groups"]
    p = _scores(s["logits"].double(), s["score"])
    key = p if s["b"] is None else p + s["b"].double()
    if G > 1:
        by = key.view(T, G, E // G)
        best = torch.sort(by, dim=2, descending=True).values[:, :, :s["group_top"]].sum(2)
        keep = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :s["top_groups"]]
        mask = torch.ones((T, G), dtype=torch.bool, device=key.device).scatter_(1, keep, False)
        key = by.masked_fill(mask[:, :, None], -math.inf).view(T, E)
    idx = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    w = p.gather(1, idx)
    if s["renorm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    return idx.to(torch.int32), (w * s["scale"]).float()


def _route_grad(s):
    idx, dg = s["topk"].long(), s["dg"]
    p = _scores(s["logits"], s["score"])
    w = p.gather(1, idx)
    ds = dg * s["scale"]
    if s["renorm"]:
        S = w.sum(1, keepdim=True) + 1e-20
        ds = (ds - (ds * w).sum(1, keepdim=True) / S) / S
    if s["score"] == "sigmoid":
        return torch.zeros_like(p).scatter_(1, idx, ds * w * (1 - w))
    return p * (torch.zeros_like(p).scatter_(1, idx, ds) - (ds * w).sum(1, keepdim=True))


def _rows(q, s):
    """fp32 values of rows with 1 x 128 scales ([blocks][rows])."""
    return (q.float().view(q.shape[0], -1, 128) * s.t()[:, :, None]).view(q.shape)


def _blocks(q, s):
    """fp32 values of [..., N, K] with 128 x 128 scales."""
    full = s.repeat_interleave(128, -2)[..., :q.shape[-2], :]
    return (q.float().view(*q.shape[:-1], -1, 128) * full[..., None]).view(q.shape)


def _gemm(s):
    a = _rows(s["a"], s["sa"])
    b = _rows(s["b"], s["sb"]) if s["block"] == 1 else _blocks(s["b"], s["sb"])
    c = a @ b.t()
    return c.to(torch.bfloat16) if s["out"] == "bf16" else c


def _experts(s):
    n, E, L = s["T"] * s["k"], s["E"], s["L"]
    off = s["off"].long()
    pos = torch.arange(n, device=off.device)
    e = torch.searchsorted(off[1:], pos, right=True)
    at = e * s["most"] + pos - off[e]  # row of the padded [E][most] layout
    q, sc = _quantize(s["xs"], 1, False)
    u = torch.zeros((E * s["most"], L), dtype=torch.float32, device=off.device)
    u[at] = _rows(q, sc)
    u = u.view(E, s["most"], L)
    gate = u @ _blocks(s["wg"], s["swg"]).transpose(1, 2)
    up = u @ _blocks(s["wu"], s["swu"]).transpose(1, 2)
    h = (gate * torch.sigmoid(gate) * up).view(E * s["most"], -1)
    q, sc = _quantize(h, 1, False)
    o = _rows(q, sc).view(E, s["most"], -1) @ _blocks(s["wd"], s["swd"]).transpose(1, 2)
    return o.view(E * s["most"], L)[at].to(torch.bfloat16)


# ------------------------------------------------------------ the package


def _own(s):
    import routing_capacity_dispatch_amd as rcd
    op = s["op"]
    if op in ("route", "route_grad"):
        cfg = rcd.make_config(s["T"], 64, 64, s["E"], 1, s["k"], 64)
        if op == "route":
            sc = rcd.scoring(s["score"], n_groups=s["groups"], top_groups=s["top_groups"], group_top=s["group_top"],
                             renormalise=s["renorm"], scale=s["scale"])
            return rcd.route_scored(cfg, sc, s["logits"], s["b"])
        sc = rcd.scoring(s["score"], renormalise=s["renorm"], scale=s["scale"])
        return rcd.route_scored_backward(cfg, sc, s["logits"], s["topk"], s["dg"])
    if op == "quantize":
        return rcd.quantize(s["x"], block_rows=s["block"], transpose=s["transpose"])
    if op == "gemm":
        return rcd.gemm_quant(s["a"], s["sa"], s["b"], s["sb"], block_rows=s["block"],
                              out_dtype=torch.bfloat16 if s["out"] == "bf16" else torch.float32)
    cfg = rcd.make_config(s["T"], 64, s["L"], s["E"], 1, s["k"], s["F"])
    return rcd.experts_dropless_quant(cfg, s["xs"], s["off"], (s["wg"], s["swg"]), (s["wu"], s["swu"]),
                                      (s["wd"], s["swd"]))


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    if op == "route":
        return _route(state)
    if op == "route_grad":
        return _route_grad(state)
    if op == "quantize":
        return _quantize(state["x"], state["block"], state["transpose"])
    if op == "gemm":
        return _gemm(state)
    return _experts(state)


# ------------------------------------------------------------------- work


def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return dict(bytes=T * E * 4 + T * k * 8 + (E * 4 if case["bias"] else 0), flops=T * E * 4)
    if op == "route_grad":
        T, E, k = case["T"], case["E"], case["k"]
        read = E if case["score"] == "softmax" else k
        return dict(bytes=T * (read * 4 + k * 8 + E * 4), flops=T * read * 6)
    if op == "quantize":
        n = case["rows"] * case["cols"]
        return dict(bytes=n * (3 if case["dtype"] == "bf16" else 5) + n // (128 * case["block"]) * 4, flops=n * 3)
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        scales = M * K // 32 + N * K // (32 * case["block"])
        return dict(bytes=M * K + N * K + scales + M * N * (2 if case["out"] == "bf16" else 4), flops=2 * M * N * K)
    T, k, E, L, F = (case[n] for n in ("T", "k", "E", "L", "F"))
    busy = E * (1 - (1 - k / E) ** T)  # experts that have rows, about
    return dict(bytes=int(busy * 3 * L * F) + T * k * L * 4, flops=6 * T * k * L * F)


# ------------------------------------------------------------- 64-bit values


def _round64(v):
    """float64 to the nearest e4m3 value, ties to even, through the list of its 127 magnitudes."""
    mags = torch.tensor([(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7)
                         for e in range(16) for m in range(8)][:127], dtype=torch.float64, device=v.device)
    a = v.abs().clamp(max=448.0)
    hi = torch.searchsorted(mags, a).clamp(max=126)  # first magnitude not below
    lo = (hi - 1).clamp(min=0)
    up, down = mags[hi] - a, a - mags[lo]
    pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return torch.sign(v) * mags[pick]


def _quantize64(x, block, transpose=False):
    """Rounded values and scales of x in float64: block maxima by index, row block by row block."""
    x = x.double().t() if transpose else x.double()
    R, K = x.shape
    kb = (torch.arange(K, device=x.device) // 128).expand(R, K)
    amax = torch.zeros((R, -(-K // 128)), dtype=torch.float64, device=x.device)
    amax.scatter_reduce_(1, kb, x.abs(), "amax")
    rb = torch.arange(R, device=x.device) // block
    by = torch.zeros((-(-R // block), amax.shape[1]), dtype=torch.float64, device=x.device)
    by.index_reduce_(0, rb, amax, "amax")
    by = by.clamp(min=TINY)
    q = torch.zeros((R, amax.shape[1] * 128), dtype=torch.float64, device=x.device)
    step = max(1, (1 << 24) // max(1, K))
    for r in range(0, R, step):
        m = by[rb[r:r + step]].gather(1, kb[r:r + step])
        q[r:r + step, :K] = _round64(x[r:r + step] * 448.0 / m)
    return q, by / 448.0


def _value64(q, s, block):
    """float64 values of quantised rows; s [row blocks][blocks along K]."""
    R, K = q.shape
    rb, kb = torch.arange(R, device=q.device) // block, torch.arange(K, device=q.device) // 128
    return q.double() * s.double()[rb][:, kb]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("route", "route_grad"):
        l = s["logits"].double()
        if case["score"] == "sigmoid":
            p = 1.0 / (1.0 + torch.exp(-l))
        else:
            p = torch.exp(l - l.max(1, keepdim=True).values)
            p = p / p.sum(1, keepdim=True)
        if op == "route":
            T, E, k, G = (case[n] for n in ("T", "E", "k", "groups"))
            key = p.clone() if s["b"] is None else p + s["b"].double()
            rest = key.view(T, G, E // G).clone()
            best = torch.zeros((T, G), dtype=torch.float64, device=key.device)
            for _ in range(min(case["group_top"], E // G)):
                m = rest.max(2)
                best += m.values
                rest.scatter_(2, m.indices[:, :, None], -math.inf)
            open_ = torch.zeros((T, G), dtype=torch.bool, device=key.device)
            for _ in range(case["top_groups"]):
                hit = best == best.max(1, keepdim=True).values
                first = hit & (hit.cumsum(1) == 1)
                open_ |= first
                best[first] = -math.inf
            key[~open_.repeat_interleave(E // G, 1)] = -math.inf
            ids = []
            for _ in range(k):
                hit = key == key.max(1, keepdim=True).values
                i = (hit & (hit.cumsum(1) == 1)).to(torch.int32).argmax(1)
                ids.append(i)
                key[torch.arange(T, device=key.device), i] = -math.inf
            idx = torch.stack(ids, 1)
            w = torch.gather(p, 1, idx)
            w = w / (w.sum(1, keepdim=True) + 1e-20) if case["renorm"] else w
            return idx.to(torch.int32), w * case["scale"]
        # the gradient through autograd of the forward formula
        ll = l.clone().requires_grad_(True)
        with torch.enable_grad():
            q = torch.sigmoid(ll) if case["score"] == "sigmoid" else torch.softmax(ll, 1)
            w = torch.gather(q, 1, s["topk"].long())
            w = w / (w.sum(1, keepdim=True) + 1e-20) if case["renorm"] else w
            (w * case["scale"] * s["dg"].double()).sum().backward()
        return ll.grad
    if op == "quantize":
        q, sc = _quantize64(s["x"], case["block"], case["transpose"])
        return q, (sc.t().contiguous() if case["block"] == 1 else sc)
    if op == "gemm":
        if 2.0 * case["M"] * case["N"] * case["K"] > 5e14:
            return None
        a = _value64(s["a"], s["sa"].t(), 1)
        b = _value64(s["b"], s["sb"].t() if case["block"] == 1 else s["sb"], case["block"])
        return torch.cat([a[i:i + 1024] @ b.t() for i in range(0, a.shape[0], 1024)])
    if 6.0 * case["T"] * case["k"] * case["L"] * case["F"] > 5e14:
        return None
    off, outs = s["off"].tolist(), []
    for e in range(case["E"]):
        if off[e] == off[e + 1]:
            continue
        u = _value64(*_quantize64(s["xs"][off[e]:off[e + 1]], 1), 1)
        g, v = (u @ _value64(s[n][e], s["s" + n][e], 128).t() for n in ("wg", "wu"))
        h = _value64(*_quantize64(g / (1.0 + torch.exp(-g)) * v, 1), 1)
        outs.append(h @ _value64(s["wd"][e], s["swd"][e], 128).t())
    return torch.cat(outs)
