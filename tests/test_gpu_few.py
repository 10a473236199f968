"""The branch for a few tokens against a plain computation in 64 bits.

Tolerances are error bounds carried through the formulas.  An fp32 sum of K
products loses (K + 8) 2^-24 of their magnitudes; an activation held in two
bf16 parts 2^-17 of itself, in three 2^-24; silu 2^-20 (1 + |a|) with slopes of
at most 1.1; a gate 2e-6; y is rounded to bf16: 2^-8 of it.  Selection and gates
are checked against the rule of moe_route on the logits that the call returns."""
import numpy as np
import pytest
import torch

import routing_capacity_dispatch_amd as rcd
from gpu_common import dev, say

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def np64(t):
    return t.detach().cpu().double().numpy()


def weights(D, L, E, F, S, Fs, seed, bias=0.01):
    g = torch.Generator(device="cpu").manual_seed(seed)

    def r(*s):
        return (torch.randn(s, generator=g) * s[-1] ** -0.5).to(torch.bfloat16)
    w = dict(w_latent=r(L, D), w_router=r(E, L), w_gate=r(E, F, L), w_up=r(E, F, L), w_down=r(E, L, F),
             w_up_proj=r(D, L))
    if S:
        w.update(ws_gate=r(S, Fs, D), ws_up=r(S, Fs, D), ws_down=r(S, D, Fs))
    if bias:
        w["router_bias"] = torch.randn(E, generator=g) * bias
    return w


def silu(a):
    return a / (1 + np.exp(-a))


def product(x, ex, w, parts):
    """x w^T and its error: x off by ex and held with 2^-17 or 2^-24, fp32 sums."""
    ax, aw = np.abs(x), np.abs(w)
    held = {1: 0.0, 2: 2.0 ** -17, 3: U}[parts]
    return x @ w.T, (ex + held * ax) @ aw.T + (parts * x.shape[1] + 8) * U * (ax @ aw.T)


def swiglu(x, ex, wg, wu, parts):
    a, ea = product(x, ex, wg, parts)
    u, eu = product(x, ex, wu, parts)
    s, es = silu(a), 1.1 * ea + 2.0 ** -20 * (1 + np.abs(a))
    return s * u, es * (np.abs(u) + eu) + np.abs(s) * eu


def check(T, D, L, E, k, F, S, Fs, seed=0, bias=0.01, res=False, x=None, w=None):
    d = dev()
    say("few", dict(T=T, D=D, L=L, E=E, k=k, F=F, S=S, Fs=Fs, bias=bias, res=res))
    w = weights(D, L, E, F, S, Fs, seed, bias) if w is None else w
    g = torch.Generator(device="cpu").manual_seed(seed + 1)
    x = torch.randn((T, D), generator=g).to(torch.bfloat16) if x is None else x
    r = torch.randn((T, D), generator=g).to(torch.bfloat16) if res else None
    cfg = rcd.make_config(T, D, L, E, 1, k, F, S, Fs, 1)
    f = rcd.ForwardFew(cfg, {n: t.to(d) for n, t in w.items()}, d, taps=True)
    f.ws.fill_(255)  # nothing in the workspace is expected to be clear
    y = f(x.to(d), None if r is None else r.to(d))
    torch.cuda.synchronize()
    verify(f, w, x, r, T, E, k, S)
    return f, y


def verify(f, w, x, r, T, E, k, S):
    n = {m: np64(t) for m, t in w.items()}
    xn = np64(x)
    z, ez = product(xn, 0.0, n["w_latent"], 1)
    lg, el = product(z, ez, n["w_router"], 3)
    logits = f.tap_t["logits"].cpu().numpy()
    assert (np.abs(logits - lg) <= el).all()
    b = w["router_bias"].numpy() if "router_bias" in w else np.zeros(E, dtype=np.float32)
    score = logits + b  # fp32
    ids = np.argsort(-score, axis=1, kind="stable")[:, :k]
    assert np.array_equal(f.tap_t["topk_idx"].cpu().numpy(), ids)
    top = np.take_along_axis(logits.astype(np.float64), ids, 1)
    gates = np.exp(top - top.max(1, keepdims=True))
    gates /= gates.sum(1, keepdims=True)
    assert np.abs(np64(f.tap_t["gates"]) - gates).max() <= 2e-6
    lat, elat = np.zeros_like(z), np.zeros_like(z)
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            h, eh = swiglu(z[t:t + 1], ez[t:t + 1], n["w_gate"][e], n["w_up"][e], 2)
            o, eo = product(h, eh, n["w_down"][e], 2)
            lat[t] += gates[t, j] * o[0]
            elat[t] += gates[t, j] * eo[0] + (2e-6 + 2.0 ** -20) * np.abs(o[0])
    y, ey = product(lat, elat, n["w_up_proj"], 2)
    for s in range(S):
        h, eh = swiglu(xn, 0.0, n["ws_gate"][s], n["ws_up"][s], 1)
        p, ep = product(h, eh, n["ws_down"][s], 2)
        y, ey = y + p, ey + ep
    if r is not None:
        y = y + np64(r)
    assert (np.abs(np64(f.y) - y) <= ey + (2.0 ** -8 + 8 * U) * (np.abs(y) + ey)).all()


@pytest.mark.parametrize("T", [1, 2, 3, 4, 7, 8, 15, 16])
def test_tokens(T):
    check(T, 256, 128, 24, 4, 192, 2, 128, seed=T, res=T % 2 == 0)


@pytest.mark.parametrize("T,D,L,E,k,F,S,Fs", [
    (1, 64, 64, 1, 1, 64, 0, 0), (16, 64, 64, 1, 1, 64, 1, 64), (5, 64, 128, 5, 5, 64, 0, 0),
    (16, 128, 64, 17, 2, 320, 3, 192), (4, 192, 448, 1024, 8, 64, 1, 64), (16, 128, 64, 64, 64, 64, 0, 0),
    (2, 64, 64, 1000, 64, 64, 1, 576), (9, 1088, 704, 33, 7, 832, 1, 1216), (3, 128, 64, 500, 1, 1984, 0, 0),
    (16, 64, 64, 200, 33, 64, 2, 64), (1, 2048, 1024, 16, 8, 1024, 2, 1024)])
@pytest.mark.parametrize("bias", [0.0, 0.3])
def test_sizes(T, D, L, E, k, F, S, Fs, bias):
    check(T, D, L, E, k, F, S, Fs, seed=D + E, bias=bias, res=S == 1)


def test_equal_scores_and_equal_tokens():
    """Experts in equal pairs (the lower index first), and 16 equal tokens: one expert takes them all."""
    w = weights(128, 64, 12, 64, 1, 64, 3, bias=0.0)
    w["w_router"] = w["w_router"][:6].repeat_interleave(2, 0).contiguous()
    x = torch.randn((1, 128), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    check(16, 128, 64, 12, 3, 64, 1, 64, x=x.expand(16, -1).contiguous(), w=w)
    check(1, 128, 64, 12, 3, 64, 1, 64, x=x, w=w)
    # x = 0: every logit is 0
    check(4, 128, 64, 12, 5, 64, 1, 64, x=torch.zeros(4, 128, dtype=torch.bfloat16), w=w)


def test_as_the_dropless_forward():
    """The same layer by moe_forward_dropless, on tokens for which both take the same experts."""
    d = dev()
    T, D, L, E, k, F, S, Fs = 16, 512, 256, 32, 4, 256, 2, 256
    w = {n: t.to(d) for n, t in weights(D, L, E, F, S, Fs, 5).items()}
    x = torch.randn((T, D), generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).to(d)
    cfg = rcd.make_config(T, D, L, E, 1, k, F, S, Fs, 1)
    y, _, taps = rcd.forward_dropless(cfg, w, x, taps=True)
    f = rcd.ForwardFew(cfg, w, d, taps=True)
    y2 = f(x)
    torch.cuda.synchronize()
    same = (taps["topk_idx"] == f.tap_t["topk_idx"]).all(1)
    assert same.sum() >= T // 2
    a, b = y[same].double(), y2[same].double()
    assert float(((a - b).abs().amax(1) / b.abs().amax(1)).max()) <= 2e-2


def test_columns_of_a_workgroup():
    """Enough columns and experts for 32 columns of the experts' outputs a
    workgroup; a token's bits do not depend on it."""
    d = dev()
    T, D, L, E, k, F, S, Fs = 16, 128, 704, 48, 8, 192, 0, 0
    w = weights(D, L, E, F, S, Fs, 11)
    f, y = check(T, D, L, E, k, F, S, Fs, seed=11, w=w)
    x = torch.randn((T, D), generator=torch.Generator().manual_seed(12)).to(torch.bfloat16).to(d)
    one = rcd.ForwardFew(rcd.make_config(1, D, L, E, 1, k, F, S, Fs, 1), f.w, d)
    y = f(x).clone()
    for t in (0, 7, 15):
        assert torch.equal(one(x[t:t + 1]), y[t:t + 1])


def test_tokens_do_not_see_each_other():
    """A token's output is the same bits alone and among others, in any place."""
    d = dev()
    w = {n: t.to(d) for n, t in weights(256, 128, 20, 192, 1, 128, 7).items()}
    x = torch.randn((16, 256), generator=torch.Generator().manual_seed(8)).to(torch.bfloat16).to(d)
    y = rcd.ForwardFew(rcd.make_config(16, 256, 128, 20, 1, 3, 192, 1, 128, 1), w, d)(x)
    one = rcd.ForwardFew(rcd.make_config(1, 256, 128, 20, 1, 3, 192, 1, 128, 1), w, d)
    for t in range(16):
        assert torch.equal(one(x[t:t + 1])[0], y[t]), t
    # a token that is not a number harms no other
    x2 = x.clone()
    x2[5, 3] = float("nan")
    y2 = rcd.ForwardFew(rcd.make_config(16, 256, 128, 20, 1, 3, 192, 1, 128, 1), w, d)(x2)
    keep = torch.arange(16, device=d) != 5
    assert torch.equal(y2[keep], y[keep]) and torch.isnan(y2[5]).all()


def test_residual_in_place_and_without_taps():
    d = dev()
    w = {n: t.to(d) for n, t in weights(128, 64, 8, 64, 1, 64, 9).items()}
    x = torch.randn((6, 128), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).to(d)
    cfg = rcd.make_config(6, 128, 64, 8, 1, 2, 64, 1, 64, 1)
    f, g = rcd.ForwardFew(cfg, w, d, taps=True), rcd.ForwardFew(cfg, w, d)
    want = f(x, x).clone()
    assert torch.equal(g(x, x), want)
    g.y.copy_(x)
    assert torch.equal(g(x, g.y), want)


def test_empty():
    d = dev()
    w = {n: t.to(d) for n, t in weights(128, 64, 8, 64, 1, 64, 9).items()}
    f = rcd.ForwardFew(rcd.make_config(0, 128, 64, 8, 1, 2, 64, 1, 64, 1), w, d)
    assert f(torch.zeros(0, 128, dtype=torch.bfloat16, device=d)).shape == (0, 128)


def test_streams_and_graph():
    """Two layers on two streams at once, each with its own workspace, and both captured in one graph and in two
    that share a workspace, replayed on new inputs in turn."""
    d = dev()
    w = {n: t.to(d) for n, t in weights(512, 256, 40, 320, 2, 256, 11).items()}
    cfg = rcd.make_config(3, 512, 256, 40, 1, 4, 320, 2, 256, 1)

    def tokens(i):
        return torch.randn((3, 512), generator=torch.Generator().manual_seed(i)).to(torch.bfloat16).to(d)
    ref = rcd.ForwardFew(cfg, w, d)
    xs = [tokens(i) for i in range(4)]
    want = [ref(x).clone() for x in xs]
    a, b = rcd.ForwardFew(cfg, w, d), rcd.ForwardFew(cfg, w, d)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(20):
        with torch.cuda.stream(s):
            a(xs[0])
        with torch.cuda.stream(t):
            b(xs[1])
    torch.cuda.synchronize()
    assert torch.equal(a.y, want[0]) and torch.equal(b.y, want[1])
    b.ws, b._tail = a.ws, (*b._tail[:4], a.ws.data_ptr(), a.ws.numel())
    x = xs[0].clone()
    graphs = []
    for f in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f(x)
        graphs.append(g)
    for i in (1, 2, 3, 0):
        for g, f in zip(graphs, (a, b)):
            x.copy_(xs[i])
            f.y.zero_()
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(f.y, want[i]), i
