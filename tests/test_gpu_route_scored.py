"""route_scored and its gradient against the fp64 oracle.

Tolerances.  A gate is made of fp32 operations on scores: an exponential (one
ulp, 2^-23), 1 + e (2^-24) and a division (2^-24) put a sigmoid within 2^-22;
a softmax score also divides by a sum of at most 1024 terms in at most 70
steps, each 2^-24, so within 2^-17; the renormalising sum and quotient and the
scale add at most 2^-20.  Gradients are held to the same bound of the formula's
value on magnitudes (cancellation included).  Ids are equal."""
import numpy as np
import pytest
import torch

import routing_capacity_dispatch_amd as rcd
from gpu_common import dev, np_i, say
from oracle import scored_routing as sr

pytestmark = pytest.mark.gpu
RTOL = {"sigmoid": 2.0 ** -20, "softmax": 2.0 ** -16}
FLOOR = 2.0 ** -140  # results below fp32's normal range


def cfg_of(T, E, k):
    return rcd.make_config(T, 64, 64, E, 1, k, 64)


def check(T, E, k, logits, bias, kind, groups=1, top_groups=1, group_top=2, renorm=True, scale=2.5):
    d = dev()
    say("route_scored", T, E, k, kind, groups, top_groups, group_top, renorm)
    sc = rcd.scoring(kind, groups, top_groups, group_top, renorm, scale)
    lt = torch.from_numpy(logits).to(d)
    bt = None if bias is None else torch.from_numpy(bias).to(d)
    topk, gates = rcd.route_scored(cfg_of(T, E, k), sc, lt, bt)
    torch.cuda.synchronize()
    ids = np_i(topk)
    ref = sr.select(logits, bias, k, kind, groups, top_groups, group_top)
    assert np.array_equal(ids, ref), np.argwhere(ids != ref)[:5]
    g = gates.cpu().numpy().astype(np.float64)
    rg = sr.gates(logits, ref, kind, renorm, scale)
    assert (np.abs(g - rg) <= RTOL[kind] * np.abs(rg) + FLOOR).all(), np.abs(g - rg).max()
    # the gradient for this selection
    dg = np.random.default_rng(T + E).standard_normal((T, k)).astype(np.float32)
    dl = rcd.route_scored_backward(cfg_of(T, E, k), sc, lt, topk, torch.from_numpy(dg).to(d))
    torch.cuda.synchronize()
    rd, mag = sr.backward(logits, ref, dg, kind, renorm, scale)
    err = np.abs(dl.cpu().numpy().astype(np.float64) - rd)
    assert (err <= RTOL[kind] * mag + FLOOR).all(), (err / (mag + FLOOR)).max()


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 384, 8), (3, 5, 5), (5, 16, 1), (7, 60, 6), (64, 64, 8), (130, 65, 2),
                                   (33, 128, 4), (100, 384, 8), (17, 1000, 8), (9, 1024, 64), (5, 100, 33),
                                   (66, 256, 7), (31, 15, 3), (4, 512, 9)])
def test_matches_oracle(T, E, k, kind, renorm):
    rng = np.random.default_rng(T * 1000 + E)
    logits = (1.5 * rng.standard_normal((T, E))).astype(np.float32)
    bias = (0.05 * rng.standard_normal(E)).astype(np.float32)
    check(T, E, k, logits, bias if E % 2 else None, kind, renorm=renorm)


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("T,E,k,G,tg", [(1, 384, 8, 8, 4), (65, 384, 8, 8, 4), (40, 256, 8, 8, 4), (20, 64, 8, 8, 1),
                                        (30, 60, 6, 4, 2), (12, 12, 3, 12, 3), (10, 64, 2, 64, 40), (9, 1024, 8, 16, 5),
                                        (25, 160, 6, 8, 3), (11, 384, 20, 8, 4), (21, 96, 4, 3, 1), (8, 70, 5, 7, 2)])
def test_group_limit_matches_oracle(T, E, k, G, tg, group_top, kind):
    rng = np.random.default_rng(T * 7 + E + G)
    logits = (1.5 * rng.standard_normal((T, E))).astype(np.float32)
    bias = (0.05 * rng.standard_normal(E)).astype(np.float32)
    check(T, E, k, logits, bias, kind, G, tg, group_top)


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("G,tg", [(1, 1), (8, 3)])
def test_equal_keys_take_the_lower_index(kind, G, tg):
    rng = np.random.default_rng(5)
    # few distinct logits and biases: equal keys within and across groups
    logits = rng.choice(np.array([-1.0, 0.0, -0.0, 0.5], dtype=np.float32), size=(200, 64))
    bias = rng.choice(np.array([0.0, 0.25], dtype=np.float32), size=64)
    check(200, 64, 8, logits, bias, kind, G, tg)
    check(200, 64, 8, logits, None, kind, G, tg)
    check(3, 384, 8, np.zeros((3, 384), np.float32), None, kind, G, tg)


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("G,tg", [(1, 1), (4, 2)])
def test_keys_that_fp32_cannot_tell_apart(kind, G, tg):
    # logits one fp32 step apart near 6 (a sigmoid's slope there is 2^-9, so
    # the scores differ by 2^-30) in random order: only fp64 keys order them
    rng = np.random.default_rng(6)
    E, T = 64, 150
    steps = np.stack([rng.permutation(E) for _ in range(T)])
    logits = (np.float32(6.0) + steps.astype(np.float32) * np.float32(2.0 ** -21)).astype(np.float32)
    check(T, E, 8, logits, None, kind, G, tg)
    # ... and scores whose differences the bias nearly cancels
    l = (1.5 * rng.standard_normal((T, E))).astype(np.float32)
    l[:] = l[:1]
    s = sr.scores(l[:1], kind)[0]
    bias = (0.5 - s).astype(np.float32)  # every key within 2^-25 of 0.5
    check(T, E, 8, l, bias, kind, G, tg)


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("G,tg", [(1, 1), (4, 2)])
def test_infinite_and_extreme_logits(kind, G, tg):
    rng = np.random.default_rng(7)
    T, E = 40, 48
    l = (2 * rng.standard_normal((T, E))).astype(np.float32)
    l[:, ::3] = -np.inf                       # masked experts score 0
    l[0] = -np.inf                            # nothing left: ids in index order, gates 0
    l[1] = -np.inf
    l[1, 17] = 0.5
    l[2] = -3.4028235e38                      # the type's lowest value
    l[3, :5] = [80.0, -80.0, 30.0, -30.0, 100.0]
    l[4] = -200.0                             # sigmoid underflows in fp32
    check(T, E, 6, l, None, kind, G, tg)
    check(T, E, 6, l, None, kind, G, tg, renorm=False)
    bias = np.zeros(E, np.float32)
    bias[5:30] = -np.inf                      # never selected while others are left
    check(T, E, 6, (2 * rng.standard_normal((T, E))).astype(np.float32), bias, kind, G, tg)


def test_no_tokens():
    d = dev()
    sc = rcd.scoring("sigmoid")
    cfg = cfg_of(0, 16, 2)
    topk, gates = rcd.route_scored(cfg, sc, torch.empty((0, 16), device=d))
    assert topk.shape == (0, 2) and gates.shape == (0, 2)
    assert rcd.route_scored_backward(cfg, sc, torch.empty((0, 16), device=d), topk, gates).shape == (0, 16)


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
def test_backward_ids_outside_and_twice(kind):
    d = dev()
    rng = np.random.default_rng(8)
    T, E, k = 30, 40, 4
    l = rng.standard_normal((T, E)).astype(np.float32)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    ids[3, 1] = ids[3, 0]
    ids[4] = ids[4, 0]
    ids[5, 2], ids[6, 0], ids[7] = -1, E, [-5, 1 << 30, E + 1, -(1 << 31)]
    dg = rng.standard_normal((T, k)).astype(np.float32)
    for renorm in (False, True):
        sc = rcd.scoring(kind, renormalise=renorm, scale=1.5)
        got = rcd.route_scored_backward(cfg_of(T, E, k), sc, torch.from_numpy(l).to(d),
                                        torch.from_numpy(ids.astype(np.int32)).to(d), torch.from_numpy(dg).to(d))
        torch.cuda.synchronize()
        ref, mag = sr.backward(l, ids, dg, kind, renorm, 1.5)
        # row 7 has no expert: S is the 1e-20 of the formula and every factor is 0
        assert (np.abs(got.cpu().numpy() - ref) <= RTOL[kind] * mag + FLOOR).all()


def test_large_batch_matches_small_ones():
    # a batch of every size class gives each token what it gets alone
    d = dev()
    g = torch.Generator(device="cpu").manual_seed(9)
    T, E, k = 5000, 384, 8
    l = (1.5 * torch.randn((T, E), generator=g)).to(d)
    b = (0.05 * torch.randn(E, generator=g)).to(d)
    sc = rcd.scoring("sigmoid", 8, 4, 2, True, 2.5)
    topk, gates = rcd.route_scored(cfg_of(T, E, k), sc, l, b)
    for t in (0, 1, 2, 3, 17, 4095, 4999):
        t1, g1 = rcd.route_scored(cfg_of(1, E, k), sc, l[t:t + 1].contiguous(), b)
        assert torch.equal(t1[0], topk[t]) and torch.equal(g1[0], gates[t])
    ln, ref = l.cpu().numpy(), None
    ref = sr.select(ln[:600], b.cpu().numpy(), k, "sigmoid", 8, 4, 2)
    assert np.array_equal(np_i(topk)[:600], ref)


def test_graph_replays_and_side_stream():
    d = dev()
    g = torch.Generator(device="cpu").manual_seed(10)
    T, E, k = 300, 64, 6
    cfg, sc = cfg_of(T, E, k), rcd.scoring("softmax", 4, 2, 2, False, 1.0)
    ls = [torch.randn((T, E), generator=g).to(d) for _ in range(3)]
    b = (0.05 * torch.randn(E, generator=g)).to(d)
    dgs = [torch.randn((T, k), generator=g).to(d) for _ in range(3)]
    x, dg = ls[0].clone(), dgs[0].clone()
    out = dict(topk_idx=torch.empty((T, k), dtype=torch.int32, device=d), gates=torch.empty((T, k), device=d))
    dl = torch.empty((T, E), device=d)

    def call():
        rcd.route_scored(cfg, sc, x, b, out=out)
        rcd.route_scored_backward(cfg, sc, x, out["topk_idx"], dg, d_logits=dl)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in (0, 1, 2, 0):
        x.copy_(ls[i])
        dg.copy_(dgs[i])
        for t in (*out.values(), dl):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        t2, g2 = rcd.route_scored(cfg, sc, ls[i], b)
        d2 = rcd.route_scored_backward(cfg, sc, ls[i], t2, dgs[i])
        torch.cuda.synchronize()
        assert torch.equal(out["topk_idx"], t2) and torch.equal(out["gates"], g2) and torch.equal(dl, d2)


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("lower", [False, True])
@pytest.mark.parametrize("E,G,tg,k", [(256, 8, 1, 2), (256, 8, 2, 4), (64, 4, 2, 4), (1024, 8, 2, 8)])
def test_group_boundary_below_fp32(E, G, tg, k, lower, kind):
    # Equal scores (exact: 1/2, or 1/E), so the bias ranks the groups.  Two
    # groups' pairs of largest biases sum to 0.375 and 0.375 + 2^-26 (or
    # - 2^-26): fp32 sums of the keys cannot tell them apart, while the keys
    # themselves are far from each other.  The other tokens are ordinary.
    rng = np.random.default_rng(E + tg)
    size = E // G
    bias = (-1 - np.arange(E) / E).astype(np.float32)
    a, b = 1, G - 2  # a would win a tie
    bias[a * size + 1], bias[a * size + 5] = 0.25, 0.125
    bias[b * size + 2] = 0.15625
    bias[b * size + 4] = np.float32(0.21875 + (-1 if lower else 1) * 2.0 ** -26)
    assert float(bias[b * size + 4]) != 0.21875
    if tg == 2:  # one group above both
        bias[0], bias[1] = 0.5, 0.4375
    logits = np.zeros((21, E), dtype=np.float32)
    logits[1::3] = rng.standard_normal((7, E))
    ref = sr.select(logits, bias, k, kind, G, tg, 2)
    assert (a if lower else b) in ref[0] // size and (b if lower else a) not in ref[0] // size
    check(21, E, k, logits, bias, kind, G, tg, 2)


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("E,k,G,tg", [(64, 8, 1, 1), (64, 8, 8, 2), (384, 8, 8, 4), (60, 4, 4, 1), (60, 12, 6, 2), (1024, 64, 1, 1)])
def test_what_is_no_number_leaves_ids_in_range(E, k, G, tg, with_bias, kind):
    # ids index the dispatch's rows: they are different and inside [0, E)
    # whatever the logits are, and the other tokens are not touched
    rng = np.random.default_rng(E + k)
    l = rng.standard_normal((40, E)).astype(np.float32)
    b = (0.05 * rng.standard_normal(E)).astype(np.float32) if with_bias or G > 1 else None
    ref = sr.select(l, b, k, kind, G, tg, 2)
    bad = {2: np.nan, 5: np.inf, 11: np.nan, 12: np.inf, 13: -np.inf}
    for t, v in bad.items():
        l[t, rng.permutation(E)[:max(E // 2, E - k + 2) if t > 10 else 3]] = v
    l[17], l[18], l[19] = np.nan, np.inf, -np.inf
    odd = [*bad, 17, 18, 19]
    d = dev()
    sc = rcd.scoring(kind, G, tg, 2)

    def ids(bias):
        t, _ = rcd.route_scored(cfg_of(40, E, k), sc, torch.from_numpy(l).to(d),
                                None if bias is None else torch.from_numpy(bias).to(d))
        torch.cuda.synchronize()
        t = np_i(t)
        assert ((t >= 0) & (t < E)).all()
        assert all(len(set(r)) == k for r in t.tolist())
        return t
    keep = [t for t in range(40) if t not in odd]
    assert np.array_equal(ids(b)[keep], ref[keep])
    if b is not None:
        for v in (np.inf, np.nan):
            c = b.copy()
            c[[1, E - 2]] = v
            ids(c)
        ids(np.full(E, np.nan, dtype=np.float32))
        ids(np.full(E, np.inf, dtype=np.float32))


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k", [(1, 64, 8), (3, 384, 8), (40, 60, 6), (33, 61, 7), (9, 8, 8), (5, 1024, 8), (17, 128, 1),
                                   (6, 100, 12)])
def test_negative_zeros_are_zeros(T, E, k, kind):
    # the two zeros are one key: equal ones are taken in index order.  Every
    # other logit is negative, so that zeros are what is selected: -0.0 alone,
    # both zeros mixed, one -0.0, and -0.0 as the last key taken
    rng = np.random.default_rng(T + E + k)
    l = -np.abs(rng.standard_normal((T, E)).astype(np.float32)) - np.float32(0.1)
    check(T, E, k, np.full((T, E), -0.0, np.float32), None, kind)
    check(T, E, k, rng.choice(np.array([0.0, -0.0], np.float32), size=(T, E)), None, kind)
    check(T, E, k, rng.choice(np.array([-1.0, 0.0, -0.0], np.float32), size=(T, E)), None, kind, renorm=False)
    one = l.copy()
    one[np.arange(T), rng.integers(0, E, T)] = -0.0
    check(T, E, k, one, None, kind)
    last = l.copy()
    for t in range(T):
        at = rng.permutation(E)[:k]
        last[t, at] = 1.0 + np.arange(k)
        last[t, at[0]] = -0.0
    check(T, E, k, last, None, kind)
    if E % 4 == 0:  # every group kept: no limit
        check(T, E, k, one, None, kind, 4, 4)


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G,tg", [(64, 1, 1), (61, 1, 1), (64, 8, 2)])
def test_signalling_nans_are_taken_last(E, G, tg, kind):
    # a NaN of either kind and sign among finite logits: the ids are different
    # and in range, and the other tokens are not touched
    d = dev()
    rng = np.random.default_rng(E)
    l = rng.standard_normal((24, E)).astype(np.float32)
    ref = sr.select(l, None, 6, kind, G, tg, 2)
    bits = np.array([0x7F800001, 0xFF800001, 0x7FC00000, 0xFFC00000], dtype=np.uint32)
    for t in range(0, 24, 3):
        l.view(np.uint32)[t, rng.permutation(E)[:E // 2]] = bits[t // 3 % 4]
    topk, _ = rcd.route_scored(cfg_of(24, E, 6), rcd.scoring(kind, G, tg, 2), torch.from_numpy(l).to(d))
    torch.cuda.synchronize()
    ids = np_i(topk)
    assert ((ids >= 0) & (ids < E)).all() and all(len(set(r)) == 6 for r in ids.tolist())
    keep = [t for t in range(24) if t % 3]
    assert np.array_equal(ids[keep], ref[keep])


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G,tg,k", [(64, 8, 4, 8), (256, 8, 3, 6), (64, 4, 1, 2), (128, 16, 5, 4), (60, 6, 2, 3)])
@pytest.mark.parametrize("size", [128.0, 1000.0, 1e5])
def test_group_sums_of_large_keys_that_cancel(size, E, G, tg, k, kind):
    # one bias of +size and the others -size in every group: its two largest
    # keys nearly cancel, so their sum says nothing of how far the fp32 keys
    # are off, half a step of theirs (2^-24 size) each.  The two experts'
    # logits spread the groups' sums over a few such steps (a sigmoid's slope
    # at 0.3 is 0.24), and the rest of a group lies well below
    rng = np.random.default_rng(E + G + int(size))
    gs = E // G
    first, second = (np.arange(G) * gs + rng.permuted(np.tile(np.arange(gs), (G, 1)), axis=1)[:, :2].T)
    bias = np.full(E, -size, np.float32)
    bias[first] = size
    T = 64
    l = np.full((T, E), -4.0, np.float32)
    for t in range(T):
        for at in (first, second):
            l[t, at] = 0.3 + size * 2.0 ** (-22 + t % 3) * rng.standard_normal(G)
    check(T, E, k, l, bias, kind, G, tg, 2)


@pytest.mark.parametrize("E,G,tg,k", [(384, 8, 4, 8), (64, 4, 2, 6), (100, 1, 1, 5), (256, 16, 4, 8), (40, 8, 3, 8)])
@pytest.mark.parametrize("spread", [6.0, 16.0, 60.0, 400.0])
@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
def test_sharp_scores_match_oracle(spread, E, G, tg, k, kind):
    # Most scores are far below the largest, down to those that fp32 and fp64
    # exponentials turn to 0; pairs of neighbouring logits among them.
    # Ids are equal.  Gates and gradients within RTOL of their magnitudes, and
    # what a score below fp32's normal range, a multiple of 2^-149 and so off
    # by up to 2 of those (its exponential's and its product's rounding),
    # makes of it: a gate scale s / S moves by scale 2^-148 / S for its own s
    # and by at most as much for each of the k in S; a gradient ds s (1 - s)
    # by |ds| 2^-148 for its own s and, through S and the sum of dg s, by at
    # most 3 k |ds| (s / S) 2^-148, s / S <= 1, |ds| the largest of the token.
    def check(T, E, k, logits, bias, kind, groups, top_groups):
        d = dev()
        say("sharp", E, k, kind, groups, top_groups, bias is not None)
        sc = rcd.scoring(kind, groups, top_groups, 2, True, 2.5)
        lt = torch.from_numpy(logits).to(d)
        topk, gates = rcd.route_scored(cfg_of(T, E, k), sc, lt, None if bias is None else torch.from_numpy(bias).to(d))
        torch.cuda.synchronize()
        ref = sr.select(logits, bias, k, kind, groups, top_groups, 2)
        assert np.array_equal(np_i(topk), ref)
        S = np.take_along_axis(sr.scores(logits, kind), ref, axis=1).sum(axis=1, keepdims=True) + 1e-20
        rg = sr.gates(logits, ref, kind, True, 2.5)
        err = np.abs(gates.cpu().numpy().astype(np.float64) - rg)
        assert (err <= RTOL[kind] * rg + FLOOR + (k + 1) * 2.5 * 2.0 ** -148 / S).all()
        dg = np.random.default_rng(T + E).standard_normal((T, k)).astype(np.float32)
        dl = rcd.route_scored_backward(cfg_of(T, E, k), sc, lt, topk, torch.from_numpy(dg).to(d))
        torch.cuda.synchronize()
        rd, mag = sr.backward(logits, ref, dg, kind, True, 2.5)
        ds = 2 * 2.5 * np.abs(dg).max(axis=1, keepdims=True) / S
        err = np.abs(dl.cpu().numpy().astype(np.float64) - rd)
        assert (err <= RTOL[kind] * mag + FLOOR + (3 * k + 1) * 2.0 ** -148 * ds).all()
    rng = np.random.default_rng(E + int(spread))
    l = (spread * rng.standard_normal((50, E))).astype(np.float32)
    pair = rng.permutation(E)[:E // 4 * 2].reshape(2, -1)
    l[::2, pair[1]] = np.nextafter(l[::2, pair[0]], np.float32(np.inf))
    low = l - l.max(axis=1, keepdims=True)
    tiny = (2.0 ** -20 * rng.standard_normal(E)).astype(np.float32)
    for x in (l, low, (low - 30).astype(np.float32)):
        for b in (None, tiny, (0.05 * rng.standard_normal(E)).astype(np.float32)):
            check(50, E, k, x, b, kind, G, tg)


def test_sharp_softmax_scores_keep_the_pace():
    # errors of fp32 scores shrink with the scores, so a batch of sharp ones
    # settles its tokens as a batch of flat ones does (the whole-wavefront
    # fp64 selection of a third of them takes five times as long)
    d = dev()
    T, E, k = 16384, 384, 8
    g = torch.Generator(device=d).manual_seed(3)
    n = torch.randn((T, E), generator=g, device=d)
    cfg, sc = cfg_of(T, E, k), rcd.scoring("softmax", 8, 4)
    out = dict(topk_idx=torch.empty((T, k), dtype=torch.int32, device=d), gates=torch.empty((T, k), device=d))

    def us(l):
        times = []
        for _ in range(9):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for _ in range(20):
                rcd.route_scored(cfg, sc, l, None, out=out)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b) * 50)
        return sorted(times)[4]
    us(n)
    flat, sharp = us(1.5 * n), us(16.0 * n)
    say("softmax scores, flat and sharp, us", flat, sharp)
    assert sharp <= 2.5 * flat


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G,tg,k", [(64, 8, 3, 6), (256, 16, 5, 8), (60, 6, 2, 4)])
def test_group_sums_past_fp32(E, G, tg, k, kind):
    # two biases of a group whose sum is no fp32 number: still ordered as real
    # numbers, in both directions
    rng = np.random.default_rng(E)
    gs = E // G
    bias = (0.05 * rng.standard_normal(E)).astype(np.float32)
    for sign in (1.0, -1.0):
        b = bias.copy()
        for g in rng.permutation(G)[:G - 1]:
            if sign > 0:
                b[g * gs + rng.permutation(gs)[:2]] = rng.uniform(1.8e38, 2.9e38, 2).astype(np.float32)
            else:
                b[g * gs:(g + 1) * gs] = -rng.uniform(1.8e38, 2.9e38, gs).astype(np.float32)
        l = (1.5 * rng.standard_normal((30, E))).astype(np.float32)
        check(30, E, k, l, b, kind, G, tg, 2)
