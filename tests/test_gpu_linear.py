"""Linear layers with their epilogue and their gradients against a plain
computation in 64 bits.

Tolerances.  A product of bf16 values is exact in fp32; sums of K of them in
any order lose at most (K + 8) 2^-24 of the summed magnitudes, bias included.
The activations' slope is at most 1.13, and the fp32 activation itself is off by
2^-20 (1 + |u|) at most (an exponential, a reciprocal, an erf of a few ulp
each).  A rounding to bf16 loses 2^-8 of the value at most, one to fp32 2^-24.
d = dy act'(pre) is rounded to bf16 for the products unless it is dy itself."""
import numpy as np
import pytest
import torch

import routing_capacity_dispatch_amd as rcd
from gpu_common import dev, say

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def np64(t):
    return t.detach().cpu().double().numpy()


def act64(u, act):
    from scipy.special import erf
    with np.errstate(over="ignore"):
        return {"none": u, "relu": np.maximum(u, 0), "silu": u / (1 + np.exp(-u)),
                "gelu": 0.5 * u * (1 + erf(u / np.sqrt(2)))}[act]


def slope64(u, act):
    from scipy.special import erf
    if act == "none":
        return np.ones_like(u)
    if act == "relu":
        return (u > 0).astype(np.float64)
    if act == "silu":
        p = 1 / (1 + np.exp(-u))
        return p * (1 + u * (1 - p))
    return 0.5 * (1 + erf(u / np.sqrt(2))) + u * np.exp(-0.5 * u * u) / np.sqrt(2 * np.pi)


def rand(shape, seed, dtype=BF, scale=1.0):
    g = torch.Generator(device="cpu").manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def held(t, d, shift=0, pad=0):
    """t on the device inside a larger buffer of NaN: rows `pad` values further apart, the first `shift` values in.
    Returns the view, and the buffer with a mask of what lies outside the view."""
    rows, cols = t.shape
    buf = torch.full((shift + rows * (cols + pad) + 32,), float("nan"), dtype=t.dtype, device=d)
    v = buf[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols] if rows and cols else \
        t.to(d).reshape(rows, cols)
    v.copy_(t)
    return v, buf


def untouched(buf, shift, rows, cols, pad):
    """Every value of buf outside the [rows, cols] view is still NaN."""
    b = buf.clone()
    b[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols] = float("nan")
    return bool(torch.isnan(b.float()).all())


def half(dtype):
    return 2.0 ** -8 if dtype == BF else 2.0 ** -24


def check_linear(M, N, K, act="none", bias=None, res=False, out=BF, pre=False, shift=0, pad=0, seed=0, inplace=False):
    d = dev()
    say("linear", M, N, K, act, bias, res, out, pre, "shift", shift, "pad", pad)
    xs, ws = rand((M, K), seed), rand((N, K), seed + 1, scale=max(K, 1) ** -0.5)
    b = rand((N,), seed + 2, bias, 0.5) if bias else None
    rs = rand((M, N), seed + 3, out) if res else None
    x, _ = held(xs, d, shift, pad)
    w, _ = held(ws, d, shift, pad)
    r = held(rs, d, shift, pad)[0] if res else None
    y, buf = held(torch.zeros(M, N, dtype=out), d, shift, pad)
    if inplace:
        y.copy_(rs)
        r = y
    got = rcd.linear(x, w, None if b is None else b.to(d), act=act, residual=r, out_dtype=out, save_pre=pre, out=y)
    torch.cuda.synchronize()
    got, kept = got if pre else (got, None)
    assert got.data_ptr() == y.data_ptr()
    if M and N:
        assert untouched(buf, shift, M, N, pad)
    xn, wn = np64(xs), np64(ws)
    u = xn @ wn.T
    mag = np.abs(xn) @ np.abs(wn).T
    if b is not None:
        u, mag = u + np64(b), mag + np.abs(np64(b))
    eu = (K + 8) * 2.0 ** -24 * mag
    ref = act64(u, act)
    e = 1.13 * eu + (2.0 ** -20 * (1 + np.abs(u)) if act in ("silu", "gelu") else 0)
    if res:
        ref = ref + np64(rs)
    e = e + half(out) * (np.abs(ref) + e) + 2.0 ** -24 * np.abs(ref)
    assert (np.abs(np64(got) - ref) <= e).all()
    if pre:
        assert (np.abs(np64(kept) - u) <= eu + half(BF) * (np.abs(u) + eu)).all()


# rows: one, below and at a block of 16, the last few-row kernel, the first tile, past a tile; K: below a chunk, odd,
# at and past a K tile
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 1), (1, 64, 128), (1, 1000, 2048), (3, 17, 5), (15, 100, 129), (16, 48, 64), (17, 33, 1000), (33, 250, 96),
    (64, 128, 256), (65, 128, 64), (65, 1, 7), (100, 129, 8), (127, 255, 65), (128, 128, 128), (130, 300, 1250),
    (257, 513, 72), (300, 40, 4000), (1000, 1000, 31), (17, 6144, 700), (40, 2048, 1600), (640, 640, 1300),
    (500, 900, 2050)])
@pytest.mark.parametrize("out", [BF, F32])
def test_linear_sizes(M, N, K, out):
    check_linear(M, N, K, "silu", BF, True, out, True, seed=M + N + K)


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("bias", [None, BF, F32])
@pytest.mark.parametrize("M", [5, 200])
def test_linear_epilogues(act, bias, M):
    check_linear(M, 136, 192, act, bias, False, BF, act != "none", seed=7)
    check_linear(M, 136, 192, act, bias, True, F32, False, seed=8)


# rows of no alignment, of 16 bytes and strided; the neighbours are NaN
@pytest.mark.parametrize("shift,pad", [(0, 8), (1, 0), (3, 5), (8, 24)])
@pytest.mark.parametrize("M", [1, 40, 190])
@pytest.mark.parametrize("out", [BF, F32])
def test_linear_strides(shift, pad, M, out):
    check_linear(M, 200, 136, "gelu", F32, True, out, True, shift, pad, seed=11)
    check_linear(M, 77, 131, "none", None, False, out, False, shift, pad, seed=12)


# whole rounds of large tiles, with ends inside a tile, and K shared by many workgroups
@pytest.mark.parametrize("M,N,K", [(3500, 3601, 200), (4096, 3328, 64), (72, 64, 40000),
                                   (200, 136, 20003), (2100, 2000, 130)])
def test_linear_large_and_shared(M, N, K):
    check_linear(M, N, K, "relu", BF, True, BF, True, seed=3)


@pytest.mark.parametrize("M", [4, 150])
def test_linear_residual_in_place(M):
    check_linear(M, 64, 64, "none", None, True, BF, inplace=True)
    check_linear(M, 72, 64, "silu", None, True, F32, inplace=True)


@pytest.mark.parametrize("M,N,K", [(0, 5, 8), (5, 0, 8), (5, 8, 0), (100, 24, 0), (0, 0, 0)])
def test_linear_empty(M, N, K):
    check_linear(M, N, K, "gelu", BF, True, BF, True)


def test_linear_infinities_stay_in_their_row():
    d = dev()
    for M, K in ((8, 100), (200, 104)):
        x, w = rand((M, K), 1).to(d), rand((64, K), 2).to(d)
        ref = rcd.linear(x, w, act="gelu")
        x[3, K - 1] = float("inf")
        x[5, 0] = float("nan")
        y = rcd.linear(x, w, act="gelu")
        keep = torch.ones(M, dtype=torch.bool, device=d)
        keep[3] = keep[5] = False
        assert torch.equal(y[keep], ref[keep]) and torch.isnan(y[5]).all()
        assert torch.isinf(rcd.linear(x, w)[3]).all()


def check_grad(M, N, K, act="silu", dt=BF, shift=0, pad=0, seed=0, need=(True, True, True)):
    d = dev()
    say("linear_backward", M, N, K, act, dt, "shift", shift, "pad", pad, need)
    xs, ws = rand((M, K), seed), rand((N, K), seed + 1, scale=max(N, 1) ** -0.5)
    dys, ps = rand((M, N), seed + 2, dt), rand((M, N), seed + 3, scale=2.0)
    x, w, dy, p = (held(t, d, shift, pad)[0] for t in (xs, ws, dys, ps))
    odx, bx = held(torch.zeros(M, K, dtype=BF), d, shift, pad)
    odw, bw = held(torch.zeros(N, K, dtype=BF), d, shift, pad)
    dx, dw, db = rcd.linear_backward(dy, x, w, pre=None if act == "none" else p, act=act, bias=need[2],
                                     need_dx=need[0], need_dw=need[1], dx=odx, dw=odw)
    torch.cuda.synchronize()
    xn, wn, dyn, pn = np64(xs), np64(ws), np64(dys), np64(ps)
    dn = dyn * slope64(pn, act)
    ed = np.abs(dyn) * 2.0 ** -20 * (1 + np.abs(pn)) if act in ("silu", "gelu") else np.zeros_like(dn)
    er = ed + (0 if act == "none" and dt == BF else 2.0 ** -8 * (np.abs(dn) + ed))
    if need[2]:
        e = ed.sum(0) + (M + 8) * 2.0 ** -24 * np.abs(dn).sum(0)
        assert (np.abs(np64(db) - dn.sum(0)) <= e).all()
    else:
        assert db is None
    for got, buf, l, el, r, on in ((dx, bx, dn, er, wn, need[0]), (dw, bw, dn.T, er.T, xn, need[1])):
        if not on:
            assert got is None and torch.equal(torch.isnan(buf.float()).sum(), torch.isnan(bx.float() if buf is bx else bw.float()).sum())
            continue
        ref = l @ r
        e = el @ np.abs(r) + (l.shape[1] + 8) * 2.0 ** -24 * (np.abs(l) @ np.abs(r))
        assert (np.abs(np64(got) - ref) <= e + 2.0 ** -8 * (np.abs(ref) + e)).all()
        if got.numel():
            assert untouched(buf, shift, got.shape[0], got.shape[1], pad)


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 100, 64), (16, 24, 40), (63, 8, 129), (64, 128, 128), (100, 131, 77),
                                   (129, 257, 300), (1000, 65, 130), (700, 520, 260), (3000, 33, 16)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_backward_sizes(M, N, K, dt):
    check_grad(M, N, K, "silu", dt, seed=M + N)
    check_grad(M, N, K, "none", dt, seed=M + N)


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("shift,pad", [(0, 0), (0, 8), (1, 0), (5, 3)])
def test_backward_strides(act, shift, pad):
    check_grad(150, 72, 88, act, BF, shift, pad, seed=5)
    check_grad(70, 51, 133, act, F32, shift, pad, seed=6)


@pytest.mark.parametrize("need", [(True, False, False), (False, True, False), (False, False, True), (True, True, False),
                                  (False, False, False)])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_backward_parts(need, act):
    check_grad(96, 48, 56, act, BF, need=need)


# the large tiles of both products
def test_backward_large():
    check_grad(3600, 3400, 272, "gelu", BF, seed=9)
    check_grad(264, 3700, 3400, "relu", BF, seed=10)


@pytest.mark.parametrize("M,N,K", [(0, 6, 8), (6, 0, 8), (6, 8, 0), (0, 0, 0)])
def test_backward_empty(M, N, K):
    d = dev()
    z = lambda r, c: torch.zeros(r, c, dtype=BF, device=d)  # noqa: E731
    for act in ("none", "silu"):
        dx, dw, db = rcd.linear_backward(z(M, N), z(M, K), z(N, K), pre=z(M, N), act=act,
                                         dx=torch.full((M, K), 7.0, dtype=BF, device=d),
                                         dw=torch.full((N, K), 7.0, dtype=BF, device=d),
                                         db=torch.full((N,), 7.0, device=d))
        torch.cuda.synchronize()
        assert (dx == 0).all() and (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_training_step_against_differences(act):
    """Forward, then backward from what it kept: the change of a loss along a direction, by central differences of
    the 64-bit layer, against <gradient, direction>."""
    d = dev()
    M, N, K = 130, 72, 96
    xs, ws, bs = rand((M, K), 1), rand((N, K), 2, scale=K ** -0.5), rand((N,), 3, F32, 0.3)
    c = rand((M, N), 4)  # loss = <c, y>
    _, pre = rcd.linear(xs.to(d), ws.to(d), bs.to(d), act=act, residual=c.to(d), save_pre=True)
    dx, dw, db = rcd.linear_backward(c.to(d), xs.to(d), ws.to(d), pre=pre, act=act)
    torch.cuda.synchronize()
    X, W, B, Cn = np64(xs), np64(ws), np64(bs), np64(c)

    def loss(x, w, b):
        return float((Cn * act64(x @ w.T + b, act)).sum())
    rng = np.random.RandomState(0)
    h = 1e-5
    for got, i in ((dx, 0), (dw, 1), (db, 2)):
        v = rng.standard_normal(tuple(got.shape))
        at = [X, W, B]
        hi, lo = list(at), list(at)
        hi[i], lo[i] = at[i] + h * v, at[i] - h * v
        slope = (loss(*hi) - loss(*lo)) / (2 * h)
        g = np64(got)
        # pre, d and the gradient are each rounded to bf16: under 2^-8 (1 + 2 + 1) of each term, whose signs are random:
        # a tenth of the sum of magnitudes times that bounds the sum with room
        assert abs((g * v).sum() - slope) <= 4 * 2.0 ** -8 * np.sqrt((np.abs(g * v) ** 2).sum()) * 4 + 1e-3


def test_streams_and_graph():
    """On another stream than the tensors' own, and captured once and replayed on new inputs, both bit for bit."""
    d = dev()
    for M, K in ((5, 300), (150, 301)):
        x, w, b = rand((M, K), 1).to(d), rand((90, K), 2).to(d), rand((90,), 3).to(d)
        r, dy = rand((M, 90), 4).to(d), rand((M, 90), 5).to(d)

        def step():
            y, pre = rcd.linear(x, w, b, act="silu", residual=r, save_pre=True)
            return [y, pre, *rcd.linear_backward(dy, x, w, pre=pre, act="silu")]
        want = [t.clone() for t in step()]
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got = step()
        s.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = step()
        for i in range(3):
            x.copy_(rand((M, K), 20 + i))
            want = [t.clone() for t in step()]
            for t in got:
                t.zero_()
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(got, want)), i


def test_workspace_of_the_caller():
    d = dev()
    x, w = rand((100, 30001), 1).to(d), rand((40, 30001), 2).to(d)
    ref = rcd.linear(x, w)
    ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device=d)
    assert torch.equal(rcd.linear(x, w, ws=ws), ref)
    with pytest.raises(rcd.MoeError, match="WORKSPACE"):
        rcd.linear(x, w, ws=ws[:256])
    with pytest.raises(ValueError):
        rcd.linear(x, w, ws=ws.cpu())
