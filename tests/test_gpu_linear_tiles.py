"""Every kernel of the linear layers and of their gradients against 64 bits (of
the same operands, on the GPU), at the sizes of forms.py, with every epilogue,
strides, residuals in place, values that are no numbers, and captured.

Tolerances are those of test_gpu_linear.py: (K + 8) 2^-24 of the summed
magnitudes, slopes of at most 1.13, 2^-20 (1 + |u|) for an activation, half a
step for a rounding."""
import pytest
import torch

import forms
import routing_capacity_dispatch_amd as rcd
from gpu_common import dev, say

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
EPILOGUES = [  # act, bias, residual, out, pre-activation kept, residual in place, (shift, pad) of outputs and residual
    ("gelu", F32, True, F32, True, False, (0, 0)), ("none", BF, False, BF, False, False, (1, 5)),
    ("silu", None, True, BF, True, True, (8, 8)), ("relu", F32, True, BF, True, False, (3, 1)),
    ("none", None, True, F32, False, True, (1, 3))]


def rand(gen, shape, dtype=BF, scale=1.0):
    return (torch.randn(shape, generator=gen, device=gen.device) * scale).to(dtype)


def held(t, at, fill=float("nan")):
    """t inside a larger buffer of NaN: rows at[1] values further apart, the first at[0] values in."""
    rows, cols = t.shape
    buf = torch.full((at[0] + rows * (cols + at[1]) + 32,), fill, dtype=t.dtype, device=t.device)
    v = buf[at[0]:at[0] + rows * (cols + at[1])].view(rows, cols + at[1])[:, :cols]
    v.copy_(t)
    return v, buf


def outside_is_nan(v, buf):
    b = buf.clone()
    b.as_strided(v.shape, v.stride(), v.storage_offset()).fill_(float("nan"))
    return bool(torch.isnan(b).all())


def act64(u, act):
    return {"none": lambda: u, "relu": lambda: u.clamp(min=0), "silu": lambda: u / (1 + torch.exp(-u)),
            "gelu": lambda: 0.5 * u * (1 + torch.erf(u * 0.5 ** 0.5))}[act]()


def slope64(u, act):
    if act == "none":
        return torch.ones_like(u)
    if act == "relu":
        return (u > 0).double()
    if act == "silu":
        p = 1 / (1 + torch.exp(-u))
        return p * (1 + u * (1 - p))
    return 0.5 * (1 + torch.erf(u * 0.5 ** 0.5)) + u * torch.exp(-0.5 * u * u) * (2 * torch.pi) ** -0.5


def half(dtype):
    return 2.0 ** -8 if dtype == BF else 2.0 ** -24


@pytest.mark.parametrize("form,size,x_at,w_at", forms.LINEAR)
def test_forward(form, size, x_at, w_at):
    d = dev()
    M, N, K = size
    say("linear", form, size, x_at, w_at)
    gen = torch.Generator(device=d).manual_seed(M + N + K)
    x, _ = held(rand(gen, (M, K)), x_at)
    w, _ = held(rand(gen, (N, K), scale=K ** -0.5), w_at)
    # a user's tensors start on 16 bytes by themselves
    assert x.data_ptr() % 16 == 2 * x_at[0] % 16 and w.data_ptr() % 16 == 2 * w_at[0] % 16
    u0 = x.double() @ w.double().t()
    mag0 = x.double().abs() @ w.double().abs().t()
    b0, r0 = rand(gen, (N,), F32, 0.5), rand(gen, (M, N), F32)
    for act, bias, res, out, pre, inplace, o_at in EPILOGUES:
        b = None if bias is None else b0.to(bias)
        r = held(r0.to(out), o_at)[0] if res else None
        y, buf = held(r0.to(out) if inplace else torch.zeros((M, N), dtype=out, device=d), o_at)
        got = rcd.linear(x, w, b, act=act, residual=y if inplace else r, out_dtype=out, save_pre=pre, out=y)
        torch.cuda.synchronize()
        got, kept = got if pre else (got, None)
        assert got.data_ptr() == y.data_ptr() and outside_is_nan(y, buf)
        u = u0 if b is None else u0 + b.double()
        eu = (K + 8) * 2.0 ** -24 * (mag0 if b is None else mag0 + b.double().abs())
        ref = act64(u, act)
        e = 1.13 * eu + (2.0 ** -20 * (1 + u.abs()) if act in ("silu", "gelu") else 0)
        if res:
            ref = ref + r0.to(out).double()
        e = e + half(out) * (ref.abs() + e) + 2.0 ** -24 * ref.abs()
        assert ((got.double() - ref).abs() <= e).all(), act
        if pre:
            assert ((kept.double() - u).abs() <= eu + half(BF) * (u.abs() + eu)).all(), act


@pytest.mark.parametrize("form,size,x_at,w_at", forms.LINEAR)
def test_forward_not_numbers_and_captured(form, size, x_at, w_at):
    """What is no number stays in its row and column; two calls and a replayed one give the same bits."""
    d = dev()
    M, N, K = size
    say("linear", form, size, "not numbers, graph")
    gen = torch.Generator(device=d).manual_seed(M * 3 + N)
    xs, ws = rand(gen, (M, K)), rand(gen, (N, K), scale=K ** -0.5)
    x, w, b, r = held(xs, x_at)[0], held(ws, w_at)[0], rand(gen, (N,)), rand(gen, (M, N))

    def step():
        return rcd.linear(x, w, b, act="silu", residual=r, save_pre=True)
    want = [t.clone() for t in step()]
    assert all(torch.equal(p, q) for p, q in zip(step(), want))
    rows, cols = [M // 3, M - 1], [N // 2, N - 1]
    x[rows[0], K - 1] = float("nan")
    x[rows[1], 0] = float("nan")
    w[cols[0], K // 2] = float("inf")
    w[cols[1], K - 1] = float("nan")
    got = step()
    inside = torch.ones((M, N), dtype=torch.bool, device=d)
    inside[rows] = False
    inside[:, cols] = False
    for p, q in zip(got, want):
        assert torch.equal(p[inside], q[inside])
        assert torch.isnan(p[rows]).all() and torch.isnan(p[:, cols[1]]).all()
        assert not torch.isfinite(p[:, cols[0]].float()).all()
    x.copy_(xs)
    w.copy_(ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(3):
        x.copy_(xs.roll(i + 1, 0))
        want = [t.clone() for t in step()]
        for t in got:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want)), i


def gradients(case):
    form, act, fp32, (M, N, K), x_at, w_at, pad_dy = case
    d = dev()
    gen = torch.Generator(device=d).manual_seed(M + 2 * N + 3 * K)
    x, _ = held(rand(gen, (M, K)), x_at)
    w, _ = held(rand(gen, (N, K), scale=N ** -0.5), w_at)
    dy, _ = held(rand(gen, (M, N), F32 if fp32 else BF), (0, pad_dy))
    pre = rand(gen, (M, N), scale=2.0)
    return act, x, w, dy, pre


@pytest.mark.parametrize("case", forms.BACKWARD, ids=lambda c: c[0])
def test_backward(case):
    say("linear_backward", *case)
    act, x, w, dy, pre = gradients(case)
    (M, N), K = dy.shape, x.shape[1]
    odx, bx = held(torch.zeros((M, K), dtype=BF, device=x.device), case[4])
    odw, bw = held(torch.zeros((N, K), dtype=BF, device=x.device), case[5])
    dx, dw, db = rcd.linear_backward(dy, x, w, pre=pre, act=act, dx=odx, dw=odw)
    torch.cuda.synchronize()
    assert outside_is_nan(odx, bx) and outside_is_nan(odw, bw)
    g, p = dy.double(), pre.double()
    dn = g * slope64(p, act)
    ed = g.abs() * 2.0 ** -20 * (1 + p.abs()) if act in ("silu", "gelu") else torch.zeros_like(dn)
    er = ed + (0 if act == "none" and dy.dtype == BF else 2.0 ** -8 * (dn.abs() + ed))
    assert ((db.double() - dn.sum(0)).abs() <= ed.sum(0) + (M + 8) * 2.0 ** -24 * dn.abs().sum(0)).all()
    for got, l, el, r in ((dx, dn, er, w.double()), (dw, dn.t(), er.t(), x.double())):
        ref, mag = l @ r, l.abs() @ r.abs()
        e = el @ r.abs() + (l.shape[1] + 8) * 2.0 ** -24 * mag
        assert ((got.double() - ref).abs() <= e + 2.0 ** -8 * (ref.abs() + e)).all()
        # the bound above counts every rounding of d as the worst; in norm they are under half a step each, as is the
        # result's own, and random: 2^-8 (half a step, relative) / sqrt 3 twice, a fifth more for sums of few
        norm = 1.2 * 2.0 ** -8 * (2 / 3) ** 0.5 * float(torch.linalg.vector_norm(ref))
        assert float(torch.linalg.vector_norm(got.double() - ref)) <= norm


@pytest.mark.parametrize("case", forms.BACKWARD, ids=lambda c: c[0])
def test_backward_parts_and_captured(case):
    """Each gradient alone is within its sums' error and a rounding of the one made with the others, what was not asked for stays
    untouched, and a replay gives an eager call's bits."""
    say("linear_backward parts", *case)
    act, x, w, dy, pre = gradients(case)
    (M, N), K = dy.shape, x.shape[1]

    def step(**kw):
        return rcd.linear_backward(dy, x, w, pre=pre, act=act, **kw)
    want = [t.clone() for t in step()]
    assert all(torch.equal(p, q) for p, q in zip(step(), want))
    shapes = ((M, K), (N, K), (N,))
    dn = dy.double().abs() * (slope64(pre.double(), act).abs() * (1 + 2.0 ** -7) + 2.0 ** -18)
    mags = (dn @ w.double().abs(), dn.t() @ x.double().abs(), dn.sum(0))
    for i in range(3):
        outs = [torch.full(s, 7.0, dtype=F32 if j == 2 else BF, device=x.device) for j, s in enumerate(shapes)]
        got = step(need_dx=i == 0, need_dw=i == 1, bias=i == 2, dx=outs[0], dw=outs[1], db=outs[2])
        torch.cuda.synchronize()
        for j in range(3):
            if j != i:
                assert got[j] is None and bool((outs[j] == 7.0).all())
        # other tiles or shares of K sum in another order: each sum's own error, and half a step of bf16 each
        a, b = got[i].double(), want[i].double()
        near = 2 * ((N, M, M)[i] + 8) * 2.0 ** -24 * mags[i]
        step_ = 0.0 if i == 2 else 2.0 ** -8 * (a.abs() + b.abs())
        assert got[i].data_ptr() == outs[i].data_ptr() and ((a - b).abs() <= near + step_).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    first = dy.clone()
    for i in range(3):
        dy.copy_(first.roll(i + 1, 0))
        want = [t.clone() for t in step()]
        for t in got:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want)), i
