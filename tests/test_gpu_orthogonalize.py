"""moe_orthogonalize against the fp64 oracle.

Tolerances.  The oracle's emulation makes the kernel's roundings with exact
sums.  fp32 sums of K products move a value by sqrt(K) 2^-24 of its terms and
with it, now and then, an fp16 rounding to the other side: the probability is
about that over 2^-11, each time 2^-10 off, so the parts of the norm that
differ are under 2^-10 sqrt(sqrt(K) 2^-13) = 1e-4 (K = 8192) a product; fifteen
products, amplified by at most 3.5: 15^0.5 * 3.5 * 1e-4 = 1.4e-3 for the worst
spectrum, in the 2-norm.  The result's rounding to bf16 is 2^-8 of each value
at most.  The emulation itself is within 1.5e-3 of the norm of the definition
(test_oracle_newton_schulz.py)."""
import numpy as np
import pytest
import torch

import routing_capacity_dispatch_amd as rcd
from gpu_common import dev, say
from oracle import newton_schulz as ns
from test_oracle_newton_schulz import spectra

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
FLIPS, ARITHMETIC, ROUND = 1.4e-3, 1.5e-3, 2.0 ** -8


def np64(t):
    return t.detach().cpu().double().numpy()


def compare(got, g, **kw):
    emu, ref = ns.emulated(g, **kw), ns.exact(g, **kw)
    n = np.linalg.norm(ref)
    assert np.isfinite(got).all()
    assert np.linalg.norm(got - emu) <= FLIPS * n + ROUND * np.linalg.norm(emu) + 1e-30
    assert np.linalg.norm(got - ref) <= (FLIPS + ARITHMETIC) * n + ROUND * n + 1e-30


def rand(shape, seed, dtype=F32, scale=1.0):
    g = torch.Generator(device="cpu").manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


# one value, rows and columns, below and past a K tile, a tile and a block of 8, tall and wide
@pytest.mark.parametrize("shape", [(1, 1), (1, 70), (70, 1), (3, 5), (8, 8), (63, 65), (64, 64), (128, 128), (129, 127),
                                   (100, 260), (260, 100), (333, 1000), (1000, 333), (65, 2000)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_shapes(shape, dtype):
    d = dev()
    say("orthogonalize", shape, dtype)
    g = rand((3, *shape), sum(shape), dtype)
    got = rcd.orthogonalize(g.to(d))
    assert got.dtype == BF and got.shape == g.shape
    one = rcd.orthogonalize(g[1].to(d))
    torch.cuda.synchronize()
    assert torch.equal(one, got[1])
    for i in range(3):
        compare(np64(got[i]), np64(g[i]))


@pytest.mark.parametrize("shape", [(96, 200), (200, 96), (256, 256)])
def test_spectra(shape):
    d = dev()
    for name, g in spectra(*shape):
        say("orthogonalize", shape, name)
        t = torch.from_numpy(g).float()
        compare(np64(rcd.orthogonalize(t.to(d))), np64(t))


# the large tiles: whole ones, ends inside them, several matrices
@pytest.mark.parametrize("B,shape", [(64, (512, 513)), (20, (1030, 1000)), (1, (4100, 4097)), (16, (1024, 1100))])
def test_large(B, shape):
    """The norm of a product with a random block, and single matrices, in 64 bits on the GPU."""
    d = dev()
    say("orthogonalize large", B, shape)
    g = torch.randn((B, *shape), generator=torch.Generator(device=d).manual_seed(5), device=d)
    got = rcd.orthogonalize(g)
    torch.cuda.synchronize()
    for i in sorted({0, B // 2, B - 1}):
        x = g[i].double()
        x = x.t() if shape[0] > shape[1] else x
        x = x / (torch.linalg.vector_norm(x) + 1e-7)
        for _ in range(5):
            a, b, c = ns.USUAL
            p = x @ x.t()
            x = a * x + (b * p + c * (p @ p)) @ x
        x = x.t() if shape[0] > shape[1] else x
        err = float(torch.linalg.vector_norm(got[i].double() - x) / torch.linalg.vector_norm(x))
        assert err <= FLIPS + ARITHMETIC + ROUND, err


@pytest.mark.parametrize("kw", [dict(steps=1), dict(steps=2), dict(steps=10, coeffs=(1.5, -0.5, 0.0)),
                                dict(steps=3, coeffs=((4.0, -6.0, 2.5), (3.4445, -4.775, 2.0315), (1.875, -1.25, 0.375))),
                                dict(steps=2, scale=-0.2), dict(steps=2, eps=0.0), dict(steps=1, eps=10.0),
                                dict(steps=2, coeffs=(1.0, 0.0, 0.0)), dict(steps=2, coeffs=(0.0, 0.0, 0.0)),
                                dict(steps=4, coeffs=(4.0, 0.0, 0.0))])
def test_parameters(kw):
    d = dev()
    for shape in ((40, 72), (150, 64)):
        say("orthogonalize", shape, kw)
        g = rand(shape, 3)
        got = np64(rcd.orthogonalize(g.to(d), **kw))
        # the polynomials' own growth is larger here: the emulation is what counts
        emu = ns.emulated(np64(g), **kw)
        assert np.linalg.norm(got - emu) <= (FLIPS + ROUND) * np.linalg.norm(emu) + 1e-30


def test_coefficients_that_diverge_are_refused():
    g = rand((40, 72), 3).to(dev())
    with pytest.raises(rcd.MoeError, match="UNSUPPORTED"):
        rcd.orthogonalize(g, steps=4, coeffs=(40.0, -3.0, 0.1))


# two halves of many large matrices, one phase apart: even and odd numbers, wide
# and tall, one step (its first phase is its last but two)
@pytest.mark.parametrize("B,shape,steps", [(52, (1000, 1100), 5), (47, (1100, 1000), 5), (40, (1024, 1100), 1),
                                           (45, (1100, 1024), 2), (32, (1024, 2048), 5), (35, (1000, 2000), 5),
                                           (35, (2000, 1000), 1), (32, (2048, 1024), 2)])
def test_halves(B, shape, steps):
    d = dev()
    say("orthogonalize halves", B, shape, steps)
    g = torch.randn((B, *shape), generator=torch.Generator(device=d).manual_seed(6), device=d)
    got = rcd.orthogonalize(g, steps=steps)
    torch.cuda.synchronize()
    for i in sorted({0, B // 2 - 1, B // 2, (B + 1) // 2, B - 1}):
        x = g[i].double()
        x = x.t() if shape[0] > shape[1] else x
        x = x / (torch.linalg.vector_norm(x) + 1e-7)
        for _ in range(steps):
            a, b, c = ns.USUAL
            p = x @ x.t()
            x = a * x + (b * p + c * (p @ p)) @ x
        x = x.t() if shape[0] > shape[1] else x
        err = float(torch.linalg.vector_norm(got[i].double() - x) / torch.linalg.vector_norm(x))
        assert err <= FLIPS + ARITHMETIC + ROUND, err


@pytest.mark.parametrize("scale", [1e-30, 1e-20, 1e15, 3e30])
def test_magnitudes(scale):
    """Sums of squares that leave fp32's range."""
    d = dev()
    g = rand((50, 80), 9, F32, scale)
    compare(np64(rcd.orthogonalize(g.to(d), eps=0.0)), np64(g), eps=0.0)


def test_zeros_and_neighbours():
    """A matrix of zeros gives zeros, its neighbours are as without it, and one with a NaN harms none."""
    d = dev()
    g = rand((4, 70, 90), 2).to(d)
    ref = rcd.orthogonalize(g)
    h = g.clone()
    h[1] = 0
    h[2, 3, 4] = float("nan")
    for eps in (1e-7, 0.0):
        got = rcd.orthogonalize(h, eps=eps)
        assert (got[1] == 0).all()
        assert eps == 0.0 or (torch.equal(got[0], ref[0]) and torch.equal(got[3], ref[3]))


@pytest.mark.parametrize("shape", [(40, 72), (72, 40), (130, 130)])
@pytest.mark.parametrize("shift,pad", [(0, 8), (1, 0), (3, 5)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_strides(shape, shift, pad, dtype):
    d = dev()
    M, N = shape
    B = 2
    g = rand((B, M, N), 4, dtype)

    def held(dtype):
        buf = torch.full((shift + B * (M + 1) * (N + pad) + 16,), float("nan"), dtype=dtype, device=d)
        return buf, buf[shift:shift + B * (M + 1) * (N + pad)].view(B, M + 1, N + pad)[:, :M, :N]
    _, v = held(dtype)
    v.copy_(g)
    buf, o = held(BF)
    got = rcd.orthogonalize(v, out=o)
    torch.cuda.synchronize()
    assert got.data_ptr() == o.data_ptr() and torch.equal(o, rcd.orthogonalize(g.to(d)))
    o.fill_(float("nan"))
    assert torch.isnan(buf.float()).all()


def test_in_place():
    d = dev()
    for shape in ((90, 72), (72, 90)):
        g = rand((3, *shape), 4, BF).to(d)
        ref = rcd.orthogonalize(g)
        assert rcd.orthogonalize(g, out=g) is g and torch.equal(g, ref)


def test_groups_of_a_large_batch():
    """More matrices than one group takes, each as if alone; sizes of zero."""
    d = dev()
    g = rand((8192 + 77, 6, 9), 1).to(d)
    got = rcd.orthogonalize(g)
    for i in (0, 8191, 8192, 8268):
        assert torch.equal(got[i], rcd.orthogonalize(g[i]))
    for shape in ((0, 4, 4), (2, 0, 4), (2, 4, 0)):
        assert rcd.orthogonalize(torch.zeros(shape, device=d)).shape == shape


def test_streams_and_graph():
    d = dev()
    for shape in ((2, 140, 200), (1, 300, 64)):
        g = rand(shape, 1).to(d)
        want = rcd.orthogonalize(g)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got = rcd.orthogonalize(g)
        s.synchronize()
        assert torch.equal(got, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = rcd.orthogonalize(g)
        for i in range(3):
            g.copy_(rand(shape, 10 + i))
            want = rcd.orthogonalize(g)
            got.zero_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(got, want), i
