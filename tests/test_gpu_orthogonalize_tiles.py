"""Every kernel of the orthogonalised updates against 64 bits on the GPU, at the
sizes of forms.py; zeros beside other matrices for any eps.  Tolerances are
those of test_gpu_orthogonalize_rows.py."""
import pytest
import torch

import forms
import routing_capacity_dispatch_amd as rcd
from gpu_common import dev, say
from test_gpu_orthogonalize import FLIPS, ROUND
from test_gpu_orthogonalize_rows import definition
from test_oracle_newton_schulz_rows import GENERAL

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form,size", forms.ORTHOGONALIZE)
@pytest.mark.parametrize("steps", [1, 5])
def test_forms(form, size, steps):
    d = dev()
    B, M, N = size
    say("orthogonalize", form, size, steps)
    gen = torch.Generator(device=d).manual_seed(B + M)
    buf = torch.full((B, M, N + 8), float("nan"), device=d)
    g = buf[:, :, :N]
    g.copy_(torch.randn(size, generator=gen, device=d))
    out = torch.full((B, M, N + 8), float("nan"), dtype=torch.bfloat16, device=d)
    got = rcd.orthogonalize(g, steps=steps, out=out[:, :, :N])
    torch.cuda.synchronize()
    assert torch.isnan(out[:, :, N:].float()).all()
    for i in sorted({0, B // 2 - 1 if B > 1 else 0, B // 2, B - 1}):
        ref = definition(g[i], steps)
        err = float(torch.linalg.vector_norm(got[i].double() - ref) / torch.linalg.vector_norm(ref))
        assert err <= GENERAL + FLIPS + ROUND, (i, err)
    assert torch.equal(got, rcd.orthogonalize(g, steps=steps))


@pytest.mark.parametrize("form,size", [c for c in forms.ORTHOGONALIZE if c[1][0] > 2])
@pytest.mark.parametrize("eps", [1e-7, 0.0])
def test_zeros_and_not_numbers_harm_no_neighbour(form, size, eps):
    d = dev()
    B, M, N = size
    say("orthogonalize zeros", form, size, eps)
    g = torch.randn(size, generator=torch.Generator(device=d).manual_seed(M), device=d)
    ref = rcd.orthogonalize(g, eps=eps)
    g[0] = 0
    g[B - 1, M - 1, N // 2] = float("nan")
    got = rcd.orthogonalize(g, eps=eps)
    torch.cuda.synchronize()
    assert (got[0] == 0).all() and torch.equal(got[1:B - 1], ref[1:B - 1]) and torch.isnan(got[B - 1]).all()


@pytest.mark.parametrize("form,size", [c for c in forms.ORTHOGONALIZE if c[1][0] in (1, 3, 6, 7)])
def test_captured(form, size):
    d = dev()
    say("orthogonalize graph", form, size)
    gen = torch.Generator(device=d).manual_seed(3)
    g = torch.randn(size, generator=gen, device=d)
    rcd.orthogonalize(g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = rcd.orthogonalize(g)
    for i in range(3):
        g.copy_(torch.randn(size, generator=gen, device=d))
        want = rcd.orthogonalize(g)
        got.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want), i
