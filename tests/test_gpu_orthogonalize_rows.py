"""moe_orthogonalize where a few rows or values carry the matrix.

Tolerances.  The arithmetic's distance from the definition is the bound of each
kind (test_oracle_newton_schulz_rows.py, from exact sums); fp32 sums add
FLIPS = 1.4e-3 of the norm at most (test_gpu_orthogonalize.py derives it), the
rounding to bf16 2^-8 of each value."""
import numpy as np
import pytest
import torch

import routing_capacity_dispatch_amd as rcd
from gpu_common import dev, say
from oracle import newton_schulz as ns
from test_gpu_orthogonalize import FLIPS, ROUND, np64
from test_oracle_newton_schulz_rows import FEW, GENERAL, few_rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(100, 260), (256, 256), (300, 700), (700, 300), (512, 512)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_few_rows_carry_the_matrix(shape, dtype):
    d = dev()
    m, n = min(shape), max(shape)
    kinds = list(few_rows(m, n, seed=m + n))
    g = torch.from_numpy(np.stack([g if shape[0] <= shape[1] else g.T for _, g, _ in kinds])).to(dtype).contiguous()
    say("orthogonalize few rows", shape, dtype)
    got = rcd.orthogonalize(g.to(d))
    torch.cuda.synchronize()
    for i, (name, _, bound) in enumerate(kinds):
        ref = ns.exact(np64(g[i]))
        # matrices of bf16 values are others than those of the bound, and small ones are held in both numbers
        err = np.linalg.norm(np64(got[i]) - ref) / np.linalg.norm(ref)
        assert err <= bound + FLIPS + ROUND, (name, err)


def definition(x, steps):
    """In 64 bits on the GPU."""
    x = x.double()
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    x = x / (torch.linalg.vector_norm(x) + 1e-7)
    for _ in range(steps):
        a, b, c = ns.USUAL
        p = x @ x.t()
        x = a * x + (b * p + c * (p @ p)) @ x
    return x.t() if tall else x


# every size of tiles, wide and tall
@pytest.mark.parametrize("B,shape", [(3, (700, 900)), (6, (1000, 1000)), (6, (1000, 1300)), (4, (2048, 2048)),
                                     (4, (2100, 2000)), (8, (2048, 4096)), (9, (4090, 2000))])
@pytest.mark.parametrize("steps", [5, 2])
def test_large(B, shape, steps):
    d = dev()
    say("orthogonalize few rows, large", B, shape, steps)
    gen = torch.Generator(device=d).manual_seed(B)
    m, n = min(shape), max(shape)

    def rand(*s):
        return torch.randn(s, generator=gen, device=d)
    g = torch.zeros((B, m, n), device=d)
    for i in range(B):
        if i % 3 == 0:
            g[i, torch.randperm(m, generator=gen, device=d)[:2 + 14 * (i % 2)]] = rand(2 + 14 * (i % 2), 1) @ rand(1, n)
        elif i % 3 == 1:
            g[i] = torch.exp(rand(m, 1)) * rand(m, 1) @ rand(1, n) + 1e-3 * rand(m, n)
        else:
            g[i] = rand(m, n)
    if shape[0] > shape[1]:
        g = g.transpose(1, 2).contiguous()
    got = rcd.orthogonalize(g, steps=steps)
    torch.cuda.synchronize()
    for i in sorted({0, 1, 2, B - 3, B - 2, B - 1}):
        ref = definition(g[i], steps)
        err = float(torch.linalg.vector_norm(got[i].double() - ref) / torch.linalg.vector_norm(ref))
        assert err <= (GENERAL if i % 3 == 2 else FEW) + FLIPS + ROUND, (i, err)
