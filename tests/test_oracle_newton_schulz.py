"""The Newton-Schulz oracle against singular values, and how far the GPU's
arithmetic (fp16 operands, fp32 X and diagonals) is from it."""
import numpy as np
import pytest

from oracle import newton_schulz as ns

RNG = np.random.RandomState


def spectra(m, n, seed=0):
    r = RNG(seed)
    k = min(m, n)
    g = r.standard_normal
    yield "gaussian", g((m, n))
    yield "decaying", (g((m, k)) / np.arange(1, k + 1)) @ g((k, n))
    yield "few directions", g((m, min(k, 8))) @ g((min(k, 8), n)) + 0.01 * g((m, n))
    yield "one direction", g((m, 1)) @ g((1, n)) + 1e-3 * g((m, n))
    yield "half the rank", g((m, (k + 1) // 2)) @ g(((k + 1) // 2, n)) + 1e-3 * g((m, n))
    yield "rows of zeros", np.where(np.arange(m)[:, None] < (m + 1) // 2, g((m, n)), 0)


@pytest.mark.parametrize("shape", [(1, 1), (1, 9), (9, 1), (8, 8), (20, 33), (33, 20)])
def test_definition_is_a_polynomial_of_the_singular_values(shape):
    for name, g in spectra(*shape):
        for co, steps in ((ns.USUAL, 5), ((1.5, -0.5, 0.0), 3), (((2.0, -1.5, 0.5), (1.5, -0.5, 0.0)), 2)):
            a, b = ns.exact(g, steps, co, scale=0.3), ns.by_singular_values(g, steps, co, scale=0.3)
            assert np.abs(a - b).max() <= 1e-11, name
    assert (ns.exact(np.zeros(shape)) == 0).all()


def test_singular_values_end_near_one():
    g = RNG(1).standard_normal((40, 64))
    s = np.linalg.svd(ns.exact(g), compute_uv=False)
    assert 0.6 < s.min() and s.max() < 1.3


@pytest.mark.parametrize("shape", [(1, 1), (2, 3), (16, 16), (17, 33), (64, 64), (100, 260), (300, 128), (256, 256)])
def test_roundings_of_the_kernels_arithmetic(shape):
    """At most 1.5e-3 of the norm, on every spectrum: what the header promises."""
    for name, g in spectra(*shape):
        a, b = ns.exact(g), ns.emulated(g)
        assert np.linalg.norm(a - b) <= 1.5e-3 * np.linalg.norm(a), name
