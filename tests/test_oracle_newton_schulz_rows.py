"""How far the GPU's arithmetic is from the definition where a few rows or
values carry the matrix, in the form for sides of 256 and more (products that
take X's first fp16 number only)."""
import numpy as np
import pytest

from oracle import newton_schulz as ns

RNG = np.random.RandomState
# what the header promises: in general, where a few rows or values of one magnitude carry the matrix, a handful of values
GENERAL, FEW, HANDFUL = 2e-3, 3.5e-3, 5e-3


def few_rows(m, n, seed=0):
    """name, matrix, bound."""
    r = RNG(seed)
    g = r.standard_normal

    def rows(count, rank):
        a = np.zeros((m, n))
        a[r.choice(m, count, False)] = g((count, rank)) @ g((rank, n))
        return a
    for count in (1, 2, 3, 4, 16):
        yield f"one direction in {count} rows", rows(count, 1), FEW
    yield "two directions in 8 rows", rows(8, 2), FEW
    yield "one direction in 64 rows", rows(64, 1), GENERAL
    for s in (1, 2):
        yield f"one direction, lognormal rows {s}", \
            np.exp(s * g((m, 1))) * g((m, 1)) @ g((1, n)) + 1e-3 * g((m, n)), FEW
    yield "four directions, lognormal rows", np.exp(g((m, 1))) * (g((m, 4)) @ g((4, n))) + 1e-3 * g((m, n)), GENERAL
    yield "lognormal rows", np.exp(2 * g((m, 1))) * g((m, n)), GENERAL
    yield "a row and a weak direction", np.where(np.arange(m)[:, None] == 0, g((1, n)), 0) + 0.01 * g((m, 1)) @ g((1, n)), GENERAL
    two = np.zeros((m, n))
    two[:, r.choice(n, 2, False)] = g((m, 1)) @ g((1, 2))
    yield "one direction in 2 columns", two, FEW
    for rank in (1, 4):
        a = np.zeros((m, n))
        a[np.ix_(r.choice(m, 4, False), r.choice(n, 4, False))] = g((4, rank)) @ g((rank, 4))
        yield f"{rank} directions in 16 values", a, HANDFUL
    yield "one magnitude", np.where(np.arange(m)[:, None] < m // 2, g((1, n)), g((1, n))) * r.choice([-1.0, 1.0], (m, 1)), FEW
    yield "orthogonal rows", np.eye(m, n) * np.geomspace(1, 1e-4, m)[:, None], GENERAL


@pytest.mark.parametrize("shape", [(256, 256), (256, 700), (512, 512)])
def test_few_rows_carry_the_matrix(shape):
    for seed in (0, 1):
        for name, g, bound in few_rows(*shape, seed=seed):
            a, b = ns.exact(g), ns.emulated(g)
            assert np.linalg.norm(a - b) <= bound * np.linalg.norm(a), name


def test_weights_of_the_second_number():
    """1 in the last step, in the others 1 over the gains of the later ones: the slope at 0 for the usual coefficients,
    the largest anywhere for others, and never more than 1."""
    a = ns.USUAL[0]
    assert np.allclose(ns.weights_of_low([ns.USUAL] * 3), [a ** -2, 1 / a, 1.0])
    assert ns.weights_of_low([(0.5, 0.0, 0.0)] * 3) == [1.0] * 3
    assert np.allclose(ns.weights_of_low([(1.0, 0.0, 0.0), (1.0, 1.0, 0.0)]), [1 / (2 + 1 / 32), 1.0], rtol=1e-3)
