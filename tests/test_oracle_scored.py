"""Pins of the scored-routing oracle (CPU only)."""
import itertools

import numpy as np
import pytest

import oracle
from oracle import scored_routing as sr


def test_scores_of_known_logits():
    l = np.array([[0.0, np.log(3.0), -np.inf]])
    assert np.allclose(sr.scores(l, "sigmoid"), [[0.5, 0.75, 0.0]])
    assert np.allclose(sr.scores(l, "softmax"), [[0.25, 0.75, 0.0]])
    assert (sr.scores(np.full((1, 3), -np.inf), "softmax") == 0).all()


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
def test_without_bias_the_order_is_that_of_the_logits(kind):
    rng = np.random.default_rng(0)
    l = rng.standard_normal((20, 24)).astype(np.float32)
    assert np.array_equal(sr.select(l, None, 5, kind), oracle.route_topk(l, np.zeros(24, np.float32), 5))


def test_group_limit_by_brute_force():
    rng = np.random.default_rng(1)
    l = rng.standard_normal((30, 12))
    b = 0.2 * rng.standard_normal(12)
    key = sr.scores(l, "sigmoid") + b
    got = sr.select(l, b, 3, "sigmoid", n_groups=4, top_groups=2, group_top=2)
    for t in range(30):
        best = max(itertools.combinations(range(4), 2),
                   key=lambda c: sum(np.sort(key[t, 3 * g:3 * g + 3])[-2:].sum() for g in c))
        inside = [e for g in best for e in range(3 * g, 3 * g + 3)]
        assert list(got[t]) == sorted(inside, key=lambda e: -key[t, e])[:3]


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renormalise", [False, True])
def test_backward_against_differences(kind, renormalise):
    rng = np.random.default_rng(2)
    l = rng.standard_normal((4, 9))
    idx = np.stack([rng.permutation(9)[:3] for _ in range(4)])
    dg = rng.standard_normal((4, 3))
    got, mag = sr.backward(l, idx, dg, kind, renormalise, 2.5)
    h = 1e-6
    for t in range(4):
        for e in range(9):
            lp, lm = l.copy(), l.copy()
            lp[t, e] += h
            lm[t, e] -= h
            d = (sr.gates(lp, idx, kind, renormalise, 2.5) - sr.gates(lm, idx, kind, renormalise, 2.5)) / (2 * h)
            # central differences: truncation h^2, rounding 2^-52 / h of values below 2.5
            assert abs((d * dg).sum() - got[t, e]) < 1e-8
    assert (mag >= np.abs(got) - 1e-15).all()
