"""Pins of the oracle's distillation loss for teachers that are no plain distribution over different ids: slots that name one
id, and probabilities that pass 1 together."""

import math

import numpy as np
import pytest

from oracle import distill as d


def test_slots_of_one_id_are_one_outcome():
    """A certain token named twice, halves of it, or many parts: the loss of the token named once."""
    x = np.random.default_rng(1).normal(0, 2, 9)
    once = d.row(x, np.array([4]), np.array([1.0]), None, 1.0)
    for parts in ([0.5, 0.5], [0.9, 0.1], [0.25] * 4):
        twice = d.row(x, np.full(len(parts), 4), np.log(parts), None, 1.0)
        assert abs(twice[0] - once[0]) <= 1e-12 and np.allclose(twice[3], once[3], rtol=0, atol=1e-12)
    ids, y = np.array([3, 6, 3, 1, 6]), np.random.default_rng(2).normal(0, 1, 5)
    merged = np.array([np.logaddexp(y[0], y[2]), np.logaddexp(y[1], y[4]), y[3]])
    lse = float(np.logaddexp.reduce(y)) + 0.4
    for z in (None, lse):
        for t in (1.0, 0.7):
            w = merged if t == 1.0 else t * np.array([np.logaddexp(y[0] / t, y[2] / t), np.logaddexp(y[1] / t, y[4] / t), y[3] / t])
            a, b = d.row(x, ids, y, z if z is None else z / t + 1, t), d.row(x, np.array([3, 6, 1]), w, z if z is None else z / t + 1, t)
            assert abs(a[0] - b[0]) <= 1e-12 and np.allclose(a[3], b[3], rtol=0, atol=1e-12)


def test_the_loss_is_never_below_zero():
    """A divergence of one distribution from another, whatever slots share an id."""
    g = np.random.default_rng(3)
    for _ in range(50):
        ids, y = g.integers(0, 5, 8), g.normal(0, 2, 8)
        x = g.normal(0, 2, 6)
        assert d.row(x, ids, y, None, 1.0)[0] >= 0
        assert d.row(x, ids, y, float(np.logaddexp.reduce(y)) + 0.2, 1.0)[0] >= 0


@pytest.mark.parametrize("temperature", [1.0, 2.5])
def test_gradient_where_the_teacher_passes_one(temperature):
    """A log-sum-exp that is too small (of another temperature, or of part of the row): the gradient is still the difference."""
    g = np.random.default_rng(4)
    for shift in (-1.0, -0.4, -1e-3):
        x, y, ids = g.normal(0, 2, 8), g.normal(0, 1, 4), g.permutation(8)[:4]
        lse = float(np.logaddexp.reduce(y / temperature)) + shift
        loss, _, _, grad = d.row(x, ids, y, lse, temperature)
        assert math.isfinite(loss)
        for v in range(8):
            up, down = x.copy(), x.copy()
            up[v] += 1e-5
            down[v] -= 1e-5
            diff = (d.row(up, ids, y, lse, temperature)[0] - d.row(down, ids, y, lse, temperature)[0]) / 2e-5
            assert abs(diff - grad[v]) <= 1e-8
