"""Pins of the oracle's distillation loss for teachers that are no plain distribution over different ids: slots that name one
id, and probabilities that pass 1 together."""


import numpy as np

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
