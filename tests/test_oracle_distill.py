"""Pins of the oracle's distillation loss, policy gradient and their gradients: differences, closed forms, brute force, and
planted mistakes that a pin must catch."""

import math

import numpy as np
import pytest

from oracle import distill as d
from oracle import rollout_is as ris


def _row(seed, v=9, k=4, used=3):
    g = np.random.default_rng(seed)
    ids = g.permutation(v)[:k]
    ids[used:] = -1
    y = g.normal(0, 2, k)
    return g.normal(0, 2, v), ids, y, math.log(np.exp(y[:used]).sum()) + 0.3


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("temperature", [1.0, 2.5])
def test_gradient_is_the_difference(tail, temperature):
    for seed in range(5):
        x, ids, y, lse = _row(seed)
        lse = math.log(np.exp(y[:3] / temperature).sum()) + 0.3 if tail else None
        grad = d.row(x, ids, y, lse, temperature)[3]
        for v in range(x.size):
            up, down = x.copy(), x.copy()
            up[v] += 1e-5
            down[v] -= 1e-5
            diff = (d.row(up, ids, y, lse, temperature)[0] - d.row(down, ids, y, lse, temperature)[0]) / 2e-5
            assert abs(diff - grad[v]) <= 1e-8


def test_loss_is_the_divergence_of_whole_distributions():
    """All of the vocabulary in the list, or the rest of it lumped: Kullback and Leibler's divergence, by loops."""
    g = np.random.default_rng(0)
    x, y = g.normal(0, 2, 6), g.normal(0, 2, 6)
    p, q = np.exp(y) / np.exp(y).sum(), np.exp(x) / np.exp(x).sum()
    whole = sum(p[i] * math.log(p[i] / q[i]) for i in range(6))
    for lse in (None, math.log(np.exp(y).sum())):
        assert abs(d.row(x, np.arange(6), y, lse, 1.0)[0] - whole) <= 1e-12
    two = p[1] * math.log(p[1] / q[1]) + (1 - p[1]) * math.log((1 - p[1]) / (1 - q[1]))
    assert abs(d.row(x, np.array([1]), y[1:2], math.log(np.exp(y).sum()), 1.0)[0] - two) <= 1e-12


def test_closed_forms():
    x, ids, y, lse = _row(3)
    assert abs(d.row(y, np.arange(4), y, None, 1.0)[0]) <= 1e-15  # the student is the teacher
    one = d.row(x, np.array([2]), np.array([5.0]), None, 1.0)  # one id: the cross entropy
    assert abs(one[0] + ris.token_logprobs(x[None], np.array([2]))[0]) <= 1e-12
    assert d.row(x, np.array([-1, -1]), y[:2], lse, 1.0)[:3] == (0.0, 0.0, 0.0)
    twice = d.row(x, np.array([2, 2, 5]), np.array([1.0, 1.0, 0.5]), None, 1.0)  # equal slots add up
    once = d.row(x, np.array([2, 5]), np.array([1.0 + math.log(2), 0.5]), None, 1.0)
    assert np.allclose(twice[3], once[3], rtol=0, atol=1e-15)
    assert abs(d.row(x, ids, y, lse, 1.0)[3].sum()) <= 1e-15  # a constant added to the logits changes nothing
    masked = x.copy()
    masked[ids[0]] = -np.inf
    assert d.row(masked, ids, y, lse, 1.0)[0] == np.inf
    assert d.row(np.full(5, -np.inf), np.array([1]), np.array([0.0]), None, 1.0)[3].tolist() == [0, -1, 0, 0, 0]


def test_policy_gradient_is_the_difference():
    g = np.random.default_rng(4)
    x, tokens, adv = g.normal(0, 2, (3, 7)), np.array([2, -1, 6]), g.normal(0, 1, 3)
    rollout = ris.token_logprobs(x, tokens) + g.normal(0, 0.5, 3)
    logp, w, grad = d.policy_gradient(x, tokens, adv, rollout, 1.2)
    assert w.max() <= 1.2 and w[1] == logp[1] == 0.0 and not grad[1].any()

    def loss(z):
        return -np.sum(adv * w * ris.token_logprobs(z, tokens))

    for t in range(3):
        for v in range(7):
            up, down = x.copy(), x.copy()
            up[t, v] += 1e-5
            down[t, v] -= 1e-5
            assert abs((loss(up) - loss(down)) / 2e-5 - grad[t, v]) <= 1e-8
    assert d.policy_gradient(x, tokens, adv)[1].tolist() == [1, 0, 1]


@pytest.mark.parametrize("mistake", ["rest", "temperature", "duplicates"])
def test_planted_mistakes_are_caught(monkeypatch, mistake):
    teacher, row = d.teacher, d.row
    if mistake == "rest":
        monkeypatch.setattr(d, "teacher", lambda *a: teacher(*a)[:3] + (0.0,))
        with pytest.raises(AssertionError):
            test_loss_is_the_divergence_of_whole_distributions()
    elif mistake == "temperature":
        monkeypatch.setattr(d, "row", lambda *a: row(*a)[:3] + (row(*a)[3] * a[4],))
        with pytest.raises(AssertionError):
            test_gradient_is_the_difference(False, 2.5)
    else:
        monkeypatch.setattr(d, "teacher", lambda ids, *a: (lambda r: (np.unique(r[0]),) + tuple(x[:np.unique(r[0]).size] for x in r[1:3]) + r[3:])(teacher(ids, *a)))
        with pytest.raises(AssertionError):
            test_closed_forms()
