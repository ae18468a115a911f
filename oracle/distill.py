"""Losses over rows of logits and their gradients: distillation from a
teacher's top logits, and the policy gradient of the tokens a rollout took.

Test infrastructure only (see the package docstring).

With x a row of logits, t the temperature, q = softmax(x / t), and the
teacher's logits y_j at the ids i_j (a negative id is no slot, the p_j of slots
that name one id add up to one outcome's):

* without the teacher's log-sum-exp: ``p_j = e^{y_j / t} / sum_i e^{y_i / t}``;
* with it: ``p_j = e^{y_j / t - lse}``, and what is missing, ``p_r = max(0, 1 -
  sum_j p_j)``, is one outcome more beside the student's probability outside
  the ids, ``q_r``; where that is 0, a ``p_r`` of up to 2^-16 counts as rounding;
  a log-sum-exp that is too small for its slots makes ``sum_j p_j > 1``, which
  is taken as given;
* ``loss = sum_j p_j (ln p_j - ln q_{i_j}) [+ p_r (ln p_r - ln q_r)]`` with
  0 ln 0 = 0; its gradient in the logits.

A row without a slot has no teacher: loss and gradient 0.  A row of logits
that are all -inf has q = 0.  Everything is float64.
"""

import numpy as np

from .rollout_is import is_weights, token_logprobs


def _lse(x: np.ndarray) -> float:
    m = np.max(x, initial=-np.inf)
    return float(m + np.log(np.sum(np.exp(x - m)))) if np.isfinite(m) else -np.inf


def teacher(ids: np.ndarray, y: np.ndarray, lse, temperature: float):
    """(ids, p, ln p, p_r) of one row's used slots."""
    used = ids >= 0
    y = np.asarray(y, np.float64)[used] / temperature
    lnp = y - (_lse(y) if lse is None else float(lse))
    p = np.exp(lnp)
    return np.asarray(ids)[used].astype(np.int64), p, lnp, 0.0 if lse is None else max(0.0, 1.0 - float(p.sum()))


def row(x: np.ndarray, ids: np.ndarray, y: np.ndarray, lse, temperature: float):
    """(loss, lse, lse outside the ids, dloss/dx) of one row."""
    z = np.asarray(x, np.float64) / temperature
    ids, p, lnp, rest = teacher(np.asarray(ids), y, lse, temperature)
    if ids.size == 0:
        return 0.0, 0.0, 0.0, np.zeros_like(z)
    total = _lse(z)
    q = np.exp(z - total) if total > -np.inf else np.zeros_like(z)
    lnq = z - (total if total > -np.inf else 0.0)
    inside = np.zeros(z.shape, bool)
    inside[ids] = True
    outside = total if lse is None else _lse(z[~inside])
    some = p > 0
    whole = np.full(z.shape, -np.inf)  # ln of what the teacher gives an id
    np.logaddexp.at(whole, ids, lnp)
    loss = float(np.sum(p[some] * (whole[ids[some]] - lnq[ids[some]])))
    grad = q * (1.0 if lse is None else max(1.0, float(p.sum())))
    np.add.at(grad, ids, -p)
    if outside == -np.inf and rest <= 2.0 ** -16:
        rest = 0.0
    if lse is not None and rest > 0:
        loss += rest * (np.log(rest) - (outside - (total if total > -np.inf else 0.0)))
        if outside > -np.inf:
            grad[~inside] -= rest * np.exp(z[~inside] - outside)
    return loss, total, outside, grad / temperature


def distill(x, ids, y, lse=None, temperature: float = 1.0):
    """(loss [T], stats [T, 2], dloss/dlogits [T, V]) of rows of logits."""
    out = [row(x[t], ids[t], y[t], None if lse is None else lse[t], temperature) for t in range(len(x))]
    loss = np.array([o[0] for o in out], np.float64)
    stats = np.array([o[1:3] for o in out], np.float64).reshape(-1, 2)
    return loss, stats, np.array([o[3] for o in out], np.float64).reshape(len(out), -1)


def policy_gradient(x, tokens, advantages, rollout_logp=None, cap: float = 0.0):
    """(logp [T], w [T], d(-sum A w logp)/dlogits [T, V]), w held fixed; zeros where the token is negative."""
    x = np.asarray(x, np.float64)
    tokens = np.asarray(tokens, np.int64)
    live = tokens >= 0
    logp = token_logprobs(x, tokens)
    w = live.astype(np.float64) if rollout_logp is None else is_weights(logp, rollout_logp, tokens, cap)
    grad = np.zeros_like(x)
    for t in np.nonzero(live)[0]:
        grad[t] = np.exp(x[t] - _lse(x[t]))
        grad[t, tokens[t]] -= 1.0
        grad[t] *= w[t] * float(advantages[t])
    return logp, w, grad
