"""Verification of drafted tokens against the target's probabilities, from
given random numbers.

Test infrastructure only (see the package docstring).

With p_i and q_i the softmax of the target's and the draft model's logits over
the temperature, drafts are taken in order while ``u_i q_i(d_i) < p_i(d_i)``; at
the first refusal the next token is ``argmax_v max(p_i(v) - q_i(v), 0) / e_v``,
behind the last draft ``argmax_v p_n(v) / e_v`` (the lowest index of equals).
Drafts without probabilities are ``q_i = [v = d_i]``.  At temperature 0 a draft
is taken if it is the target's likeliest token, which is also the next token.
For u uniform and e exponential the tokens are distributed as drawn from p.

Everything is float64 on the logits' values; drafts are decided by logarithms, as
their probabilities may be below float64's range (e^-7000 at a temperature of
0.001) where their quotient is not.
"""

import numpy as np


def softmax(x: np.ndarray) -> np.ndarray:
    x = np.asarray(x, np.float64)
    e = np.exp(x - np.max(x))
    return e / e.sum()


def log_softmax(x: np.ndarray) -> np.ndarray:
    x = np.asarray(x, np.float64)
    x = x - np.max(x)
    return x - np.log(np.exp(x).sum())


def sequence(target, drafts, uniforms=None, noise=None, draft_logits=None, temperature: float = 1.0):
    """(tokens, accepted, logp, margin) of one sequence: ``target`` [n + 1, V], ``drafts`` [n].

    ``margin`` is how far, relatively, the closest of its decisions is from going the other way."""
    target = np.asarray(target, np.float64)
    n = len(drafts)
    for i, d in enumerate(drafts):
        if d < 0 or d >= target.shape[1]:
            n = i
            break
    t = temperature if temperature > 0 else 1.0
    tokens, logp, margin = [], [], np.inf
    for i in range(n + 1):
        p = softmax(target[i] / t)
        q = None
        if i < n:
            d = int(drafts[i])
            if temperature == 0:
                ok = d == int(np.argmax(target[i]))
            else:
                q, lnq = np.eye(1, p.size, d)[0], 0.0
                if draft_logits is not None:
                    y = np.asarray(draft_logits[i], np.float64) / t
                    q, lnq = softmax(y), log_softmax(y)[d]
                with np.errstate(divide="ignore"):
                    left, right = np.log(float(uniforms[i])) + lnq, log_softmax(target[i] / t)[d]
                ok = left < right
                if np.isfinite(left) and np.isfinite(right):  # with a 0 on either side nothing is near
                    margin = min(margin, -np.expm1(-abs(left - right)))
            if ok:
                tokens.append(d)
                logp.append(float(log_softmax(target[i] / t)[d]))
                continue
        if temperature == 0:
            token = int(np.argmax(target[i]))
        else:
            r = p if q is None else np.maximum(p - q, 0.0)
            if not r.any():
                r = p
            score = r / np.asarray(noise, np.float64)
            token = int(np.argmax(score))
            # an error of eps in p and q moves a score by eps (p + q) / e
            blur = score if q is None else (p + q) / np.asarray(noise, np.float64)
            gap = (score[token] - score) / (blur[token] + blur + 1e-300)
            gap[token] = np.inf
            margin = min(margin, float(gap.min()))
        return tokens + [token], i, logp + [float(np.log(p[token]))], margin
    raise AssertionError


def batch(target, drafts, counts, uniforms=None, noise=None, draft_logits=None, temperature: float = 1.0):
    """(tokens [T + B], accepted [B], logp [T + B], margin [B]) of sequences with counts[b] drafts each."""
    tokens, logp, accepted, margins = [], [], [], []
    at = 0
    for b, n in enumerate(counts):
        rows = slice(at, at + n)
        tok, a, lp, margin = sequence(target[at + b:at + b + n + 1], drafts[rows],
                                      None if uniforms is None else uniforms[rows], None if noise is None else noise[b],
                                      None if draft_logits is None else draft_logits[rows], temperature)
        tokens += tok + [-1] * (n + 1 - len(tok))
        logp += lp + [0.0] * (n + 1 - len(lp))
        accepted.append(a)
        margins.append(margin)
        at += n
    return np.array(tokens, np.int64), np.array(accepted, np.int64), np.array(logp, np.float64), np.array(margins)
