"""Pins of the oracle's verification of drafts: the distribution of what comes out, closed forms, and planted mistakes."""

import numpy as np
import pytest

from oracle import verify as v


def _frequencies(lookup, trials=20000):
    """How often each token comes first, with drafts drawn from q (or always token 1), and the target's probabilities."""
    g = np.random.default_rng(5)
    target, draft = np.array([[0.3, 1.0, -1.0, 0.7], [0.0, 0.0, 0.0, 0.0]]), np.array([[1.2, -0.5, 0.4, 0.1]])
    q = v.softmax(draft[0])
    count = np.zeros(4)
    for _ in range(trials):
        d = [1] if lookup else [g.choice(4, p=q)]
        tokens, *_ = v.sequence(target, d, g.random(1), g.exponential(size=4), None if lookup else draft)
        count[tokens[0]] += 1
    return count / trials, v.softmax(target[0])


@pytest.mark.parametrize("lookup", [False, True])
def test_tokens_are_distributed_as_the_target(lookup):
    got, p = _frequencies(lookup)
    assert np.all(np.abs(got - p) <= 5 * np.sqrt(p * (1 - p) / 20000))


def test_closed_forms():
    g = np.random.default_rng(1)
    x, e = g.normal(0, 2, (4, 6)), g.exponential(size=6)
    tokens, accepted, logp, _ = v.sequence(x, [3, 0, 5], np.full(3, 0.999), e, x[:3])  # q = p: all are taken
    assert accepted == 3 and tokens[:3] == [3, 0, 5] and tokens[3] == int(np.argmax(v.softmax(x[3]) / e))
    assert np.allclose(logp, [np.log(v.softmax(x[i])[t]) for i, t in enumerate(tokens)])
    masked = x.copy()
    masked[1, 0] = -np.inf  # a token that the target rules out is refused whatever u is
    tokens, accepted, _, _ = v.sequence(masked, [3, 0, 5], np.zeros(3), e, x[:3])
    assert accepted == 1 and tokens[1] != 0
    tokens, accepted, _, _ = v.sequence(x, [3, -1, 5], np.zeros(3), e, x[:3])  # no draft behind the first
    assert accepted == 1 and tokens[1] == int(np.argmax(v.softmax(x[1]) / e))
    ties = np.array([[1.0, 2.0, 2.0], [0.0, -1.0, 0.0]])
    assert v.sequence(ties, [1], temperature=0)[0] == [1, 0] and v.sequence(ties, [2], temperature=0)[0] == [1]


def test_batch_places():
    g = np.random.default_rng(2)
    x = g.normal(0, 1, (5, 4))
    tokens, accepted, logp, _ = v.batch(x, np.array([int(np.argmax(x[0])), 9]), [2, 0, 0], temperature=0.0)
    assert tokens[2] == -1 and accepted.tolist() == [1, 0, 0] and logp[2] == 0.0
    assert tokens[1] == np.argmax(x[1]) and tokens[3] == np.argmax(x[3]) and tokens[4] == np.argmax(x[4])


@pytest.mark.parametrize("mistake", ["p instead of what is left", "flipped test"])
def test_planted_mistakes_are_caught(monkeypatch, mistake):
    right = v.sequence

    def wrong(target, drafts, uniforms, noise, draft_logits=None, temperature=1.0):
        if mistake == "flipped test":
            return right(target, drafts, 1.0 - np.sqrt(uniforms), noise, draft_logits, temperature)
        got = right(target, drafts, uniforms, noise, draft_logits, temperature)
        return got if got[1] == len(drafts) else ([int(np.argmax(v.softmax(target[got[1]]) / noise))],) + got[1:]

    monkeypatch.setattr(v, "sequence", wrong)
    with pytest.raises(AssertionError):
        test_tokens_are_distributed_as_the_target(False)
