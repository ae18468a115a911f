"""Verification of drafts at the ends of its ranges: rows whose sums stand at references of different kinds, uniforms of 0, and
drafts whose margin is below rounding, of which the rest of the output is checked.

A sum is kept at a whole power of two near its largest logit where that is below 2^20 in base 2, at the logit itself beyond.
Decisions and tolerances are those of test_gpu_verify_drafts.py: the oracle's wherever its margin is above NEAR."""

import math

import numpy as np
import pytest
import torch

from oracle import verify

from .test_gpu_verify_drafts import BF16, DEV, EPS, FP32, LSE, NEAR, _case, _check, _run, q  # noqa: F401

pytestmark = pytest.mark.gpu


def _edge(temperature):
    """The logit whose base-2 exponent is 2^20."""
    return 2.0 ** 20 * temperature * math.log(2)


def _given(target, draft, drafts, uniforms, noise, temperature):
    """Sequences of one draft each."""
    n = len(drafts)
    return dict(target=target.to(DEV), draft_logits=None if draft is None else draft.to(DEV), counts=[1] * n,
                drafts=torch.tensor(drafts, dtype=torch.int32, device=DEV),
                uniforms=torch.as_tensor(uniforms, dtype=torch.float32).to(DEV), noise=noise.to(DEV), temperature=temperature)


@pytest.mark.parametrize("temperature", [1e-5, 1e-4])
@pytest.mark.parametrize("tie", [False, True])
def test_rows_on_either_side(q, temperature, tie):  # noqa: F811
    """The draft is the likeliest token of both rows, one of which is beyond the edge: p / q is 1, or 1/2 with a tie in the target."""
    far, near = [1.03, 1.24, 2.75, -1.03, -2.75], [0.895, 0.69, 0.964, 0.45, 0.0, -0.9, -0.69]
    pairs = [(a, b) for a in far for b in near] + [(b, a) for a in far for b in near]
    us = [0.3, 0.45, 0.52, 0.6, 0.69, 0.72, 0.8, 0.9, 0.99]
    v, rows = 40, [(a, b, u) for a, b in pairs for u in us]
    target, draft = torch.empty(2 * len(rows), v), torch.empty(len(rows), v)
    for i, (a, b, _) in enumerate(rows):
        for row, top in ((target[2 * i], a), (draft[i], b)):
            row[:] = (top - 0.5) * _edge(temperature)
            row[7] = top * _edge(temperature)
        target[2 * i, 30 if tie else 7] = target[2 * i, 7]
        target[2 * i + 1] = target[2 * i]
    noise = torch.empty(len(rows), v).exponential_(generator=torch.Generator().manual_seed(1)).clamp(min=1e-3)
    s = _given(target, draft, [7] * len(rows), [u for *_, u in rows], noise, temperature)
    _, accepted, _ = _check(q, s, enough=0.99)
    want = torch.tensor([u < (0.5 if tie else 1.0) for *_, u in rows])
    assert torch.equal(accepted.cpu().bool(), want)


@pytest.mark.parametrize("form", ["model", "lookup"])
@pytest.mark.parametrize("temperature", [1e-5, 1e-4])
@pytest.mark.parametrize("sign", [1, -1])
def test_rows_across_the_edge(q, form, temperature, sign):  # noqa: F811
    """Rows within a few temperatures of the edge: parts of one row are summed at references of both kinds."""
    g = torch.Generator().manual_seed(2)
    n, v = 24, 40000
    at = sign * _edge(temperature) + temperature * torch.linspace(-3, 12, 2 * n)[:, None]
    target = (at - temperature * 6 * torch.rand(2 * n, v, generator=g))
    draft = (at[::2] - temperature * 6 * torch.rand(n, v, generator=g))
    gumbel = -torch.log(-torch.log(torch.rand(n, v, generator=g).clamp(1e-9, 1 - 1e-7)))
    drafts = ((draft if form == "model" else target[::2]) / temperature + gumbel).argmax(-1).tolist()
    noise = torch.empty(n, v).exponential_(generator=g).clamp(min=1e-20)
    u = torch.rand(n, generator=g) * (1.0 if form == "model" else 2.0 / v)
    s = _given(target, draft if form == "model" else None, drafts, u, noise, temperature)
    _check(q, s, enough=0.6)


@pytest.mark.parametrize("form", ["model", "lookup"])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("temperature", [1e-3, 1.0])
def test_uniforms_of_zero(q, form, dtype, temperature):  # noqa: F811
    """0 q < p takes every draft that the target does not rule out, however unlikely: p / q down to e^-4000 here."""
    g = torch.Generator().manual_seed(3)
    n, v = 12, 500
    target, draft = torch.randn(2 * n, v, generator=g).to(dtype), torch.randn(n, v, generator=g).to(dtype)
    target[::2, 17] = -4.0 if temperature < 1 else -300.0
    draft[:, 17] = 5.0
    target[4::8, 17] = -torch.inf
    noise = torch.empty(n, v).exponential_(generator=g).clamp(min=1e-3)
    s = _given(target, draft if form == "model" else None, [17] * n, torch.zeros(n), noise, temperature)
    _, accepted, _ = _check(q, s, enough=0.7)
    assert accepted.tolist() == [0 if b % 4 == 2 else 1 for b in range(n)]


@pytest.mark.parametrize("v", [700, 704])
def test_same_logits_nearer_than_rounding(q, v):  # noqa: F811
    """q = p and u the largest below 1: a draft may go either way where rows start unalike, but what is given out holds together,
    and every log-probability is the oracle's of its token."""
    s = _case([5] * 12, v, BF16, "model", 7)
    s["draft_logits"] = s["target"][[i for i in range(72) if i % 6 != 5]].contiguous()
    s["uniforms"].fill_(1 - 2.0 ** -24)
    tokens, accepted, logp = (x.cpu().numpy() for x in _run(q, s))
    tokens, logp, drafts = tokens.reshape(12, 6), logp.reshape(12, 6), s["drafts"].cpu().numpy().reshape(12, 5)
    target, noise = s["target"].double().cpu().numpy().reshape(12, 6, v), s["noise"].double().cpu().numpy()
    if v == 704:
        assert (accepted == 5).all()
    for b in range(12):
        n = int(accepted[b])
        assert 0 <= n <= 5 and tokens[b, :n].tolist() == drafts[b, :n].tolist() and (tokens[b, n + 1:] == -1).all()
        assert not logp[b, n + 1:].any() and 0 <= tokens[b, n] < v
        for i in range(n + 1):
            want = verify.log_softmax(target[b, i])[tokens[b, i]]
            assert abs(logp[b, i] - want) <= LSE + 3 * EPS * abs(want)
        if n == 5:  # behind the last draft: by p and the noise
            score = verify.softmax(target[b, 5]) / noise[b]
            assert score[tokens[b, 5]] >= score.max() * (1 - NEAR)


def test_lookups_follow_the_target(q):  # noqa: F811
    """The frequencies of looked-up first tokens are p's whatever the drafts are, among them always one token (5 sigma)."""
    n, v = 20000, 6
    g = torch.Generator(device=DEV).manual_seed(12)
    x = torch.tensor([0.3, 1.0, -1.0, 0.7, 0.0, -2.0], device=DEV)
    p = torch.softmax(x.double(), -1)
    for drafts in (torch.full((n,), 1), torch.full((n,), 5), torch.arange(n) % v):
        tokens, _, _ = q.verify_drafts(x.expand(2 * n, v).contiguous(), drafts.to(torch.int32).to(DEV),
                                       uniforms=torch.rand(n, generator=g, device=DEV),
                                       noise=torch.empty(n, v, device=DEV).exponential_(generator=g))
        got = torch.bincount(tokens[::2].long(), minlength=v).double() / n
        assert torch.all((got - p).abs() <= 5 * torch.sqrt(p * (1 - p) / n))
