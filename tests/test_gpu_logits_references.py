"""Losses over logits at temperatures where sums stand at references of both kinds (test_gpu_verify_references.py says which),
with a tail and without, beside and across the edge between them.

Bounds, those of test_gpu_logits_loss.py's extreme temperatures: of a loss every logarithm is rounded by itself, 3 EPS of (y -
y_max) / t and (x - x_max) / t each, and 8 EPS of the whole grant both; a rest of the teacher's is off by P of 1.  What is
known by its fp32 log-sum-exp is off by 3 EPS of that: its own rounding, that of its product with t and that of a difference."""

import math

import numpy as np
import pytest
import torch

from oracle import distill

from .test_gpu_logits_loss import DEV, EPS, LSE, P, _close, q  # noqa: F401

pytestmark = pytest.mark.gpu
T_ROWS, V, K = 8, 5001, 12


def _given(temperature, sign, tail):
    """Rows whose ids and whose other logits reach the edge, one side of it or the other, or stand far apart about it."""
    g = torch.Generator().manual_seed(5)
    edge, t = sign * 2.0 ** 20 * temperature * math.log(2), temperature
    tops = [(edge * 1.002, edge * 0.999), (edge * 0.999, edge * 1.002), (edge + 3 * t, edge - 2 * t), (edge - 2 * t, edge + 3 * t),
            (edge, edge), (edge + 40 * t, edge + 37 * t), (edge - 40 * t, edge - 44 * t), (edge * 2, edge * 2 - 3 * t)]
    ids = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(T_ROWS)])
    x = torch.empty(T_ROWS, V)
    y = torch.empty(T_ROWS, K)
    for row, (at, rest) in enumerate(tops):
        x[row] = rest - 6 * t * torch.rand(V, generator=g)
        x[row, ids[row]] = at - 6 * t * torch.rand(K, generator=g)
        y[row] = at + t * (2 * torch.rand(K, generator=g) - 3)
    lse = (torch.logsumexp(y.double() / t, -1) + 0.7).float() if tail else None
    return x.to(DEV), ids.to(torch.int32).to(DEV), y.to(DEV), None if lse is None else lse.to(DEV)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("temperature", [1e-5, 1e-4])
def test_losses_about_the_edge(q, temperature, sign, tail):  # noqa: F811
    x, ids, y, lse = _given(temperature, sign, tail)
    grad, st = torch.ones(T_ROWS, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    host = lambda a: None if a is None else a.cpu().numpy().astype(np.float64)  # noqa: E731
    loss, stats, ref = distill.distill(host(x), ids.cpu().numpy(), host(y), host(lse), temperature)
    more = dict(top_lse=lse, temperature=temperature, dev_status=st)
    got, got_stats = q.distill_topk(x, ids, y, **more)
    again, d = q.distill_topk_grad(x, ids, y, grad, **more)
    back = q.distill_topk_backward(x, ids, y, got_stats, grad, **more)
    l_bound = 4 * (LSE + P) + 8 * EPS * np.abs(loss)
    _close(got, loss, l_bound, "loss")
    _close(again, loss, l_bound, "loss with its gradient")
    _close(got_stats, stats, LSE + 3 * EPS * np.abs(stats), "stats")
    scale = (LSE + P + 3 * EPS * 100) * 2 / temperature
    _close(d, ref, scale + np.abs(ref) * EPS, "gradient")
    known = np.expm1(3 * EPS * np.abs(stats).max(-1, keepdims=True)) * 3 / temperature
    _close(back, ref, scale + known + np.abs(ref) * EPS, "backward")
    assert q.get_last_device_status(st) == 0


@pytest.mark.parametrize("temperature", [1e-6, 1e-3, 1e3, 1e6])
def test_extreme_temperatures_with_a_tail(q, temperature):  # noqa: F811
    """Ordinary logits over all temperatures; the teacher's log-sum-exp leaves it a rest."""
    g = torch.Generator().manual_seed(6)
    x = 2.5 * torch.randn(5, 3001, generator=g)
    x[3, ::2] = -torch.inf
    ids = torch.stack([torch.randperm(1500, generator=g)[:K] for _ in range(5)]) * 2 + 1
    y = x.gather(1, ids) + 0.8 * torch.randn(5, K, generator=g)
    lse = (torch.logsumexp(y.double() / temperature, -1) + torch.tensor([0.1, 0.5, 1.0, 2.0, 4.0])).float()
    x, ids, y, lse = x.to(DEV), ids.to(torch.int32).to(DEV), y.to(DEV), lse.to(DEV)
    host = lambda a: a.cpu().numpy().astype(np.float64)  # noqa: E731
    loss, stats, ref = distill.distill(host(x), ids.cpu().numpy(), host(y), host(lse), temperature)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    more = dict(top_lse=lse, temperature=temperature, dev_status=st)
    got, got_stats = q.distill_topk(x, ids, y, **more)
    again, d = q.distill_topk_grad(x, ids, y, torch.ones(5, device=DEV), **more)
    l_bound = 4 * (LSE + P) + 8 * EPS * np.abs(loss)
    _close(got, loss, l_bound, "loss")
    _close(again, loss, l_bound, "loss with its gradient")
    _close(got_stats, stats, LSE + 3 * EPS * np.abs(stats), "stats")
    _close(d, ref, (LSE + P + 3 * EPS * 100) * 2 / temperature + np.abs(ref) * EPS, "gradient")
    assert q.get_last_device_status(st) == 0
