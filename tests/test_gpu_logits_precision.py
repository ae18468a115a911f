"""How near losses of about 0.1 and log-sum-exps of 20 to 30 come to the float64 oracle: what temperatures in double,
exponents in two parts and two-part sums at the ids are there for.

Rows whose 64 ids hold most, so that the bounds are small.  What is outside them, a share r, is off by the hardware's exponentials
(2^-22), their arguments' rounding (20 2^-24 ln 2) and the sum's 24 additions in sequence (4096 elements over 128 threads, 2^-24
each): 2.5e-6 of itself, which is 2.5e-6 r of the whole sum, and of a tail's logarithm that times the teacher's rest.  At the ids
an exponential is within 2^-24 and the two-part sum exact; the logarithm, and the difference that is rounded as a small number, 2^-24
each: 1.8e-7.  A log-sum-exp is rounded besides, by 2^-20 below 32.  (An exponent of 30 that is rounded alone is off by 2^-20 =
9.5e-7 at each id, a temperature of 0.8 in 32 bits by 1.5e-8 of itself, 4e-7 and more at such logits.)"""

import math

import numpy as np
import pytest
import torch

from oracle import distill

from .test_gpu_logits_loss import BF16, DEV, FP32, q  # noqa: F401

pytestmark = pytest.mark.gpu
V, K, T_ROWS, OUTSIDE, IDS = 4096, 64, 40, 2.5e-6, 1.8e-7


@pytest.mark.parametrize("temperature", [0.8, 1.0])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("tail", [False, True])
def test_losses_and_log_sum_exps(q, dtype, temperature, tail):  # noqa: F811
    g = torch.Generator().manual_seed(71)
    t = temperature
    outside = t * (17 / t + 1.5 / t ** 2 + math.log(0.08 * K / V))  # a normal's mean is e^(s^2 / 2) above its middle's
    x = outside + torch.randn(T_ROWS, V, generator=g)
    ids = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(T_ROWS)])
    x.scatter_(1, ids, 17 + 2 * torch.randn(T_ROWS, K, generator=g).clamp(-2.5, 2.5))
    x = x.to(dtype)
    y = x.float() + 0.4 * t * torch.randn(T_ROWS, V, generator=g)
    top = y.gather(1, ids)
    lse = torch.logsumexp(y.double() / t, -1).float()
    loss, stats, _ = distill.distill(x.double().numpy(), ids.numpy(), top.double().numpy(), lse.double().numpy() if tail else None, t)
    total = torch.logsumexp(x.double() / t, -1).numpy()
    r = 1 - np.exp(torch.logsumexp(x.double().gather(1, ids) / t, -1).numpy() - total)
    rest = np.array([max(0.0, 1 - np.exp(top[i].double().numpy() / t - float(lse[i])).sum()) for i in range(T_ROWS)]) if tail else 0.0
    assert 0.03 < np.median(loss) < 0.3 and total.max() < 32 and np.median(r) < 0.15
    x, ids, top, lse = x.to(DEV), ids.to(torch.int32).to(DEV), top.to(DEV), lse.to(DEV) if tail else None
    more = dict(top_lse=lse, temperature=t)
    got, got_stats = q.distill_topk(x, ids, top, **more)
    again, _ = q.distill_topk_grad(x, ids, top, torch.ones(T_ROWS, device=DEV), **more)
    for a in (got, again):
        assert np.all(np.abs(a.double().cpu().numpy() - loss) <= OUTSIDE * (r + rest) + IDS)
    off = np.abs(got_stats.double().cpu().numpy() - stats)
    assert np.all(off[:, 0] <= OUTSIDE * r + IDS + 2.0 ** -20)
    if tail:
        assert np.all(off[:, 1] <= OUTSIDE + 2.0 ** -20)


@pytest.mark.parametrize("temperature", [0.8, 1.0])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("tail", [False, True])
def test_two_ids_hold_all(q, dtype, temperature, tail):  # noqa: F811
    """Rows of two ids about 26 t whose errors do not average out: nothing is outside them but what a tail's logarithm is of.

    Off by: the exponentials at the ids, 2^-24; the logarithm's small part, 2^-25; y - x, below 2, over t, 1.25 2^-24; that with the
    log-sum-exps' difference, 2^-24; the two products and their sum, 2^-24: 2.9e-7.  A tail's logarithm is off by 2.5e-6 as
    above, times the rest of 0.03.  Mistakes that these bounds have to find, planted in the oracle: exponents of 37
    rounded once, and a temperature in 32 bits beside a log-sum-exp that is not."""
    g = torch.Generator().manual_seed(72)
    t, n, v = temperature, 200, 513
    x = 4 + torch.randn(n, v, generator=g)
    ids = torch.stack([torch.randperm(v, generator=g)[:2] for _ in range(n)])
    x.scatter_(1, ids, 26 * t + 0.5 * torch.randn(n, 2, generator=g).clamp(-2, 2))
    x = x.to(dtype)
    top = x.float().gather(1, ids) + t * torch.tensor([0.4, -1.2]) + 0.05 * torch.randn(n, 2, generator=g)
    lse = (torch.logsumexp(top.double() / t, -1) + 0.03).float() if tail else None
    host = lambda a: None if a is None else a.double().numpy()  # noqa: E731

    def of(scaled, temperature=1.0, y=host(top) / t):
        return distill.distill(scaled, ids.numpy(), y, host(lse), temperature)[0]

    loss = of(host(x) / t)
    bound = np.full(n, 2.9e-7 + (OUTSIDE * 0.03 if tail else 0.0))
    once = (x.float() * np.float32(math.log2(math.e) / t)).double().numpy() * math.log(2)
    assert (np.abs(of(once) - loss) > bound).sum() >= 5
    if tail and t != 1.0:
        t32 = float(np.float32(t))
        assert (np.abs(of(host(x) / t32, y=host(top) / t32) - loss) > bound).sum() >= 5
    x, ids_, top, lse_ = x.to(DEV), ids.to(torch.int32).to(DEV), top.to(DEV), None if lse is None else lse.to(DEV)
    more = dict(top_lse=lse_, temperature=t)
    got, _ = q.distill_topk(x, ids_, top, **more)
    again, _ = q.distill_topk_grad(x, ids_, top, torch.ones(n, device=DEV), **more)
    for a in (got, again):
        assert np.all(np.abs(a.double().cpu().numpy() - loss) <= bound)
