"""Teachers that are no plain distribution over different ids, against the float64 oracle and against differences of the
losses: slots that name one id, and probabilities that pass 1 together.  Bounds are test_gpu_logits_loss.py's."""

import pytest
import torch

from .test_gpu_logits_loss import BF16, DEV, FP32, LSE, P, _check, _rows, _teacher, q  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("k", [2, 3, 64, 1024])
def test_a_certain_token_named_often(q, dtype, k):  # noqa: F811
    """k equal slots of one id are that id with probability 1: the loss is -ln q, and 0 where the student is certain too."""
    x, _ = _rows(3, 2001, dtype, 1)
    x[1] = -torch.inf
    x[1, 5] = 1.0
    ids = torch.full((3, k), 5, dtype=torch.int32, device=DEV)
    top = torch.full((3, k), 2.0, device=DEV)
    want = (torch.logsumexp(x.double(), -1) - x[:, 5].double()).cpu()
    loss, _ = q.distill_topk(x, ids, top)
    again, d = q.distill_topk_grad(x, ids, top, torch.ones(3, device=DEV))
    for got in (loss, again):
        assert torch.all((got.double().cpu() - want).abs() <= LSE + P * (1 + want))
    # (p and q each within P of 1, and a bf16's rounding of what is left)
    assert abs(float(d[1, 5])) <= 2 * P


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_slots_of_one_id(q, dtype, tail):  # noqa: F811
    """Pairs far apart in probability, triples, and slots of p = 0, over rows of one CTA and of several."""
    for t, v in ((4, 900), (2, 60000), (400, 333)):
        x, _ = _rows(t, v, dtype, v)
        ids, top, _ = _teacher(x, 60, 6, 1.0, False)
        ids[:, 1:30:2] = ids[:, 0:30:2]
        ids[:, 40:42] = ids[:, 39:40]
        top[:, 0:10] += 4
        top[:, 20:24:2] = -torch.inf
        lse = torch.logsumexp(torch.where(ids >= 0, top.double(), -torch.inf), -1).float() + 0.2 if tail else None
        _check(q, x, ids, top, lse, 1.0)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("temperature", [1.0, 0.7])
@pytest.mark.parametrize("shift", [-1e-6, -1e-3, -0.4, -1.0])
def test_probabilities_that_pass_one(q, dtype, temperature, shift):  # noqa: F811
    """The teacher's log-sum-exp is smaller than that of its slots alone: there is no rest, and the gradient is the loss's."""
    for t, v, k in ((5, 1203, 20), (2, 60000, 64), (400, 333, 7)):
        x, _ = _rows(t, v, dtype, v)
        ids, top, _ = _teacher(x, k, 6, temperature, False)
        lse = (torch.logsumexp(torch.where(ids >= 0, top.double() / temperature, -torch.inf), -1) + shift).float()
        _check(q, x, ids, top, lse, temperature)


@pytest.mark.parametrize("shift", [-0.4, -1.0])
def test_their_gradient_is_the_difference(q, shift):  # noqa: F811
    """As test_gpu_drafted_update.py takes it, of a loss with the teacher's probabilities summing to e^-shift."""
    g = torch.Generator().manual_seed(3)
    t, v, k, h = 7, 1500, 40, 0.05
    x = (2 * torch.randn(t, v, generator=g)).to(DEV)
    y = x.cpu() + torch.randn(t, v, generator=g)
    top, ids = torch.topk(y, k, -1)
    more = dict(top_lse=(torch.logsumexp(top, -1) + shift).to(DEV))
    top, ids = top.to(DEV), ids.to(torch.int32).to(DEV)
    d = torch.where(y > y.median(), 1.0, -1.0).to(DEV) * torch.rand(t, v, generator=g).to(DEV)
    loss, grad = q.distill_topk_grad(x, ids, top, torch.ones(t, device=DEV), **more)
    sides = [q.distill_topk(x + s * h * d, ids, top, **more)[0].double() for s in (1, -1)]
    along = (grad.double() * d.double()).sum(-1)
    size = (grad.abs().double() * d.abs().double()).sum(-1)
    # a loss is off by (LSE + P) (2 M + loss) at a mass of M = e^-shift, the difference by h^2 / 6 of M + 1 third cumulants below 1
    m = float(torch.exp(torch.tensor(-shift)))
    bound = (LSE + P) * (2 * m + loss.double().abs()) / h + h * h / 6 * (m + 1) + (LSE + P) * (2 + size)
    assert torch.all(((sides[0] - sides[1]) / (2 * h) - along).abs() <= bound)
