"""What the calls on rows of logits report, beside what test_gpu_logits_loss.py asks of them: the gradient from known
log-sum-exps, teachers and rollouts without numbers, and rows that are not read."""

import numpy as np
import pytest
import torch

from .test_gpu_logits_loss import BF16, DEV, FP32, _check, _rows, _teacher, q  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture
def status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def _flags(q, status, call):  # noqa: F811
    status.zero_()
    call()
    return q.get_last_device_status(status)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("t,v,pad", [(4, 601, 0), (3, 40000, 0), (400, 70, 1)])
def test_backward(q, status, t, v, pad, dtype, tail):  # noqa: F811
    """A NaN or +inf in a row or in its log-sum-exps, wherever it stands, in place and to rows that start elsewhere."""
    x, _ = _rows(t, v, dtype, 1, pad)
    ids, top, lse = _teacher(x, 6, 2, 1.0, tail)
    grad = torch.ones(t, device=DEV)
    _, stats = q.distill_topk(x, ids, top, top_lse=lse)
    more = dict(top_lse=lse, dev_status=status)
    outs = [lambda y: y, lambda y: torch.empty(t, v + 1, dtype=dtype, device=DEV)[:, :v], lambda y: torch.empty_like(y)]
    assert all(_flags(q, status, lambda: q.distill_topk_backward(x.clone(), ids, top, stats, grad, dlogits=o(x.clone()), **more)) == 0
               for o in outs)
    for bad in (float("nan"), float("inf")):
        for at in (0, 1, v // 2, v - 2, v - 1, int(ids[t - 1, 3])):
            for out in outs:
                y = x.clone()
                y[t - 1, at] = bad
                assert _flags(q, status, lambda: q.distill_topk_backward(y, ids, top, stats, grad, dlogits=out(y), **more)) == q.DEV_NONFINITE, (bad, at)
        for column in (0, 1) if tail else (0,):
            s = stats.clone()
            s[t - 1, column] = bad
            assert _flags(q, status, lambda: q.distill_topk_backward(x, ids, top, s, grad, **more)) == q.DEV_NONFINITE, (bad, column)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_finite_rows_raise_nothing(q, status, dtype, tail):  # noqa: F811
    """Masks, rows of -inf, the type's lowest and large values are no NaN or +inf: no call reports them."""
    x, _ = _rows(7, 3001, dtype, 3)
    ids, top, lse = _teacher(x, 12, 4, 1.0, tail)
    x[0, 5:] = -torch.inf
    x[1] = -torch.inf
    x[2, 7:] = torch.finfo(dtype).min
    x[3] -= 3000
    x[4] += 3000
    x[5] = 0
    x[6, ids[6].long()] -= 300
    grad, tokens = torch.linspace(-1, 1, 7, device=DEV), ids[:, 0].contiguous()
    more = dict(top_lse=lse, dev_status=status)
    _, stats = q.distill_topk(x, ids, top, **more)
    for call in (lambda: q.distill_topk(x, ids, top, **more), lambda: q.distill_topk_grad(x, ids, top, grad, **more),
                 lambda: q.distill_topk_backward(x, ids, top, stats, grad, **more),
                 lambda: q.token_logprobs_is_grad(x, tokens, grad, dev_status=status)):
        assert _flags(q, status, call) == 0


def test_rows_that_are_not_read(q, status):  # noqa: F811
    """NaN in a row without a teacher or token, and in its log-sum-exps, and behind the vocabulary: nothing is reported."""
    x, _ = _rows(6, 900, BF16, 5, pad=9)  # (the padding is NaN)
    ids, top, lse = _teacher(x, 5, 6, 1.0, True, idle=2)
    x[::2] = float("nan")
    grad, tokens = torch.ones(6, device=DEV), ids[:, 3].contiguous()
    more = dict(top_lse=lse, dev_status=status)
    _, stats = q.distill_topk(x, ids, top, **more)
    stats[::2] = float("nan")
    for call in (lambda: q.distill_topk(x, ids, top, **more), lambda: q.distill_topk_grad(x, ids, top, grad, **more),
                 lambda: q.distill_topk_backward(x, ids, top, stats, grad, **more),
                 lambda: q.token_logprobs_is_grad(x, tokens, grad, dev_status=status)):
        assert _flags(q, status, call) == 0


def test_teachers_of_nothing(q, status):  # noqa: F811
    """All of a row's slots at -inf: no distribution among them, which is reported; with the teacher's log-sum-exp all of it is
    rest."""
    x, _ = _rows(4, 700, BF16, 7)
    ids, top, lse = _teacher(x, 5, 8, 1.0, True)
    grad = torch.ones(4, device=DEV)
    _, stats = q.distill_topk(x, ids, top)
    top[2] = -torch.inf
    for call in (lambda: q.distill_topk(x, ids, top, dev_status=status), lambda: q.distill_topk_grad(x, ids, top, grad, dev_status=status),
                 lambda: q.distill_topk_backward(x, ids, top, stats, grad, dev_status=status)):
        assert _flags(q, status, call) == q.DEV_NONFINITE
    _check(q, x, ids, top, lse, 1.0)


@pytest.mark.parametrize("cap", [0.0, 1.5])
def test_weights_without_a_number(q, status, cap):  # noqa: F811
    """A rollout's log-probability that is NaN, or -inf where the token is masked here too: the weight is NaN, capped or not, and
    reported; a weight of +inf without a cap as well, and with one it is the cap."""
    x, _ = _rows(5, 300, BF16, 9)
    x[2, 11] = -torch.inf
    tokens = torch.tensor([4, 8, 11, 15, 16], dtype=torch.int32, device=DEV)
    adv = torch.ones(5, device=DEV)
    rollout = torch.tensor([-3.0, float("nan"), -torch.inf, -4.0, -5.0], device=DEV)
    got = {}
    assert _flags(q, status, lambda: got.update(r=q.token_logprobs_is_grad(x, tokens, adv, rollout, cap, dev_status=status))) == q.DEV_NONFINITE
    logp, w, d = got["r"]
    assert torch.isnan(w).tolist() == [False, True, True, False, False]
    assert torch.isnan(d).any(1).tolist() == [False, True, True, False, False]
    want = torch.exp(logp.double() - rollout.double())[[0, 3, 4]]
    want = want.clamp(max=cap) if cap else want
    assert np.allclose(w.double()[[0, 3, 4]].cpu().numpy(), want.cpu().numpy(), rtol=1e-6, atol=0)
    rollout = torch.tensor([-3.0, -torch.inf, -3.0, -4.0, -5.0], device=DEV)
    flags = _flags(q, status, lambda: got.update(r=q.token_logprobs_is_grad(x, tokens, adv, rollout, cap, dev_status=status)))
    assert flags == (0 if cap else q.DEV_NONFINITE) and float(got["r"][1][1]) == (cap or np.inf)
