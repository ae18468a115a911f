"""Gradients over the logits themselves where a row's sums are taken twice: logits at the ids, or the token's, are so far below the
row's that the first reference does not serve, or the row is beyond 2^20 in base 2.  Bit for bit what other memory gets."""

import pytest
import torch

from .test_gpu_logits_loss import BF16, DEV, FP32, _rows, _teacher, q  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("t,v,pad", [(1, 40000, 0), (3, 32003, 0), (9, 1001, 1), (400, 9001, 0), (5, 128256, 0)])
def test_rows_that_are_summed_twice(q, t, v, pad, dtype, tail):  # noqa: F811
    x, _ = _rows(t, v, dtype, v, pad)
    ids, top, lse = _teacher(x, 33, 6, 1.0, tail)
    x.scatter_(1, ids.clamp(min=0).long(), -150.0)  # e^150 of a reference there
    x[t // 2] += 1e6
    grad, tokens = torch.linspace(-1, 1, t, device=DEV) if t > 1 else torch.ones(1, device=DEV), ids[:, 5].contiguous()
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    more = dict(top_lse=lse, dev_status=st)
    loss, want = q.distill_topk_grad(x, ids, top, grad, **more)
    _, stats = q.distill_topk(x, ids, top, **more)
    back = q.distill_topk_backward(x, ids, top, stats, grad, **more)
    logp, w, policy = q.token_logprobs_is_grad(x, tokens, grad, grad, 2.0, dev_status=st)
    assert q.get_last_device_status(st) == 0 and torch.isfinite(want).all() and torch.isfinite(policy).all()
    for _ in range(3):
        for call, ref, also in ((lambda o: q.distill_topk_grad(o, ids, top, grad, dlogits=o, **more), want, loss),
                                (lambda o: (loss, q.distill_topk_backward(o, ids, top, stats, grad, dlogits=o, **more)), back, loss),
                                (lambda o: q.token_logprobs_is_grad(o, tokens, grad, grad, 2.0, dlogits=o, dev_status=st)[::2], policy, logp)):
            own = torch.empty_strided(x.shape, x.stride(), dtype=dtype, device=DEV).copy_(x)
            first, d = call(own)
            assert d.data_ptr() == own.data_ptr() and torch.equal(own, ref) and torch.equal(first, also)
