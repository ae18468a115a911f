"""Losses of masks by the type's lowest value where a teacher gives them something: p 3.4e38 / t is a number as long as it is below
fp32's largest, though (x - x_max) / t, or that in base 2, is not."""

import numpy as np
import pytest
import torch

from oracle import distill

from .test_gpu_logits_loss import BF16, DEV, EPS, FP32, LSE, P, _close, _rows, _teacher, q  # noqa: F401

pytestmark = pytest.mark.gpu


def _check(q, x, ids, top, lse, temperature):  # noqa: F811
    """A loss is off by P of a share and P of 1 of the rest, each times what it is multiplied with, and 8 EPS of itself."""
    host = lambda a: None if a is None else a.double().cpu().numpy()  # noqa: E731
    want, stats, _ = distill.distill(host(x), ids.cpu().numpy(), host(top), host(lse), temperature)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    more = dict(top_lse=lse, temperature=temperature, dev_status=st)
    loss, _ = q.distill_topk(x, ids, top, **more)
    again, d = q.distill_topk_grad(x, ids, top, torch.ones(x.shape[0], device=DEV), **more)
    far = np.array([abs(float(torch.finfo(x.dtype).min)) / temperature if abs(w) > 1e30 else 0.0 for w in want])
    bound = 2 * (LSE + P) * (1 + np.abs(want)) + 8 * EPS * np.abs(want) + (P * far if lse is not None else 0.0)
    _close(loss, want, bound, "loss")
    _close(again, want, bound, "loss with its gradient")
    assert torch.isfinite(d).all() and q.get_last_device_status(st) == 0
    return loss


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("temperature", [0.3, 0.8, 1.0, 1.3, 3.0])
def test_an_id_at_the_lowest_value(q, dtype, temperature, tail):  # noqa: F811
    """Of a tenth of the teacher's mass: a loss of 3e37 / t."""
    x, _ = _rows(5, 3001, dtype, 1)
    ids, top, _ = _teacher(x, 12, 2, temperature, False)
    ids[1] = ids[2]
    x[torch.arange(5), ids[:, 4].long()] = torch.finfo(dtype).min
    others = torch.logsumexp(torch.cat([top[:, :4], top[:, 5:]], 1).double() / temperature, -1)
    top[:, 4] = (temperature * (others - np.log(9))).float()
    lse = (torch.logsumexp(top.double() / temperature, -1) + 0.2).float() if tail else None
    loss = _check(q, x, ids, top, lse, temperature)
    assert torch.isfinite(loss).all() and (loss > 5e36).all()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("temperature", [0.3, 0.8, 1.0, 1.3, 3.0])
def test_nothing_but_the_lowest_value_outside_the_ids(q, dtype, temperature):  # noqa: F811
    """Of a teacher with a rest of 0.01 to 0.2."""
    x, _ = _rows(5, 3001, dtype, 3)
    ids, top, _ = _teacher(x, 12, 4, temperature, False)
    ids[1] = ids[2]
    keep = x.gather(1, ids.long())
    x[:] = torch.finfo(dtype).min
    x.scatter_(1, ids.long(), keep)
    lse = (torch.logsumexp(top.double() / temperature, -1) + torch.tensor([0.01, 0.02, 0.05, 0.1, 0.2], device=DEV)).float()
    loss = _check(q, x, ids, top, lse, temperature)
    assert torch.isfinite(loss).all() and (loss > 1e35).all()
