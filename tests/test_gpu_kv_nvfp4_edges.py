"""The paged NVFP4 cache at the ends of its arguments: positions at the ends of 32 bits, offsets that leave the rows,
calls without rows, queries that are not finite."""

import numpy as np
import pytest
import torch

from .test_gpu_kv_nvfp4 import Bed, _dev, q  # noqa: F401

pytestmark = pytest.mark.gpu
DEV = "cuda"
LOWEST = -2 ** 31


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("news", [[1, 3, 2], [40, 300, 60], [2, 300, 1]])
@pytest.mark.parametrize("low", [LOWEST, LOWEST + 5, -2 ** 30 - 1, -2 ** 30, -1000])
def test_positions_far_below_zero(q, dim, news, low):  # noqa: F811
    """Sequences whose rows all stand before the first token see nothing; the one between them is as in a call of its own."""
    bed = Bed(q, [200, 400, 90], 2, dim, 16, 30)
    t, st = sum(news), _dev([0])
    x = torch.randn(t, 8, dim, device=DEV).to(torch.bfloat16)
    cu = np.concatenate([[0], np.cumsum(news)])
    pos = [low, 400 - news[1], low]
    out, lse = q.attention_nvfp4(x, bed.cache, _dev(pos), cu=_dev(cu), max_new=max(news), return_lse=True, dev_status=st)
    mid = slice(cu[1], cu[2])
    alone = q.attention_nvfp4(x[mid].contiguous(), bed.cache, _dev([0, pos[1], 0]), cu=_dev([0, 0, news[1], news[1]]),
                              max_new=max(news), return_lse=True, dev_status=st)
    k, v = q.kv_read_nvfp4(bed.cache, _dev(pos), cu=_dev(cu), rows=t, dev_status=st)
    before = [z.clone() for z in bed.cache.tensors[:4]]
    rows = torch.randn(t, 2, dim, device=DEV).to(torch.bfloat16)
    q.kv_append_nvfp4(rows, rows, bed.cache, _dev([low] * 3), cu=_dev(cu), dev_status=st)
    assert q.get_last_device_status(st) == 0
    for s in (slice(0, cu[1]), slice(cu[2], t)):
        assert not out[s].any() and torch.isneginf(lse[s]).all() and not k[s].any() and not v[s].any()
    # the cut of the work may differ between the calls, so bits may: two bf16 roundings apart
    assert torch.isfinite(lse[mid]).all() and (lse[mid] - alone[1]).abs().max() < 1e-4
    assert (out[mid] - alone[0]).float().abs().max() <= 2 ** -6 * alone[0].float().abs().max()
    assert all(torch.equal(a, b) for a, b in zip(before, bed.cache.tensors[:4]))
