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


T = 12
OFFSETS = [  # offsets of two sequences, and the rows that belong to a sequence with sound ones
    ([0, 6, 50], range(0, 6)), ([-3, 6, 12], range(6, 12)), ([0, 12, 13], range(0, 12)), ([-1, 0, 12], range(0, 12)), ([5, 40, 60], []),
    ([0, 6, 12], range(0, 12)), ([2, 2, 9], range(2, 9))]


def _guarded(shape, dtype):
    """A tensor of sevens inside a larger one, and a check that what lies around it stays."""
    n = int(np.prod(shape))
    whole = torch.full((n + 4096,), 7, dtype=dtype, device=DEV)
    return whole[2048:2048 + n].view(shape), lambda: bool((whole[:2048] == 7).all() and (whole[2048 + n:] == 7).all())


@pytest.mark.parametrize("cu,sound", OFFSETS)
def test_append_and_read_tell_offsets_that_leave_the_rows(q, cu, sound):  # noqa: F811
    """Such a sequence's rows are not written and read zeros; the others are as ever."""
    bad = not 0 <= cu[0] <= cu[1] <= cu[2] <= T
    cache = q.KvCacheNvfp4.empty(8, 2, 16, 64, _dev([[0, 1, 2, 3], [4, 5, 6, 7]]))
    x = torch.randn(T, 2, 64, device=DEV).to(torch.bfloat16)
    st, pos = _dev([0]), _dev([1, 20])
    q.kv_append_nvfp4(x, x, cache, pos, cu=_dev(cu), dev_status=st)
    assert q.get_last_device_status(st) == (q.DEV_BAD_INDEX if bad else 0)
    places = {(int(t >= cu[1]), [1, 20][t >= cu[1]] + t - cu[t >= cu[1]]): t for t in sound}  # (sequence, position): row
    for s in (0, 1):
        for p in range(64):
            there = bool(cache.tensors[1][4 * s + p // 16, :, p % 16].any())
            assert there == ((s, p) in places), (s, p)
    full = torch.randn(128, 2, 64, device=DEV).to(torch.bfloat16)
    q.kv_append_nvfp4(full, full, cache, _dev([0, 0]), cu=_dev([0, 64, 128]))
    (k, k_ok), (v, v_ok) = _guarded((T, 2, 64), torch.bfloat16), _guarded((T, 2, 64), torch.bfloat16)
    st.zero_()
    q.kv_read_nvfp4(cache, pos, cu=_dev(cu), k=k, v=v, dev_status=st)
    assert q.get_last_device_status(st) == (q.DEV_BAD_INDEX if bad else 0) and k_ok() and v_ok()
    want = torch.cat(q.kv_read_nvfp4(cache, _dev([0, 0]), cu=_dev([0, 64, 128]), rows=128)[:1])
    rows = {t: 64 * s + p for (s, p), t in places.items()}
    for t in range(T):
        assert torch.equal(k[t], want[rows[t]]) if t in rows else not k[t].any()


@pytest.mark.parametrize("cu", [[0, 9, 4], [0, 13, 4], [7, 3, 12]])
def test_descending_offsets_are_told(q, cu):  # noqa: F811
    """What rows such offsets name is not said; nothing outside the call's rows is touched."""
    cache = q.KvCacheNvfp4.empty(8, 2, 16, 64, _dev([[0, 1, 2, 3], [4, 5, 6, 7]]))
    x = torch.randn(T, 2, 64, device=DEV).to(torch.bfloat16)
    for call in (lambda st: q.kv_append_nvfp4(x, x, cache, _dev([1, 20]), cu=_dev(cu), dev_status=st),
                 lambda st: q.kv_read_nvfp4(cache, _dev([1, 20]), cu=_dev(cu), k=k, v=v, dev_status=st)):
        (k, k_ok), (v, v_ok), st = _guarded((T, 2, 64), torch.bfloat16), _guarded((T, 2, 64), torch.bfloat16), _dev([0])
        call(st)
        assert q.get_last_device_status(st) == q.DEV_BAD_INDEX and k_ok() and v_ok()


@pytest.mark.parametrize("cu", [[0, 6, 50], [-3, 6, 12], [0, 9, 4], [5, 40, 60]])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (80, 1)])
def test_attention_stays_inside_the_rows(q, cu, hq, hkv):  # noqa: F811
    """Offsets that leave the rows or descend: flagged, and nothing around out and lse is written (both kernels)."""
    bed = Bed(q, [40, 200], hkv, 64, 16, 24)
    x = torch.randn(T, hq, 64, device=DEV).to(torch.bfloat16)
    (out, out_ok), (lse, lse_ok), st = _guarded((T, hq, 64), torch.bfloat16), _guarded((T, hq), torch.float32), _dev([0])
    q.attention_nvfp4(x, bed.cache, _dev([30, 180]), cu=_dev(cu), max_new=12, out=out, lse=lse, dev_status=st)
    assert q.get_last_device_status(st) & q.DEV_BAD_INDEX and out_ok() and lse_ok()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("b,hkv", [(2, 2), (600, 8)])
def test_no_rows_a_sequence_beside_rows_of_nobody(q, dim, b, hkv):  # noqa: F811
    """max_new = 0 over a cache of more than a range's tokens, with few items and with many: the rows are left alone, and
    a sequence that does bring one is told."""
    cache = q.KvCacheNvfp4.empty(20, hkv, 16, dim, torch.zeros(b, 20, dtype=torch.int32, device=DEV))
    x = torch.randn(5, 2 * hkv, dim, device=DEV).to(torch.bfloat16)
    for at, cu in ((0, [3] * (b + 1)), (q.DEV_BAD_INDEX, [0] * b + [1])):
        (out, out_ok), (lse, lse_ok), st = _guarded(tuple(x.shape), torch.bfloat16), _guarded((5, 2 * hkv), torch.float32), _dev([0])
        q.attention_nvfp4(x, cache, _dev([40] * b), cu=_dev(cu), max_new=0, out=out, lse=lse, dev_status=st)
        assert q.get_last_device_status(st) == at and out_ok() and lse_ok()
        assert (out == 7).all() and (lse == 7).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens,news", [([60, 30], [1, 1]), ([3000, 30], [1, 2]), ([9000, 20], [1, 4]), ([700, 90], [40, 60]), ([5000, 40], [300, 1])])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_queries_that_are_not_finite(q, dim, lens, news, value):  # noqa: F811
    """Such a row comes out as NaN, its log-sum-exp too (not as a row that sees nothing); every other row is as without it.
    Items in one piece, in a few and in many, both kernels."""
    bed = Bed(q, lens, 2, dim, 16, 31)
    t = sum(news)
    x = torch.randn(t, 8, dim, device=DEV).to(torch.bfloat16)
    pos, cu = _dev([n - m for n, m in zip(lens, news)]), _dev([0, news[0], t])
    want = q.attention_nvfp4(x, bed.cache, pos, cu=cu, max_new=max(news), return_lse=True)
    hit = torch.zeros(t, 8, dtype=torch.bool, device=DEV)
    for row, head in ((0, 3), (t - 1, 6)):
        x[row, head, 17] = value
        hit[row, head] = True
    st = _dev([0])
    out, lse = q.attention_nvfp4(x, bed.cache, pos, cu=cu, max_new=max(news), return_lse=True, dev_status=st)
    assert q.get_last_device_status(st) == q.DEV_NONFINITE
    assert torch.isnan(lse[hit]).all() and torch.isnan(out[hit]).all()
    assert torch.equal(out[~hit], want[0][~hit]) and torch.equal(lse[~hit], want[1][~hit])
