"""The many-rows attention kernel where a row's running reference moves inside a key tile of 128 tokens: what the tile's
earlier chunks of 32 tokens left is read back, scaled and used.

Keys are one value in channel 0 and the query is one there, with scale = ln 2, so a token's score in base 2 is its key.
Values of chunk c lie in their own 16 channels, so an output shows one chunk's weights alone.  The tolerance is that of
attention over this cache: a weight is off by 2^-11 (f16) and by its score's 2^-20 M + 2^-21, outputs by 2^-9 of themselves,
and 2^-32 of the row's largest weight for each token; all doubled, M the largest sum of |q_d k_d| scale."""

import numpy as np
import pytest
import torch

from oracle import kv_nvfp4 as kv
from oracle.formats import bf16_rne

from .conftest import to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOKENS, CHUNK = 300, 32


@pytest.fixture(scope="module")
def q():
    from quantized_rl_rollout_gb300 import build, qrr

    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    qrr.lib()
    return qrr


def _keys(dim, chunks):
    """Key rows [TOKENS, 1, dim] whose chunk c of the first tile has the score chunks[c]; zero behind it."""
    k = torch.zeros(TOKENS, 1, dim)
    for c, score in enumerate(chunks):
        k[CHUNK * c:CHUNK * (c + 1), 0, 0] = score
    return k


def _values(dim, seed):
    """Values [TOKENS, 1, dim]: token t's lie in the 16 channels of its chunk (of the first tile; the rest in chunk 3's)."""
    v = torch.zeros(TOKENS, 1, dim)
    g = torch.Generator().manual_seed(seed)
    for t in range(TOKENS):
        c = min(t // CHUNK, 3)
        v[t, 0, 16 * c:16 * c + 16] = torch.randn(16, generator=g).abs() + 0.5
    return v


def _check(q, k, v, rows=40, hq=8, runs=1, on_grid=True):
    """``rows`` last tokens' attention over all of it, against the oracle; every run the same bits.  ``on_grid``: the keys
    are meant to be kept as they are."""
    dim = k.shape[-1]
    k, v = k.to(torch.bfloat16).to(DEV), v.to(torch.bfloat16).to(DEV)
    pages = -(-TOKENS // 64)
    cache = q.KvCacheNvfp4.empty(pages, 1, 64, dim, torch.arange(pages, dtype=torch.int32, device=DEV)[None])
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    q.kv_append_nvfp4(k, v, cache, i32([0]), cu=i32([0, TOKENS]))
    x = torch.zeros(rows, hq, dim, device=DEV)
    x[..., 0] = 1
    x = x.to(torch.bfloat16)
    scale = float(np.log(2.0))
    first = None
    for _ in range(runs):
        out, lse = q.attention_nvfp4(x, cache, i32([TOKENS - rows]), cu=i32([0, rows]), max_new=rows, scale=scale, return_lse=True)
        if first is None:
            first = out, lse
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    one = np.ones(1, np.float32)
    kd, vd = (kv.kv_values(*kv.kv_quantize(to_np(z), one), one) for z in (k, v))
    assert not on_grid or np.array_equal(kd[..., 0], bf16_rne(to_np(k)[..., 0]))
    want, want_lse, spread = kv.attention(to_np(x), kd, vd, TOKENS - rows, scale)
    tol = 2 ** -18 * (np.abs(kd).max() * scale + 1)
    assert (np.abs(to_np(first[1]) - want_lse) <= tol).all()
    bound = 2 ** -8 * np.abs(want) + (2 ** -10 + tol) * spread + 2 ** -31 * np.abs(vd).sum(0) + 1e-30
    off = np.abs(to_np(first[0]) - want) / bound
    assert off.max() <= 1, off.max((0, 1))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("chunks", [(0, 9, 18, 27), (0, 18, 18, 36), (0, 0, 12, 24), (0, 15, 0, 0), (-12, 0, 0, 9)])
def test_reference_moves_from_chunk_to_chunk(q, dim, chunks):
    _check(q, _keys(dim, chunks), _values(dim, 1), runs=50)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("top", [13.5, 15, 22.5, 24, 27, 30])
def test_heavy_weights_under_a_far_larger_score(q, dim, top):
    """Chunk 1's scores (7.5) are just under what would move the reference (-7), so their weights are f16's largest; one
    score of ``top`` in chunk 2 moves it far.  What is left of chunk 1's weights, down to 2^-30 of the row's largest, is
    seen alone in its channels."""
    k = _keys(dim, (0, 7.5))
    k[2 * CHUNK + 5, 0, 0] = top
    _check(q, k, _values(dim, 2))
    for t in range(CHUNK, 2 * CHUNK):  # several tiles, other shares of the row's weights
        k[t, 0, 0] = (0, 1.5, 3, 4.5, 6, 7.5)[t % 6]
    k[200, 0, 0] = top + 6
    _check(q, k, _values(dim, 3), on_grid=False)
