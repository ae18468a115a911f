"""The paged NVFP4 key/value cache and attention over it, in float64.

Test infrastructure only (see the package docstring).

What it follows.  QeRL keeps the policy in NVFP4 during rollout ("QeRL: Beyond
Efficiency", abstract), and NVIDIA's FP8 recipe extends low precision from the
linear layers to the KV cache and the attention operations ("NVIDIA NeMo RL
behaalt 48% ...", section "Praktische prestatiewinsten").  Readings:

* a cached row (one token, one KV head, D values) takes the weights' NVFP4
  layout, with a caller's global scale per head in the place of the tensor
  scale (``nvfp4.quantize_rows``);
* a table maps position p of sequence b to slot p % page of page
  ``table[b][p // page]``;
* row cu[b] + i of a call stands at position pos[b] + i, and its attention sees
  the positions 0 .. pos[b] + i; query head h reads KV head h // (Hq / Hkv).
"""

import numpy as np

from . import nvfp4
from .formats import e2m1_value, e4m3_value


def kv_quantize(rows, gs):
    """Codes [T, Hkv, D/2] and E4M3 scales [T, Hkv, D/16] of rows [T, Hkv, D]; gs [Hkv]."""
    rows = np.asarray(rows, np.float32)
    t, hkv, d = rows.shape
    codes, scales = np.zeros((t, hkv, d // 2), np.uint8), np.zeros((t, hkv, d // 16), np.uint8)
    for h in range(hkv):
        codes[:, h], scales[:, h] = nvfp4.quantize_rows(rows[:, h], np.float32(gs[h]))
    return codes, scales


def kv_values(codes, scales, gs):
    """float64 values [..., Hkv, D] (exact) of codes [..., Hkv, D/2] and scales; gs [Hkv]."""
    v = e2m1_value(nvfp4.unpack_nibbles(codes)).astype(np.float64)
    return v * np.repeat(e4m3_value(scales).astype(np.float64), 16, axis=-1) * np.asarray(gs, np.float64)[:, None]


def gather(pool, table_row, count):
    """The first ``count`` positions' rows [count, Hkv, x] of a sequence from a page pool [pages, Hkv, page, x]."""
    page = pool.shape[2]
    p = np.arange(count)
    return pool[table_row[p // page], :, p % page]


def attention(q, k, v, pos, scale):
    """(out [n, Hq, D], lse [n, Hq], spread [n, Hq, D]) of one sequence's rows q [n, Hq, D] over values k, v [L, Hkv, D].

    ``spread`` is sum_j p_j |v_j| / sum_j p_j: what a relative error of the weights is multiplied by."""
    q = np.asarray(q, np.float64)
    n, hq, d = q.shape
    g = hq // k.shape[1]
    out, lse, spread = np.zeros((n, hq, d)), np.full((n, hq), -np.inf), np.zeros((n, hq, d))
    for i in range(n):
        seen = min(pos + i + 1, k.shape[0])
        if seen <= 0:
            continue
        for h in range(hq):
            s = (k[:seen, h // g] @ q[i, h]) * scale
            m = s.max()
            p = np.exp(s - m)
            lse[i, h] = m + np.log(p.sum())
            p /= p.sum()
            out[i, h] = p @ v[:seen, h // g]
            spread[i, h] = p @ np.abs(v[:seen, h // g])
    return out, lse, spread
