"""Pins of the NVFP4-cache oracle: the rows' rule against the weight quantizer, one visible token, equal keys, a
row that sees nothing, brute force in plain Python, and the order of pages."""

import math

import numpy as np

from oracle import kv_nvfp4 as kv
from oracle import nvfp4
from oracle.formats import bf16_rne


def _rows(g, *shape):
    return bf16_rne(g.standard_normal(shape).astype(np.float32))


def test_rows_follow_the_weight_rule():
    g = np.random.default_rng(0)
    x = _rows(g, 6, 1, 64)
    codes, scales, s_t = nvfp4.quantize(x[:, 0])
    got = kv.kv_quantize(x, [s_t])
    assert np.array_equal(got[0][:, 0], codes) and np.array_equal(got[1][:, 0], scales)
    assert np.array_equal(kv.kv_values(*got, [s_t])[:, 0], nvfp4.dequantize(codes, scales, s_t))


def test_closed_forms():
    g = np.random.default_rng(1)
    k, v = g.standard_normal((5, 2, 16)), g.standard_normal((5, 2, 16))
    q = g.standard_normal((3, 4, 16))
    out, lse, _ = kv.attention(q, k, v, -1, 0.25)  # the first row sees nothing, the second one token
    assert not out[0].any() and np.isneginf(lse[0]).all()
    assert np.allclose(out[1], np.repeat(v[0], 2, axis=0))
    assert np.allclose(lse[1], [(q[1, h] @ k[0, h // 2]) * 0.25 for h in range(4)])
    k[:] = k[0]
    out, _, spread = kv.attention(q[:1], k, v, 4, 0.25)
    assert np.allclose(out[0], np.repeat(v.mean(0), 2, axis=0))
    assert np.allclose(spread[0], np.repeat(np.abs(v).mean(0), 2, axis=0))


def test_brute_force():
    g = np.random.default_rng(2)
    k, v, q = g.standard_normal((4, 1, 8)), g.standard_normal((4, 1, 8)), g.standard_normal((2, 3, 8))
    out, lse, _ = kv.attention(q, k, v, 1, 0.5)
    for i in range(2):
        for h in range(3):
            w = [math.exp(0.5 * sum(q[i, h, d] * k[j, 0, d] for d in range(8))) for j in range(2 + i)]
            assert math.isclose(lse[i, h], math.log(sum(w)), rel_tol=1e-12)
            for d in range(8):
                assert math.isclose(out[i, h, d], sum(w[j] * v[j, 0, d] for j in range(2 + i)) / sum(w), rel_tol=1e-9)


def test_gather_walks_the_pages():
    pool = np.arange(3 * 2 * 4).reshape(3, 2, 4, 1)
    got = kv.gather(pool, np.array([2, 0]), 6)
    assert got[:, 0, 0].tolist() == [16, 17, 18, 19, 0, 1] and got[:, 1, 0].tolist() == [20, 21, 22, 23, 4, 5]
