"""Host-only checks of the NVFP4-cache entry points: bad descriptions and arguments are refused before anything is
launched.  No call here reaches a GPU."""

import ctypes

import pytest

FAKE = 0x10000  # a 16-byte-aligned non-null address that is never dereferenced


@pytest.fixture(scope="module")
def qrr():
    from quantized_rl_rollout_gb300 import build, qrr

    build.build()
    qrr.lib()
    return qrr


def _desc(qrr, **change):
    d = dict(k_codes=FAKE, k_scales=FAKE, v_codes=FAKE, v_scales=FAKE, k_gs=None, v_gs=None, page_table=FAKE, num_pages=4,
             Hkv=2, page=16, D=128, B=3, max_pages=2)
    d.update(change)
    return qrr.KvNvfp4Desc(*[d[f] for f, _ in qrr.KvNvfp4Desc._fields_])


def _calls(qrr, desc, T=3, cu=None, pos=FAKE, k=FAKE, ld=256, q=FAKE, ld_q=1024, hq=8, max_new=1, scale=0.1, out=FAKE, ws=FAKE,
           ws_bytes=1 << 40):
    lib, c = qrr.lib(), ctypes.addressof(desc)
    return (lib.qrr_kv_append_nvfp4(c, k, FAKE, T, ld, 256, cu, pos, None, None),
            lib.qrr_kv_read_nvfp4(c, T, cu, pos, k, FAKE, None, None),
            lib.qrr_attention_nvfp4(c, q, T, ld_q, hq, cu, pos, max_new, scale, out, None, ws, ws_bytes, None, None))


@pytest.mark.parametrize("change,status", [
    (dict(D=96), 2), (dict(D=256), 2), (dict(page=8), 2), (dict(page=48), 2), (dict(page=0), 1), (dict(Hkv=-1), 1),
    (dict(B=-1), 1), (dict(num_pages=-4), 1), (dict(max_pages=1 << 27), 2), (dict(page_table=None), 1),
    (dict(k_codes=None), 1), (dict(v_scales=None), 1), (dict(k_codes=FAKE + 8), 3), (dict(v_scales=FAKE + 8), 3),
    (dict(k_gs=FAKE + 2), 3), (dict(page_table=FAKE + 1), 3)])
def test_cache_descriptions(qrr, change, status):
    assert _calls(qrr, _desc(qrr, **change)) == (status,) * 3


def test_rows(qrr):
    d = _desc(qrr)
    assert _calls(qrr, d, T=4) == (1,) * 3  # one row a sequence without cu
    assert _calls(qrr, d, T=-1) == (1,) * 3
    assert _calls(qrr, d, pos=None) == (1,) * 3
    assert _calls(qrr, d, T=(1 << 30) + 1, cu=FAKE) == (2,) * 3
    assert _calls(qrr, d, cu=FAKE + 2) == (3,) * 3
    lib = qrr.lib()
    assert lib.qrr_kv_append_nvfp4(None, FAKE, FAKE, 1, 256, 256, None, FAKE, None, None) == 1
    assert lib.qrr_kv_read_nvfp4(None, 1, None, FAKE, FAKE, FAKE, None, None) == 1


def test_arguments(qrr):
    d = _desc(qrr)
    assert _calls(qrr, d, k=None)[:2] == (1, 1)
    assert _calls(qrr, d, k=FAKE + 8)[:2] == (3, 3)
    assert _calls(qrr, d, ld=248)[0] == 1 and _calls(qrr, d, ld=260)[0] == 3
    for change, status in [(dict(hq=7), 2), (dict(hq=-8), 1), (dict(max_new=2), 1), (dict(max_new=-1), 1), (dict(scale=0.0), 1),
                           (dict(scale=-1.0), 1), (dict(scale=float("inf")), 1), (dict(scale=float("nan")), 1),
                           (dict(q=None), 1), (dict(out=None), 1), (dict(q=FAKE + 8), 3), (dict(out=FAKE + 2), 3),
                           (dict(ld_q=1000), 1), (dict(ld_q=1028), 3), (dict(ws=None), 4), (dict(ws_bytes=64), 4),
                           (dict(ws=FAKE + 8), 3)]:
        assert _calls(qrr, d, **change)[2] == status, change
    assert qrr.lib().qrr_attention_nvfp4_workspace_bytes(None, 1, 8, 1) == 0
    assert qrr.lib().qrr_attention_nvfp4_workspace_bytes(ctypes.addressof(d), -1, 8, 1) == 0


def test_injected_fault(qrr, monkeypatch):
    monkeypatch.setenv("QRR_INJECT_FAULT", "cuda")
    assert _calls(qrr, _desc(qrr)) == (5,) * 3
