"""Calls on a side stream beside work that is queued on the current one: each call's own buffers are its own."""

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def q():
    from quantized_rl_rollout_gb300 import build, qrr

    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    qrr.lib()
    return qrr


@pytest.mark.parametrize("handle", [False, True])
def test_nvfp4_attention_and_read(q, handle):
    """No synchronization between the calls; a prompt's attention takes long enough for the next to be queued behind it."""
    n, page = 2048, 64
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    cache = q.KvCacheNvfp4.empty(n // page, 2, page, 128, torch.arange(n // page, dtype=torch.int32, device=DEV)[None])
    kv = [torch.randn(n, 2, 128, device=DEV).to(torch.bfloat16) for _ in range(2)]
    x = [torch.randn(n, 16, 128, device=DEV).to(torch.bfloat16) for _ in range(2)]
    pos, cu = i32([0]), i32([0, n])
    q.kv_append_nvfp4(*kv, cache, pos, cu=cu)

    def call(i, stream=None):
        return q.attention_nvfp4(x[i], cache, pos, cu=cu, max_new=n, return_lse=True, stream=stream) + q.kv_read_nvfp4(
            cache, pos, cu=cu, rows=n, stream=stream)

    want = [call(0), call(1)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    given = side.cuda_stream if handle else side
    for _ in range(20):
        a = [call(0) for _ in range(3)]
        b = call(1, given)
        c = call(0)
        torch.cuda.synchronize()
        for got, i in [(g, 0) for g in a] + [(b, 1), (c, 0)]:
            assert all(torch.equal(y, z) for y, z in zip(got, want[i]))
        del a, b, c, got


def test_linear_and_fp8_attention(q):
    """The linear (prefill and decode) and the FP8 cache's attention."""
    from quantized_rl_rollout_gb300 import inputs

    codes, scales, ts = q.quantize_nvfp4(inputs.weight(2048, 2048, 1, device=DEV))
    xs = [[inputs.activations(m, 2048, 2 + i, device=DEV) for i in range(2)] for m in (4, 1024)]
    b, lmax = 64, 2048
    kq, ks = q.quantize_fp8_a1x128(inputs.activations(b * 2 * lmax, 128, 5, device=DEV))
    kv = (kq.view(b, 2, lmax, 128), ks.view(b, 2, lmax)) * 2
    qs = [inputs.activations(b * 8, 128, 6 + i, device=DEV).view(b, 8, 128) for i in range(2)]
    lens = torch.full((b,), lmax, dtype=torch.int32, device=DEV)

    def call(i, stream=None):
        return [q.linear_nvfp4_lora(x[i], codes, scales, ts, stream=stream) for x in xs] + [
            q.attention_decode_fp8(qs[i], *kv, lens, stream=stream)]

    want = [call(0), call(1)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(20):
        got = [(call(0), 0), (call(0), 0), (call(1, side), 1), (call(0), 0)]
        torch.cuda.synchronize()
        for g, i in got:
            assert all(torch.equal(y, z) for y, z in zip(g, want[i]))
        del got, g


@pytest.mark.parametrize("news", [[1, 3, 2], [4, 1, 1], [40, 300, 60]])
def test_arguments_made_in_the_call(q, news):
    """Every tensor of the calls a temporary: results are those with the tensors held, a sequence that sees nothing first."""
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    n = 400
    cache = q.KvCacheNvfp4.empty(3 * 25, 2, 16, 64, torch.arange(75, dtype=torch.int32, device=DEV).view(3, 25))
    kv = torch.randn(3 * n, 2, 64, device=DEV).to(torch.bfloat16)
    ends = [0, n, 2 * n, 3 * n]
    q.kv_append_nvfp4(kv.clone(), kv.clone(), cache, i32([0, 0, 0]), cu=i32(ends))
    whole = torch.cat(q.kv_read_nvfp4(cache, i32([0, 0, 0]), cu=i32(ends), rows=3 * n))
    t = sum(news)
    x, pos, cu = torch.randn(t, 8, 64, device=DEV).to(torch.bfloat16), i32([-news[0], n - news[1], 5]), i32([0, news[0], news[0] + news[1], t])
    held = i32(ends)
    assert torch.equal(whole, torch.cat(q.kv_read_nvfp4(cache, i32([0, 0, 0]), cu=held, rows=3 * n)))
    want = q.attention_nvfp4(x, cache, pos, cu=cu, max_new=max(news), return_lse=True)
    assert torch.isneginf(want[1][:news[0]]).all() and torch.isfinite(want[1][news[0]:]).all() and want[1][news[0]:].max() < 20
    for _ in range(30):
        got = q.attention_nvfp4(x.clone(), cache, pos.clone(), cu=cu.clone(), max_new=max(news), return_lse=True)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del got


@pytest.mark.parametrize("handle", [0, 1, 2])
def test_default_streams_by_their_handles(q, handle):
    """A call on the default stream, or a thread's own, while another stream is current."""
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    cache = q.KvCacheNvfp4.empty(8, 2, 64, 128, i32([list(range(8))]))
    kv = torch.randn(512, 2, 128, device=DEV).to(torch.bfloat16)
    x = torch.randn(512, 8, 128, device=DEV).to(torch.bfloat16)
    pos, cu = i32([0]), i32([0, 512])
    q.kv_append_nvfp4(kv, kv, cache, pos, cu=cu)
    want = q.attention_nvfp4(x, cache, pos, cu=cu, max_new=512, return_lse=True)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = [q.attention_nvfp4(x, cache, pos, cu=cu, max_new=512, return_lse=True, stream=s) for s in (handle, None, handle)]
        torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))
