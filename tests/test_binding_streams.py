"""Buffers that the binding makes for a call on another stream come from that stream's memory: a block of the current
stream's could still be in use there.  Host only: the stream, the allocator and the library are stand-ins."""

import contextlib
import weakref

import pytest
import torch

from quantized_rl_rollout_gb300 import qrr


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


class Tensor:
    """What the binding looks at, of a CUDA tensor with one head of 64 values a row."""

    is_cuda, device = True, "cuda:0"

    def __init__(self, shape, dtype, under=None):
        self.shape, self.dtype, self.under, self.recorded = torch.Size(shape), dtype, under, []

    def is_contiguous(self):
        return True

    def stride(self):
        return tuple(int(torch.Size(self.shape[i + 1:]).numel()) for i in range(len(self.shape)))

    def numel(self):
        return self.shape.numel()

    def dim(self):
        return len(self.shape)

    def data_ptr(self):
        return 0x10000

    def record_stream(self, stream):
        self.recorded.append(stream.cuda_stream)


CURRENT, SIDE = Stream(11), Stream(22)


@pytest.fixture
def made(monkeypatch):
    """Every tensor that is allocated, with the stream that was current then."""
    now, made = [CURRENT], []

    @contextlib.contextmanager
    def stream(s):
        now.append(s)
        yield
        now.pop()

    def empty(*shape, dtype=None, device=None):
        made.append(Tensor(shape[0] if len(shape) == 1 and not isinstance(shape[0], int) else shape, dtype, now[-1].cuda_stream))
        return made[-1]

    class Lib:
        def __getattr__(self, name):
            return lambda *a: 1000 if name.endswith("_bytes") else 0

    def external(handle):
        """As the real one: 0 makes a stream of its own, and the other two default handles cannot be used."""
        assert handle not in (1, 2), "invalid StreamId"
        return Stream(handle or 99)

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", external)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda *a: Stream(0))
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: now[-1])
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: now[-1].cuda_stream, raising=False)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(qrr, "lib", lambda: Lib())
    return made


@pytest.fixture
def cache(made):
    u8 = [Tensor((4, 1, 16, n), torch.uint8) for n in (32, 4, 32, 4)]
    return qrr.KvCacheNvfp4(*u8, Tensor((2, 2), torch.int32))


POS, X = Tensor((2,), torch.int32), Tensor((2, 1, 64), torch.bfloat16)


@pytest.mark.parametrize("stream", [SIDE, 22])
def test_nvfp4_cache_calls(cache, made, stream):
    got = qrr.attention_nvfp4(X, cache, POS, return_lse=True, stream=stream)
    assert len(made) == 3 and [t.under for t in made] == [22] * 3  # out, lse, workspace
    # what the caller gets may be used on their own stream as well
    assert [t.recorded for t in got] == [[11]] * 2
    del made[:]
    got = qrr.kv_read_nvfp4(cache, POS, stream=stream)
    assert [t.under for t in made] == [22] * 2 and [t.recorded for t in got] == [[11]] * 2


@pytest.mark.parametrize("stream", [0, 1, 2])
def test_default_streams_by_their_handles(cache, made, monkeypatch, stream):
    """The default stream (0, or by its name 1) and a thread's (2), which waits for it and is waited for by it, take the
    default stream's memory; where that is the current one, the call is as without a stream."""
    got = qrr.attention_nvfp4(X, cache, POS, return_lse=True, stream=stream)
    qrr.linear_nvfp4_lora(_bf16(2, 64), *W, stream=stream)
    assert len(made) == 5 and [t.under for t in made] == [0] * 5 and [t.recorded for t in got] == [[11]] * 2
    del made[:]
    monkeypatch.setattr(CURRENT, "cuda_stream", 0)
    qrr.attention_nvfp4(X, cache, POS, return_lse=True, stream=stream)
    qrr.linear_nvfp4_lora(_bf16(2, 64), *W, stream=stream)
    assert len(made) == 5 and all(t.under == 0 and not t.recorded for t in made)


@pytest.mark.parametrize("stream", [None, CURRENT, 11])
def test_nvfp4_cache_calls_on_the_current_stream(cache, made, stream):
    qrr.attention_nvfp4(X, cache, POS, return_lse=True, stream=stream)
    qrr.kv_read_nvfp4(cache, POS, stream=stream)
    assert len(made) == 5 and all(t.under == 11 and not t.recorded for t in made)


def _bf16(*shape):
    return Tensor(shape, torch.bfloat16)


W = [Tensor((128, 32), torch.uint8), Tensor((128, 4), torch.uint8), Tensor((1,), torch.float32)]
CALLS = {
    "quantize_nvfp4": (4, lambda s: qrr.quantize_nvfp4(_bf16(128, 64), stream=s)),
    "linear": (2, lambda s: qrr.linear_nvfp4_lora(_bf16(2, 64), *W, stream=s)),
    "linear_noalloc": (1, lambda s: qrr.linear_nvfp4_lora_noalloc(_bf16(2, 64), *W, stream=s)),
    "grouped": (2, lambda s: qrr.linear_nvfp4_lora_grouped([dict(x=_bf16(2, 64), codes=W[0], scales=W[1], tensor_scale=W[2])], stream=s)),
    "fp8 weight": (2, lambda s: qrr.quantize_fp8_w128x128(_bf16(128, 128), stream=s)),
    "fp8 activation": (2, lambda s: qrr.quantize_fp8_a1x128(_bf16(2, 128), stream=s)),
    "fp8 gemm": (1, lambda s: qrr.gemm_fp8_blockwise(Tensor((2, 128), torch.uint8), Tensor((2, 1), torch.float32), Tensor((128, 128), torch.uint8),
                                                    Tensor((1, 1), torch.float32), stream=s)),
    "requantize": (1, lambda s: qrr.requantize_weights([_bf16(128, 64)], [W], stream=s)),
    "requantize aqn": (1, lambda s: qrr.requantize_weights_aqn([_bf16(128, 64)], [W], 0.1, 1, 2, stream=s)),
    "aqn probe": (1, lambda s: qrr.aqn_noise_probe(8, 1, 0, 0, stream=s)),
    "round probe": (1, lambda s: qrr.round_probe(Tensor((8,), torch.float32), 0, stream=s)),
    "logprobs": (2, lambda s: qrr.token_logprobs_is(_bf16(2, 64), Tensor((2,), torch.int32), Tensor((2,), torch.float32), stream=s)),
    "lora backward": (4, lambda s: qrr.lora_backward_nvfp4(_bf16(2, 128), _bf16(2, 64), *W, _bf16(8, 64), _bf16(128, 8), stream=s)),
    "fp8 attention": (2, lambda s: qrr.attention_decode_fp8(_bf16(2, 4, 128), Tensor((2, 4, 16, 128), torch.uint8), W[2], W[0], W[2],
                                                            Tensor((2,), torch.int32), stream=s)),
}


@pytest.mark.parametrize("name", CALLS)
def test_other_calls(made, monkeypatch, name):
    monkeypatch.setattr(torch, "empty_like", lambda t: torch.empty(*t.shape, dtype=t.dtype))
    count, call = CALLS[name]
    for stream, under in ((SIDE, 22), (22, 22), (None, 11), (CURRENT, 11)):
        del made[:]
        call(stream)
        assert [t.under for t in made] == [under] * count


NVFP4_CALLS = {
    "qrr_kv_append_nvfp4": lambda cache, make: qrr.kv_append_nvfp4(make(X), make(X), cache, make(POS), cu=make(CU), dev_status=make(ST)),
    "qrr_kv_read_nvfp4": lambda cache, make: qrr.kv_read_nvfp4(cache, make(POS), cu=make(CU), rows=2, dev_status=make(ST)),
    "qrr_attention_nvfp4": lambda cache, make: qrr.attention_nvfp4(make(X), cache, make(POS), cu=make(CU), max_new=2, return_lse=True,
                                                                   dev_status=make(ST)),
}
CU, ST = Tensor((3,), torch.int32), Tensor((1,), torch.int32)


@pytest.mark.parametrize("name", NVFP4_CALLS)
def test_arguments_live_until_the_launch(cache, made, monkeypatch, name):
    """Tensors that only the call holds (made in its argument list) keep their memory until it has launched: the call's
    own buffers would be put there otherwise, and written while the offsets are read."""
    refs, seen = [], []

    def make(like):
        t = Tensor(like.shape, like.dtype)
        refs.append(weakref.ref(t))
        return t

    def alive(*a, **k):
        seen.append([r() is not None for r in refs])

    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: (alive(), empty(*a, **k))[1])

    class Lib:
        def __getattr__(self, entry):
            return lambda *a: 1000 if entry.endswith("_bytes") else (alive() if entry == name else None, 0)[1]

    monkeypatch.setattr(qrr, "lib", lambda: Lib())
    NVFP4_CALLS[name](cache, make)
    assert seen and all(all(s) for s in seen), seen
