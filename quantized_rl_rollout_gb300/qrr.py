"""Thin ctypes binding of the C ABI in ``include/qrr.h``.

Each Python function has the name of the C entry point without its ``qrr_``
prefix and only marshals arguments: it checks dtypes and contiguity, allocates
outputs and workspace with torch when the caller passes none, and hands raw
device pointers and the current CUDA stream to the library.  Every step of the
computation runs in the library's kernels; there is no other code path, and a
missing library is an error.
"""

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_qrr.so")

SCALE_FP32 = 0
SCALE_POW2 = 1
FORMAT_NVFP4 = 0
FORMAT_FP8_W128 = 1
DEV_NONFINITE = 0x1
DEV_TIMEOUT = 0x2
DEV_SCALE_RANGE = 0x4
DEV_BAD_INDEX = 0x8
DTYPE_BF16 = 0
DTYPE_FP32 = 1
OP_QUANTIZE_NVFP4 = 0
OP_LINEAR_NVFP4_LORA = 1
OP_REQUANTIZE_WEIGHTS = 2
OP_QUANTIZE_FP8 = 3
OP_GEMM_FP8 = 4
OP_LORA_BACKWARD = 5

_c_i64 = ctypes.c_int64
_c_i32 = ctypes.c_int32
_c_p = ctypes.c_void_p
_c_sz = ctypes.c_size_t


class WeightDesc(ctypes.Structure):
    """Mirror of ``qrr_weight_desc``."""

    _fields_ = [("W", _c_p), ("N", _c_i64), ("K", _c_i64), ("codes", _c_p), ("scales", _c_p),
                ("tensor_scale", _c_p)]


class LinearDesc(ctypes.Structure):
    """Mirror of ``qrr_linear_desc``."""

    _fields_ = [("x", _c_p), ("N", _c_i64), ("K", _c_i64), ("codes", _c_p), ("scales", _c_p),
                ("tensor_scale", _c_p), ("lora_A", _c_p), ("lora_B", _c_p), ("r", _c_i32), ("alpha", ctypes.c_float),
                ("y", _c_p)]


class KvNvfp4Desc(ctypes.Structure):
    """Mirror of ``qrr_kv_nvfp4``."""

    _fields_ = [("k_codes", _c_p), ("k_scales", _c_p), ("v_codes", _c_p), ("v_scales", _c_p), ("k_gs", _c_p),
                ("v_gs", _c_p), ("page_table", _c_p), ("num_pages", _c_i32), ("Hkv", _c_i32), ("page", _c_i32),
                ("D", _c_i32), ("B", _c_i32), ("max_pages", _c_i32)]


# symbol -> (restype, argtypes)
SIGNATURES = {
    "qrr_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "qrr_abi_version": (ctypes.c_int, []),
    "qrr_quantize_nvfp4_workspace_bytes": (_c_sz, []),
    "qrr_quantize_nvfp4": (ctypes.c_int, [_c_p, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_p, _c_sz, _c_p, _c_p]),
    "qrr_linear_nvfp4_lora_workspace_bytes": (_c_sz, [_c_i64, _c_i64, _c_i64, _c_i32]),
    "qrr_linear_nvfp4_lora": (ctypes.c_int, [_c_p, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_i64, _c_p, _c_p, _c_i32,
                                             ctypes.c_float, _c_p, _c_p, _c_sz, _c_p, _c_p]),
    "qrr_noalloc_scratch_bytes": (_c_sz, []),
    "qrr_linear_nvfp4_lora_noalloc": (ctypes.c_int, [_c_p, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_i64, _c_p, _c_p,
                                                     _c_i32, ctypes.c_float, _c_p, _c_p, _c_p]),
    "qrr_linear_nvfp4_lora_grouped_workspace_bytes": (_c_sz, [ctypes.POINTER(LinearDesc), _c_i32, _c_i64]),
    "qrr_linear_nvfp4_lora_grouped": (ctypes.c_int, [ctypes.POINTER(LinearDesc), _c_i32, _c_i64, _c_p, _c_sz, _c_p,
                                                     _c_p]),
    "qrr_quantize_fp8_w128x128": (ctypes.c_int, [_c_p, _c_i64, _c_i64, _c_p, _c_p, _c_i32, _c_p, _c_p]),
    "qrr_quantize_fp8_a1x128": (ctypes.c_int, [_c_p, _c_i64, _c_i64, _c_p, _c_p, _c_i32, _c_p, _c_p]),
    "qrr_gemm_fp8_blockwise": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_p, _c_i64, _c_i64, _c_i64, _c_p, _c_i32, _c_p,
                                              _c_p]),
    "qrr_requantize_workspace_bytes": (_c_sz, [_c_i32]),
    "qrr_requantize_weights": (ctypes.c_int, [ctypes.POINTER(WeightDesc), _c_i32, _c_i32, _c_i32, _c_p, _c_sz, _c_p,
                                              _c_p]),
    "qrr_round_probe": (ctypes.c_int, [_c_p, _c_i64, _c_i32, _c_p, _c_p]),
    "qrr_get_last_device_status": (ctypes.c_int, [_c_p, _c_p, _c_p]),
    "qrr_kv_append_fp8": (ctypes.c_int, [_c_p, _c_p, _c_i32, _c_i32, _c_p, _c_p, _c_p, _c_p, _c_p, _c_i32, _c_i32, _c_p,
                                         _c_p]),
    "qrr_attention_decode_fp8_workspace_bytes": (_c_sz, [_c_i32, _c_i32, _c_i32]),
    "qrr_attention_decode_fp8": (ctypes.c_int, [_c_p, _c_i32, _c_i32, _c_i32, _c_p, _c_p, _c_p, _c_p, _c_p, _c_i32, _c_p,
                                                _c_p, _c_sz, _c_p, _c_p]),
    "qrr_kv_append_nvfp4": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_p]),
    "qrr_kv_read_nvfp4": (ctypes.c_int, [_c_p, _c_i64, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p]),
    "qrr_attention_nvfp4_workspace_bytes": (_c_sz, [_c_p, _c_i64, _c_i32, _c_i32]),
    "qrr_attention_nvfp4": (ctypes.c_int, [_c_p, _c_p, _c_i64, _c_i64, _c_i32, _c_p, _c_p, _c_i32, ctypes.c_float, _c_p,
                                           _c_p, _c_p, _c_sz, _c_p, _c_p]),
    "qrr_lora_backward_workspace_bytes": (_c_sz, [_c_i64, _c_i64, _c_i64, _c_i32]),
    "qrr_lora_backward_nvfp4": (ctypes.c_int, [_c_p, _c_i64, _c_i64, _c_p, _c_i64, _c_p, _c_p, _c_p, _c_p, _c_p, _c_i32,
                                               ctypes.c_float, _c_p, _c_p, _c_p, _c_p, _c_sz, _c_p, _c_p]),
    "qrr_requantize_weights_aqn": (ctypes.c_int, [ctypes.POINTER(WeightDesc), _c_i32, _c_i32, _c_i32, ctypes.c_float,
                                                  ctypes.c_uint64, _c_i32, _c_p, _c_sz, _c_p, _c_p]),
    "qrr_aqn_sigma": (ctypes.c_float, [_c_i32, _c_i32, ctypes.c_double, ctypes.c_double]),
    "qrr_aqn_noise_probe": (ctypes.c_int, [_c_p, _c_i64, _c_i64, ctypes.c_uint64, _c_i32, _c_i32, _c_p]),
    "qrr_token_logprobs_is": (ctypes.c_int, [_c_p, _c_i64, _c_i64, _c_p, _c_p, ctypes.c_float, _c_p, _c_p, _c_p,
                                             _c_p]),
    "qrr_distill_topk": (ctypes.c_int, [_c_p, _c_i32, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_i32, _c_p, ctypes.c_double, _c_p,
                                        _c_p, _c_p, _c_p]),
    "qrr_distill_topk_backward": (ctypes.c_int, [_c_p, _c_i32, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_i32, _c_p,
                                                 ctypes.c_double, _c_p, _c_p, _c_p, _c_i64, _c_p, _c_p]),
    "qrr_distill_topk_grad": (ctypes.c_int, [_c_p, _c_i32, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_i32, _c_p, ctypes.c_double,
                                             _c_p, _c_p, _c_p, _c_i64, _c_p, _c_p]),
    "qrr_token_logprobs_is_grad": (ctypes.c_int, [_c_p, _c_i32, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_p, ctypes.c_float,
                                                  _c_p, _c_p, _c_p, _c_i64, _c_p, _c_p]),
    "qrr_verify_drafts_workspace_bytes": (_c_sz, [_c_i64, _c_i32, _c_i64, _c_i32]),
    "qrr_verify_drafts": (ctypes.c_int, [_c_p, _c_i64, _c_p, _c_i64, _c_i32, _c_i64, _c_i32, _c_i64, _c_p, _c_p, _c_p, _c_p,
                                         _c_i64, ctypes.c_double, _c_p, _c_p, _c_p, _c_p, _c_sz, _c_p, _c_p]),
    "qrr_workspace_bytes": (_c_sz, [_c_i32, _c_i64, _c_i64, _c_i64, _c_i32]),
    "qrr_wait_probe": (ctypes.c_int, [_c_i64, _c_i32, _c_p, _c_p, _c_p]),
    "qrr_stream_probe": (ctypes.c_int, [_c_p, _c_i64, _c_i64, _c_p, _c_p]),
    "qrr_plan_decode_units": (_c_i64, [_c_i64, _c_i32, _c_p, _c_p, _c_p, _c_i32, _c_p, _c_i32, _c_p, _c_p]),
}

_lib = None


class QrrError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_name(status)}")


def lib() -> ctypes.CDLL:
    """The loaded library (loaded on first use); raises if it is not built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"the CUDA library {LIB_PATH} is not built; run __graft_entry__.build() "
                               "(there is no CPU fallback)")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def status_name(status: int) -> str:
    return lib().qrr_status_string(int(status)).decode()


def _check(status: int, what: str):
    if status != 0:
        raise QrrError(status, what)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:  # torch.cuda.current_stream().cuda_stream, without making the Python object (2.9 us)
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _need(t, dtype, name):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _on_stream(shape, dtype, device, stream, returned=True):
    """A new tensor for a call on ``stream`` (None: the current one), from that stream's memory: a block of the current
    stream's may still be in use by work queued there.  ``returned``: the caller may go on with it on the current stream."""
    handle = None if stream is None else _stream(stream)
    if handle in (0, 1, 2):  # the default stream, and a thread's own, which is ordered with it both ways
        handle = 0
    if handle is None or handle == _stream(None):
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if returned:
        t.record_stream(torch.cuda.current_stream())
    return t


def _workspace(nbytes: int, device, stream):
    return _on_stream((max(int(nbytes), 256),), torch.uint8, device, stream, returned=False)


# ---------------------------------------------------------------------------

def quantize_nvfp4(W, codes=None, scales=None, tensor_scale=None, workspace=None, dev_status=None, stream=None):
    """NVFP4 quantization of a bf16 [N, K] weight -> (codes, scales, tensor_scale)."""
    _need(W, torch.bfloat16, "W")
    n, k = W.shape
    dev = W.device
    codes = _on_stream((n, k // 2), torch.uint8, dev, stream) if codes is None else codes
    scales = _on_stream((n, k // 16), torch.uint8, dev, stream) if scales is None else scales
    tensor_scale = _on_stream((1,), torch.float32, dev, stream) if tensor_scale is None else tensor_scale
    ws_bytes = lib().qrr_quantize_nvfp4_workspace_bytes()
    workspace = _workspace(ws_bytes, dev, stream) if workspace is None else workspace
    _check(lib().qrr_quantize_nvfp4(_ptr(W), n, k, _ptr(codes), _ptr(scales), _ptr(tensor_scale), _ptr(workspace),
                                    workspace.numel(), _ptr(dev_status), _stream(stream)), "qrr_quantize_nvfp4")
    return codes, scales, tensor_scale


def linear_nvfp4_lora_workspace_bytes(M, N, K, r) -> int:
    return int(lib().qrr_linear_nvfp4_lora_workspace_bytes(M, N, K, r))


def linear_nvfp4_lora(x, codes, scales, tensor_scale, lora_A=None, lora_B=None, alpha=0.0, y=None, workspace=None,
                      dev_status=None, stream=None):
    """y = x . dequant(W)^T + (alpha/r) (x . A^T) . B^T in bf16."""
    _need(x, torch.bfloat16, "x")
    m, k = x.shape
    n = codes.shape[0]
    r = 0 if lora_A is None or lora_B is None else int(lora_A.shape[0])
    y = _on_stream((m, n), torch.bfloat16, x.device, stream) if y is None else y
    if workspace is None:
        workspace = _workspace(linear_nvfp4_lora_workspace_bytes(m, n, k, r), x.device, stream)
    _check(lib().qrr_linear_nvfp4_lora(_ptr(x), m, k, _ptr(codes), _ptr(scales), _ptr(tensor_scale), n,
                                       _ptr(lora_A), _ptr(lora_B), r, float(alpha), _ptr(y), _ptr(workspace),
                                       workspace.numel(), _ptr(dev_status), _stream(stream)),
           "qrr_linear_nvfp4_lora")
    return y


def linear_nvfp4_lora_noalloc(x, codes, scales, tensor_scale, lora_A=None, lora_B=None, alpha=0.0, y=None,
                              dev_status=None, stream=None):
    """Same as ``linear_nvfp4_lora`` but on the library's built-in scratch (no workspace)."""
    _need(x, torch.bfloat16, "x")
    m, k = x.shape
    n = codes.shape[0]
    r = 0 if lora_A is None or lora_B is None else int(lora_A.shape[0])
    y = _on_stream((m, n), torch.bfloat16, x.device, stream) if y is None else y
    _check(lib().qrr_linear_nvfp4_lora_noalloc(_ptr(x), m, k, _ptr(codes), _ptr(scales), _ptr(tensor_scale), n,
                                               _ptr(lora_A), _ptr(lora_B), r, float(alpha), _ptr(y),
                                               _ptr(dev_status), _stream(stream)), "qrr_linear_nvfp4_lora_noalloc")
    return y


def _linear_descs(layers, stream=None):
    descs = (LinearDesc * len(layers))()
    m = None
    for i, d in enumerate(layers):
        x, codes, scales, ts = d["x"], d["codes"], d["scales"], d["tensor_scale"]
        _need(x, torch.bfloat16, f"layers[{i}].x")
        a, b = d.get("lora_A"), d.get("lora_B")
        r = 0 if a is None or b is None else int(a.shape[0])
        if m is None:
            m = x.shape[0]
        elif x.shape[0] != m:
            raise ValueError("every layer of a grouped call has the same token count")
        if d.get("y") is None:
            d["y"] = _on_stream((m, codes.shape[0]), torch.bfloat16, x.device, stream)
        descs[i] = LinearDesc(_ptr(x), codes.shape[0], x.shape[1], _ptr(codes), _ptr(scales), _ptr(ts), _ptr(a),
                              _ptr(b), r, float(d.get("alpha", 0.0)), _ptr(d["y"]))
    return descs, (m or 0)


def linear_nvfp4_lora_grouped_workspace_bytes(layers) -> int:
    descs, m = _linear_descs(layers)
    return int(lib().qrr_linear_nvfp4_lora_grouped_workspace_bytes(descs, len(layers), m))


def linear_nvfp4_lora_grouped(layers, workspace=None, dev_status=None, stream=None):
    """Run up to 8 layers sharing the token count in one grouped call.

    ``layers`` is a list of dicts with keys x, codes, scales, tensor_scale and
    optionally lora_A, lora_B, alpha, y (allocated when absent).  Returns the
    list of outputs.
    """
    descs, m = _linear_descs(layers, stream)
    if workspace is None:
        nbytes = lib().qrr_linear_nvfp4_lora_grouped_workspace_bytes(descs, len(layers), m)
        workspace = _workspace(nbytes, layers[0]["x"].device, stream)
    _check(lib().qrr_linear_nvfp4_lora_grouped(descs, len(layers), m, _ptr(workspace), workspace.numel(),
                                               _ptr(dev_status), _stream(stream)), "qrr_linear_nvfp4_lora_grouped")
    return [d["y"] for d in layers]


class GroupedLinear:
    """A grouped linear call prepared once, for the decode loop's case of
    fixed buffers: the layers' tensors (x, weights, adapters, y) and the
    workspace are bound at construction, checked once, and ``run()`` only
    launches.  Refill x in place between runs; y is rewritten by each run.
    (Buffers made here belong to the stream that is current now: a ``run`` on
    another stream has to be ordered behind its work.)
    The numbers are those of ``linear_nvfp4_lora_grouped`` on the same
    tensors, bit for bit (it is the same C call)."""

    def __init__(self, layers, workspace=None):
        self.layers = layers
        self.descs, self.m = _linear_descs(layers)
        nbytes = int(lib().qrr_linear_nvfp4_lora_grouped_workspace_bytes(self.descs, len(layers), self.m))
        if workspace is None:
            workspace = _workspace(nbytes, layers[0]["x"].device, None)
        elif workspace.numel() < nbytes:
            raise ValueError(f"workspace of {workspace.numel()} bytes, the call needs {nbytes}")
        self.workspace = workspace
        self.outputs = [d["y"] for d in layers]
        self._args = (self.descs, len(layers), self.m, _ptr(workspace), workspace.numel())
        self._fn = lib().qrr_linear_nvfp4_lora_grouped

    def run(self, dev_status=None, stream=None):
        _check(self._fn(*self._args, _ptr(dev_status), _stream(stream)), "qrr_linear_nvfp4_lora_grouped")
        return self.outputs


def quantize_fp8_w128x128(W, mode=SCALE_FP32, q=None, scales=None, dev_status=None, stream=None):
    _need(W, torch.bfloat16, "W")
    n, k = W.shape
    q = _on_stream((n, k), torch.uint8, W.device, stream) if q is None else q
    scales = _on_stream(((n + 127) // 128, k // 128), torch.float32, W.device, stream) if scales is None else scales
    _check(lib().qrr_quantize_fp8_w128x128(_ptr(W), n, k, _ptr(q), _ptr(scales), int(mode), _ptr(dev_status),
                                           _stream(stream)), "qrr_quantize_fp8_w128x128")
    return q, scales


def quantize_fp8_a1x128(x, mode=SCALE_FP32, q=None, scales=None, dev_status=None, stream=None):
    _need(x, torch.bfloat16, "x")
    m, k = x.shape
    q = _on_stream((m, k), torch.uint8, x.device, stream) if q is None else q
    scales = _on_stream((m, k // 128), torch.float32, x.device, stream) if scales is None else scales
    _check(lib().qrr_quantize_fp8_a1x128(_ptr(x), m, k, _ptr(q), _ptr(scales), int(mode), _ptr(dev_status),
                                         _stream(stream)), "qrr_quantize_fp8_a1x128")
    return q, scales


def gemm_fp8_blockwise(qa, sa, qw, sw, mode=SCALE_FP32, y=None, dev_status=None, stream=None):
    m, k = qa.shape
    n = qw.shape[0]
    y = _on_stream((m, n), torch.bfloat16, qa.device, stream) if y is None else y
    _check(lib().qrr_gemm_fp8_blockwise(_ptr(qa), _ptr(sa), _ptr(qw), _ptr(sw), m, n, k, _ptr(y), int(mode),
                                        _ptr(dev_status), _stream(stream)), "qrr_gemm_fp8_blockwise")
    return y


def _weight_descs(weights, outputs, fmt):
    count = len(weights)
    descs = (WeightDesc * max(count, 1))()
    for i, (w, out) in enumerate(zip(weights, outputs)):
        _need(w, torch.bfloat16, f"weights[{i}]")
        ts = out[2] if fmt == FORMAT_NVFP4 else None
        descs[i] = WeightDesc(_ptr(w), w.shape[0], w.shape[1], _ptr(out[0]), _ptr(out[1]), _ptr(ts))
    return descs, count


def requantize_weights(weights, outputs, fmt=FORMAT_NVFP4, mode=SCALE_FP32, workspace=None, dev_status=None,
                       stream=None):
    """Re-quantize every bf16 weight of ``weights`` into ``outputs``.

    ``outputs[i]`` is ``(codes, scales, tensor_scale)`` for NVFP4 or
    ``(q, scales)`` for FP8 128x128.
    """
    descs, count = _weight_descs(weights, outputs, fmt)
    dev = weights[0].device if count else torch.device("cuda")
    if workspace is None:
        workspace = _workspace(lib().qrr_requantize_workspace_bytes(count), dev, stream)
    _check(lib().qrr_requantize_weights(descs, count, int(fmt), int(mode), _ptr(workspace), workspace.numel(),
                                        _ptr(dev_status), _stream(stream)), "qrr_requantize_weights")
    return outputs


def requantize_weights_aqn(weights, outputs, sigma, seed, step, fmt=FORMAT_NVFP4, mode=SCALE_FP32, workspace=None,
                           dev_status=None, stream=None):
    """``requantize_weights`` of the noisy masters bf16(W + sigma z) (see ``qrr_requantize_weights_aqn``)."""
    descs, count = _weight_descs(weights, outputs, fmt)
    dev = weights[0].device if count else torch.device("cuda")
    if workspace is None:
        workspace = _workspace(lib().qrr_requantize_workspace_bytes(count), dev, stream)
    _check(lib().qrr_requantize_weights_aqn(descs, count, int(fmt), int(mode), float(sigma), int(seed), int(step),
                                            _ptr(workspace), workspace.numel(), _ptr(dev_status), _stream(stream)),
           "qrr_requantize_weights_aqn")
    return outputs


def aqn_sigma(step, steps, sigma_start, sigma_end) -> float:
    return float(lib().qrr_aqn_sigma(int(step), int(steps), float(sigma_start), float(sigma_end)))


def aqn_noise_probe(n, seed, tensor, step, start=0, out=None, stream=None):
    out = _on_stream((n,), torch.float32, "cuda", stream) if out is None else out
    _check(lib().qrr_aqn_noise_probe(_ptr(out), int(n), int(start), int(seed), int(tensor), int(step),
                                     _stream(stream)), "qrr_aqn_noise_probe")
    return out


def round_probe(values, fmt, out=None, stream=None):
    _need(values, torch.float32, "values")
    out = _on_stream((values.numel(),), torch.uint8, values.device, stream) if out is None else out
    _check(lib().qrr_round_probe(_ptr(values), values.numel(), int(fmt), _ptr(out), _stream(stream)),
           "qrr_round_probe")
    return out


def get_last_device_status(dev_status, stream=None) -> int:
    """Host copy of the device status word once the stream's earlier work is done."""
    _need(dev_status, torch.int32, "dev_status")
    out = ctypes.c_int32(0)
    _check(lib().qrr_get_last_device_status(ctypes.addressof(out), _ptr(dev_status), _stream(stream)),
           "qrr_get_last_device_status")
    return int(out.value)


def workspace_bytes(op, M=0, N=0, K=0, r=0) -> int:
    return int(lib().qrr_workspace_bytes(int(op), int(M), int(N), int(K), int(r)))


def plan_decode_units(M, shapes, grid, max_units=4096):
    """The decode launch's unit table for layers ``shapes`` = [(N, K, r), ...]
    at M tokens on ``grid`` CTAs (host only; see ``qrr_plan_decode_units``).

    Returns ``(units, offsets)``: a list of decoded units (dicts with layer,
    m_tile, n_tile, pieces, c0, nk, piece, lora) and the per-CTA offsets."""
    n = len(shapes)
    Ns = (ctypes.c_int64 * n)(*[int(s[0]) for s in shapes])
    Ks = (ctypes.c_int64 * n)(*[int(s[1]) for s in shapes])
    rs = (ctypes.c_int32 * n)(*[int(s[2]) for s in shapes])
    units = (ctypes.c_uint32 * (2 * max_units))()
    offsets = (ctypes.c_uint16 * (int(grid) + 1))()
    used = ctypes.c_int32(0)
    got = lib().qrr_plan_decode_units(int(M), n, ctypes.addressof(Ns), ctypes.addressof(Ks), ctypes.addressof(rs),
                                      int(grid), ctypes.addressof(units), int(max_units), ctypes.addressof(offsets),
                                      ctypes.addressof(used))
    if got < 0:
        raise QrrError(int(-got), "qrr_plan_decode_units")
    out = []
    for i in range(got):
        w0, w1 = units[2 * i], units[2 * i + 1]
        out.append(dict(layer=w0 & 0xF, m_tile=(w0 >> 4) & 0xF, n_tile=(w0 >> 8) & 0xFFFF, pieces=w0 >> 24,
                        c0=w1 & 0xFFF, nk=(w1 >> 12) & 0x7FF, piece=(w1 >> 23) & 0xFF, lora=w1 >> 31))
    return out, [int(offsets[b]) for b in range(used.value + 1)]


def wait_probe(limit_cycles, arrive, dev_status, cycles=None, stream=None):
    """Run the bounded-wait probe (see ``qrr_wait_probe``)."""
    _need(dev_status, torch.int32, "dev_status")
    if cycles is not None:
        _need(cycles, torch.int64, "cycles")
    _check(lib().qrr_wait_probe(int(limit_cycles), int(arrive), _ptr(dev_status), _ptr(cycles), _stream(stream)),
           "qrr_wait_probe")


def stream_probe(data, dev_status=None, stream=None):
    """Stream a uint8 [rows, row_bytes] matrix through the TMA ring of the
    decode kernels with no arithmetic (see ``qrr_stream_probe``)."""
    _need(data, torch.uint8, "data")
    if data.dim() != 2:
        raise ValueError("stream_probe: data must be a 2-D uint8 tensor")
    if dev_status is not None:
        _need(dev_status, torch.int32, "dev_status")
    _check(lib().qrr_stream_probe(_ptr(data), data.shape[0], data.shape[1], _ptr(dev_status), _stream(stream)),
           "qrr_stream_probe")


def token_logprobs_is(logits, tokens, rollout_logp=None, cap=0.0, logp=None, w=None, dev_status=None, stream=None):
    """Token log-probabilities (and, given the rollout's, importance weights).

    Returns ``logp`` or ``(logp, w)`` when ``rollout_logp`` is given."""
    _need(logits, torch.bfloat16, "logits")
    _need(tokens, torch.int32, "tokens")
    t, v = logits.shape
    logp = _on_stream((t,), torch.float32, logits.device, stream) if logp is None else logp
    if rollout_logp is not None:
        _need(rollout_logp, torch.float32, "rollout_logp")
        w = _on_stream((t,), torch.float32, logits.device, stream) if w is None else w
    _check(lib().qrr_token_logprobs_is(_ptr(logits), t, v, _ptr(tokens), _ptr(rollout_logp), float(cap), _ptr(logp),
                                       _ptr(w) if rollout_logp is not None else None, _ptr(dev_status),
                                       _stream(stream)), "qrr_token_logprobs_is")
    return logp if rollout_logp is None else (logp, w)


_DTYPES = {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_FP32}


def _logit_rows(x, rows, v, name, dtype=None):
    """(dtype number, row stride) of logits [rows, v] whose rows are contiguous (a slice of wider rows will do)."""
    if x.dtype not in _DTYPES or not x.is_cuda or (dtype is not None and x.dtype != dtype):
        raise TypeError(f"{name} must be a CUDA {'bfloat16 or float32' if dtype is None else dtype} tensor, got {x.dtype}")
    if x.shape != (rows, v):
        raise ValueError(f"{name} must be {[rows, v]}, got {list(x.shape)}")
    s = x.stride()
    if (v > 1 and s[1] != 1) or (rows > 1 and s[0] < v):
        raise ValueError(f"{name}: rows must be contiguous and must not overlap")
    return _DTYPES[x.dtype], s[0] if rows > 1 else v


def _vector(x, n, dtype, name, device):
    """Address of a contiguous vector of n values (None stays)."""
    if x is None:
        return None
    if x.dtype != dtype or not x.is_contiguous() or x.numel() != n or not x.is_cuda:
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor of {n} values")
    if x.device != device:
        raise ValueError(f"{name} is on {x.device}, the logits on {device}")
    return x.data_ptr()


def _status(x, device):
    """Address of a status word (None stays)."""
    if x is None:
        return None
    if x.dtype != torch.int32 or x.numel() < 1 or x.device != device:
        raise ValueError(f"dev_status must be an int32 tensor on {device}")
    return x.data_ptr()


def _output(x, shape, n, dtype, name, device, stream):
    """(tensor, address) of an output of n values: the caller's, or a new one."""
    if x is None:
        x = _on_stream(shape, dtype, device, stream)
        return x, x.data_ptr()
    return x, _vector(x, n, dtype, name, device)


def _same_device(device, *tensors):
    if device.index != torch._C._cuda_getDevice():
        raise ValueError(f"the logits are on {device}, which is not the current device")
    for t in tensors:
        if t is not None and t.device != device:
            raise ValueError(f"every tensor must be on {device}, got one on {t.device}")


def _loss_rows(logits, dlogits, stream, grad=True):
    """Of a call on rows of logits: (T, V, dtype number, row stride) and the gradient's tensor with its row stride."""
    if logits.dim() != 2:
        raise ValueError(f"logits must be [T, V], got {list(logits.shape)}")
    t, v = logits.shape
    dtype, ld = _logit_rows(logits, t, v, "logits")
    _same_device(logits.device, dlogits)
    if not grad:
        return (dtype, t, v, ld), None, 0
    if dlogits is None:
        return (dtype, t, v, ld), _on_stream((t, v), logits.dtype, logits.device, stream), v
    return (dtype, t, v, ld), dlogits, _logit_rows(dlogits, t, v, "dlogits", logits.dtype)[1]


def _teacher(top_ids, top_logits, top_lse, temperature, t, device):
    if top_ids.dim() != 2 or top_ids.shape[0] != t or top_logits.shape != top_ids.shape:
        raise ValueError(f"top_ids and top_logits must both be [{t}, k], got {list(top_ids.shape)} and {list(top_logits.shape)}")
    n = top_ids.numel()
    return (_vector(top_ids, n, torch.int32, "top_ids", device), _vector(top_logits, n, torch.float32, "top_logits", device),
            top_ids.shape[1], _vector(top_lse, t, torch.float32, "top_lse", device), float(temperature))


def distill_topk(logits, top_ids, top_logits, top_lse=None, temperature=1.0, loss=None, stats=None, dev_status=None,
                 stream=None):
    """Distillation from a teacher's top logits: (loss fp32 [T], stats fp32 [T, 2] for ``distill_topk_backward``).

    ``logits`` bf16 or fp32 [T, V]; ``top_ids`` int32 and ``top_logits`` fp32 [T, k], a negative id an unused slot;
    ``top_lse`` fp32 [T]: the log-sum-exp of the teacher's whole row over the temperature, for a tail (see
    ``qrr_distill_topk``)."""
    rows, _, _ = _loss_rows(logits, None, stream, grad=False)
    t, dev = rows[1], logits.device
    teacher = _teacher(top_ids, top_logits, top_lse, temperature, t, dev)
    loss, loss_ptr = _output(loss, (t,), t, torch.float32, "loss", dev, stream)
    stats, stats_ptr = _output(stats, (t, 2), 2 * t, torch.float32, "stats", dev, stream)
    _check(lib().qrr_distill_topk(logits.data_ptr(), *rows, *teacher, loss_ptr, stats_ptr, _status(dev_status, dev), _stream(stream)),
           "qrr_distill_topk")
    return loss, stats


def distill_topk_backward(logits, top_ids, top_logits, stats, grad, top_lse=None, temperature=1.0, dlogits=None,
                          dev_status=None, stream=None):
    """dlogits [T, V] = grad[t] dloss[t]/dlogits in the logits' type, from the ``stats`` of ``distill_topk`` with the same
    arguments; ``dlogits`` may be ``logits`` itself."""
    rows, dlogits, ldd = _loss_rows(logits, dlogits, stream)
    t, dev = rows[1], logits.device
    teacher = _teacher(top_ids, top_logits, top_lse, temperature, t, dev)
    _check(lib().qrr_distill_topk_backward(logits.data_ptr(), *rows, *teacher, _vector(stats, 2 * t, torch.float32, "stats", dev),
                                           _vector(grad, t, torch.float32, "grad", dev), dlogits.data_ptr(), ldd,
                                           _status(dev_status, dev), _stream(stream)), "qrr_distill_topk_backward")
    return dlogits


def distill_topk_grad(logits, top_ids, top_logits, grad, top_lse=None, temperature=1.0, loss=None, dlogits=None,
                      dev_status=None, stream=None):
    """(loss, dlogits) of ``distill_topk`` and ``distill_topk_backward`` at once, where the rows' weights ``grad`` are known
    beforehand: the logits are read from memory once, and a second time from L2 mostly."""
    rows, dlogits, ldd = _loss_rows(logits, dlogits, stream)
    t, dev = rows[1], logits.device
    teacher = _teacher(top_ids, top_logits, top_lse, temperature, t, dev)
    loss, loss_ptr = _output(loss, (t,), t, torch.float32, "loss", dev, stream)
    _check(lib().qrr_distill_topk_grad(logits.data_ptr(), *rows, *teacher, _vector(grad, t, torch.float32, "grad", dev),
                                       loss_ptr, dlogits.data_ptr(), ldd, _status(dev_status, dev),
                                       _stream(stream)), "qrr_distill_topk_grad")
    return loss, dlogits


def token_logprobs_is_grad(logits, tokens, advantages, rollout_logp=None, cap=0.0, logp=None, w=None, dlogits=None,
                           dev_status=None, stream=None):
    """(logp, w, dlogits): ``token_logprobs_is`` and the gradient of -sum A w logp in the logits (bf16 or fp32) at once, w
    held fixed (None, for 1, without ``rollout_logp``); ``dlogits`` may be ``logits`` itself.  At temperature 1: of a rollout at
    another one, take the logits over it, and the gradient over it again."""
    rows, dlogits, ldd = _loss_rows(logits, dlogits, stream)
    t, dev = rows[1], logits.device
    logp, logp_ptr = _output(logp, (t,), t, torch.float32, "logp", dev, stream)
    w, w_ptr = (None, None) if rollout_logp is None else _output(w, (t,), t, torch.float32, "w", dev, stream)
    _check(lib().qrr_token_logprobs_is_grad(logits.data_ptr(), *rows, _vector(tokens, t, torch.int32, "tokens", dev),
                                            _vector(advantages, t, torch.float32, "advantages", dev),
                                            _vector(rollout_logp, t, torch.float32, "rollout_logp", dev), float(cap),
                                            logp_ptr, w_ptr, dlogits.data_ptr(), ldd, _status(dev_status, dev), _stream(stream)),
           "qrr_token_logprobs_is_grad")
    return logp, w, dlogits


def verify_drafts(target, drafts, uniforms=None, noise=None, draft_logits=None, cu=None, temperature=1.0, tokens=None,
                  accepted=None, logp=None, workspace=None, dev_status=None, stream=None):
    """Test drafted tokens against the target's probabilities and draw the token that follows (see ``qrr_verify_drafts``).

    ``target`` logits [T + B, V] (bf16 or fp32), ``drafts`` int32 [T]: sequence b has the drafts cu[b] .. cu[b + 1] - 1 (as
    many as any other without ``cu``) and one row more, from cu[b] + b on.  ``draft_logits`` [T, V] is None for drafts
    without probabilities; ``uniforms`` fp32 [T] in [0, 1) and ``noise`` fp32 [B, V], exponential, are not needed at
    temperature 0.  Returns (tokens int32 [T + B], -1 behind the last of a sequence; accepted int32 [B]; logp fp32
    [T + B])."""
    if target.dim() != 2:
        raise ValueError(f"target must be [T + B, V], got {list(target.shape)}")
    rows, v = target.shape
    t = drafts.numel()
    b, dev = rows - t, target.device
    if b < 0:
        raise ValueError(f"target must have a row more than drafts for every sequence: {rows} rows, {t} drafts")
    dtype, ld_target = _logit_rows(target, rows, v, "target")
    ld_draft = ld_noise = 0
    if temperature == 0:
        draft_logits = uniforms = noise = None
    else:
        if (t and uniforms is None) or (b and noise is None):
            raise ValueError("uniforms and noise are needed but at temperature 0")
        if draft_logits is not None:
            ld_draft = _logit_rows(draft_logits, t, v, "draft_logits", target.dtype)[1]
        if noise is not None:
            ld_noise = _logit_rows(noise, b, v, "noise", torch.float32)[1]
    _same_device(dev, draft_logits, noise)
    cu_ptr = _vector(cu, b + 1, torch.int32, "cu", dev)
    tokens, tokens_ptr = _output(tokens, (rows,), rows, torch.int32, "tokens", dev, stream)
    accepted, accepted_ptr = _output(accepted, (b,), b, torch.int32, "accepted", dev, stream)
    logp, logp_ptr = _output(logp, (rows,), rows, torch.float32, "logp", dev, stream)
    if workspace is None:
        workspace = _workspace(lib().qrr_verify_drafts_workspace_bytes(t, b, v, dtype), dev, stream)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    _check(lib().qrr_verify_drafts(target.data_ptr(), ld_target, _ptr(draft_logits), ld_draft, dtype, t, b, v,
                                   _vector(drafts, t, torch.int32, "drafts", dev), cu_ptr,
                                   _vector(uniforms, t, torch.float32, "uniforms", dev), _ptr(noise), ld_noise,
                                   float(temperature), tokens_ptr, accepted_ptr, logp_ptr, workspace.data_ptr(),
                                   workspace.numel(), _status(dev_status, dev), _stream(stream)), "qrr_verify_drafts")
    return tokens, accepted, logp


def lora_backward_workspace_bytes(M, N, K, r) -> int:
    return int(lib().qrr_lora_backward_workspace_bytes(M, N, K, r))


def lora_backward_nvfp4(dy, x, codes, scales, tensor_scale, lora_A=None, lora_B=None, alpha=0.0, dx=None, dA=None,
                        dB=None, workspace=None, dev_status=None, stream=None):
    """(dX bf16 [M, K], dA fp32 [r, K], dB fp32 [N, r]) of the linear's backward
    through the frozen NVFP4 weight (dA, dB None without an adapter)."""
    _need(dy, torch.bfloat16, "dy")
    m, n = dy.shape
    k = codes.shape[1] * 2
    r = 0 if lora_A is None or lora_B is None else int(lora_A.shape[0])
    dev = dy.device
    dx = _on_stream((m, k), torch.bfloat16, dev, stream) if dx is None else dx
    if r:
        _need(x, torch.bfloat16, "x")
        dA = _on_stream((r, k), torch.float32, dev, stream) if dA is None else dA
        dB = _on_stream((n, r), torch.float32, dev, stream) if dB is None else dB
    if workspace is None:
        workspace = _workspace(lora_backward_workspace_bytes(m, n, k, r), dev, stream)
    _check(lib().qrr_lora_backward_nvfp4(_ptr(dy), m, n, _ptr(x), k, _ptr(codes), _ptr(scales), _ptr(tensor_scale),
                                         _ptr(lora_A), _ptr(lora_B), r, float(alpha), _ptr(dx),
                                         _ptr(dA) if r else None, _ptr(dB) if r else None, _ptr(workspace),
                                         workspace.numel(), _ptr(dev_status), _stream(stream)),
           "qrr_lora_backward_nvfp4")
    return dx, (dA if r else None), (dB if r else None)


def kv_append_fp8(k_new, v_new, pos, k_cache, k_scales, v_cache, v_scales, mode=SCALE_FP32, dev_status=None,
                  stream=None):
    """Quantize one decode step's key/value rows [B, Hkv, 128] into slot pos[b] of the FP8 caches."""
    _need(k_new, torch.bfloat16, "k_new")
    _need(v_new, torch.bfloat16, "v_new")
    _need(pos, torch.int32, "pos")
    b, hkv, _ = k_new.shape
    lmax = k_cache.shape[2]
    _check(lib().qrr_kv_append_fp8(_ptr(k_new), _ptr(v_new), b, hkv, _ptr(pos), _ptr(k_cache), _ptr(k_scales),
                                   _ptr(v_cache), _ptr(v_scales), lmax, int(mode), _ptr(dev_status), _stream(stream)),
           "qrr_kv_append_fp8")


def attention_decode_fp8(q, k_cache, k_scales, v_cache, v_scales, lens, out=None, workspace=None, dev_status=None,
                         stream=None):
    """o [B, Hq, 128] bf16 of decode attention over the FP8 caches [B, Hkv, Lmax, 128]."""
    _need(q, torch.bfloat16, "q")
    _need(lens, torch.int32, "lens")
    b, hq, _ = q.shape
    hkv, lmax = k_cache.shape[1], k_cache.shape[2]
    out = _on_stream(q.shape, q.dtype, q.device, stream) if out is None else out
    if workspace is None:
        workspace = _workspace(lib().qrr_attention_decode_fp8_workspace_bytes(b, hq, lmax), q.device, stream)
    _check(lib().qrr_attention_decode_fp8(_ptr(q), b, hq, hkv, _ptr(k_cache), _ptr(k_scales), _ptr(v_cache),
                                          _ptr(v_scales), _ptr(lens), lmax, _ptr(out), _ptr(workspace),
                                          workspace.numel(), _ptr(dev_status), _stream(stream)),
           "qrr_attention_decode_fp8")
    return out


class KvCacheNvfp4:
    """A paged NVFP4 key/value cache over buffers of the caller's, checked once.

    ``k_codes``, ``v_codes`` uint8 [pages, Hkv, page, D/2]; ``k_scales``,
    ``v_scales`` uint8 [pages, Hkv, page, D/16]; ``page_table`` int32
    [B, max_pages]; ``k_gs``, ``v_gs`` fp32 [Hkv] global scales or None (1).
    The tensors are kept, not copied: their contents may change between calls
    (new pages in the table, say), their storage may not."""

    def __init__(self, k_codes, k_scales, v_codes, v_scales, page_table, k_gs=None, v_gs=None):
        for t, name in ((k_codes, "k_codes"), (k_scales, "k_scales"), (v_codes, "v_codes"), (v_scales, "v_scales")):
            _need(t, torch.uint8, name)
        _need(page_table, torch.int32, "page_table")
        if k_codes.dim() != 4 or page_table.dim() != 2:
            raise ValueError("k_codes must be [pages, Hkv, page, D/2] and page_table [B, max_pages]")
        pages, hkv, page, half = k_codes.shape
        if v_codes.shape != k_codes.shape:
            raise ValueError("k_codes and v_codes must have the same shape")
        for t, name in ((k_scales, "k_scales"), (v_scales, "v_scales")):
            if tuple(t.shape) != (pages, hkv, page, half // 8):
                raise ValueError(f"{name} must be {[pages, hkv, page, half // 8]}, got {list(t.shape)}")
        for t, name in ((k_gs, "k_gs"), (v_gs, "v_gs")):
            if t is not None:
                _need(t, torch.float32, name)
                if t.numel() != hkv:
                    raise ValueError(f"{name} must have one value a KV head")
        self.tensors = (k_codes, k_scales, v_codes, v_scales, page_table, k_gs, v_gs)
        self.device = k_codes.device
        self.pages, self.hkv, self.page, self.dim = pages, hkv, page, 2 * half
        self.batch, self.max_pages = page_table.shape
        self._workspace_bytes = {}  # of attention, by (query heads, max_new)
        self.desc = KvNvfp4Desc(_ptr(k_codes), _ptr(k_scales), _ptr(v_codes), _ptr(v_scales), _ptr(k_gs), _ptr(v_gs),
                                _ptr(page_table), pages, hkv, page, 2 * half, self.batch, self.max_pages)
        self._addr = ctypes.addressof(self.desc)

    @classmethod
    def empty(cls, pages, hkv, page, dim, page_table, k_gs=None, v_gs=None):
        """A cache with buffers of its own, all zeros."""
        dev = page_table.device
        codes = [torch.zeros(pages, hkv, page, dim // 2, dtype=torch.uint8, device=dev) for _ in range(2)]
        scales = [torch.zeros(pages, hkv, page, dim // 16, dtype=torch.uint8, device=dev) for _ in range(2)]
        return cls(codes[0], scales[0], codes[1], scales[1], page_table, k_gs, v_gs)


def _kv_rows(cache, pos, cu, t):
    """Address of ``cu`` (None without).  The caller keeps the tensor to the end of its call: it may be a temporary, whose
    memory a buffer of the call would take."""
    if pos.dtype is not torch.int32 or not pos.is_cuda or not pos.is_contiguous() or pos.numel() != cache.batch:
        raise ValueError(f"pos must be a contiguous CUDA int32 tensor of {cache.batch} values")
    if cu is None:
        if t != cache.batch:
            raise ValueError(f"without cu there is one row a sequence: {cache.batch}, got {t}")
        return None
    if cu.dtype is not torch.int32 or not cu.is_cuda or not cu.is_contiguous() or cu.numel() != cache.batch + 1:
        raise ValueError(f"cu must be a contiguous CUDA int32 tensor of {cache.batch + 1} values")
    return cu.data_ptr()


def _head_rows(x, heads, dim, name):
    """Row stride of bf16 rows [T, heads, dim] whose heads are contiguous (a slice of a wider projection will do)."""
    if x.dtype is not torch.bfloat16 or not x.is_cuda:
        raise TypeError(f"{name} must be a CUDA bfloat16 tensor")
    shape = x.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise ValueError(f"{name} must be [T, {heads}, {dim}], got {list(shape)}")
    s = x.stride()
    if s[2] != 1 or (heads > 1 and s[1] != dim):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    return s[0] if shape[0] > 1 else heads * dim


def _result(given, shape, dtype, device, stream, name):
    """An output: the caller's tensor, checked, or a new one."""
    if given is None:
        return _on_stream(shape, dtype, device, stream)
    if given.dtype is not dtype or not given.is_cuda or not given.is_contiguous() or given.shape != shape:
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor {list(shape)}")
    return given


def kv_append_nvfp4(k_new, v_new, cache, pos, cu=None, dev_status=None, stream=None):
    """Quantize rows [T, Hkv, D] of keys and values into the cache: sequence b's rows cu[b] .. cu[b + 1] - 1 (row b
    alone without ``cu``) at the positions pos[b], pos[b] + 1, ... (see ``qrr_kv_append_nvfp4``)."""
    ld_k = _head_rows(k_new, cache.hkv, cache.dim, "k_new")
    ld_v = _head_rows(v_new, cache.hkv, cache.dim, "v_new")
    t = k_new.shape[0]
    if v_new.shape[0] != t:
        raise ValueError("k_new and v_new must have the same rows")
    cu_ptr = _kv_rows(cache, pos, cu, t)
    _check(lib().qrr_kv_append_nvfp4(cache._addr, k_new.data_ptr(), v_new.data_ptr(), t, ld_k, ld_v, cu_ptr, pos.data_ptr(),
                                     _ptr(dev_status), _stream(stream)), "qrr_kv_append_nvfp4")


def kv_read_nvfp4(cache, pos, cu=None, rows=None, k=None, v=None, dev_status=None, stream=None):
    """(k, v) bf16 [rows, Hkv, D]: the cached values at pos[b], pos[b] + 1, ... of every sequence, as many as ``cu``
    gives it (one without ``cu``); ``rows`` is cu[B], which the host cannot see without waiting for the GPU."""
    if rows is None:
        if cu is not None and k is None:
            raise ValueError("rows is needed with cu")
        rows = cache.batch if k is None else k.shape[0]
    cu_ptr = _kv_rows(cache, pos, cu, rows)
    shape = (rows, cache.hkv, cache.dim)
    k = _result(k, shape, torch.bfloat16, cache.device, stream, "k")
    v = _result(v, shape, torch.bfloat16, cache.device, stream, "v")
    _check(lib().qrr_kv_read_nvfp4(cache._addr, rows, cu_ptr, pos.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(dev_status),
                                   _stream(stream)), "qrr_kv_read_nvfp4")
    return k, v


def attention_nvfp4_workspace_bytes(cache, rows, hq, max_new=1) -> int:
    return int(lib().qrr_attention_nvfp4_workspace_bytes(cache._addr, int(rows), int(hq), int(max_new)))


def attention_nvfp4(q, cache, pos, cu=None, max_new=None, scale=None, return_lse=False, out=None, lse=None,
                    workspace=None, dev_status=None, stream=None):
    """Attention of query rows q [T, Hq, D] over the NVFP4 cache: row cu[b] + i sees the positions up to pos[b] + i.

    ``max_new`` bounds the rows of a sequence (needed with ``cu``); ``scale`` is
    1/sqrt(D) unless given.  Returns out bf16 [T, Hq, D], or (out, lse fp32
    [T, Hq]) when ``return_lse`` is set or ``lse`` is given."""
    shape = q.shape
    if len(shape) != 3:
        raise ValueError(f"q must be [T, Hq, D], got {list(shape)}")
    t, hq, d = shape
    ld_q = _head_rows(q, hq, cache.dim, "q")
    if max_new is None:
        if cu is not None:
            raise ValueError("max_new is needed with cu")
        max_new = 1
    cu_ptr = _kv_rows(cache, pos, cu, t)
    device = cache.device
    out = _result(out, shape, torch.bfloat16, device, stream, "out")
    if return_lse or lse is not None:
        lse = _result(lse, (t, hq), torch.float32, device, stream, "lse")
    if workspace is None:
        need = cache._workspace_bytes.get((hq, max_new))
        if need is None:  # it goes by the cache's shape and these two
            need = cache._workspace_bytes[hq, max_new] = max(attention_nvfp4_workspace_bytes(cache, t, hq, max_new), 256)
        workspace = _on_stream((need,), torch.uint8, device, stream, returned=False)
    _check(lib().qrr_attention_nvfp4(cache._addr, q.data_ptr(), t, ld_q, hq, cu_ptr, pos.data_ptr(), max_new,
                                     d ** -0.5 if scale is None else scale, out.data_ptr(), _ptr(lse),
                                     workspace.data_ptr(), workspace.numel(), _ptr(dev_status), _stream(stream)),
           "qrr_attention_nvfp4")
    return out if lse is None else (out, lse)
