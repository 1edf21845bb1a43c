"""GB300-native W8A8 / W4A8 online-activation-quantized linear layer.

A thin binding over the C ABI of ``libcider.so`` (declared in
``include/cider.h``).  Each function here has the name of the C entry point it
calls, takes PyTorch CUDA tensors, allocates the outputs with PyTorch on the
input's device, and passes raw pointers and the current CUDA stream.  Every
step of the computation runs in the library's CUDA kernels; there is no CPU or
PyTorch fallback: if the library is missing or the GPU is not sm_103, calls
raise.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

import torch

from . import inputs  # noqa: F401  (seeded synthetic inputs, no arithmetic)

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libcider.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "cider.h")

CIDER_OK = 0
CIDER_PER_CHANNEL = 0
CIDER_PER_GROUP = 1
CIDER_F16 = 0
CIDER_BF16 = 1
CIDER_F32 = 2
_DTYPES = {torch.float16: CIDER_F16, torch.bfloat16: CIDER_BF16}
STATUS_NAMES = {0: "CIDER_OK", 1: "CIDER_ERR_INVALID_ARGUMENT", 2: "CIDER_ERR_MISALIGNED",
                3: "CIDER_ERR_UNSUPPORTED_DEVICE", 4: "CIDER_ERR_CUDA", 5: "CIDER_ERR_TIMEOUT",
                6: "CIDER_ERR_INDEX"}

_lib = None
_lock = threading.Lock()


class CiderError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        msg = _load().cider_status_string(status).decode()
        super().__init__(f"{fn} failed with status {status}: {msg}")


def _declare(lib):
    p, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    sig = {
        "cider_is_available": ([], i32),
        "cider_status_string": ([i32], ctypes.c_char_p),
        "cider_version": ([], i32),
        "cider_quantize_act": ([p, i64, i64, p, p, p], i32),
        "cider_quantize_act_bf16": ([p, i64, i64, p, p, p], i32),
        "cider_int4_from_offset_binary": ([p, p, i64, p], i32),
        "cider_quantize_weight_int8": ([p, i64, i64, i32, p, p, p], i32),
        "cider_quantize_weight_int4": ([p, i64, i64, i32, p, p, p], i32),
        "cider_quantize_weight_int8_clip": ([p, i64, i64, i32, ctypes.c_double, p, p, p], i32),
        "cider_quantize_weight_int4_clip": ([p, i64, i64, i32, ctypes.c_double, p, p, p], i32),
        "cider_w8a8_linear": ([p, i64, i64, i64, p, p, i32, i32, p, p], i32),
        "cider_w4a8_linear": ([p, i64, i64, i64, p, p, i32, i32, p, p], i32),
        "cider_w8a8_linear_bf16": ([p, i64, i64, i64, p, p, i32, i32, p, p], i32),
        "cider_w4a8_linear_bf16": ([p, i64, i64, i64, p, p, i32, i32, p, p], i32),
        "cider_w8a8_linear_ex": ([p, i32, i64, i64, i64, p, p, i32, i32, p, i32, p], i32),
        "cider_w4a8_linear_ex": ([p, i32, i64, i64, i64, p, p, i32, i32, p, i32, p], i32),
        "cider_w8a8_linear_prequant": ([p, p, i64, i64, i64, p, p, i32, i32, p, p], i32),
        "cider_w4a8_linear_prequant": ([p, p, i64, i64, i64, p, p, i32, i32, p, p], i32),
        "cider_w8a8_accumulators": ([p, i64, i64, i64, p, i32, p, p], i32),
        "cider_w4a8_accumulators": ([p, i64, i64, i64, p, i32, p, p], i32),
        "cider_check_device_error": ([p], i32),
        "cider_trim_scratch_pool": ([i64, p], i32),
        "cider_timing_begin": ([i64], i32),
        "cider_timing_end": ([ctypes.POINTER(i64), ctypes.POINTER(ctypes.c_double)], i32),
        "cider_debug_wait_timeout": ([i64, p], i32),
        "cider_debug_pair_schedule": ([i64, i64, i64, i32, i64, p, p, p], i32),
        "cider_debug_small_m_slices": ([i64, i64, i64, i32, i32, i32, p], i32),
        "cider_kv_append": ([p, i64, p, i64, p, i64, i32, p, i64, p], i32),
        "cider_kv_read": ([p, i64, p, i64, p, p, i64, i64, p, p, i32, p], i32),
        "cider_kv_compact": ([p, p, i64, p, p, i64, p, i64, p], i32),
        "cider_tree_attention": ([p, i64, p, i64, i32, i64, i64, p, i64, p, p, i64, i64, p,
                                  ctypes.c_float, p, p], i32),
        "cider_verify_drafts": ([p, i64, i32, p, p, p, i64, i64, i64, i64, p, p, p, p, p, p, p, p],
                                i32),
        "cider_debug_verify_timeout": ([p, i64, i32, p, p, p, i64, i64, i64, i64, p, p, p, p, p, p, p,
                                        i64, ctypes.c_int32, p], i32),
        "cider_quantize_fp4": ([p, i32, i64, p, p], i32),
        "cider_dequantize_fp4": ([p, p, i32, p], i32),
        "cider_w4a4_linear": ([p, i32, i64, i64, p, p, i32, p], i32),
        "cider_w4a4_linear_prequant": ([p, p, p, i32, p], i32),
        "cider_w4a4_gated_linear": ([p, i32, i64, i64, p, p, i32, p, i32, p], i32),
        "cider_w4a4_gated_linear_prequant": ([p, p, p, i32, p, i32, p], i32),
        "cider_w4a4_feed_forward": ([p, i32, i64, i64, p, p, p, i32, p, i32, p], i32),
        "cider_debug_small_m_launch": ([i64, i64, i64, i32, i32, i32, i32, p], i32),
    }
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    return lib


def _load():
    """Load libcider.so (built in-tree by ``_build.build()``); raise if absent."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"libcider.so not found at {LIB_PATH}: build it first with "
                    "`python -m w4a8_quantized_linear_gb300._build` (needs nvcc); "
                    "there is no fallback implementation")
            _lib = _declare(ctypes.CDLL(LIB_PATH))
    return _lib


def library():
    """The loaded ctypes library (for callers that want the raw C ABI)."""
    return _load()


def _check(fn: str, status: int):
    if status != CIDER_OK:
        raise CiderError(fn, status)


# The current stream's handle, of a device index, and the current device's index.
# The functions behind current_stream() and current_device() save a few
# microseconds a call; a PyTorch without CUDA lacks them.
_raw_stream = (getattr(torch._C, "_cuda_getCurrentRawStream", None)
               or (lambda dev: torch.cuda.current_stream(dev).cuda_stream))
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _launch(call, dev: int, args: tuple):
    """Call an entry point of the library with `args`, the last of them a stream of
    the device that its tensors are on.  The library launches on the current
    device, so that one is made current."""
    if _current_device() == dev:
        status = call(*args)
    else:
        with torch.cuda.device(dev):
            status = call(*args)
    if status:
        _check(call.__name__, status)


def _call(fn: str, t: torch.Tensor, *args):
    """_launch with the current stream of t's device."""
    dev = t.get_device()
    _launch(getattr(_lib or _load(), fn), dev, args + (_raw_stream(dev),))


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _need(t: torch.Tensor, dtype, name: str, ndim: int):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


# ----------------------------------------------------------------------------- API
def cider_is_available() -> bool:
    return bool(_load().cider_is_available())


def _quantize_act(fn, x, dtype):
    _need(x, dtype, "x", 2)
    M, K = x.shape
    qa = torch.empty((M, K), dtype=torch.int8, device=x.device)
    sa = torch.empty((M,), dtype=torch.float32, device=x.device)
    _call(fn, x, _ptr(x), M, K, _ptr(qa), _ptr(sa))
    return qa, sa


def cider_quantize_act(x: torch.Tensor):
    """x fp16 [M, K] -> (qa int8 [M, K], sa fp32 [M])."""
    return _quantize_act("cider_quantize_act", x, torch.float16)


def cider_quantize_act_bf16(x: torch.Tensor):
    """x bf16 [M, K] -> (qa int8 [M, K], sa fp32 [M])."""
    return _quantize_act("cider_quantize_act_bf16", x, torch.bfloat16)


def cider_int4_from_offset_binary(packed: torch.Tensor, out=None):
    """uint8 INT4 bytes stored offset-binary (nibble u = value + 8) -> the
    library's two's complement packing (out may be packed itself)."""
    if not isinstance(packed, torch.Tensor) or not packed.is_cuda or packed.dtype != torch.uint8:
        raise TypeError("packed must be a CUDA uint8 tensor")
    if not packed.is_contiguous():
        raise ValueError("packed must be contiguous")
    dst = out if out is not None else torch.empty_like(packed)
    _call("cider_int4_from_offset_binary", packed, _ptr(packed), _ptr(dst), packed.numel())
    return dst


def cider_quantize_weight_int8(w: torch.Tensor, group_size: int = 0, clip_percentile=None):
    """w fp32 [N, K] -> (qw int8 [N, K], sw fp32 [N, G]); min-max scales, or
    percentile-clipped ones when ``clip_percentile`` (in (0, 100]) is given."""
    _need(w, torch.float32, "w", 2)
    N, K = w.shape
    G = K // group_size if group_size else 1
    qw = torch.empty((N, K), dtype=torch.int8, device=w.device)
    sw = torch.empty((N, G), dtype=torch.float32, device=w.device)
    if clip_percentile is None:
        _call("cider_quantize_weight_int8", w, _ptr(w), N, K, group_size, _ptr(qw), _ptr(sw))
    else:
        _call("cider_quantize_weight_int8_clip", w, _ptr(w), N, K, group_size,
              float(clip_percentile), _ptr(qw), _ptr(sw))
    return qw, sw


def cider_quantize_weight_int4(w: torch.Tensor, group_size: int = 0, clip_percentile=None):
    """w fp32 [N, K] -> (packed uint8 [N, K/2], sw fp32 [N, G]); min-max or
    percentile-clipped scales as for the INT8 quantizer."""
    _need(w, torch.float32, "w", 2)
    N, K = w.shape
    G = K // group_size if group_size else 1
    qp = torch.empty((N, K // 2), dtype=torch.uint8, device=w.device)
    sw = torch.empty((N, G), dtype=torch.float32, device=w.device)
    if clip_percentile is None:
        _call("cider_quantize_weight_int4", w, _ptr(w), N, K, group_size, _ptr(qp), _ptr(sw))
    else:
        _call("cider_quantize_weight_int4_clip", w, _ptr(w), N, K, group_size,
              float(clip_percentile), _ptr(qp), _ptr(sw))
    return qp, sw


def _gran(group_size: int) -> int:
    return CIDER_PER_GROUP if group_size else CIDER_PER_CHANNEL


def _linear(fn, x, qw, sw, group_size, int4, out=None, x_dtype=torch.float16):
    _need(x, x_dtype, "x", 2)
    _need(qw, torch.uint8 if int4 else torch.int8, "qw", 2)
    M, K = x.shape
    N = qw.shape[0]
    if qw.shape[1] != (K // 2 if int4 else K):
        raise ValueError("weight width does not match K")
    sw = sw.reshape(N, -1)
    _need(sw, torch.float32, "sw", 2)
    y = out if out is not None else torch.empty((M, N), dtype=torch.float16, device=x.device)
    _call(fn, x, _ptr(x), M, N, K, _ptr(qw), _ptr(sw), _gran(group_size), group_size, _ptr(y))
    return y


def cider_w8a8_linear(x, qw, sw, group_size: int = 0, out=None):
    """y fp16 [M, N] = W8A8 linear of x fp16 [M, K] with qw int8 [N, K] and
    scales sw fp32 [N] (group_size 0) or [N, K/group_size]."""
    return _linear("cider_w8a8_linear", x, qw, sw, group_size, False, out)


def cider_w4a8_linear(x, qw_packed, sw, group_size: int = 0, out=None):
    """W4A8 linear with qw_packed uint8 [N, K/2]."""
    return _linear("cider_w4a8_linear", x, qw_packed, sw, group_size, True, out)


def cider_w8a8_linear_bf16(x, qw, sw, group_size: int = 0, out=None):
    """As cider_w8a8_linear for x bf16 [M, K]; y is fp16."""
    return _linear("cider_w8a8_linear_bf16", x, qw, sw, group_size, False, out, torch.bfloat16)


def cider_w4a8_linear_bf16(x, qw_packed, sw, group_size: int = 0, out=None):
    """As cider_w4a8_linear for x bf16 [M, K]; y is fp16."""
    return _linear("cider_w4a8_linear_bf16", x, qw_packed, sw, group_size, True, out,
                   torch.bfloat16)


def _linear_ex(fn, x, qw, sw, group_size, int4, y_dtype, out):
    if x.dtype not in _DTYPES or y_dtype not in _DTYPES:
        raise TypeError("x and y must be float16 or bfloat16")
    _need(x, x.dtype, "x", 2)
    _need(qw, torch.uint8 if int4 else torch.int8, "qw", 2)
    M, K = x.shape
    N = qw.shape[0]
    if qw.shape[1] != (K // 2 if int4 else K):
        raise ValueError("weight width does not match K")
    sw = sw.reshape(N, -1)
    _need(sw, torch.float32, "sw", 2)
    y = out if out is not None else torch.empty((M, N), dtype=y_dtype, device=x.device)
    _need(y, y_dtype, "out", 2)
    _call(fn, x, _ptr(x), _DTYPES[x.dtype], M, N, K, _ptr(qw), _ptr(sw), _gran(group_size),
          group_size, _ptr(y), _DTYPES[y_dtype])
    return y


def cider_w8a8_linear_ex(x, qw, sw, group_size: int = 0, y_dtype=torch.float16, out=None):
    """W8A8 linear with x fp16 or bf16 [M, K] and y of ``y_dtype`` (fp16 or
    bf16, the fp32 result rounded once to it)."""
    return _linear_ex("cider_w8a8_linear_ex", x, qw, sw, group_size, False, y_dtype, out)


def cider_w4a8_linear_ex(x, qw_packed, sw, group_size: int = 0, y_dtype=torch.float16, out=None):
    """W4A8 linear with x fp16 or bf16 [M, K] and y of ``y_dtype``."""
    return _linear_ex("cider_w4a8_linear_ex", x, qw_packed, sw, group_size, True, y_dtype, out)


def _linear_prequant(fn, qa, sa, qw, sw, group_size, int4, out=None):
    _need(qa, torch.int8, "qa", 2)
    _need(sa, torch.float32, "sa", 1)
    _need(qw, torch.uint8 if int4 else torch.int8, "qw", 2)
    M, K = qa.shape
    N = qw.shape[0]
    sw = sw.reshape(N, -1)
    _need(sw, torch.float32, "sw", 2)
    y = out if out is not None else torch.empty((M, N), dtype=torch.float16, device=qa.device)
    _call(fn, qa, _ptr(qa), _ptr(sa), M, N, K, _ptr(qw), _ptr(sw), _gran(group_size), group_size,
          _ptr(y))
    return y


def cider_w8a8_linear_prequant(qa, sa, qw, sw, group_size: int = 0, out=None):
    return _linear_prequant("cider_w8a8_linear_prequant", qa, sa, qw, sw, group_size, False, out)


def cider_w4a8_linear_prequant(qa, sa, qw_packed, sw, group_size: int = 0, out=None):
    return _linear_prequant("cider_w4a8_linear_prequant", qa, sa, qw_packed, sw, group_size, True,
                            out)


def _accumulators(fn, qa, qw, group_size, int4):
    _need(qa, torch.int8, "qa", 2)
    _need(qw, torch.uint8 if int4 else torch.int8, "qw", 2)
    M, K = qa.shape
    N = qw.shape[0]
    G = K // group_size if group_size else 1
    acc = torch.empty((M, N, G), dtype=torch.int32, device=qa.device)
    _call(fn, qa, _ptr(qa), M, N, K, _ptr(qw), group_size, _ptr(acc))
    return acc


def cider_w8a8_accumulators(qa, qw, group_size: int = 0):
    """Exact int32 accumulators [M, N, G] of the same kernels."""
    return _accumulators("cider_w8a8_accumulators", qa, qw, group_size, False)


def cider_w4a8_accumulators(qa, qw_packed, group_size: int = 0):
    return _accumulators("cider_w4a8_accumulators", qa, qw_packed, group_size, True)


def cider_check_device_error(device=None) -> int:
    """Synchronize the current stream and return (and clear) the status of
    the library's device error word: 0 (CIDER_OK), 5 (CIDER_ERR_TIMEOUT) or 6
    (CIDER_ERR_INDEX: a page, slot, offset, count or token was out of range)."""
    with torch.cuda.device(device):   # the error word is the current device's; None: as it is
        s = torch.cuda.current_stream()
        return int(_load().cider_check_device_error(ctypes.c_void_p(s.cuda_stream)))


def cider_trim_scratch_pool(keep_bytes: int = 0, device=None) -> None:
    """Return the library's pooled scratch memory beyond ``keep_bytes`` to the
    device (after the current stream's queued calls have run)."""
    with torch.cuda.device(device):
        s = torch.cuda.current_stream()
        _check("cider_trim_scratch_pool",
               _load().cider_trim_scratch_pool(int(keep_bytes), ctypes.c_void_p(s.cuda_stream)))


def cider_debug_wait_timeout(max_polls: int, device=None) -> int:
    with torch.cuda.device(device):
        s = torch.cuda.current_stream()
        return int(_load().cider_debug_wait_timeout(int(max_polls), ctypes.c_void_p(s.cuda_stream)))


def cider_timing_begin(capacity: int) -> None:
    """Time the integer-GEMM kernel of the next `capacity` linear calls made
    from this thread (CUDA events recorded by the library around each launch)."""
    _check("cider_timing_begin", _load().cider_timing_begin(int(capacity)))


def cider_timing_end():
    """-> (number of timed launches, their summed device time in ms)."""
    n = ctypes.c_int64(0)
    ms = ctypes.c_double(0.0)
    _check("cider_timing_end", _load().cider_timing_end(ctypes.byref(n), ctypes.byref(ms)))
    return int(n.value), float(ms.value)


def cider_debug_pair_schedule(M: int, N: int, K: int, pairs: int):
    """Work split of the per-channel tensor-core GEMM (host arithmetic only).
    -> (info dict, list of (pair, tile, kb0, kb1, kind, row0, row1))."""
    info = (ctypes.c_int32 * 6)()
    count = ctypes.c_int64(0)
    lib = _load()
    _check("cider_debug_pair_schedule",
           lib.cider_debug_pair_schedule(M, N, K, pairs, 0, None, ctypes.byref(count), info))
    rows = (ctypes.c_int32 * (7 * max(count.value, 1)))()
    _check("cider_debug_pair_schedule",
           lib.cider_debug_pair_schedule(M, N, K, pairs, count.value, rows, ctypes.byref(count),
                                         info))
    keys = ("pairs", "whole_tiles", "cut_tiles", "pieces", "blocks_per_tile", "tiles")
    units = [tuple(rows[7 * i:7 * i + 7]) for i in range(count.value)]
    return dict(zip(keys, list(info))), units


def cider_debug_small_m_launch(M: int, N: int, K: int, bits: int, group_size: int,
                               split_allowed: bool, num_sms: int) -> dict:
    """Launch sizes of the small-M path for this linear (host arithmetic only)."""
    info = (ctypes.c_int32 * 10)()
    _check("cider_debug_small_m_launch",
           _load().cider_debug_small_m_launch(M, N, K, 1 if bits == 4 else 0, group_size,
                                              1 if split_allowed else 0, num_sms, info))
    keys = ("mb", "mma", "slices", "tiles_per_slice", "staged_codes", "pitch", "ring_slots",
            "smem", "smem_cap", "codes_per_tile")
    return dict(zip(keys, list(info)))


def cider_debug_small_m_slices(M: int, N: int, K: int, bits: int, group_size: int,
                               num_sms: int) -> int:
    """K slices of the small-M path for this linear (host arithmetic only)."""
    out = ctypes.c_int32(0)
    _check("cider_debug_small_m_slices",
           _load().cider_debug_small_m_slices(M, N, K, 1 if bits == 4 else 0, group_size,
                                              num_sms, ctypes.byref(out)))
    return int(out.value)


# ------------------------------------------------- quantized key/value cache
_CACHE = struct.Struct("@PPPPqqiiii")   # cider_kv_cache_t


def cider_kv_cache(layers: int, pages: int, heads: int, head_dim: int, page_size: int = 64,
                   bits: int = 8, device="cuda"):
    """An empty paged cache: (k, k_scale, v, v_scale) with codes int8 [layers,
    pages, heads, page_size, head_dim] (bits 8) or uint8 [..., head_dim / 2]
    (bits 4) and scales fp32 [layers, pages, heads, page_size]."""
    if bits not in (8, 4):
        raise ValueError("bits must be 8 or 4")
    shape = (layers, pages, heads, page_size)
    width, kind = (head_dim, torch.int8) if bits == 8 else (head_dim // 2, torch.uint8)
    out = []
    for _ in range(2):
        out += [torch.zeros(shape + (width,), dtype=kind, device=device),
                torch.ones(shape, dtype=torch.float32, device=device)]
    return tuple(out)


# The checks below run on every call of a decoding step, whose kernels take a few
# microseconds: each tensor is passed by one chained condition, and only a
# tensor that fails it goes through the function that says what is wrong.
_I32, _I64, _F32, _I8, _U8 = torch.int32, torch.int64, torch.float32, torch.int8, torch.uint8


def _refuse_cache(cache):
    k, ks, v, vs = cache
    for t in (k, ks, v, vs):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError("cache must be CUDA tensors")
    if k.dtype not in (_I8, _U8) or v.dtype != k.dtype:
        raise TypeError("cache codes must be int8 or (packed INT4) uint8")
    if ks.dtype != _F32 or vs.dtype != _F32:
        raise TypeError("cache scales must be float32")
    if k.dim() != 5 or v.shape != k.shape or ks.shape != k.shape[:-1] or vs.shape != k.shape[:-1]:
        raise ValueError("cache tensors do not match")
    if not all(t.is_contiguous() for t in (k, ks, v, vs)):
        raise ValueError("cache must be contiguous")
    raise ValueError("cache tensors are on different devices")


def _cache_args(cache):
    """-> (cider_kv_cache_t as bytes, device index, heads, head_dim, layers)."""
    k, ks, v, vs = cache
    try:
        shape, kind, dev = k.shape, k.dtype, k.get_device()
        if not (len(shape) == 5 and (kind is _I8 or kind is _U8) and v.dtype is kind and ks.dtype is _F32
                and vs.dtype is _F32 and v.shape == shape and dev >= 0 and ks.get_device() == dev
                and v.get_device() == dev and vs.get_device() == dev and k.is_contiguous()
                and v.is_contiguous() and ks.is_contiguous() and vs.is_contiguous()
                and ks.shape == shape[:4] and vs.shape == shape[:4]):
            _refuse_cache(cache)
    except AttributeError:   # not all are tensors
        _refuse_cache(cache)
    layers, pages, heads, page, width = shape
    bits, dim = (8, width) if kind is _I8 else (4, 2 * width)
    return (_CACHE.pack(k.data_ptr(), ks.data_ptr(), v.data_ptr(), vs.data_ptr(), layers, pages,
                        heads, page, dim, bits), dev, heads, dim, layers)


def _rows(t, name, heads, dim, dev):
    """dtype and token stride of a [tokens, heads, dim] tensor with dense heads."""
    if not getattr(t, "is_cuda", False):
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype not in _DTYPES:
        raise TypeError(f"{name} must be float16 or bfloat16, got {t.dtype}")
    shape = t.shape
    if len(shape) != 3 or shape[2] != dim or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} has shape {tuple(shape)}, the cache {heads} heads of {dim}")
    n, h, d = shape
    token, row, one = t.stride()
    if one != 1 or (h > 1 and row != d):
        raise ValueError(f"{name}'s heads must be contiguous within a token")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on another device")
    return _DTYPES[t.dtype], token if n > 1 else h * d


def _flat(t, dtype, name, shape, dev):
    """A contiguous tensor of this type and shape on this device -> its pointer."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:   # not a tensor
        pass
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != dtype:
        raise TypeError(f"{name} must be a CUDA {dtype} tensor")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} is on another device")


def _size(t, name, dims):
    """The last dimension of a vector (dims 1) or a matrix (2)."""
    try:
        shape = t.shape
    except AttributeError:
        raise TypeError(f"{name} must be a CUDA tensor") from None
    if len(shape) != dims:
        raise ValueError(f"{name} must have {dims} dimension{'s' * (dims > 1)}, got {tuple(shape)}")
    return shape[-1]


def cider_kv_append(k, v, slots, cache, layer: int = 0) -> None:
    """Quantize k, v [tokens, heads, D] (fp16 or bf16, any token stride) into
    slots int64 [tokens] (page * page_size + row, negative: skip) of a layer."""
    c, dev, heads, dim, _ = _cache_args(cache)
    dt, ks = _rows(k, "k", heads, dim, dev)
    dv, vs = _rows(v, "v", heads, dim, dev)
    n = k.shape[0]
    if dv != dt or v.shape[0] != n:
        raise ValueError("k and v must have the same type and tokens")
    sp = _flat(slots, _I64, "slots", (n,), dev)
    _launch((_lib or _load()).cider_kv_append, dev, (c, layer, k.data_ptr(), ks, v.data_ptr(), vs,
            dt, sp, n, _raw_stream(dev)))


def cider_kv_read(cache, table, starts, offsets, tokens: int, dtype=torch.float16, layer=None,
                  out=None):
    """-> (k, v) of `dtype` [tokens, heads, D] ([layers, tokens, heads, D] for
    layer None): request b's positions starts[b], starts[b] + 1, ... for its
    output rows offsets[b] .. offsets[b + 1]."""
    c, dev, heads, dim, layers = _cache_args(cache)
    n, width = _size(starts, "starts", 1), _size(table, "table", 2)
    tp = _flat(table, _I32, "table", (n, width), dev)
    sp = _flat(starts, _I32, "starts", (n,), dev)
    op = _flat(offsets, _I32, "offsets", (n + 1,), dev)
    shape = (tokens, heads, dim) if layer is not None else (layers, tokens, heads, dim)
    if dtype not in _DTYPES:
        raise TypeError("dtype must be float16 or bfloat16")
    # the C entry reads -1 as all layers, for which `shape` has no room
    if layer is not None and layer < 0:
        raise ValueError(f"layer must be None (all layers) or at least 0, got {layer}")
    if out is None:
        # zeros where nothing is launched, as below
        make = torch.empty if n and cache[0].shape[1] else torch.zeros
        place = cache[0].device
        k, v = out = make(shape, dtype=dtype, device=place), make(shape, dtype=dtype, device=place)
        kp, vp = k.data_ptr(), v.data_ptr()
    else:
        kp = _flat(out[0], dtype, "out[0]", shape, dev)
        vp = _flat(out[1], dtype, "out[1]", shape, dev)
        if not n or not cache[0].numel():   # nothing is launched for an empty problem
            out[0].zero_()
            out[1].zero_()
    _launch((_lib or _load()).cider_kv_read, dev, (c, -1 if layer is None else layer, tp, width, sp,
            op, n, tokens, kp, vp, _DTYPES[dtype], _raw_stream(dev)))
    return out


def cider_kv_compact(cache, table, starts, path, kept) -> None:
    """In every layer, move request b's row at position starts[b] + path[b, i]
    to starts[b] + i for i < kept[b]."""
    c, dev, _, _, _ = _cache_args(cache)
    n, width, most = _size(starts, "starts", 1), _size(table, "table", 2), _size(path, "path", 2)
    tp = _flat(table, _I32, "table", (n, width), dev)
    sp = _flat(starts, _I32, "starts", (n,), dev)
    pp = _flat(path, _I32, "path", (n, most), dev)
    kp = _flat(kept, _I32, "kept", (n,), dev)
    _launch((_lib or _load()).cider_kv_compact, dev, (c, tp, width, sp, pp, most, kp, n,
            _raw_stream(dev)))


def cider_tree_attention(q, cache, table, lengths, offsets, max_nodes: int, tree=None, scale=None,
                         layer: int = 0, out=None):
    """Attention of each request's last tokens q [tokens, q_heads, D] over its
    cached positions (lengths int32 [requests], the new tokens included).
    tree int64 [tokens]: which of its request's new tokens a token sees (None:
    itself and the earlier ones).  -> out [tokens, q_heads, D] of q's type; rows
    that no request owns are zeros."""
    c, dev, heads, dim, _ = _cache_args(cache)
    dt, qs = _rows(q, "q", None, dim, dev)
    shape = q.shape
    n, b, width = shape[0], _size(lengths, "lengths", 1), _size(table, "table", 2)
    tp = _flat(table, _I32, "table", (b, width), dev)
    lp = _flat(lengths, _I32, "lengths", (b,), dev)
    op = _flat(offsets, _I32, "offsets", (b + 1,), dev)
    mp = None if tree is None else _flat(tree, _I64, "tree", (n,), dev)
    if out is None:
        out = torch.empty(shape, dtype=q.dtype, device=q.device)
        yp = out.data_ptr()
    else:
        yp = _flat(out, q.dtype, "out", shape, dev)
    if not b or not cache[0].numel():   # nothing is launched for an empty problem
        return out.zero_()
    _launch((_lib or _load()).cider_tree_attention, dev, (c, layer, q.data_ptr(), qs, dt, n,
            shape[1], tp, width, lp, op, b, max_nodes, mp, dim ** -0.5 if scale is None else scale,
            yp, _raw_stream(dev)))
    return out


def cider_verify_drafts(logits, tokens, parents, offsets, uniforms, noise, max_nodes: int,
                        draft_probs=None, temperature=None):
    """Accept or reject each request's drafted tokens against the target's
    logits [nodes, vocab] (fp16 or bf16, any row stride), with the given random
    numbers.  -> (count int32 [requests], path int32 [requests, max_nodes],
    next int32 [requests])."""
    if not getattr(logits, "is_cuda", False):
        raise TypeError("logits must be a CUDA tensor")
    dev = logits.get_device()
    if logits.dtype not in _DTYPES:
        raise TypeError("logits must be float16 or bfloat16")
    vocab = _size(logits, "logits", 2)
    n = logits.shape[0]
    stride, one = logits.stride()
    if one != 1 and vocab > 1:
        raise ValueError("logits must have contiguous rows")
    b = _size(offsets, "offsets", 1) - 1
    tp = _flat(tokens, _I32, "tokens", (n,), dev)
    pp = _flat(parents, _I32, "parents", (n,), dev)
    op = _flat(offsets, _I32, "offsets", (b + 1,), dev)
    up = _flat(uniforms, _F32, "uniforms", (n,), dev)
    ep = _flat(noise, _F32, "noise", (b, vocab), dev)
    dp = None if draft_probs is None else _flat(draft_probs, _F32, "draft_probs", (n, vocab), dev)
    wp = None if temperature is None else _flat(temperature, _F32, "temperature", (b,), dev)
    place = logits.device
    path = torch.empty((b, max_nodes), dtype=_I32, device=place)
    count = torch.empty((b,), dtype=_I32, device=place)
    nxt = torch.empty((b,), dtype=_I32, device=place)
    _launch((_lib or _load()).cider_verify_drafts, dev, (logits.data_ptr(),
            stride if n > 1 else vocab, _DTYPES[logits.dtype], tp, pp, op, b, n, vocab, max_nodes,
            up, ep, dp, wp, count.data_ptr(), path.data_ptr(), nxt.data_ptr(), _raw_stream(dev)))
    return count, path, nxt


# ------------------------------------------ microscaled 4-bit floating point
_FP4 = struct.Struct("@PPPqqi4x")   # cider_fp4_t
_ACTIVATIONS = {"silu": 0, "gelu": 1}
_WIDE = {torch.float16: CIDER_F16, torch.bfloat16: CIDER_BF16, torch.float32: CIDER_F32}


def _refuse_fp4(q, block_size, name):
    if block_size not in (16, 32):
        raise ValueError(f"block_size must be 16 or 32, got {block_size}")
    if not isinstance(q, (tuple, list)) or len(q) != 3:
        raise TypeError(f"{name} must be (codes, scales, row_scale)")
    codes, scales, row = q
    for t, part in ((codes, "codes"), (scales, "scales")) + (((row, "row_scale"),) if row is not None else ()):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name}'s {part} must be a CUDA tensor")
    if codes.dtype != _U8 or scales.dtype != _U8:
        raise TypeError(f"{name}'s codes and scales must be uint8")
    if row is not None and row.dtype != _F32:
        raise TypeError(f"{name}'s row_scale must be float32")
    if codes.dim() != 2:
        raise ValueError(f"{name}'s codes must have 2 dimensions, got shape {tuple(codes.shape)}")
    if not all(t is None or t.is_contiguous() for t in q):
        raise ValueError(f"{name} must be contiguous")
    if any(t is not None and t.get_device() != codes.get_device() for t in q):
        raise ValueError(f"{name}'s tensors are on different devices")
    rows, cols = codes.shape[0], 2 * codes.shape[1]
    raise ValueError(f"{name}: codes {tuple(codes.shape)} of block size {block_size} need scales "
                     f"{_scale_shape(rows, cols, block_size)} and row_scale {(rows,)} (or None), got "
                     f"{tuple(scales.shape)} and {None if row is None else tuple(row.shape)}")


def _scale_shape(rows, cols, block_size):
    return (rows + 127) // 128, -(-cols // (4 * block_size)), 512


def _fp4_args(q, block_size, name, dev=None):
    """-> (cider_fp4_t as bytes, device index, rows, cols)."""
    try:
        codes, scales, row = q
        rows, half = codes.shape
        place = codes.get_device()
        if not (codes.dtype is _U8 and scales.dtype is _U8 and place >= 0 and scales.get_device() == place
                and (block_size == 16 or block_size == 32)
                and scales.shape == ((rows + 127) >> 7, -(-half // (2 * block_size)), 512)
                and codes.is_contiguous() and scales.is_contiguous()
                and (row is None or (row.dtype is _F32 and row.shape == (rows,) and row.get_device() == place
                                     and row.is_contiguous()))):
            _refuse_fp4(q, block_size, name)
    except (AttributeError, TypeError, ValueError):   # not a triple of tensors
        _refuse_fp4(q, block_size, name)
    if dev is not None and place != dev:
        raise ValueError(f"{name} is on another device")
    return (_FP4.pack(codes.data_ptr(), scales.data_ptr(), 0 if row is None else row.data_ptr(), rows, 2 * half,
                      block_size), place, rows, 2 * half)


def _wide_rows(x, cols, kinds, dev):
    """Type, row stride and rows of a matrix [rows, cols] with dense rows on this device (None: any)."""
    try:
        kind, place = kinds[x.dtype], x.get_device()
        n, k = x.shape
        stride, one = x.stride()
        if (one == 1 or k == 1) and (cols is None or k == cols) and place >= 0 and (dev is None or place == dev):
            return kind, stride if n > 1 else k, n
    except (AttributeError, KeyError, ValueError):
        pass
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError("x must be a CUDA tensor")
    if x.dtype not in kinds:
        raise TypeError(f"x must be one of {', '.join(str(t) for t in kinds)}, got {x.dtype}")
    if x.dim() != 2 or (cols is not None and x.shape[1] != cols):
        raise ValueError(f"x must have shape [rows, {'cols' if cols is None else cols}], got {tuple(x.shape)}")
    if x.stride(1) != 1:
        raise ValueError("x must have contiguous rows")
    raise ValueError("x is on another device")


def _result(out, shape, dtype, like, name):
    """The given output, or a new one on the device of `like`, and its pointer."""
    if dtype not in _DTYPES:
        raise TypeError(f"{name}'s type must be float16 or bfloat16")
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=like.device)
        return out, out.data_ptr()
    return out, _flat(out, dtype, name, shape, like.get_device())


def cider_quantize_fp4(x: torch.Tensor, block_size: int = 32):
    """x fp16, bf16 or fp32 [rows, cols] (any row stride) -> (codes uint8 [rows, cols / 2],
    scales uint8 [ceil(rows / 128), ceil(cols / (4 block_size)), 512], row_scale):
    4-bit floating point (E2M1) with an E8M0 scale per 32 values (row_scale None),
    or an E4M3 scale per 16 values and row_scale fp32 [rows]."""
    if block_size not in (16, 32):
        raise ValueError(f"block_size must be 16 or 32, got {block_size}")
    kind, stride, rows = _wide_rows(x, None, _WIDE, None)
    cols, place = x.shape[1], x.device
    q = (torch.empty((rows, cols // 2), dtype=_U8, device=place),
         torch.empty(_scale_shape(rows, cols, block_size), dtype=_U8, device=place),
         torch.empty((rows,), dtype=_F32, device=place) if block_size == 16 else None)
    c = _FP4.pack(q[0].data_ptr(), q[1].data_ptr(), 0 if q[2] is None else q[2].data_ptr(), rows, cols, block_size)
    dev = x.get_device()
    _launch((_lib or _load()).cider_quantize_fp4, dev, (x.data_ptr(), kind, stride, c, _raw_stream(dev)))
    return q


def cider_dequantize_fp4(q, block_size: int = 32, dtype=torch.float16, out=None):
    """The values of a quantized matrix (codes, scales, row_scale) -> [rows, cols] of
    `dtype` (fp16, bf16 or fp32)."""
    c, dev, rows, cols = _fp4_args(q, block_size, "q")
    if dtype not in _WIDE:
        raise TypeError("dtype must be float16, bfloat16 or float32")
    if out is None:
        out = torch.empty((rows, cols), dtype=dtype, device=q[0].device)
        xp = out.data_ptr()
    else:
        xp = _flat(out, dtype, "out", (rows, cols), dev)
    _launch((_lib or _load()).cider_dequantize_fp4, dev, (c, xp, _WIDE[dtype], _raw_stream(dev)))
    return out


def cider_w4a4_linear(x, w, block_size: int = 32, y_dtype=None, out=None):
    """y [M, N] of y_dtype (None: x's) = x w^T for x fp16 or bf16 [M, K] (any row
    stride), quantized by the call, and w = cider_quantize_fp4(weights [N, K])."""
    c, dev, n, k = _fp4_args(w, block_size, "w")
    kind, stride, m = _wide_rows(x, k, _DTYPES, dev)
    y_dtype = x.dtype if y_dtype is None else y_dtype
    y, yp = _result(out, (m, n), y_dtype, w[0], "out")
    _launch((_lib or _load()).cider_w4a4_linear, dev, (x.data_ptr(), kind, stride, m, c, yp, _DTYPES[y_dtype],
            _raw_stream(dev)))
    return y


def cider_w4a4_linear_prequant(qx, w, block_size: int = 32, y_dtype=torch.float16, out=None):
    """As cider_w4a4_linear for rows that cider_quantize_fp4 has quantized already."""
    c, dev, n, k = _fp4_args(w, block_size, "w")
    a, _, m, kx = _fp4_args(qx, block_size, "qx", dev)
    if kx != k:
        raise ValueError(f"qx has {kx} columns, w {k}")
    y, yp = _result(out, (m, n), y_dtype, w[0], "out")
    _launch((_lib or _load()).cider_w4a4_linear_prequant, dev, (a, c, yp, _DTYPES[y_dtype], _raw_stream(dev)))
    return y


def _gate_up(gate, up, block_size, activation):
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation must be one of {', '.join(_ACTIVATIONS)}, got {activation!r}")
    g, dev, f, k = _fp4_args(gate, block_size, "gate")
    u, _, fu, ku = _fp4_args(up, block_size, "up", dev)
    if (fu, ku) != (f, k):
        raise ValueError(f"gate is {f} x {k}, up {fu} x {ku}")
    return g, u, dev, f, k, _ACTIVATIONS[activation]


def cider_w4a4_gated_linear(x, gate, up, block_size: int = 32, activation="silu", h_dtype=None, out=None):
    """h [M, F] of h_dtype (None: x's) = act(x gate^T) * (x up^T): the first half of a
    gated feed-forward block.  activation: "silu", or "gelu" (by its tanh form)."""
    g, u, dev, f, k, act = _gate_up(gate, up, block_size, activation)
    kind, stride, m = _wide_rows(x, k, _DTYPES, dev)
    h_dtype = x.dtype if h_dtype is None else h_dtype
    h, hp = _result(out, (m, f), h_dtype, gate[0], "out")
    _launch((_lib or _load()).cider_w4a4_gated_linear, dev, (x.data_ptr(), kind, stride, m, g, u, act, hp,
            _DTYPES[h_dtype], _raw_stream(dev)))
    return h


def cider_w4a4_gated_linear_prequant(qx, gate, up, block_size: int = 32, activation="silu",
                                     h_dtype=torch.float16, out=None):
    """As cider_w4a4_gated_linear for rows that cider_quantize_fp4 has quantized already."""
    g, u, dev, f, k, act = _gate_up(gate, up, block_size, activation)
    a, _, m, kx = _fp4_args(qx, block_size, "qx", dev)
    if kx != k:
        raise ValueError(f"qx has {kx} columns, gate {k}")
    h, hp = _result(out, (m, f), h_dtype, gate[0], "out")
    _launch((_lib or _load()).cider_w4a4_gated_linear_prequant, dev, (a, g, u, act, hp, _DTYPES[h_dtype],
            _raw_stream(dev)))
    return h


def cider_w4a4_feed_forward(x, gate, up, down, block_size: int = 32, activation="silu", y_dtype=None, out=None):
    """y [M, N] of y_dtype (None: x's) = h down^T, h = act(x gate^T) * (x up^T) rounded
    to x's type and quantized: a whole gated feed-forward block."""
    g, u, dev, f, k, act = _gate_up(gate, up, block_size, activation)
    d, _, n, fd = _fp4_args(down, block_size, "down", dev)
    if fd != f:
        raise ValueError(f"down has {fd} columns, gate {f} rows")
    kind, stride, m = _wide_rows(x, k, _DTYPES, dev)
    y_dtype = x.dtype if y_dtype is None else y_dtype
    y, yp = _result(out, (m, n), y_dtype, gate[0], "out")
    _launch((_lib or _load()).cider_w4a4_feed_forward, dev, (x.data_ptr(), kind, stride, m, g, u, d, act, yp,
            _DTYPES[y_dtype], _raw_stream(dev)))
    return y
