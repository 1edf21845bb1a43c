"""The entry points of 4-bit floating point over recording launchers (tests/fp4_calls.cu): which kernels a call launches,
and on which memory."""
import ctypes
import functools
import os
import subprocess
import tempfile

from w4a8_quantized_linear_gb300 import _build

HERE = os.path.dirname(os.path.abspath(__file__))
SCRATCH, QUANTIZE, FEW, PAIRS = range(4)
NAMES = ("kind bytes wide codes scales row y to_codes to_scales to_row stride m n k gated dependent").split()


class Record(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in NAMES]


class Fp4(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("row_scale", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("block_size", ctypes.c_int32)]


@functools.cache
def library():
    with tempfile.TemporaryDirectory() as d:
        out = os.path.join(d, "calls.so")
        subprocess.run([_build._nvcc(), *_build.ARCH, *_build.NVCC_FLAGS, "-I", _build.CSRC, "-shared", "-o", out,
                        os.path.join(HERE, "fp4_calls.cu")], check=True, capture_output=True)
        loaded = ctypes.CDLL(out)
    p, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    loaded.calls_begin.argtypes = [i64, i32, i32]
    loaded.calls_records.restype = p
    loaded.cider_w4a4_linear.argtypes = [p, i32, i64, i64, p, p, i32, p]
    loaded.cider_w4a4_gated_linear.argtypes = [p, i32, i64, i64, p, p, i32, p, i32, p]
    loaded.cider_w4a4_feed_forward.argtypes = [p, i32, i64, i64, p, p, p, i32, p, i32, p]
    return loaded


def weights(rows, cols, block):
    """A matrix far away from everything else."""
    far = 0x100000000000
    return Fp4(far, far + (1 << 40), None, rows, cols, block)


def made(lib):
    """What the launchers have written down since calls_begin."""
    n = lib.calls_made()
    return [Record.from_buffer_copy(r) for r in (Record * n).from_address(lib.calls_records())] if n else []


def product_kernels(m, n, k, block, gated, sms):
    """The kernel (FEW or PAIRS) of a linear or gated product of m tokens."""
    lib = library()
    w = weights(n, k, block)
    lib.calls_begin(0x700000000000, sms, 0)
    x, y, r = 0x200000000000, 0x300000000000, ctypes.byref
    status = (lib.cider_w4a4_gated_linear(x, 0, k, m, r(w), r(w), 0, y, 0, None) if gated
              else lib.cider_w4a4_linear(x, 0, k, m, r(w), y, 0, None))
    assert status == 0
    return made(lib)[-1].kind


def first_on_pairs(n, k, block, gated, sms):
    """The fewest tokens whose product runs on pairs."""
    m = 1
    while product_kernels(m, n, k, block, gated, sms) != PAIRS:
        m += 1
    return m
