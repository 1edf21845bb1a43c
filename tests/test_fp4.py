"""Microscaled 4-bit floating point: quantization bit for bit, products against
64 bits, refusals."""
import ctypes
import zlib

import pytest
import torch

import w4a8_quantized_linear_gb300 as cider
from tests import fp4_reference as ref

gpu = pytest.mark.gpu
TYPES = [torch.float16, torch.bfloat16, torch.float32]
OK, INVALID, MISALIGNED, UNSUPPORTED = 0, 1, 2, 3


def normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def generator(*key):
    return torch.Generator(device="cuda").manual_seed(zlib.crc32(repr(key).encode()))


def activations(gen, rows, cols, dtype=torch.float32):
    x = normal(gen, rows, cols)
    x[:, torch.randperm(cols, generator=gen, device="cuda")[: max(1, cols // 50)]] *= 20
    return x.to(dtype)


def clean():
    assert cider.cider_check_device_error() == 0


# ------------------------------------------------------------ the reference itself
def test_reference_grids_and_powers():
    assert ref.VALUES.tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    g = ref.e4m3_grid()
    assert len(g) == 127 and g[-1] == 448 and bool((g[1:] > g[:-1]).all())
    assert torch.equal(g, torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double())
    q = torch.tensor([0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.1, 9.0], dtype=torch.float64)
    assert ref.nearest(q, ref.VALUES).tolist() == [0, 1, 2, 2, 4, 4, 6, 6, 7, 7]
    a = torch.tensor([6.0, 6.0001, 3.0, 3.0001, 2688.0, 1e-44], dtype=torch.float64)
    assert ref.power_at_least(a, 6.0, -127).tolist() == [0, 1, -1, 0, 9, -127]


# ------------------------------------------------------------ quantization
@gpu
@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 64), (3, 96), (127, 512), (129, 544), (130, 2080), (2, 16384), (3, 16416),
                                       (257, 4096)])
def test_quantize_bit_for_bit(rows, cols, dtype, block):
    gen = generator(rows, cols, str(dtype), block)
    x = normal(gen, rows, cols) * torch.exp(normal(gen, rows, 1))
    x[:, cols // 3] *= 50
    x[rows // 2] = 0
    x[-1, :32] = 0
    x = x.to(dtype)
    q = cider.cider_quantize_fp4(x, block)
    codes, held, row = ref.quantize(x, block)
    assert torch.equal(q[1], ref.tiles(held))
    assert (q[2] is None) == (row is None) and (row is None or torch.equal(q[2], row))
    got = torch.stack((q[0] & 15, q[0] >> 4), -1).flatten(1).long()
    assert torch.equal(got, codes)
    for back in TYPES:
        v = cider.cider_dequantize_fp4(q, block, back)
        # code x scale is exact in 32 bits, and so is the product with a power of two
        assert torch.equal(v, ref.values(q, block).float().to(back))
    clean()


@gpu
@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows,cols", [(5, 4064), (1300, 4128), (700, 8160), (350, 12320), (3, 16416), (200, 20512), (2, 32768),
                                       (3, 32800)])
def test_quantize_long_rows_bit_for_bit(rows, cols, dtype, block):
    gen = generator(rows, cols, str(dtype), block)
    wide = (normal(gen, rows, cols + 32) * torch.exp(normal(gen, rows, 1))).to(dtype)
    x = wide[:, 16:16 + cols]
    x[:, cols // 3] *= 50
    x[rows // 2, cols // 2:] = 0
    x[0, cols - 1] = 400   # the last unit holds the row's maximum
    q = cider.cider_quantize_fp4(x, block)
    codes, held, row = ref.quantize(x, block)
    assert torch.equal(q[1], ref.tiles(held))
    assert (q[2] is None) == (row is None) and (row is None or torch.equal(q[2], row))
    assert torch.equal(torch.stack((q[0] & 15, q[0] >> 4), -1).flatten(1).long(), codes)
    clean()


@gpu
@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_quantize_edges(dtype, block):
    """Ties of every code, the largest and the smallest numbers, borders of the scales, signed zeros."""
    big = torch.finfo(dtype).max
    tiny = torch.finfo(dtype).tiny
    rows = []
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0]
    for s in (1.0, 0.75, 1.125, 1.875, 2.0 ** -10, 1344.0):
        rows.append([t * s for t in ties] * 2 + [-t * s for t in ties] * 2)
    rows.append([2688.0] + [6.0 * 2.0 ** -9 * j for j in range(31)])
    rows.append([2704.0] + [0.01 * j for j in range(31)])
    rows.append([big, -big] + [1.0] * 30)
    rows.append([tiny, -tiny] + [tiny / 4] * 30)
    rows.append([-0.0, 0.0] * 16)
    rows.append([6.0, 3.0, 12.0, 1.5] * 8)
    rows.append([6.0 + 6.0 / 128] + [3.0] * 31)
    x = torch.tensor(rows, dtype=torch.float64).to(dtype).cuda()
    x = torch.cat((x, x.flip(0)), 1).contiguous()
    q = cider.cider_quantize_fp4(x, block)
    codes, held, row = ref.quantize(x, block)
    assert torch.equal(q[1], ref.tiles(held))
    assert row is None or torch.equal(q[2], row)
    assert torch.equal(torch.stack((q[0] & 15, q[0] >> 4), -1).flatten(1).long(), codes)
    clean()


@gpu
@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("cols", [64, 16416])
def test_not_finite_values_make_their_block_or_row_nan(block, value, cols):
    gen = generator(block, str(value), cols)
    x = normal(gen, 5, cols).half()
    x[2, 37] = value
    q = cider.cider_quantize_fp4(x, block)
    v = cider.cider_dequantize_fp4(q, block, torch.float32)
    want = torch.zeros_like(v, dtype=torch.bool)
    want[2, slice(None) if block == 16 else slice(32, 64)] = True
    assert torch.equal(torch.isnan(v), want)
    # and the outputs that need it; the others are numbers, or infinite where 16 bits do not hold them (a product of two
    # sums of 16416 products of size one passes 65504)
    w = ref.matrix(normal(gen, 24, cols), block)
    y = cider.cider_w4a4_linear(x, w, block)
    assert bool(torch.isnan(y[2]).all()) and not bool(torch.isnan(y[[0, 1, 3, 4]]).any())
    h = cider.cider_w4a4_gated_linear(x, w, w, block)
    assert bool(torch.isnan(h[2]).all()) and not bool(torch.isnan(h[[0, 1, 3, 4]]).any())
    clean()


@gpu
@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_quantize_strided_rows(dtype, block):
    gen = generator(str(dtype), block)
    both = normal(gen, 70, 3 * 160).to(dtype)
    x = both[:, 160:320]
    a, b = cider.cider_quantize_fp4(x, block), cider.cider_quantize_fp4(x.contiguous(), block)
    assert all(s is t or torch.equal(s, t) for s, t in zip(a, b))
    w = ref.matrix(normal(gen, 40, 160), block)
    if dtype != torch.float32:
        assert torch.equal(cider.cider_w4a4_linear(x, w, block), cider.cider_w4a4_linear(x.contiguous(), w, block))
        last = both[69:, 160:320]
        assert torch.equal(cider.cider_w4a4_linear(last, w, block), cider.cider_w4a4_linear(last.clone(), w, block))
    clean()


# ------------------------------------------------------------ products
@gpu
@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("m,n,k", [(1, 8, 32), (1, 128, 64), (16, 136, 96), (17, 264, 256), (100, 120, 160), (129, 256, 288),
                                   (130, 520, 512), (300, 392, 544)])
def test_linear_of_exact_values(m, n, k, block):
    """Values that four bits hold: nothing is rounded but the output, so it is exact."""
    gen = generator(m, n, k, block)
    pick = lambda r: ref.VALUES.float().cuda()[torch.randint(0, 8, (r, k), generator=gen, device="cuda")] * (
        1 - 2 * torch.randint(0, 2, (r, k), generator=gen, device="cuda"))
    x, w = pick(m), pick(n)
    x[:, ::16], w[:, ::16] = 6.0, -6.0
    y = cider.cider_w4a4_linear(x.half(), cider.cider_quantize_fp4(w, block), block, y_dtype=torch.bfloat16)
    assert torch.equal(y, (x.double() @ w.double().T).float().bfloat16())
    clean()


def close(y, want, bound):
    bad = (y.double() - want).abs() > bound
    assert not bool(bad.any()), (int(bad.sum()), float(((y.double() - want).abs() / bound).max()))


@gpu
@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("dtype", TYPES[:2], ids=str)
@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 33, 64, 65, 127, 128, 129, 200, 256, 257, 300, 513])
@pytest.mark.parametrize("n,k", [(8, 32), (200, 2080), (1000, 736)])
def test_linear(m, n, k, dtype, block):
    gen = generator(m, n, k, str(dtype), block)
    x, w = activations(gen, m, k, dtype), ref.matrix(0.05 * normal(gen, n, k), block)
    y = cider.cider_w4a4_linear(x, w, block)
    a, b = ref.values(ref.matrix(x, block), block), ref.values(w, block)
    want = a @ b.T
    close(y, want, ref.sum_bound(a, b) + ref.half_step(dtype, want) * (1 + 2.0 ** -10))
    clean()


@gpu
@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("m", [1, 16, 31, 100, 128, 130, 256, 260, 513])
@pytest.mark.parametrize("f,k", [(8, 64), (392, 1056), (136, 2080)])
def test_gated_linear(m, f, k, act, block):
    gen = generator(m, f, k, act, block)
    dtype = torch.float16 if (m + f) % 3 else torch.bfloat16
    x = activations(gen, m, k, dtype)
    gate, up = (ref.matrix(0.03 * normal(gen, f, k), block) for _ in range(2))
    h = cider.cider_w4a4_gated_linear(x, gate, up, block, act)
    a, gv, uv = (ref.values(q, block) for q in (ref.matrix(x, block), gate, up))
    g, u = a @ gv.T, a @ uv.T
    eg, eu = ref.sum_bound(a, gv), ref.sum_bound(a, uv)
    want = ref.activate(g, act) * u
    # the activation's slope is at most 1.13; e^x and the reciprocal are off by 2 ulp each, e^x's argument (with t's
    # cube, |t| grows at most three times as fast as g) by a few ulp of itself, at most 128 before the result vanishes
    bound = 1.13 * eg * (u.abs() + eu) + ref.activate(g.abs(), act).abs() * eu + want.abs() * 2.0 ** -14 + 2.0 ** -40
    close(h, want, bound + ref.half_step(dtype, want) * (1 + 2.0 ** -10))
    clean()


@gpu
@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("m,k,f,n", [(1, 64, 96, 8), (16, 512, 288, 200), (61, 416, 1056, 416), (128, 256, 512, 256), (129, 256, 512, 256),
                                     (300, 288, 544, 264)])
def test_feed_forward_is_its_two_products(m, k, f, n, block):
    gen = generator(m, k, f, n, block)
    for dtype, y_dtype, act in ((torch.float16, torch.float16, "silu"), (torch.bfloat16, torch.float16, "gelu")):
        x = activations(gen, m, k, dtype)
        gate, up = (cider.cider_quantize_fp4(0.03 * normal(gen, f, k), block) for _ in range(2))
        down = cider.cider_quantize_fp4(0.03 * normal(gen, n, f), block)
        y = cider.cider_w4a4_feed_forward(x, gate, up, down, block, act, y_dtype=y_dtype)
        h = cider.cider_w4a4_gated_linear(x, gate, up, block, act)
        assert torch.equal(y, cider.cider_w4a4_linear(h, down, block, y_dtype=y_dtype))
        qh = cider.cider_quantize_fp4(h, block)
        a, b = ref.values(ref.matrix(h, block), block), ref.values(down, block)
        assert torch.equal(ref.values(qh, block), a)
        close(y, a @ b.T, ref.sum_bound(a, b) + ref.half_step(y_dtype, a @ b.T) * (1 + 2.0 ** -10))
    clean()


@gpu
@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("m", [1, 40, 200, 700])
def test_quantized_input_shared_by_projections(m, block):
    gen = generator(m, block)
    x = activations(gen, m, 512, torch.bfloat16)
    a, b = (cider.cider_quantize_fp4(0.05 * normal(gen, 264, 512), block) for _ in range(2))
    qx = cider.cider_quantize_fp4(x, block)
    assert torch.equal(cider.cider_w4a4_linear_prequant(qx, a, block, torch.bfloat16), cider.cider_w4a4_linear(x, a, block))
    assert torch.equal(cider.cider_w4a4_gated_linear_prequant(qx, a, b, block, "gelu", torch.bfloat16),
                       cider.cider_w4a4_gated_linear(x, a, b, block, "gelu"))
    clean()


@gpu
@pytest.mark.parametrize("m", [3, 150])
def test_given_row_scales_and_none(m):
    """Any positive row scales, on either block size; None counts as ones."""
    gen = generator(m)
    x, w = activations(gen, m, 288), 0.05 * normal(gen, 72, 288)
    for block in (16, 32):
        (xc, xs, _), (wc, ws, _) = ref.matrix(x, block), ref.matrix(w, block)
        rx, rw = torch.rand(m, generator=gen, device="cuda") + 0.3, torch.rand(72, generator=gen, device="cuda") + 0.3
        for qx, qw in (((xc, xs, rx), (wc, ws, rw)), ((xc, xs, None), (wc, ws, rw)), ((xc, xs, None), (wc, ws, None))):
            # without their row scales the sums of block size 16 pass what fp16 holds
            y = cider.cider_w4a4_linear_prequant(qx, qw, block, torch.bfloat16)
            a, b = ref.values(qx, block), ref.values(qw, block)
            close(y, a @ b.T, ref.sum_bound(a, b) + ref.half_step(torch.bfloat16, a @ b.T) * (1 + 2.0 ** -10))
    clean()


@gpu
@pytest.mark.parametrize("m", [1, 20, 128, 300])
def test_outputs_stay_inside_their_rows(m):
    gen = generator(m)
    x, w = activations(gen, m, 96, torch.float16), cider.cider_quantize_fp4(normal(gen, 40, 96))
    room = torch.full((m * 40 + 128,), 7.0, dtype=torch.float16, device="cuda")
    y = cider.cider_w4a4_linear(x, w, out=room[64 : 64 + m * 40].view(m, 40))
    assert bool((room[:64] == 7).all()) and bool((room[64 + m * 40 :] == 7).all())
    assert torch.equal(y, cider.cider_w4a4_linear(x, w))
    h = cider.cider_w4a4_gated_linear(x, w, w, out=room[64 : 64 + m * 40].view(m, 40))
    assert bool((room[:64] == 7).all()) and bool((room[64 + m * 40 :] == 7).all())
    assert torch.equal(h, cider.cider_w4a4_gated_linear(x, w, w))
    clean()


@gpu
@pytest.mark.parametrize("m", [1, 61, 400])
def test_captured_replayed_and_on_two_streams(m):
    """A block's calls in a graph, replayed with other inputs, beside the same calls on another stream."""
    gen = generator(m)
    k, f = 512, 768
    gate, up = (cider.cider_quantize_fp4(0.03 * normal(gen, f, k), 16) for _ in range(2))
    down = cider.cider_quantize_fp4(0.03 * normal(gen, k, f), 16)
    xs = [activations(gen, m, k, torch.bfloat16) for _ in range(4)]
    want = [cider.cider_w4a4_feed_forward(x, gate, up, down, 16) for x in xs]
    x = xs[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = cider.cider_w4a4_feed_forward(x, gate, up, down, 16)
    for i in range(8):
        x.copy_(xs[i % 4])
        graph.replay()
        with torch.cuda.stream(side):
            z = cider.cider_w4a4_feed_forward(xs[3 - i % 4], gate, up, down, 16)
        torch.cuda.synchronize()
        assert torch.equal(y, want[i % 4]) and torch.equal(z, want[3 - i % 4])
    clean()


@gpu
@pytest.mark.parametrize("block", [16, 32])
def test_empty(block):
    w = cider.cider_quantize_fp4(torch.ones(40, 64, device="cuda"), block)
    none = cider.cider_quantize_fp4(torch.ones(0, 64, device="cuda"), block)
    assert none[0].shape == (0, 32) and none[1].shape[0] == 0
    x = torch.ones(3, 64, dtype=torch.float16, device="cuda")
    assert cider.cider_w4a4_linear(x[:0], w, block).shape == (0, 40)
    assert cider.cider_w4a4_linear(x, none, block).shape == (3, 0)
    assert cider.cider_w4a4_linear_prequant(none, w, block).shape == (0, 40)
    assert cider.cider_w4a4_gated_linear(x[:0], w, w, block).shape == (0, 40)
    assert cider.cider_dequantize_fp4(none, block).shape == (0, 64)
    clean()


# ------------------------------------------------------------ refusals
class Fp4(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("row_scale", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("block_size", ctypes.c_int32)]


def mat(rows=128, cols=64, block=32, **kw):
    f = dict(codes=4096, scales=8192, row_scale=None, rows=rows, cols=cols, block_size=block)
    f.update(kw)
    return Fp4(**f)


@pytest.fixture
def lib(monkeypatch):
    from w4a8_quantized_linear_gb300 import _build
    _build.build()
    monkeypatch.setenv("CIDER_FORCE_UNSUPPORTED", "1")
    return cider.library()


def test_struct_size():
    assert ctypes.sizeof(Fp4) == cider._FP4.size


@pytest.mark.parametrize("bad", [dict(codes=None), dict(scales=None), dict(rows=-1), dict(cols=0), dict(cols=48), dict(cols=16),
                                 dict(cols=131104), dict(block=8), dict(block=64)], ids=str)
def test_matrices_that_are_refused(lib, bad):
    r = ctypes.byref
    q = mat(**bad)
    assert lib.cider_quantize_fp4(4096, 0, 131104, r(q), None) == INVALID
    assert lib.cider_dequantize_fp4(r(q), 4096, 0, None) == INVALID
    if bad.get("rows") != -1:
        assert lib.cider_w4a4_linear(4096, 0, 131104, 4, r(q), 4096, 0, None) == INVALID
    assert lib.cider_w4a4_linear_prequant(r(q), r(mat()), 4096, 0, None) == INVALID
    assert lib.cider_w4a4_gated_linear(4096, 0, 64, 4, r(mat()), r(q), 0, 4096, 0, None) == INVALID


def test_arguments_that_are_refused(lib):
    r = ctypes.byref
    w, other, odd = mat(), mat(block=16), mat(rows=100)
    quant, linear = lib.cider_quantize_fp4, lib.cider_w4a4_linear
    assert quant(4096, 0, 64, r(w), None) == UNSUPPORTED
    assert quant(4096, 2, 64, r(w), None) == UNSUPPORTED
    assert quant(4096, 3, 64, r(w), None) == INVALID
    assert quant(4096, 0, 60, r(w), None) == INVALID
    assert quant(4096, 0, 68, r(w), None) == INVALID       # 136 bytes
    assert quant(4096, 2, 68, r(w), None) == UNSUPPORTED   # 272 bytes
    assert quant(None, 0, 64, r(w), None) == INVALID
    assert quant(4096, 0, 64, None, None) == INVALID
    assert quant(4096, 0, 64, r(mat(row_scale=4096)), None) == INVALID     # a scale that block size 32 does not have
    assert quant(4096, 0, 64, r(other), None) == INVALID                   # none where 16 has one
    assert quant(4096, 0, 64, r(mat(block=16, row_scale=4098)), None) == MISALIGNED
    assert quant(4104, 0, 64, r(w), None) == MISALIGNED
    assert quant(4096, 0, 64, r(mat(codes=4104)), None) == MISALIGNED
    assert linear(4096, 0, 64, 4, r(w), 4096, 1, None) == UNSUPPORTED
    assert linear(4096, 2, 64, 4, r(w), 4096, 1, None) == INVALID          # fp32 activations
    assert linear(4096, 0, 64, 4, r(w), 4096, 2, None) == INVALID
    assert linear(4096, 0, 64, -1, r(w), 4096, 0, None) == INVALID
    assert linear(4096, 0, 64, 4, r(odd), 4096, 0, None) == INVALID        # N % 8
    assert linear(4096, 0, 64, 4, r(w), None, 0, None) == INVALID
    assert linear(4096, 0, 64, 4, None, 4096, 0, None) == INVALID
    assert linear(4096, 0, 64, 4, r(w), 4104, 0, None) == MISALIGNED
    assert linear(4096, 0, 64, 0, r(w), None, 0, None) == OK               # nothing to do
    assert lib.cider_w4a4_linear_prequant(r(other), r(w), 4096, 0, None) == INVALID
    assert lib.cider_w4a4_linear_prequant(r(mat(cols=96)), r(w), 4096, 0, None) == INVALID
    assert lib.cider_w4a4_linear_prequant(None, r(w), 4096, 0, None) == INVALID
    gated = lib.cider_w4a4_gated_linear
    assert gated(4096, 0, 64, 4, r(w), r(w), 1, 4096, 0, None) == UNSUPPORTED
    assert gated(4096, 0, 64, 4, r(w), r(w), 2, 4096, 0, None) == INVALID
    assert gated(4096, 0, 64, 4, r(w), r(mat(rows=136)), 0, 4096, 0, None) == INVALID
    assert gated(4096, 0, 64, 4, r(w), r(other), 0, 4096, 0, None) == INVALID
    forward = lib.cider_w4a4_feed_forward
    assert forward(4096, 0, 64, 4, r(w), r(w), r(mat(cols=128)), 0, 4096, 0, None) == UNSUPPORTED
    assert forward(4096, 0, 64, 4, r(w), r(w), r(mat(cols=96)), 0, 4096, 0, None) == INVALID
    assert forward(4096, 0, 64, 4, r(w), r(w), r(mat(cols=128, rows=100)), 0, 4096, 0, None) == INVALID
    assert forward(4096, 0, 64, 4, r(w), r(w), None, 0, 4096, 0, None) == INVALID


def test_binding_refuses_what_is_not_a_cuda_matrix():
    x = torch.ones(4, 64)
    with pytest.raises(TypeError):
        cider.cider_quantize_fp4(x)
    with pytest.raises(ValueError):
        cider.cider_quantize_fp4(x, 64)
    q = (torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(1, 1, 512, dtype=torch.uint8), None)
    for bad in (q, None, (1, 2, 3), q[:2]):
        with pytest.raises(TypeError):
            cider.cider_w4a4_linear(x, bad)
        with pytest.raises(TypeError):
            cider.cider_dequantize_fp4(bad)


@gpu
def test_binding_refusals():
    x = torch.ones(4, 256, dtype=torch.float16, device="cuda")
    w = cider.cider_quantize_fp4(torch.ones(40, 256, device="cuda"))
    w16 = cider.cider_quantize_fp4(torch.ones(40, 256, device="cuda"), 16)
    for bad in ((w, 16), (w16, 32), ((w[0], w[1][:, :1], None), 32), ((w[0][:, :64].contiguous(), w[1], None), 32),
                ((w16[0], w16[1], w16[2][:8]), 16)):
        with pytest.raises(ValueError):
            cider.cider_w4a4_linear(x, *bad)
    for bad in ((w[0].to(torch.int8), w[1], None), (w[0], w[1].to(torch.int8), None), (w16[0], w16[1], w16[2].double())):
        with pytest.raises(TypeError):
            cider.cider_w4a4_linear(x, bad)
    for bad in (x[:, :32], x[0], x.t()):
        with pytest.raises(ValueError):
            cider.cider_w4a4_linear(bad, w)
    with pytest.raises(TypeError):
        cider.cider_w4a4_linear(x.float(), w)
    with pytest.raises(TypeError):
        cider.cider_w4a4_linear(x, w, y_dtype=torch.float32)
    with pytest.raises(TypeError):
        cider.cider_w4a4_linear(x, w, out=torch.empty(4, 40, device="cuda"))
    with pytest.raises(ValueError):
        cider.cider_w4a4_linear(x, w, out=torch.empty(4, 48, dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        cider.cider_w4a4_gated_linear(x, w, w, activation="relu")
    with pytest.raises(ValueError):
        cider.cider_w4a4_gated_linear(x, w, cider.cider_quantize_fp4(torch.ones(48, 256, device="cuda")))
    with pytest.raises(cider.CiderError):   # 52 outputs: not a multiple of 8
        cider.cider_w4a4_linear(x, cider.cider_quantize_fp4(torch.ones(52, 256, device="cuda")))
    with pytest.raises(cider.CiderError):   # rows that start 8 bytes behind a 16-byte boundary
        cider.cider_quantize_fp4(torch.ones(4, 72, dtype=torch.float16, device="cuda")[:, 4:68])
    clean()


@gpu
@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("dtype", TYPES[:2], ids=str)
@pytest.mark.parametrize("m,n,k", [(1, 128, 4096), (2, 264, 10240), (5, 2560, 10240), (13, 520, 1056), (16, 256, 4096), (16, 136, 4128),
                                   (16, 2560, 10240), (3, 72, 36896), (1, 40, 131072)])
def test_few_tokens_have_the_bits_of_quantized_ones(m, n, k, dtype, block):
    """One launch that quantizes the rows itself, and two that do not: the same codes and sums."""
    gen = generator(m, n, k, str(dtype), block)
    x = activations(gen, m, k, dtype)
    x[m // 2, : min(k, 96)] = 0
    w, u = (cider.cider_quantize_fp4(0.05 * normal(gen, n, k), block) for _ in range(2))
    qx = cider.cider_quantize_fp4(x, block)
    assert torch.equal(cider.cider_w4a4_linear(x, w, block), cider.cider_w4a4_linear_prequant(qx, w, block, dtype))
    assert torch.equal(cider.cider_w4a4_gated_linear(x, w, u, block), cider.cider_w4a4_gated_linear_prequant(qx, w, u, block, "silu", dtype))
    a, b = ref.values(ref.matrix(x, block), block), ref.values(w, block)
    y = cider.cider_w4a4_linear(x, w, block)
    close(y, a @ b.T, ref.sum_bound(a, b) + ref.half_step(dtype, a @ b.T) * (1 + 2.0 ** -10))
    clean()


@gpu
@pytest.mark.parametrize("dtype", TYPES[1:], ids=str)
@pytest.mark.parametrize("power", [-125, -112, -101, -99, 60, 99, 101, 112])
def test_quantize_rows_far_from_one(dtype, power):
    """Rows whose scales, or their products with the blocks', come near the ends of fp32."""
    gen = generator(str(dtype), power)
    x = (normal(gen, 40, 96) * torch.exp2(-20 * torch.rand(40, 96, generator=gen, device="cuda"))).double()
    x = (x * 2.0 ** power).to(dtype)
    for block in (16, 32):
        q = cider.cider_quantize_fp4(x, block)
        codes, held, row = ref.quantize(x, block)
        assert torch.equal(q[1], ref.tiles(held)) and (row is None or torch.equal(q[2], row))
        assert torch.equal(torch.stack((q[0] & 15, q[0] >> 4), -1).flatten(1).long(), codes)
    clean()


@gpu
@pytest.mark.parametrize("dtype", TYPES[:2], ids=str)
@pytest.mark.parametrize("m", [1, 7, 16, 40, 128, 129, 515])
@pytest.mark.parametrize("f", [32, 96, 160, 224, 416, 1056])
def test_hidden_values_are_quantized_as_by_the_quantizer(m, f, dtype):
    """Widths that end inside a step of 64, a tile of four blocks and a tile of 128 rows; a hidden value that is not
    finite, blocks of zeros."""
    gen = generator(m, f, str(dtype))
    x = activations(gen, m, 128, dtype)
    g, u = 0.05 * normal(gen, f, 128), 0.05 * normal(gen, f, 128)
    u[: min(32, f - 1)] = 0
    g[f - 1] = 1e6 if dtype == torch.float16 else 1e30   # h passes what the type holds, where x's sum is above zero
    u[f - 1] = 1e6 if dtype == torch.float16 else 1e30
    gate, up = cider.cider_quantize_fp4(g), cider.cider_quantize_fp4(u)
    down = cider.cider_quantize_fp4(normal(gen, 40, f))
    y = cider.cider_w4a4_feed_forward(x, gate, up, down)
    h = cider.cider_w4a4_gated_linear(x, gate, up)
    want = cider.cider_w4a4_linear(h, down)
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    assert torch.equal(y.nan_to_num(), want.nan_to_num())
    clean()


@gpu
@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("m", [1, 16, 50, 128, 300])
def test_output_on_the_input(m, block):
    gen = generator(m, block)
    w, u = (cider.cider_quantize_fp4(0.05 * normal(gen, 2560, 2560), block) for _ in range(2))
    for call in (lambda x, **kw: cider.cider_w4a4_linear(x, w, block, **kw),
                 lambda x, **kw: cider.cider_w4a4_gated_linear(x, w, u, block, **kw),
                 lambda x, **kw: cider.cider_w4a4_feed_forward(x, w, u, w, block, **kw)):
        x = activations(gen, m, 2560, torch.bfloat16)
        want = call(x)
        for _ in range(3):
            z = x.clone()
            assert call(z, out=z) is z and torch.equal(z, want)
    clean()


@gpu
def test_calls_on_three_streams_at_once():
    """Kernels of every form beside each other: clusters that share SMs, pairs, quantization."""
    gen = generator(3)
    k, f = 1024, 2048
    gate, up = (cider.cider_quantize_fp4(0.03 * normal(gen, f, k), 16) for _ in range(2))
    down = cider.cider_quantize_fp4(0.03 * normal(gen, k, f), 16)
    sizes = (1, 16, 33, 100, 200, 600)
    xs = [activations(gen, m, k, torch.float16) for m in sizes]
    call = lambda x: cider.cider_w4a4_feed_forward(x, gate, up, down, 16)
    want = [call(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for i in range(40):
        for j, s in enumerate(streams):
            with torch.cuda.stream(s):
                n = (i * 5 + j * 2) % len(xs)
                got.append((n, call(xs[n])))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[n]) for n, y in got)
    clean()


@gpu
@pytest.mark.parametrize("block", [16, 32])
def test_rows_whose_offsets_pass_32_bits(block):
    """Rows of x 2^31 elements apart, matrices of more than 2^32 elements, outputs of more than 2^31."""
    gen = generator(block)
    far = torch.empty((2 << 31) + 4096, dtype=torch.float16, device="cuda")
    w = cider.cider_quantize_fp4(0.05 * normal(gen, 24, 288), block)
    x = far.as_strided((3, 288), (1 << 31, 1))
    x.copy_(activations(gen, 3, 288, torch.float16))
    near = x.contiguous()
    a, b = cider.cider_quantize_fp4(x, block), cider.cider_quantize_fp4(near, block)
    assert all(s is t or torch.equal(s, t) for s, t in zip(a, b))
    assert torch.equal(cider.cider_w4a4_linear(x, w, block), cider.cider_w4a4_linear(near, w, block))
    del far, x
    rows, cols = 33000, 131072
    big = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    big[-130:] = normal(gen, 130, cols).bfloat16()
    q = cider.cider_quantize_fp4(big, block)
    tail = big[-130:].clone()
    codes, held, row = ref.quantize(tail, block)
    assert torch.equal(torch.stack((q[0][-130:] & 15, q[0][-130:] >> 4), -1).flatten(1).long(), codes)
    assert row is None or torch.equal(q[2][-130:], row)
    back = cider.cider_dequantize_fp4(q, block, torch.bfloat16, out=big)
    mine = ref.matrix(tail, block)
    assert torch.equal(back[-130:].double(), ref.values(mine, block))
    # the weights' last rows, through both kernels
    for m in (2, 200):
        x = activations(gen, m, cols, torch.bfloat16)
        y = cider.cider_w4a4_linear(x, q, block)
        v, u = ref.values(ref.matrix(x, block), block), ref.values(mine, block)
        close(y[:, -130:], v @ u.T, ref.sum_bound(v, u) + ref.half_step(torch.bfloat16, v @ u.T) * (1 + 2.0 ** -10))
    del big, back, q
    x, w = activations(gen, 70000, 64, torch.float16), cider.cider_quantize_fp4(normal(gen, 32768, 64), block)
    y = cider.cider_w4a4_linear(x, w, block)
    assert y.numel() > 1 << 31
    assert torch.equal(y[-300:], cider.cider_w4a4_linear(x[-300:], w, block))
    clean()


# ------------------------------------------------------------ sizes that fill the GPU with pairs' tiles
@gpu
@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("m,n,k", [(257, 5000, 288), (300, 9800, 544), (1030, 2600, 2080), (700, 3208, 96), (513, 4808, 32),
                                   (65, 12296, 736), (2100, 1272, 64)])
def test_many_tokens(m, n, k, block):
    gen = generator(m, n, k, block)
    for dtype in TYPES[:2]:
        x, w = activations(gen, m, k, dtype), ref.matrix(0.05 * normal(gen, n, k), block)
        y = cider.cider_w4a4_linear(x, w, block)
        a, b = ref.values(ref.matrix(x, block), block), ref.values(w, block)
        want = a @ b.T
        close(y, want, ref.sum_bound(a, b) + ref.half_step(dtype, want) * (1 + 2.0 ** -10))
    # values that four bits hold: exact
    pick = lambda r: ref.VALUES.float().cuda()[torch.randint(0, 8, (r, k), generator=gen, device="cuda")] * (
        1 - 2 * torch.randint(0, 2, (r, k), generator=gen, device="cuda"))
    x, w = pick(m), pick(n)
    x[:, ::16], w[:, ::16] = 6.0, -6.0
    y = cider.cider_w4a4_linear(x.half(), cider.cider_quantize_fp4(w, block), block, y_dtype=torch.bfloat16)
    assert torch.equal(y, (x.double() @ w.double().T).float().bfloat16())
    clean()


@gpu
@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("m,f,k,act", [(300, 2600, 1056, "silu"), (129, 9736, 160, "gelu"), (700, 1304, 2080, "silu"), (260, 5000, 64, "gelu")])
def test_gated_linear_of_many_tokens(m, f, k, act, block):
    gen = generator(m, f, k, act, block)
    for dtype in TYPES[:2]:
        x = activations(gen, m, k, dtype)
        gate, up = (ref.matrix(0.03 * normal(gen, f, k), block) for _ in range(2))
        h = cider.cider_w4a4_gated_linear(x, gate, up, block, act)
        a, gv, uv = (ref.values(q, block) for q in (ref.matrix(x, block), gate, up))
        g, u = a @ gv.T, a @ uv.T
        eg, eu = ref.sum_bound(a, gv), ref.sum_bound(a, uv)
        want = ref.activate(g, act) * u
        bound = 1.13 * eg * (u.abs() + eu) + ref.activate(g.abs(), act).abs() * eu + want.abs() * 2.0 ** -14 + 2.0 ** -40
        close(h, want, bound + ref.half_step(dtype, want) * (1 + 2.0 ** -10))
    clean()


@gpu
@pytest.mark.parametrize("block", [16, 32])
def test_many_tokens_edges(block):
    """Neighbours of the output, rows that are not finite, row scales of the caller's, the whole block, twice the same bits."""
    gen = generator(block)
    m, n, k = 300, 5000, 96
    x, w = activations(gen, m, k, torch.bfloat16), cider.cider_quantize_fp4(0.05 * normal(gen, n, k), block)
    room = torch.full((m * n + 128,), 7.0, dtype=torch.bfloat16, device="cuda")
    y = cider.cider_w4a4_linear(x, w, block, out=room[64 : 64 + m * n].view(m, n))
    assert bool((room[:64] == 7).all()) and bool((room[64 + m * n :] == 7).all())
    assert torch.equal(y, cider.cider_w4a4_linear(x, w, block))
    h = cider.cider_w4a4_gated_linear(x, w, w, block, out=room[64 : 64 + m * n].view(m, n))
    assert bool((room[:64] == 7).all()) and bool((room[64 + m * n :] == 7).all())
    assert torch.equal(h, cider.cider_w4a4_gated_linear(x, w, w, block))
    z = x.clone()
    z[[5, 299], 40] = torch.tensor([float("nan"), float("inf")], device="cuda").bfloat16()
    bad = torch.zeros(m, dtype=torch.bool, device="cuda")
    bad[[5, 299]] = True
    for call in (lambda v: cider.cider_w4a4_linear(v, w, block), lambda v: cider.cider_w4a4_gated_linear(v, w, w, block)):
        got, want = call(z), call(x)
        assert bool(torch.isnan(got[bad]).all()) and torch.equal(got[~bad], want[~bad])
    (xc, xs, _), (wc, ws, _) = cider.cider_quantize_fp4(x, block), w
    rx, rw = torch.rand(m, generator=gen, device="cuda") + 0.3, torch.rand(n, generator=gen, device="cuda") + 0.3
    for qx, qw in (((xc, xs, rx), (wc, ws, rw)), ((xc, xs, None), (wc, ws, rw)), ((xc, xs, None), (wc, ws, None))):
        y = cider.cider_w4a4_linear_prequant(qx, qw, block, torch.bfloat16)
        a, b = ref.values(qx, block), ref.values(qw, block)
        close(y, a @ b.T, ref.sum_bound(a, b) + ref.half_step(torch.bfloat16, a @ b.T) * (1 + 2.0 ** -10))
    f = 9760   # ends in the middle of a step of 64
    gate, up = (cider.cider_quantize_fp4(0.03 * normal(gen, f, k), block) for _ in range(2))
    down = cider.cider_quantize_fp4(0.03 * normal(gen, 264, f), block)
    y = cider.cider_w4a4_feed_forward(x, gate, up, down, block)
    assert torch.equal(y, cider.cider_w4a4_linear(cider.cider_w4a4_gated_linear(x, gate, up, block), down, block))
    clean()
