"""Which launches the calls of 4-bit floating point make, and on which memory: the entry points' own code
over launchers that only write down their arguments, so that no GPU is needed and every address can be made up."""
import ctypes
import itertools

import pytest

from tests.fp4_calls import FEW, PAIRS, QUANTIZE, SCRATCH, first_on_pairs, library, made, product_kernels, weights

BASE = 0x700000000000


@pytest.fixture(scope="module")
def lib():
    return library()


def up(v, unit):
    return -(-v // unit) * unit


def held(rows, cols, block, codes, scales, row):
    """The ranges of a quantized matrix."""
    tiles = -(-cols // (4 * block))
    r = [(codes, codes + rows * cols // 2), (scales, scales + up(rows, 128) // 128 * tiles * 512)]
    return r + ([(row, row + 4 * rows)] if block == 16 else [])


def apart(a, b):
    return a[1] <= b[0] or b[1] <= a[0]


def check(records, block, x, stride, m, y, out):
    """Every launch but the last writes scratch only; nothing is written where it or a later launch still reads; what is
    read is x, or what an earlier launch wrote."""
    room = (0, 0)
    wide, quantized = {x}, set()
    launches = [r for r in records if r.kind != SCRATCH]
    for r in records:
        if r.kind == SCRATCH:
            assert room == (0, 0), "one allocation"
            room = (r.y, r.y + r.bytes)
    for i, r in enumerate(launches):
        if r.wide:
            assert r.wide in wide
            pitch = stride if r.wide == x else r.k
            assert r.stride == pitch
            reads = [(r.wide, r.wide + 2 * ((r.m - 1) * pitch + r.k))]
        else:
            assert (r.codes, r.scales, r.row) in quantized
            reads = held(r.m, r.k, block, r.codes, r.scales, r.row)
        if r.to_codes:
            writes = held(r.m, r.n if r.kind != QUANTIZE else r.k, block, r.to_codes, r.to_scales, r.to_row)
            quantized.add((r.to_codes, r.to_scales, r.to_row))
        else:
            writes = [(r.y, r.y + 2 * r.m * r.n)]
            wide.add(r.y)
        last = i == len(launches) - 1
        assert (r.y == y) == last
        for w in writes:
            assert last or (room[0] <= w[0] and w[1] <= room[1]), "outside of the scratch"
        # x quantized by a kernel of its own is not read by the product: a product may write on it
        assert all(apart(a, b) for a in reads + writes for b in writes if a is not b), "reads what it writes"
    return launches


CASES = [(1, 256, 512), (2, 4096, 2048), (16, 256, 1056), (16, 1024, 6144), (40, 512, 768), (61, 2048, 2048), (900, 512, 2560)]


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("fits", [0, 1])
@pytest.mark.parametrize("m,k,f", CASES)
def test_x_anywhere_around_the_scratch(lib, m, k, f, fits, block):
    """Device memory of other programs' parts lies directly before and behind the call's scratch."""
    def call(x):
        lib.calls_begin(BASE, 152, fits)
        g, d = weights(f, k, block), weights(k, f, block)
        y = 0x200000000000
        assert lib.cider_w4a4_feed_forward(x, 0, k, m, ctypes.byref(g), ctypes.byref(g), ctypes.byref(d), 0, y, 0, None) == 0
        return check(made(lib), block, x, k, m, y, k)

    far = call(0x300000000000)
    size = sum(r.bytes for r in made(lib) if r.kind == SCRATCH)
    shape = [(r.kind, bool(r.wide), bool(r.to_codes), r.dependent) for r in far]
    # every multiple of 256 bytes behind the scratch, thinned out, and the ranges before it that end at it
    steps = sorted({0, 256, 512, up(m * f, 256), up(2 * m * f, 256), up(3 * m * f, 256), up(m * f // 2, 256), 1 << 21, 1 << 22})
    for at in [BASE + up(size, 256) + s for s in steps] + [BASE - up(2 * m * k, 256) - s for s in steps]:
        assert [(r.kind, bool(r.wide), bool(r.to_codes), r.dependent) for r in call(at)] == shape


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("m,k,n", [(1, 512, 512), (16, 1024, 2560), (16, 2560, 256), (61, 512, 512), (900, 512, 2560)])
def test_y_on_x(lib, m, k, n, block):
    """The kernel that quantizes x itself is not taken where y lies on x: others still read what it writes."""
    x = 0x300000000000
    w = weights(n, k, block)
    for off, gated in itertools.product((-2 * m * n, -2 * m * n + 16, -256, 0, 256, 2 * m * k - 16, 2 * m * k), (False, True)):
        lib.calls_begin(BASE, 152, 1)
        y = x + off
        if gated:
            assert lib.cider_w4a4_gated_linear(x, 0, k, m, ctypes.byref(w), ctypes.byref(w), 0, y, 0, None) == 0
        else:
            assert lib.cider_w4a4_linear(x, 0, k, m, ctypes.byref(w), y, 0, None) == 0
        launches = check(made(lib), block, x, k, m, y, n)
        clear = off + 2 * m * n <= 0 or off >= 2 * m * k
        assert launches[-1].kind == PAIRS or (len(launches) == 1) == clear


@pytest.mark.parametrize("sms", [152, 148, 76])
@pytest.mark.parametrize("gated", [False, True])
def test_which_products_run_on_pairs(sms, gated):
    """Never up to 64 tokens; always where there are more tiles of 128 weight rows and tokens than half of the SMs."""
    for n in (8, 200, 1000, 2560, 10240, 128 * (sms // 2), 128 * (sms // 2) + 8):
        first = first_on_pairs(n, 512, 32, gated, sms)
        assert first > 64
        assert product_kernels(first - 1, n, 512, 32, gated, sms) == FEW
        half, rows = sms // 2, -(-n // 128)
        assert -(-first // 64) * rows > half and (gated or -(-first // 128) * rows > half)
        for m in (first + 1, 2 * first, 10 * first):
            assert product_kernels(m, n, 512, 16, gated, sms) == PAIRS
