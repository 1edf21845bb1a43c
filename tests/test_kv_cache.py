"""The paged, quantized key/value cache: append (codes and scales bit for bit),
read (values bit for bit), compact, and their refusals."""
import ctypes

import numpy as np
import pytest
import torch

from tests import kv_reference as ref
from tests.parity_util import require_gpu
from w4a8_quantized_linear_gb300 import _CACHE, _build

OK, INVALID, MISALIGNED, UNSUPPORTED, INDEX = 0, 1, 2, 3, 6
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------ refusals (CPU)
@pytest.fixture(scope="module")
def lib():
    _build.build()
    import w4a8_quantized_linear_gb300 as pkg
    return pkg.library()


@pytest.fixture
def no_device(monkeypatch):
    monkeypatch.setenv("CIDER_FORCE_UNSUPPORTED", "1")


P = 0x10000   # an aligned address that no call here follows


def cache_bytes(k=P, ks=P, v=P, vs=P, layers=2, pages=4, heads=2, page=16, dim=128, bits=8):
    return _CACHE.pack(k, ks, v, vs, layers, pages, heads, page, dim, bits)


def append(lib, layer=0, k=P, stride=256, v=P, v_stride=256, dtype=0, slots=P, tokens=3, **kw):
    return lib.cider_kv_append(cache_bytes(**kw), layer, k, stride, v, v_stride, dtype, slots,
                               tokens, None)


def read(lib, layer=0, table=P, width=4, starts=P, offsets=P, requests=2, tokens=5, k=P, v=P,
         dtype=0, **kw):
    return lib.cider_kv_read(cache_bytes(**kw), layer, table, width, starts, offsets, requests,
                             tokens, k, v, dtype, None)


def compact(lib, table=P, width=4, starts=P, path=P, path_width=8, kept=P, requests=2, **kw):
    return lib.cider_kv_compact(cache_bytes(**kw), table, width, starts, path, path_width, kept,
                                requests, None)


BAD_CACHES = [dict(k=0), dict(ks=0), dict(v=0), dict(vs=0), dict(layers=-1), dict(pages=-1),
              dict(heads=0), dict(page=8), dict(page=48), dict(page=256), dict(dim=96),
              dict(dim=256), dict(bits=16), dict(bits=2)]


@pytest.mark.parametrize("kw", BAD_CACHES)
def test_bad_caches_are_refused(lib, no_device, kw):
    # a pointer of the cache, given for the calls whose own k / v have the same names
    if set(kw) & {"k", "v"}:
        kw = dict(kw)
        raw = cache_bytes(**kw)
        assert lib.cider_kv_append(raw, 0, P, 256, P, 256, 0, P, 3, None) == INVALID
        assert lib.cider_kv_read(raw, 0, P, 4, P, P, 2, 5, P, P, 0, None) == INVALID
    else:
        assert append(lib, **kw) == INVALID
        assert read(lib, **kw) == INVALID
    assert compact(lib, **kw) == INVALID


@pytest.mark.parametrize("kw", [
    dict(k=0), dict(v=0), dict(slots=0), dict(layer=2), dict(layer=-1), dict(tokens=-1),
    dict(tokens=1 << 31), dict(stride=248), dict(v_stride=248), dict(stride=260), dict(dtype=2)])
def test_append_refusals(lib, no_device, kw):
    assert append(lib, **kw) == INVALID


@pytest.mark.parametrize("kw", [
    dict(table=0), dict(starts=0), dict(offsets=0), dict(k=0), dict(v=0), dict(layer=2),
    dict(layer=-2), dict(width=0), dict(requests=-1), dict(tokens=-1), dict(dtype=7)])
def test_read_refusals(lib, no_device, kw):
    assert read(lib, **kw) == INVALID


@pytest.mark.parametrize("kw", [
    dict(table=0), dict(starts=0), dict(path=0), dict(kept=0), dict(width=0), dict(path_width=0),
    dict(path_width=65), dict(requests=-1)])
def test_compact_refusals(lib, no_device, kw):
    assert compact(lib, **kw) == INVALID


def test_misaligned_and_device_and_empty(lib, no_device):
    assert append(lib, k=P + 8) == MISALIGNED
    assert append(lib, slots=P + 4) == MISALIGNED
    assert append(lib, ks=P + 4) == MISALIGNED
    assert read(lib, v=P + 2) == MISALIGNED
    assert read(lib, table=P + 2) == MISALIGNED
    assert compact(lib, kept=P + 1) == MISALIGNED
    assert append(lib) == UNSUPPORTED
    assert read(lib) == UNSUPPORTED
    assert read(lib, layer=-1) == UNSUPPORTED
    assert compact(lib) == UNSUPPORTED
    assert append(lib, tokens=0, slots=0) == OK
    assert read(lib, tokens=0) == OK
    assert read(lib, requests=0) == OK
    assert compact(lib, requests=0) == OK
    assert append(lib, pages=0) == OK
    assert lib.cider_kv_append(None, 0, P, 256, P, 256, 0, P, 3, None) == INVALID


def test_cache_struct_has_the_c_layout():
    class C(ctypes.Structure):
        _fields_ = ([(n, ctypes.c_void_p) for n in ("k", "ks", "v", "vs")]
                    + [(n, ctypes.c_int64) for n in ("layers", "pages")]
                    + [(n, ctypes.c_int32) for n in ("heads", "page", "dim", "bits")])
    assert ctypes.sizeof(C) == _CACHE.size
    assert C.from_buffer_copy(cache_bytes()).bits == 8


# --------------------------------------------------------------------- append
def rows(rng, n, heads, dim, dtype):
    """Rows of many kinds: ordinary, zero, one value, ties, the type's ends."""
    x = rng.standard_normal((n, heads, dim)).astype(np.float32)
    x *= np.exp(rng.uniform(-8, 4, (n, heads, 1))).astype(np.float32)
    flat = x.reshape(-1, dim)
    for i in range(0, len(flat), 7):
        kind = (i // 7) % 6
        if kind == 0:
            flat[i] = 0
        elif kind == 1:
            flat[i] = 0
            flat[i, i % dim] = -3.5
        elif kind == 2:   # quotients that end in .5
            flat[i] = (rng.integers(-13, 14, dim) / 2).astype(np.float32)
            flat[i, 0] = 7.0
        elif kind == 3:
            flat[i] = rng.integers(-1, 2, dim) * (65504.0 if dtype == torch.float16 else 3.3e38)
        elif kind == 4:
            flat[i] = rng.integers(-40, 41, dim) * (2.0 ** -24 if dtype == torch.float16 else 2.0 ** -133)
        else:
            flat[i] = rng.integers(-254, 255, dim) / 2
            flat[i, 0] = 127.0
    return torch.from_numpy(x).to(dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("n,heads,dim,page", [(1, 1, 64, 16), (5, 3, 128, 16), (67, 8, 128, 64),
                                              (130, 5, 64, 128), (300, 2, 128, 32)])
def test_append_codes_and_scales_bit_for_bit(n, heads, dim, page, bits, dtype):
    cider = require_gpu()
    rng = np.random.default_rng(n + bits)
    layers, pages = 2, -(-n // page) + 2
    cache = ref.Cache(rng, layers, pages, heads, dim, page, bits)
    dev = cache.device()
    before = [t.clone() for t in dev]
    # k and v are slices of one wider tensor: [tokens, 2 heads, dim]
    both = torch.cat([rows(rng, n, heads, dim, DTYPES[dtype]),
                      rows(rng, n, heads, dim, DTYPES[dtype])], 1).cuda()
    slots = rng.permutation(pages * page)[:n].astype(np.int64)
    skipped = slots.copy()
    skipped[::5] = -1 - skipped[::5]   # any negative slot is not written
    cider.cider_kv_append(both[:, :heads], both[:, heads:], torch.from_numpy(skipped).cuda(), dev,
                          layer=1)
    want = [t.cpu().numpy() for t in before]
    for w, x in ((0, both[:, :heads]), (1, both[:, heads:])):
        q, s = ref.encode(x.float().cpu().numpy(), bits)
        for i in range(n):
            if skipped[i] >= 0:
                p, r = divmod(int(skipped[i]), page)
                want[2 * w][1, p, :, r] = ref.pack(q[i], bits)
                want[2 * w + 1][1, p, :, r] = s[i]
    for t, w in zip(dev, want):
        assert np.array_equal(t.cpu().numpy().view(np.uint8), np.ascontiguousarray(w).view(np.uint8))
    assert cider.cider_check_device_error() == OK


@pytest.mark.gpu
def test_append_slot_out_of_range_is_reported_and_skipped():
    cider = require_gpu()
    rng = np.random.default_rng(0)
    cache = ref.Cache(rng, 1, 3, 2, 64, 16, 8)
    dev = cache.device()
    x = torch.randn(3, 2, 64, device="cuda").half()
    slots = torch.tensor([48, 1 << 40, -1], dtype=torch.int64, device="cuda")
    before = [t.clone() for t in dev]
    cider.cider_kv_append(x, x, slots, dev)
    assert cider.cider_check_device_error() == INDEX
    assert cider.cider_check_device_error() == OK
    assert all(torch.equal(a, b) for a, b in zip(before, dev))


# ----------------------------------------------------------------------- read
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("counts,heads,dim,page", [
    ([1], 1, 64, 16), ([0, 17, 0, 1, 64], 3, 128, 16), ([200, 333], 8, 128, 64), ([31] * 9, 5, 64, 128)])
def test_read_bit_for_bit(counts, heads, dim, page, bits, dtype):
    cider = require_gpu()
    rng = np.random.default_rng(sum(counts))
    starts = rng.integers(0, 70, len(counts)).astype(np.int32)
    table, pages = ref.table_for(rng, starts + np.array(counts), page)
    cache = ref.Cache(rng, 3, pages, heads, dim, page, bits)
    dev = cache.device()
    off = ref.offsets_of(counts)
    n = int(off[-1])
    args = [torch.from_numpy(a).cuda() for a in (table, starts, off)]

    def want(layer):
        got = np.empty((2, n, heads, dim), np.float32)
        for b, c in enumerate(counts):
            at = int(starts[b]) + np.arange(c)
            for w in range(2):
                for h in range(heads):
                    # a code times a 24-bit scale is exact in 64 bits: rounding it to 32 is the fp32 product
                    got[w, off[b]:off[b + 1], h] = cache.values(w, layer, table[b], at, h)
        return torch.from_numpy(got).to(DTYPES[dtype])

    k, v = cider.cider_kv_read(dev, *args, n, DTYPES[dtype], layer=1)
    w = want(1)
    assert torch.equal(k.cpu(), w[0]) and torch.equal(v.cpu(), w[1])
    k, v = cider.cider_kv_read(dev, *args, n, DTYPES[dtype], layer=None)
    for layer in range(3):
        w = want(layer)
        assert torch.equal(k[layer].cpu(), w[0]) and torch.equal(v[layer].cpu(), w[1])
    assert cider.cider_check_device_error() == OK


@pytest.mark.gpu
def test_read_of_missing_pages_is_zero_and_reported():
    cider = require_gpu()
    rng = np.random.default_rng(3)
    cache = ref.Cache(rng, 1, 4, 2, 64, 16, 8)
    dev = cache.device()
    table = torch.tensor([[0, -1], [1, 9]], dtype=torch.int32, device="cuda")
    starts = torch.tensor([10, 10], dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 10, 40], dtype=torch.int32, device="cuda")   # 10 + 30 > 2 pages
    k, v = cider.cider_kv_read(dev, table, starts, off, 41, torch.float16, layer=0)
    assert cider.cider_check_device_error() == INDEX
    assert k[:6].abs().sum() > 0 and k[10:16].abs().sum() > 0
    assert k[6:10].abs().sum() == 0 and v[16:].abs().sum() == 0


@pytest.mark.gpu
def test_append_then_read_on_another_stream_and_beyond_32_bits():
    """A cache whose code tensors are larger than 2^32 bytes: the last page's
    rows come back, written and read on a stream of their own."""
    cider = require_gpu()
    pages = (1 << 32) // (8 * 64 * 128) + 8
    dev = cider.cider_kv_cache(1, pages, 8, 128, 64, 8)
    x = torch.randn(70, 8, 128, device="cuda").half()
    last = pages * 64 - 70
    slots = torch.arange(last, pages * 64, device="cuda")
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    starts = torch.tensor([last], dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 70], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cider.cider_kv_append(x, -x, slots, dev)
        k, v = cider.cider_kv_read(dev, table, starts, off, 70, torch.float16, layer=0)
    torch.cuda.current_stream().wait_stream(side)
    q, s = ref.encode(x.float().cpu().numpy(), 8)
    want = torch.from_numpy((q.astype(np.float64) * s[..., None]).astype(np.float32)).half()
    assert torch.equal(k.cpu(), want) and torch.equal(v.cpu(), -want)
    assert dev[0][0, :2].abs().sum() == 0
    assert cider.cider_check_device_error() == OK


# -------------------------------------------------------------------- compact
@pytest.mark.gpu
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("nodes,heads,dim,page", [([1], 1, 64, 16), ([5, 0, 64, 2], 3, 128, 16),
                                                  ([33, 40], 2, 128, 64), ([20] * 7, 5, 64, 32)])
def test_compact_moves_rows_of_every_layer(nodes, heads, dim, page, bits):
    cider = require_gpu()
    rng = np.random.default_rng(sum(nodes))
    starts = rng.integers(0, 50, len(nodes)).astype(np.int32)
    table, pages = ref.table_for(rng, starts + np.array(nodes), page)
    cache = ref.Cache(rng, 3, pages, heads, dim, page, bits)
    dev = cache.device()
    width = max(nodes)
    path = np.full((len(nodes), width), -1, np.int32)
    kept = np.zeros(len(nodes), np.int32)
    for b, t in enumerate(nodes):
        if t:
            kept[b] = rng.integers(1, t + 1)
            path[b, :kept[b]] = np.sort(rng.permutation(t)[:kept[b]])
    if len(nodes) == 7:   # an order that is not increasing, with a row twice
        path[2, :3], kept[2] = [4, 0, 4], 3
    cider.cider_kv_compact(dev, *(torch.from_numpy(a).cuda() for a in (table, starts, path, kept)))
    want = [a.copy() for a in cache.host]
    for b in range(len(nodes)):
        for i in range(kept[b]):
            f, t = int(starts[b] + path[b, i]), int(starts[b] + i)
            for w, old in zip(want, cache.host):
                w[:, table[b, t // page], :, t % page] = old[:, table[b, f // page], :, f % page]
    for t, w in zip(dev, want):
        assert np.array_equal(t.cpu().numpy(), w)
    assert cider.cider_check_device_error() == OK


@pytest.mark.gpu
def test_compact_out_of_range_is_reported_and_skipped():
    cider = require_gpu()
    rng = np.random.default_rng(1)
    cache = ref.Cache(rng, 2, 4, 2, 64, 16, 8)
    dev = cache.device()
    before = [t.clone() for t in dev]
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table, starts = i32([0], [1], [77]), i32(8, 8, 8)
    cider.cider_kv_compact(dev, table, starts, i32([20, -1], [-1, -1], [1, 2]), i32(1, 3, 2))
    assert cider.cider_check_device_error() == INDEX
    assert all(torch.equal(a, b) for a, b in zip(before, dev))


@pytest.mark.gpu
def test_wrong_tensors_are_refused_by_the_binding():
    cider = require_gpu()
    dev = cider.cider_kv_cache(1, 4, 2, 64, 16, 8)
    x = torch.zeros(3, 2, 64, device="cuda").half()
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    with pytest.raises(TypeError):
        cider.cider_kv_append(x.float(), x.float(), slots, dev)
    with pytest.raises(TypeError):
        cider.cider_kv_append(x, x, slots.int(), dev)
    with pytest.raises(ValueError):
        cider.cider_kv_append(x[:, :1], x, slots, dev)
    with pytest.raises(ValueError):
        cider.cider_kv_append(x.transpose(1, 2), x, slots, dev)
    with pytest.raises(ValueError):
        cider.cider_kv_append(x, x[:2], slots, dev)
    with pytest.raises(ValueError):
        cider.cider_kv_append(x, x, slots, (dev[0], dev[1], dev[2][:, :2], dev[3]))
    with pytest.raises(cider.CiderError):
        cider.cider_kv_append(x, x, slots, dev, layer=1)
