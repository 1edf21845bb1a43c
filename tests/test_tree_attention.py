"""Attention of new tokens over the paged, quantized cache against a 64-bit
reference, and its refusals.

Tolerance, derived: the result is rounded once to its type (at most u |o|, u =
2^-11 for fp16's 11 significant bits, 2^-8 for bf16's 8); each weight of the values is rounded
to fp16 (2^-11 of it, so at most 2^-11 A in all, A = sum_j p_j |v_j|); a weight
below fp16's normal range is off by less than 2^-24 of the largest, over 2^15
weights less than 2^-9 A / 2^8.  The fp32 parts (128 products, the exponential
of arguments below 100, sums) stay below 1e-4 A.  Together: u |o| + 7e-4 A,
and one subnormal step of fp16."""
import numpy as np
import pytest
import torch

from tests import kv_reference as ref
from tests.parity_util import require_gpu
from w4a8_quantized_linear_gb300 import _CACHE, _build

OK, INVALID, MISALIGNED, UNSUPPORTED, INDEX = 0, 1, 2, 3, 6
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
P = 0x10000


@pytest.fixture(scope="module")
def lib():
    _build.build()
    import w4a8_quantized_linear_gb300 as pkg
    return pkg.library()


def call(lib, layer=0, q=P, stride=512, dtype=0, tokens=3, hq=4, table=P, width=4, lengths=P,
         offsets=P, requests=2, nodes=2, tree=P, scale=1.0, out=P, pages=4):
    c = _CACHE.pack(P, P, P, P, 2, pages, 2, 16, 128, 8)
    return lib.cider_tree_attention(c, layer, q, stride, dtype, tokens, hq, table, width, lengths,
                                    offsets, requests, nodes, tree, scale, out, None)


@pytest.mark.parametrize("kw", [
    dict(q=0), dict(table=0), dict(lengths=0), dict(offsets=0), dict(out=0), dict(layer=2),
    dict(layer=-1), dict(dtype=3), dict(tokens=-1), dict(hq=3), dict(hq=0), dict(width=0),
    dict(requests=-1), dict(nodes=0), dict(nodes=65), dict(stride=504), dict(stride=516),
    dict(scale=float("nan")), dict(scale=float("inf"))])
def test_refusals(lib, monkeypatch, kw):
    monkeypatch.setenv("CIDER_FORCE_UNSUPPORTED", "1")
    assert call(lib, **kw) == INVALID


def test_alignment_device_and_empty(lib, monkeypatch):
    monkeypatch.setenv("CIDER_FORCE_UNSUPPORTED", "1")
    assert call(lib, q=P + 8) == MISALIGNED
    assert call(lib, out=P + 4) == MISALIGNED
    assert call(lib, tree=P + 4) == MISALIGNED
    assert call(lib, lengths=P + 2) == MISALIGNED
    assert call(lib) == UNSUPPORTED
    assert call(lib, tree=None) == UNSUPPORTED
    assert call(lib, tokens=0, q=0, out=0) == OK
    assert call(lib, requests=0) == OK


def run(cider, rng, lengths, nodes, hq, heads, dim, page, bits, dtype, masks="tree", scale=None,
        stride=None, table_edit=None, check=True, spread=1.0):
    """lengths: context lengths of the requests, nodes: their new tokens."""
    full = np.array(lengths, np.int32) + np.array(nodes, np.int32)
    table, pages = ref.table_for(rng, full, page)
    cache = ref.Cache(rng, 2, pages, heads, dim, page, bits)
    n = int(sum(nodes))
    wide = stride or hq
    q = torch.from_numpy((spread * rng.standard_normal((n, wide, dim))).astype(np.float32)).to(DTYPES[dtype])
    q = q[:, wide - hq:]
    if masks == "tree":
        tree = [m for t in nodes if t for m in ref.random_tree(rng, t)[1]]
    elif masks == "random":   # any bits, empty rows among them, bits past the nodes
        tree = [int(rng.integers(0, 1 << 62)) & int(rng.integers(0, 1 << 62)) for _ in range(n)]
        tree = [0 if i % 4 == 1 else m | (1 << 63 if i % 3 == 0 else 0) for i, m in enumerate(tree)]
    else:
        tree = None
    off = ref.offsets_of(nodes)
    scale = dim ** -0.5 if scale is None else scale
    dev = [torch.from_numpy(a).cuda() for a in (table, full, off)]
    mask = torch.from_numpy(ref.signed(tree)).cuda() if tree is not None else None
    qd = torch.empty((n, wide, dim), dtype=DTYPES[dtype], device="cuda")[:, wide - hq:]
    qd.copy_(q)
    out = cider.cider_tree_attention(qd, cache.device(), *dev, max(max(nodes), 1), tree=mask,
                                     scale=scale, layer=1)
    assert out.dtype == DTYPES[dtype] and out.shape == (n, hq, dim)
    assert cider.cider_check_device_error() == OK
    want, size = ref.attend(q.float().numpy(), cache, table, full, off, tree, scale, layer=1)
    u = 2.0 ** -11 if dtype == "fp16" else 2.0 ** -8
    bound = u * np.abs(want) + 7e-4 * size + 2.0 ** -24
    err = np.abs(out.float().cpu().numpy().astype(np.float64) - want)
    assert np.isfinite(err).all()
    assert (err <= bound).all(), (float((err / bound).max()), np.argwhere(err > bound)[:4])
    return out, cache


@pytest.mark.gpu
@pytest.mark.parametrize("bits,dtype", [(8, "fp16"), (4, "fp16"), (8, "bf16"), (4, "bf16")])
@pytest.mark.parametrize("hq,heads,dim", [(1, 1, 64), (8, 8, 128), (16, 8, 128), (12, 4, 64),
                                          (32, 8, 128), (16, 1, 128), (20, 1, 64), (34, 2, 128)])
def test_one_token(hq, heads, dim, bits, dtype):
    cider = require_gpu()
    rng = np.random.default_rng(hq + dim)
    run(cider, rng, [0, 1, 15, 16, 17, 130, 333, 1025], [1] * 8, hq, heads, dim, 16, bits, dtype,
        masks="chain")


@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("bits,dtype", [(8, "bf16"), (4, "fp16")])
@pytest.mark.parametrize("masks", ["tree", "random", "chain"])
def test_trees(page, bits, dtype, masks):
    cider = require_gpu()
    rng = np.random.default_rng(page)
    run(cider, rng, [0, 3, 64, 127, 500], [7, 64, 1, 33, 16], 8, 2, 128, page, bits, dtype, masks)


@pytest.mark.gpu
@pytest.mark.parametrize("hq,heads,dim", [(4, 4, 64), (16, 8, 128), (32, 8, 64), (24, 8, 128),
                                          (12, 1, 64), (48, 2, 64)])
@pytest.mark.parametrize("bits", [8, 4])
def test_head_layouts_of_trees(hq, heads, dim, bits):
    cider = require_gpu()
    rng = np.random.default_rng(hq)
    run(cider, rng, [100, 37, 0], [5, 64, 21], hq, heads, dim, 32, bits, "fp16")


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("nodes", [2, 3, 4, 5, 6, 7, 8, 9])
def test_every_number_of_rows(nodes, bits, dim):
    """8 .. 36 query rows per key/value head: each form of the kernels for few
    rows, full and not, and the change to the one for many."""
    cider = require_gpu()
    rng = np.random.default_rng(nodes)
    run(cider, rng, [300, 41, 1000], [nodes, 1, nodes], 8, 2, dim, 16, bits, "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("bits,dtype", [(8, "fp16"), (4, "bf16")])
@pytest.mark.parametrize("nodes", [1, 3, 40])
def test_long_axis_and_many_requests(bits, dtype, nodes):
    """A long request beside short and empty ones: its axis is split and joined."""
    cider = require_gpu()
    rng = np.random.default_rng(nodes)
    run(cider, rng, [9000, 3, 0, 700, 1], [nodes, 0, nodes, 1, nodes], 8, 2, 128, 64, bits, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("nodes", [1, 6])
@pytest.mark.parametrize("bits,dtype,scale,page", [(8, "fp16", None, 16), (4, "bf16", 0.6, 64), (8, "bf16", 0.6, 128)])
def test_many_tiles_per_share(nodes, bits, dtype, scale, page):
    """Far more positions than the GPU has SMs: each works through many tiles and
    several requests in a row, with maxima that rise on the way."""
    cider = require_gpu()
    rng = np.random.default_rng(31 + bits)
    lengths = [int(x) for x in rng.integers(400, 1900, 40)]
    run(cider, rng, lengths, [nodes - (i % 2 if nodes > 1 else 0) for i in range(40)], 32, 8, 128, page, bits, dtype,
        scale=scale)


@pytest.mark.gpu
def test_sharp_and_flat_scores():
    """Scores far apart (one position takes all) and all equal (scale 0)."""
    cider = require_gpu()
    rng = np.random.default_rng(9)
    for bits in (8, 4):
        run(cider, rng, [400, 90], [20, 1], 8, 2, 128, 16, bits, "fp16", scale=1.0, spread=2.0)
        run(cider, rng, [400, 90], [20, 1], 8, 2, 128, 16, bits, "fp16", scale=0.0)
        run(cider, rng, [400, 90], [1, 1], 8, 2, 128, 16, bits, "bf16", scale=-0.3)


@pytest.mark.gpu
def test_query_stride_and_magnitudes():
    cider = require_gpu()
    rng = np.random.default_rng(10)
    run(cider, rng, [200], [5], 8, 4, 128, 16, 8, "bf16", stride=17)
    run(cider, rng, [200], [1], 8, 4, 64, 16, 8, "bf16", stride=9, spread=1e30, scale=1e-31)
    run(cider, rng, [200], [30], 8, 4, 64, 16, 4, "bf16", spread=1e-30, scale=1e29)
    run(cider, rng, [200], [30], 8, 4, 128, 16, 8, "fp16", spread=3000.0, scale=1e-4)


@pytest.mark.gpu
@pytest.mark.parametrize("nodes", [1, 24])
def test_what_no_token_sees_does_not_matter(nodes):
    """NaN and infinite scales past the length, in unused pages and at a
    position that the mask hides leave the result as it was."""
    cider = require_gpu()
    rng = np.random.default_rng(11)
    page, heads, dim, ctx = 16, 2, 128, 75
    full = np.array([ctx + nodes], np.int32)
    table, pages = ref.table_for(rng, full, page)
    cache = ref.Cache(rng, 1, pages, heads, dim, page, 8)
    hidden = nodes - 1 if nodes > 1 else None
    _, tree = ref.random_tree(rng, nodes)
    if hidden is not None:
        tree = [m & ~(1 << hidden) for m in tree]
    q = torch.randn(nodes, 8, dim, device="cuda").half()
    dev = [torch.from_numpy(a).cuda() for a in (table, full, ref.offsets_of([nodes]))]
    mask = torch.from_numpy(ref.signed(tree)).cuda()
    a = cider.cider_tree_attention(q, cache.device(), *dev, nodes, tree=mask)
    for bad in (np.nan, np.inf, -np.inf, 0.0):
        used = np.zeros((pages, page), bool)
        pos = np.arange(int(full[0]) if hidden is None else int(full[0]) - 1)
        used[table[0, pos // page], pos % page] = True
        for s in (1, 3):
            cache.host[s][0] = np.where(used[:, None], cache.host[s][0], np.float32(bad))
        b = cider.cider_tree_attention(q, cache.device(), *dev, nodes, tree=mask)
        assert torch.isfinite(b).all() and torch.equal(a, b), bad
    assert cider.cider_check_device_error() == OK


@pytest.mark.gpu
@pytest.mark.parametrize("nodes", [1, 12])
def test_same_inputs_same_bits(nodes):
    """Splitting and joining does not depend on which part ends first."""
    cider = require_gpu()
    dev = cider.cider_kv_cache(1, 300, 4, 128, 64, 8)
    dev[0].random_(-127, 128)
    dev[2].random_(-127, 128)
    dev[1].uniform_(0.001, 0.02)
    dev[3].uniform_(0.001, 0.02)
    table = torch.arange(300, dtype=torch.int32, device="cuda").view(2, 150)
    lengths = torch.tensor([9600, 7001], dtype=torch.int32, device="cuda")
    off = torch.tensor([0, nodes, 2 * nodes], dtype=torch.int32, device="cuda")
    q = torch.randn(2 * nodes, 16, 128, device="cuda").half()
    first = cider.cider_tree_attention(q, dev, table, lengths, off, nodes)
    for _ in range(5):
        assert torch.equal(first, cider.cider_tree_attention(q, dev, table, lengths, off, nodes))


@pytest.mark.gpu
@pytest.mark.parametrize("nodes", [1, 9])
def test_contradicting_lengths_are_reported(nodes):
    """A request longer than its table, shorter than its new tokens, or with
    more tokens than max_nodes is left out; the others are computed."""
    cider = require_gpu()
    rng = np.random.default_rng(12)
    cache = ref.Cache(rng, 1, 8, 2, 64, 16, 8)
    dev = cache.device()
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(4, 2)
    good = torch.tensor([20, 20, 20, 20], dtype=torch.int32, device="cuda")
    off = torch.arange(5, device="cuda").int() * nodes
    q = torch.randn(4 * nodes, 4, 64, device="cuda").half()
    want = cider.cider_tree_attention(q, dev, table, good, off, nodes)
    out = torch.full_like(want, 7.0)
    lengths = torch.tensor([20, 33, nodes - 1, 20], dtype=torch.int32, device="cuda")
    cider.cider_tree_attention(q, dev, table, lengths, off, nodes, out=out)
    assert cider.cider_check_device_error() == INDEX
    assert torch.equal(out[:nodes], want[:nodes]) and torch.equal(out[3 * nodes:], want[3 * nodes:])
    assert (out[nodes:3 * nodes] == 7.0).all()
    # a page that is not there is as if its positions were hidden
    hole = table.clone()
    hole[3, 0] = 99
    cider.cider_tree_attention(q, dev, hole, good, off, nodes, out=out)
    assert cider.cider_check_device_error() == INDEX
    assert torch.isfinite(out[3 * nodes:].float()).all()
    bad = torch.tensor([0, nodes, nodes, 3 * nodes, 5 * nodes], dtype=torch.int32, device="cuda")
    cider.cider_tree_attention(q, dev, table, good, bad, nodes, out=out)
    assert cider.cider_check_device_error() == INDEX
    assert torch.equal(out[:nodes], want[:nodes])


@pytest.mark.gpu
def test_cache_beyond_32_bits_and_graph_capture():
    """Pages past 2^32 bytes of codes, from a captured graph on another stream."""
    cider = require_gpu()
    heads, dim, page = 8, 128, 64
    pages = (1 << 32) // (heads * page * dim) + 40
    dev = cider.cider_kv_cache(1, pages, heads, dim, page, 8)
    small = cider.cider_kv_cache(1, 40, heads, dim, page, 8)
    for s, d in zip(small, dev):
        if s.dtype == torch.int8:
            s.random_(-127, 128)
        else:
            s.uniform_(0.001, 0.02)
        d[:, -40:] = s
    q = torch.randn(8, 16, dim, device="cuda").half()
    lengths = torch.tensor([40 * page - 3], dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    near = torch.arange(40, dtype=torch.int32, device="cuda")[None]
    far = near + (pages - 40)
    want = cider.cider_tree_attention(q, small, near, lengths, off, 8)
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cider.cider_tree_attention(q, dev, far, lengths, off, 8, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert cider.cider_check_device_error() == OK
