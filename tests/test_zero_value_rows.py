"""Positions whose value row is all zeros (scale 1, as the format has it) and
which take most of the attention, as a null token does, leave the other values
the precision that they have without them.

Tolerance as in test_tree_attention, derived there: u |o| + 7e-4 A, A = sum_j
p_j |v_j|; the largest weight that counts is the largest among the positions
that contribute to A.  Scores go to 30 here, not 100."""
import numpy as np
import pytest
import torch

from tests import kv_reference as ref
from tests.parity_util import require_gpu

OK = 0


@pytest.mark.gpu
@pytest.mark.parametrize("size", [1.0, 1e-2, 1e-4])
@pytest.mark.parametrize("above", [-8.0, 5.0, 12.0])
@pytest.mark.parametrize("bits,dtype", [(8, "bf16"), (4, "bf16"), (8, "fp16")])
@pytest.mark.parametrize("nodes", [1, 5, 16])
def test_dominant_zero_rows(nodes, bits, dtype, above, size):
    """size: of the values; above: how far the zero rows' scores lie above the
    others' largest; 4 .. 64 query rows per key/value head."""
    cider = require_gpu()
    rng = np.random.default_rng(nodes + bits)
    heads, hq, dim, page = 2, 8, 128, 16
    full = np.array([1000 + nodes, 40 + nodes], np.int32)
    table, pages = ref.table_for(rng, full, page)
    cache = ref.Cache(rng, 1, pages, heads, dim, page, bits)
    cache.host[3] *= np.float32(size)
    q = rng.standard_normal((1, 1, dim)) + 0.05 * rng.standard_normal((2 * nodes, hq, dim))
    q = torch.from_numpy(q.astype(np.float32)).to(torch.float16 if dtype == "fp16" else torch.bfloat16)
    qf = q.float().numpy().astype(np.float64)
    for b in range(2):
        for at in (0, 17, int(full[b]) - nodes - 1):   # first, in the middle, last of the context
            p, r = table[b, at // page], at % page
            for h in range(heads):
                pos = np.arange(int(full[b]))
                k = cache.values(0, 0, table[b], pos, h)
                high = (k @ qf.reshape(-1, dim).T).max() * dim ** -0.5
                mean = qf.mean((0, 1))
                row = mean * ((high + above) * dim ** 0.5 / (mean @ mean))
                code, s = ref.encode(row[None].astype(np.float32), bits)
                cache.host[0][0, p, h, r], cache.host[1][0, p, h, r] = ref.pack(code, bits)[0], s[0]
                cache.host[2][0, p, h, r], cache.host[3][0, p, h, r] = 0, 1.0
    off = ref.offsets_of([nodes, nodes])
    dev = [torch.from_numpy(a).cuda() for a in (table, full, off)]
    out = cider.cider_tree_attention(q.cuda(), cache.device(), *dev, nodes)
    assert cider.cider_check_device_error() == OK
    want, a = ref.attend(q.float().numpy(), cache, table, full, off, None, dim ** -0.5)
    u = 2.0 ** -11 if dtype == "fp16" else 2.0 ** -8
    bound = u * np.abs(want) + 7e-4 * a + (2.0 ** -24 if dtype == "fp16" else 0.0)
    err = np.abs(out.float().cpu().numpy().astype(np.float64) - want)
    assert (err <= bound).all(), float((err / np.maximum(bound, 1e-300)).max())


@pytest.mark.gpu
@pytest.mark.parametrize("nodes", [1, 16])
@pytest.mark.parametrize("bits", [8, 4])
def test_only_zero_rows(bits, nodes):
    """Nothing but zero rows, and values whose scale is exactly 1 beside them."""
    cider = require_gpu()
    rng = np.random.default_rng(bits)
    heads, hq, dim, page = 2, 8, 64, 32
    full = np.array([70 + nodes, 70 + nodes], np.int32)
    table, pages = ref.table_for(rng, full, page)
    cache = ref.Cache(rng, 1, pages, heads, dim, page, bits)
    cache.host[3][:] = 1.0
    used = table[0][table[0] >= 0]
    cache.host[2][0, used] = 0   # all of the first request's, every third of the others'
    cache.host[2][0, :, :, ::3] = 0
    q = torch.from_numpy(rng.standard_normal((2 * nodes, hq, dim)).astype(np.float32)).half()
    off = ref.offsets_of([nodes, nodes])
    out = cider.cider_tree_attention(q.cuda(), cache.device(), *[torch.from_numpy(x).cuda() for x in (table, full, off)], nodes)
    want, a = ref.attend(q.float().numpy(), cache, table, full, off, None, dim ** -0.5)
    err = np.abs(out.float().cpu().numpy().astype(np.float64) - want)
    assert (out[:nodes] == 0).all()
    assert (err <= 2.0 ** -11 * np.abs(want) + 7e-4 * a + 2.0 ** -24).all()
    assert cider.cider_check_device_error() == OK
