"""Queries of one sign, whose products with the codes' offset are many times the
scores themselves, and large scores.

Tolerance, derived: as in test_tree_attention, u |o| + 7e-4 A, with the scores'
own error in place of its 1e-4 for the fp32 parts.  The kernels add up terms of
at most 255 |q_d| (INT4: 15) sk scale per dim in fp32, D products in steps of
16: an error of at most D / 16 + 1 roundings (2^-23 each, the accumulator may be
cut, not rounded) of the largest partial sum 255 sum|q| sk scale; q itself fits
fp16 but for 2^-34 of its largest value per dim (INT4's upper codes).  A score that is off by e changes
its weight by the factor exp(e): all together change o by at most 2 e A (once in
the sum of values, once in the sum of weights)."""
import numpy as np
import pytest
import torch

from tests import kv_reference as ref
from tests.parity_util import require_gpu


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("nodes", [1, 5, 16])
@pytest.mark.parametrize("spread", [1.0, 8.0])
def test_one_signed_queries(spread, nodes, dtype, bits):
    cider = require_gpu()
    rng = np.random.default_rng(nodes + bits)
    heads, hq, dim, page = 2, 8, 128, 32
    full = np.array([700 + nodes], np.int32)
    table, pages = ref.table_for(rng, full, page)
    cache = ref.Cache(rng, 1, pages, heads, dim, page, bits)
    q = spread * np.abs(rng.standard_normal((nodes, hq, dim)))
    q = torch.from_numpy(q.astype(np.float32)).to(torch.float16 if dtype == "fp16" else torch.bfloat16)
    off = ref.offsets_of([nodes])
    out = cider.cider_tree_attention(q.cuda(), cache.device(), *[torch.from_numpy(x).cuda() for x in (table, full, off)], nodes)
    want, a = ref.attend(q.float().numpy(), cache, table, full, off, None, dim ** -0.5)
    qf = q.float().numpy().astype(np.float64)
    sk = cache.host[1].max() * dim ** -0.5
    wide = (255 if bits == 8 else 15) * np.abs(qf).sum(-1).max() * sk
    e = (dim / 16 + 1) * 2.0 ** -23 * wide + 2.0 ** -34 * np.abs(qf).max() * dim * (127 if bits == 8 else 7) * sk
    u = 2.0 ** -11 if dtype == "fp16" else 2.0 ** -8
    bound = u * np.abs(want) + (7e-4 + 2 * e) * a + 2.0 ** -24
    err = np.abs(out.float().cpu().numpy().astype(np.float64) - want)
    assert (err <= bound).all(), (float((err / bound).max()), e)
    assert cider.cider_check_device_error() == 0
