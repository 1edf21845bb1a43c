"""Rows of the attention's output that no request owns are zeros, and reported
where the device can tell; an empty problem has zeros too."""
import pytest
import torch

from tests.parity_util import require_gpu

OK, INDEX = 0, 6


def setup(cider, nodes, rows, requests=2, pages=8):
    cache = cider.cider_kv_cache(1, pages, 2, 64, 16, 8)
    for t in cache[::2]:
        t.random_(-127, 128)
    for t in cache[1::2]:
        t.uniform_(0.001, 0.02)
    table = torch.arange(2 * requests, dtype=torch.int32, device="cuda").view(requests, 2)
    lengths = torch.full((requests,), 30, dtype=torch.int32, device="cuda")
    q = torch.randn(rows, 8, 64, device="cuda").half()
    return q, cache, table, lengths


@pytest.mark.gpu
@pytest.mark.parametrize("nodes", [1, 3, 20])
@pytest.mark.parametrize("before,after", [(0, 5), (3, 0), (2, 300)])
def test_rows_outside_of_the_offsets(nodes, before, after):
    """A padded batch: 4 .. 80 query rows per key/value head, so that each
    kernel is used."""
    cider = require_gpu()
    rows = before + 2 * nodes + after
    q, cache, table, lengths = setup(cider, nodes, rows)
    offsets = before + torch.arange(3, device="cuda").int() * nodes
    own = slice(before, before + 2 * nodes)
    want = cider.cider_tree_attention(q[own], cache, table, lengths, offsets - before, nodes)
    assert cider.cider_check_device_error() == OK
    out = torch.full_like(q, 7.0)
    cider.cider_tree_attention(q, cache, table, lengths, offsets, nodes, out=out)
    assert cider.cider_check_device_error() == INDEX
    assert torch.equal(out[own], want)
    assert (out[:before] == 0).all() and (out[before + 2 * nodes:] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("empty", ["requests", "pages"])
def test_empty_problems(empty, given):
    cider = require_gpu()
    q, cache, table, lengths = setup(cider, 1, 4)
    offsets = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    if empty == "requests":
        table, lengths, offsets = table[:0], lengths[:0], offsets[:1]
    else:
        cache = cider.cider_kv_cache(1, 0, 2, 64, 16, 8)
    out = torch.full_like(q, 7.0) if given else None
    junk = [torch.full_like(q, 7.0) for _ in range(8)]   # what an allocation may find
    del junk
    got = cider.cider_tree_attention(q, cache, table, lengths, offsets, 2, out=out)
    assert (got == 0).all() and (out is None or got is out)
    assert cider.cider_check_device_error() == OK
