"""A negative number of kept rows is out of range: nothing moves, and it is
reported, as a number beyond the path's width is."""
import pytest
import torch

from tests.parity_util import require_gpu

OK, INDEX = 0, 6


@pytest.mark.gpu
def test_negative_counts_are_reported():
    cider = require_gpu()
    cache = cider.cider_kv_cache(2, 4, 2, 64, 16, 8)
    for t in cache[::2]:
        t.random_(-127, 128)
    before = [t.clone() for t in cache]
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    args = (cache, i32([0], [1]), i32(2, 2), i32([3, 4], [5, 6]))
    cider.cider_kv_compact(*args, i32(0, 0))
    assert cider.cider_check_device_error() == OK
    cider.cider_kv_compact(*args, i32(0, -1))
    assert cider.cider_check_device_error() == INDEX
    assert all(torch.equal(a, b) for a, b in zip(before, cache))
