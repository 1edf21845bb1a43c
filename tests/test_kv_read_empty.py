"""A read of an empty problem (no requests, or a cache without pages) leaves zeros
in the tensors that it is given, as in those that it makes."""
import pytest
import torch

from tests.parity_util import require_gpu


@pytest.mark.gpu
@pytest.mark.parametrize("layer", [0, None])
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("empty", ["requests", "pages"])
def test_empty_problems(empty, given, layer):
    cider = require_gpu()
    requests, pages = (0, 8) if empty == "requests" else (2, 0)
    cache = cider.cider_kv_cache(2, pages, 2, 64, 16, 8)
    table = torch.zeros(requests, 2, dtype=torch.int32, device="cuda")
    starts = torch.zeros(requests, dtype=torch.int32, device="cuda")
    offsets = torch.arange(requests + 1, dtype=torch.int32, device="cuda") * 2
    shape = (4, 2, 64) if layer is not None else (2, 4, 2, 64)
    pair = tuple(torch.full(shape, 7.0, device="cuda").half() for _ in range(2)) if given else None
    got = cider.cider_kv_read(cache, table, starts, offsets, 4, torch.float16, layer=layer, out=pair)
    assert got[0].shape == shape and (got[0] == 0).all() and (got[1] == 0).all()
    assert pair is None or all(a is b for a, b in zip(got, pair))
    assert cider.cider_check_device_error() == 0
