"""A negative layer is refused by the binding: the C entry point reads -1 as all
layers, which would be written into the room of one."""
import pytest
import torch

from tests.parity_util import require_gpu


@pytest.mark.gpu
@pytest.mark.parametrize("layer", [-1, -2])
@pytest.mark.parametrize("given", [False, True])
def test_negative_layers_are_refused(given, layer):
    cider = require_gpu()
    cache = cider.cider_kv_cache(3, 2, 2, 64, 16, 8)
    table = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    starts = torch.zeros(1, dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    out = tuple(torch.full((5, 2, 64), 7.0, device="cuda").half() for _ in range(2)) if given else None
    with pytest.raises(ValueError):
        cider.cider_kv_read(cache, table, starts, offsets, 5, torch.float16, layer=layer, out=out)
    if given:
        assert (out[0] == 7.0).all() and (out[1] == 7.0).all()
    k, _ = cider.cider_kv_read(cache, table, starts, offsets, 5, torch.float16)
    assert k.shape == (3, 5, 2, 64)
