"""What is not a tensor is refused with a TypeError, whichever argument it is, and
a tensor of another rank with a ValueError."""
import numpy as np
import pytest
import torch

from tests.parity_util import require_gpu


def calls(cider):
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = cider.cider_kv_cache(1, 4, 2, 64, 16, 8)
    x = torch.zeros(2, 2, 64, device="cuda").half()
    row = torch.zeros(2, 8, device="cuda").half()
    f = torch.ones(2, device="cuda")
    return {
        cider.cider_kv_append: dict(k=x, v=x, slots=torch.arange(2, device="cuda"), cache=cache),
        cider.cider_kv_read: dict(cache=cache, table=i32([0], [1]), starts=i32(0, 0), offsets=i32(0, 1, 2), tokens=2, layer=0),
        cider.cider_kv_compact: dict(cache=cache, table=i32([0], [1]), starts=i32(0, 0), path=i32([0], [0]), kept=i32(1, 1)),
        cider.cider_tree_attention: dict(q=x, cache=cache, table=i32([0], [1]), lengths=i32(1, 1), offsets=i32(0, 1, 2),
                                         max_nodes=1, tree=torch.ones(2, dtype=torch.int64, device="cuda"), out=x.clone()),
        cider.cider_verify_drafts: dict(logits=row, tokens=i32(0, 0), parents=i32(-1, -1), offsets=i32(0, 1, 2), uniforms=f,
                                        noise=torch.ones(2, 8, device="cuda"), max_nodes=1,
                                        draft_probs=torch.ones(2, 8, device="cuda"), temperature=f),
    }


def test_what_is_no_cache_is_refused():
    import w4a8_quantized_linear_gb300 as cider
    for cache in ((1, 2, 3, 4), (None,) * 4, tuple(np.zeros((1, 4, 2, 16, 64)) for _ in range(4)),
                  tuple(torch.zeros(1, 4, 2, 16, 64) for _ in range(4))):
        with pytest.raises(TypeError):
            cider.cider_kv_append(None, None, None, cache)
    with pytest.raises(TypeError):
        cider.cider_verify_drafts([[0.0]], None, None, None, None, None, 1)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["cider_kv_append", "cider_kv_read", "cider_kv_compact", "cider_tree_attention",
                                  "cider_verify_drafts"])
def test_every_argument(name):
    cider = require_gpu()
    call = getattr(cider, name)
    args = calls(cider)[call]
    call(**args)
    for key, value in args.items():
        if not isinstance(value, torch.Tensor):
            continue
        wrong = [[1, 2], np.zeros(tuple(value.shape), np.float32), 3.0]
        if key not in ("tree", "out", "draft_probs", "temperature"):
            wrong.append(None)
        for w in wrong:
            with pytest.raises(TypeError):
                call(**{**args, key: w})
        with pytest.raises(ValueError):
            call(**{**args, key: value[None]})
        with pytest.raises((TypeError, ValueError)):
            call(**{**args, key: value.cpu()})
    for i in range(4):
        if "cache" in args:
            cache = list(args["cache"])
            cache[i] = [1]
            with pytest.raises(TypeError):
                call(**{**args, "cache": tuple(cache)})
    assert cider.cider_check_device_error() == 0
