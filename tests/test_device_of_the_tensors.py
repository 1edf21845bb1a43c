"""The library launches on the current device: a call whose tensors are on another
one makes that current for its time, with that device's stream."""
import contextlib
import types

import pytest
import torch

import w4a8_quantized_linear_gb300 as pkg
from tests.parity_util import require_gpu


def test_launch_on_the_tensors_device(monkeypatch):
    now, seen = [0], []

    @contextlib.contextmanager
    def device(d):
        before, now[0] = now[0], d
        yield
        now[0] = before

    def cider_kv_append(*a):
        seen.append((now[0], a))
        return 0

    def cider_kv_read(*a):
        return 2

    monkeypatch.setattr(pkg, "_lib", types.SimpleNamespace(cider_status_string=lambda s: b"refused"))
    monkeypatch.setattr(pkg, "_current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    pkg._launch(cider_kv_append, 0, (1, 2))
    pkg._launch(cider_kv_append, 3, (1, 2))
    assert seen == [(0, (1, 2)), (3, (1, 2))] and now == [0]
    with pytest.raises(pkg.CiderError, match="cider_kv_read"):
        pkg._launch(cider_kv_read, 3, ())
    assert now == [0]


@pytest.mark.gpu
def test_every_call_takes_its_tensors_device(monkeypatch):
    """Seen from a process whose current device is another one."""
    cider = require_gpu()
    x = torch.randn(20, 256, device="cuda").half()
    w = torch.randn(64, 256, device="cuda")
    cache = cider.cider_kv_cache(1, 4, 2, 64, 16, 8)
    kv = torch.randn(3, 2, 64, device="cuda").half()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table, starts, offsets = i32([0, 1]), i32(0), i32(0, 3)

    def all_calls():
        q8, s8 = cider.cider_quantize_weight_int8(w, 64)
        q4, s4 = cider.cider_quantize_weight_int4(w, 0, clip_percentile=99.0)
        qa, sa = cider.cider_quantize_act(x)
        cider.cider_kv_append(kv, kv, torch.arange(3, device="cuda"), cache)
        cider.cider_kv_compact(cache, table, starts, i32([0, 2]), i32(2))
        return [q8, q4, qa, cider.cider_w8a8_linear(x, q8, s8, 64), cider.cider_w4a8_linear_ex(x, q4, s4),
                cider.cider_w8a8_linear_prequant(qa, sa, q8, s8, 64), cider.cider_w8a8_accumulators(qa, q8, 64),
                cider.cider_int4_from_offset_binary(q4), *cider.cider_kv_read(cache, table, starts, offsets, 3),
                cider.cider_tree_attention(kv, cache, table, i32(3), offsets, 3),
                *cider.cider_verify_drafts(x[:1], i32(0), i32(0), i32(0, 1), torch.zeros(1, device="cuda"),
                                           torch.ones(1, 256, device="cuda"), 1)]

    want = all_calls()
    entered = []

    class Device(torch.cuda.device):
        def __init__(self, d):
            entered.append(d)
            super().__init__(d)

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(cider, "_current_device", lambda: 1)
    got = all_calls()
    assert entered == [0] * 13
    monkeypatch.undo()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert cider.cider_check_device_error(0) == 0
