"""The waits between the CTAs that verify one request have a limit: a rank that
sends nothing ends the request with an error that the host reads, for every
thread alike, and the next call is as if nothing had happened."""
import time

import numpy as np
import pytest
import torch

from tests import test_verify_drafts as drafts
from tests.parity_util import require_gpu
from w4a8_quantized_linear_gb300 import _build

OK, INVALID, UNSUPPORTED, TIMEOUT = 0, 1, 3, 5
P = 0x10000


@pytest.mark.parametrize("wait,silent,status", [(0, 0, INVALID), (100001, 0, INVALID), (-5, 0, INVALID),
                                                (10, -2, INVALID), (10, -1, UNSUPPORTED), (10, 9, UNSUPPORTED)])
def test_refusals(monkeypatch, wait, silent, status):
    monkeypatch.setenv("CIDER_FORCE_UNSUPPORTED", "1")
    _build.build()
    import w4a8_quantized_linear_gb300 as pkg
    call = pkg.library().cider_debug_verify_timeout
    assert call(P, 1001, 0, P, P, P, 2, 5, 1001, 4, P, P, None, None, P, P, P, wait, silent, None) == status
    assert call(P, 1001, 0, P, P, P, 2, 5, 0, 4, P, P, None, None, P, P, P, 10, -1, None) == INVALID


@pytest.mark.gpu
@pytest.mark.parametrize("sampled", [False, True])
@pytest.mark.parametrize("silent", [0, 1, 7])
def test_a_rank_that_sends_nothing(silent, sampled):
    """40000 tokens and few requests: eight CTAs to a request."""
    cider = require_gpu()
    rng = np.random.default_rng(silent)
    nodes, vocab, most = [5, 0, 9, 1], 40000, 9
    d = drafts.inputs(rng, nodes, vocab, 2, sampled, "fp16", temperature=[1.0, 1.0, 0.7, 0.0])
    want = drafts.launch(cider, d, most)
    assert cider.cider_check_device_error() == OK
    dev = {k: torch.from_numpy(v).cuda() for k, v in d.items() if isinstance(v, np.ndarray)}
    logits = d["logits"].cuda()
    count = torch.full((4,), 7, dtype=torch.int32, device="cuda")
    nxt, path = count.clone(), torch.full((4, most), 7, dtype=torch.int32, device="cuda")

    def call(rank, us):
        draft = dev["draft"].data_ptr() if sampled else None
        return cider.library().cider_debug_verify_timeout(
            logits.data_ptr(), vocab, 0, dev["tokens"].data_ptr(), dev["parents"].data_ptr(), dev["offsets"].data_ptr(),
            4, sum(nodes), vocab, most, dev["uniforms"].data_ptr(), dev["noise"].data_ptr(), draft,
            dev["temperature"].data_ptr(), count.data_ptr(), path.data_ptr(), nxt.data_ptr(), us, rank,
            torch.cuda.current_stream().cuda_stream)

    begin = time.monotonic()
    assert call(silent, 1000) == OK
    assert cider.cider_check_device_error() == TIMEOUT
    assert time.monotonic() - begin < 20.0
    assert (count == 0).all() and (nxt == -1).all() and (path == -1).all()
    for rank in (-1, 8):
        assert call(rank, 100000) == OK
        assert cider.cider_check_device_error() == OK
        for got, w in zip((count, path, nxt), want):
            assert np.array_equal(got.cpu().numpy(), w)
    for got, w in zip(drafts.launch(cider, d, most), want):
        assert np.array_equal(got, w)
