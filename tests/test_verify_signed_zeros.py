"""Greedy verification: +0 and -0 are equal, so a tie of them goes to the lowest
index too."""
import pytest
import torch

from tests.parity_util import require_gpu


@pytest.mark.gpu
@pytest.mark.parametrize("vocab", [600, 601, 40000])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_tie_of_zeros(dtype, vocab):
    cider = require_gpu()
    row = torch.full((vocab,), -1.0)
    row[5], row[vocab // 2], row[vocab - 1] = -0.0, 0.0, 0.0
    logits = row.to(dtype).cuda().repeat(2, 1)
    i32 = dict(dtype=torch.int32, device="cuda")
    count, path, nxt = cider.cider_verify_drafts(
        logits, torch.tensor([0, 5], **i32), torch.tensor([-1, 0], **i32), torch.tensor([0, 2], **i32),
        torch.zeros(2, device="cuda"), torch.ones(1, vocab, device="cuda"), 2, temperature=torch.zeros(1, device="cuda"))
    assert count.tolist() == [2] and path.tolist() == [[0, 1]] and nxt.tolist() == [5]
    assert cider.cider_check_device_error() == 0
