"""The operators together, as the example runs them: with temperature 0 every
token that trees of drafts yield is the likeliest one when the text is read in
one pass, up to the rounding that lies between the two paths."""
import importlib.util
import os

import pytest
import torch

from tests.parity_util import require_gpu

EXAMPLE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "speculative_decode.py")


def load():
    spec = importlib.util.spec_from_file_location("speculative_decode", EXAMPLE)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [8, 4])
def test_trees_yield_the_likeliest_tokens(bits):
    cider = require_gpu()
    example = load()
    model = example.Decoder(vocab=504, layers=2)
    prompts = torch.randint(504, (3, 90), generator=torch.Generator().manual_seed(2)).cuda()
    text, steps = example.generate(model, prompts, 40, bits=bits)
    gap = example.gaps(model, prompts, text, bits=bits)
    assert cider.cider_check_device_error() == 0
    # logits are of size 1, their largest about 3: a wrong token is ~3 below; the
    # INT8 activations that an fp16 ulp moves to the next code are worth ~0.05
    assert gap.max() < 0.5 and gap.mean() < 0.05, (gap.max(), gap.mean())
    assert steps < 40
    singles, count = example.generate(model, prompts, 20, [-1], [0], bits=bits)
    assert count == 19
    assert example.gaps(model, prompts, singles, bits=bits).max() < 0.5


@pytest.mark.gpu
def test_sampling_runs():
    cider = require_gpu()
    example = load()
    model = example.Decoder(vocab=504, layers=1)
    prompts = torch.randint(504, (2, 20), generator=torch.Generator().manual_seed(3)).cuda()
    text, _ = example.generate(model, prompts, 12, temperature=0.8)
    assert text.shape == (2, 12) and ((text >= 0) & (text < 504)).all()
    assert cider.cider_check_device_error() == 0
