"""The products' outputs are numbers: the tests of the values against 64 bits, with a comparison that takes no NaN for
one that is near enough."""
import pytest
import torch

from tests import test_fp4
from tests.test_fp4 import test_gated_linear, test_gated_linear_of_many_tokens, test_linear, test_many_tokens  # noqa: F401


def close(y, want, bound):
    assert bool(torch.isfinite(want).all()) and bool(torch.isfinite(bound).all())
    good = (y.double() - want).abs() <= bound
    assert bool(good.all()), (int((~good).sum()), float(((y.double() - want).abs() / bound).nan_to_num(torch.inf).max()))


@pytest.fixture(autouse=True)
def strict(monkeypatch):
    monkeypatch.setattr(test_fp4, "close", close)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_the_comparison_itself(value):
    want = torch.ones(3, 5, dtype=torch.float64)
    y = want.half()
    close(y, want, torch.zeros_like(want))
    y[1, 2] = value
    with pytest.raises(AssertionError):
        close(y, want, torch.ones_like(want))
    with pytest.raises(AssertionError):
        close(want.half(), y.double(), torch.ones_like(want))
