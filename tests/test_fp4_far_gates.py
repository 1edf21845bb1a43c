"""Gates far below zero against large values on the other side: right down to where the activation is less than what fp32
holds, and nothing but that number or zero behind it."""
import pytest
import torch

import w4a8_quantized_linear_gb300 as cider
from tests import fp4_reference as ref

pytestmark = pytest.mark.gpu
COLS = 64


def rows_with_sums(sums):
    """Rows of COLS four-bit values with these sums (whole and half numbers of up to 6 COLS)."""
    left = (2 * torch.tensor(sums, dtype=torch.float64)).round().long()
    sign, left = torch.sign(left), left.abs()
    halves = torch.tensor([12, 8, 6, 4, 3, 2, 1])
    v = torch.zeros((len(sums), COLS), dtype=torch.float64)
    for j in range(COLS):
        take = halves[(left[:, None] >= halves).int().argmax(1)] * (left > 0)
        v[:, j] = sign * take / 2.0
        left = left - take
    assert bool((left == 0).all())
    return v


def matrix(v, power):
    """Rows of four-bit values v times 2^power in block size 32, as the library takes it."""
    code = ref.nearest(v.abs(), ref.VALUES) + 8 * (v < 0)
    held = (power + 127)[:, None].expand(-1, COLS // 32)
    return ref.pack(code).cuda().contiguous(), ref.tiles(held).cuda(), None


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=str)
@pytest.mark.parametrize("m,repeat", [(1, 1), (40, 1), (70, 26)], ids=["one", "some", "pairs"])
def test_far_gates(m, repeat, dtype, act):
    # up to t of -190 (the gelu's t is 1.6 (g + 0.0447 g^3))
    steps = 380 if act == "silu" else 27
    g = (-0.5 * (torch.arange(400 * repeat) % (steps + 1))).double()
    t = g if act == "silu" else (8 / torch.pi) ** 0.5 * (g + 0.044715 * g ** 3)
    # the other side makes up for the activation, as far as fp32 goes: products around 2^-6 and 2^-18
    power = (torch.clamp(-t * 1.4427, -20, 120) - (8 + 12 * (torch.arange(len(g)) % 2))).long()
    gate = matrix(rows_with_sums(g.tolist()), torch.zeros(len(g), dtype=torch.long))
    side = torch.zeros((len(g), COLS), dtype=torch.float64)
    side[:, 5] = 4.0
    up = matrix(side, power)
    x = torch.ones((m, COLS), dtype=dtype, device="cuda")
    h = cider.cider_w4a4_gated_linear(x, gate, up, 32, act)
    want = (g * torch.sigmoid(t) * 4.0 * torch.exp2(power.double())).cuda()
    # the sums are exact.  t and its product with log2 e: at most eight roundings of 2^-24; 2^x and the reciprocal: 2 ulp
    # each, four products: together less than 2^-21
    t = t.cuda()
    bound = want.abs() * (t.abs() + 2) * 2.0 ** -21 + ref.half_step(dtype, want) * (1 + 2.0 ** -10)
    # e^87 < 2^126: above t = -87 the denominator and its reciprocal are normal numbers
    bound = torch.where(t < -87, torch.maximum(bound, want.abs()), bound)
    assert bool((bound < want.abs() / 8)[(t >= -87) & (t < -80)].all()) or dtype == torch.float16
    assert bool(torch.isfinite(want).all())
    assert bool(((h.double() - want).abs() <= bound).all()), float(((h.double() - want).abs() / bound).max())
    assert cider.cider_check_device_error() == 0
