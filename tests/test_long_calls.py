"""A call may take longer than a wait inside of it may (2 s): no wait of the products on CTA pairs begins with the call."""
import pytest
import torch

import w4a8_quantized_linear_gb300 as cider

pytestmark = pytest.mark.gpu
GIB = 1 << 30


@pytest.fixture
def room():
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    stream = torch.cuda.current_stream().cuda_stream
    assert cider.library().cider_trim_scratch_pool(0, stream) == 0
    if torch.cuda.mem_get_info()[0] < 150 * GIB:
        pytest.skip("needs 150 GiB of device memory")
    yield
    torch.cuda.empty_cache()
    assert cider.library().cider_trim_scratch_pool(0, stream) == 0


def clean():
    torch.cuda.synchronize()
    assert cider.cider_check_device_error() == 0


def test_gated_product_of_four_bits(room):
    m, f, k, tail = 2560 * 128, 1 << 17, 1 << 17, 39 * 128
    codes = lambda rows: torch.randint(0, 256, (rows, k // 2), dtype=torch.uint8, device="cuda")
    scales = lambda rows, byte: torch.full((rows // 128, k // 128, 512), byte, dtype=torch.uint8, device="cuda")
    qx, gate = (codes(m), scales(m, 120), None), (codes(f), scales(f, 120), None)
    h = cider.cider_w4a4_gated_linear_prequant(qx, gate, gate)
    clean()
    few = (qx[0][m - tail:], qx[1][(m - tail) // 128:], None)
    assert torch.equal(h[m - tail:], cider.cider_w4a4_gated_linear_prequant(few, gate, gate))
    assert bool((h[m - tail:] != 0).any()) and bool(torch.isfinite(h[m - tail:]).all())
    clean()


@pytest.mark.parametrize("group", [0, 128])
def test_int8_product(room, group):
    # per channel rows as long as these are multiplied in parts that fp32 holds exactly, which takes four times as long
    m, n, k, tail = 1 << 17 if group else 1 << 15, 1 << 17, 1 << 17, 4096
    x = torch.randn((m, k), dtype=torch.float16, device="cuda")
    w = torch.randint(-127, 128, (n, k), dtype=torch.int8, device="cuda")
    s = torch.full((n, k // group if group else 1), 2.0 ** -14, device="cuda")
    y = cider.cider_w8a8_linear(x, w, s, group)
    clean()
    assert torch.equal(y[m - tail:], cider.cider_w8a8_linear(x[m - tail:], w, s, group))
    assert bool((y[m - tail:] != 0).any()) and bool(torch.isfinite(y[m - tail:]).all())
    clean()
