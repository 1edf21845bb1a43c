"""Products on CTA pairs, wherever the dispatch begins to use them: their numbers of tokens are asked of the entry points'
own code for this GPU, and so stay on pairs when the dispatch changes."""
import pytest
import torch

import w4a8_quantized_linear_gb300 as cider
from tests import fp4_reference as ref
from tests.fp4_calls import FEW, PAIRS, first_on_pairs, product_kernels
from tests.test_fp4 import activations, generator, normal
from tests.test_fp4_numbers import close

pytestmark = pytest.mark.gpu


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def both_on_pairs(k, f, n, block):
    """The fewest tokens for which both products of a feed-forward block run on pairs."""
    return max(first_on_pairs(f, k, block, True, sms()), first_on_pairs(n, f, block, False, sms()))


def clean():
    assert cider.cider_check_device_error() == 0


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("more", [0, 1, 131])
@pytest.mark.parametrize("k,f,n", [(512, 1312, 2560), (288, 2080, 1032), (1024, 3104, 1024)])
def test_feed_forward_with_both_products_on_pairs(k, f, n, more, block):
    """The second one's rows are what the first one's epilogue wrote, or the quantizer behind it."""
    gen = generator(k, f, n, more, block)
    m = both_on_pairs(k, f, n, block) + more
    for dtype, act in ((torch.float16, "gelu"), (torch.bfloat16, "silu")):
        x = activations(gen, m, k, dtype)
        gate, up = (cider.cider_quantize_fp4(0.03 * normal(gen, f, k), block) for _ in range(2))
        down = cider.cider_quantize_fp4(0.03 * normal(gen, n, f), block)
        y = cider.cider_w4a4_feed_forward(x, gate, up, down, block, act)
        h = cider.cider_w4a4_gated_linear(x, gate, up, block, act)
        assert torch.equal(y, cider.cider_w4a4_linear(h, down, block))
        a, b = ref.values(ref.matrix(h, block), block), ref.values(down, block)
        close(y, a @ b.T, ref.sum_bound(a, b) + ref.half_step(dtype, a @ b.T) * (1 + 2.0 ** -10))
    clean()


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("n,k", [(1000, 736), (2568, 512)])
def test_quantized_input(n, k, block):
    """On either side of the border: the call that quantizes, and the one of rows that are quantized already."""
    gen = generator(n, k, block)
    a, b = (cider.cider_quantize_fp4(0.05 * normal(gen, n, k), block) for _ in range(2))
    for gated in (False, True):
        first = first_on_pairs(n, k, block, gated, sms())
        for m, kernel in ((first - 1, FEW), (first, PAIRS), (2 * first + 77, PAIRS)):
            assert product_kernels(m, n, k, block, gated, sms()) == kernel
            x = activations(gen, m, k, torch.bfloat16)
            qx = cider.cider_quantize_fp4(x, block)
            if gated:
                assert torch.equal(cider.cider_w4a4_gated_linear_prequant(qx, a, b, block, "gelu", torch.bfloat16),
                                   cider.cider_w4a4_gated_linear(x, a, b, block, "gelu"))
            else:
                y = cider.cider_w4a4_linear(x, a, block)
                assert torch.equal(cider.cider_w4a4_linear_prequant(qx, a, block, torch.bfloat16), y)
                v, w = ref.values(ref.matrix(x, block), block), ref.values(a, block)
                close(y, v @ w.T, ref.sum_bound(v, w) + ref.half_step(torch.bfloat16, v @ w.T) * (1 + 2.0 ** -10))
    clean()


@pytest.mark.parametrize("block", [16, 32])
def test_captured_replayed_and_on_two_streams(block):
    """Pairs as programmatic dependents in a graph, replayed with other inputs, beside the same calls on another stream."""
    k, f = 1024, 1536
    gen = generator(block)
    m = both_on_pairs(k, f, k, block) + 40
    gate, up = (cider.cider_quantize_fp4(0.03 * normal(gen, f, k), block) for _ in range(2))
    down = cider.cider_quantize_fp4(0.03 * normal(gen, k, f), block)
    xs = [activations(gen, m, k, torch.bfloat16) for _ in range(4)]
    want = [cider.cider_w4a4_linear(cider.cider_w4a4_gated_linear(x, gate, up, block), down, block) for x in xs]
    x = xs[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = cider.cider_w4a4_feed_forward(x, gate, up, down, block)
        z = cider.cider_w4a4_feed_forward(y, gate, up, down, block)
    for i in range(12):
        x.copy_(xs[i % 4])
        graph.replay()
        with torch.cuda.stream(side):
            other = cider.cider_w4a4_feed_forward(xs[3 - i % 4], gate, up, down, block)
        torch.cuda.synchronize()
        assert torch.equal(y, want[i % 4]) and torch.equal(other, want[3 - i % 4])
        assert torch.equal(z, cider.cider_w4a4_feed_forward(want[i % 4], gate, up, down, block))
    clean()


@pytest.mark.parametrize("block", [16, 32])
def test_output_on_the_input(block):
    k = 2560
    gen = generator(block, "on")
    w, u = (cider.cider_quantize_fp4(0.05 * normal(gen, k, k), block) for _ in range(2))
    m = both_on_pairs(k, k, k, block) + 3
    for call in (lambda x, **kw: cider.cider_w4a4_linear(x, w, block, **kw),
                 lambda x, **kw: cider.cider_w4a4_gated_linear(x, w, u, block, **kw),
                 lambda x, **kw: cider.cider_w4a4_feed_forward(x, w, u, w, block, **kw)):
        x = activations(gen, m, k, torch.bfloat16)
        want = call(x)
        for _ in range(3):
            z = x.clone()
            assert call(z, out=z) is z and torch.equal(z, want)
    clean()
