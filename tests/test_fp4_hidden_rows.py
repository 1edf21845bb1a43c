"""The second product of a feed-forward block overlaps with the end of the launch that writes its rows: it reads them as
written, call for call, where the same scratch comes back with other contents."""
import zlib

import pytest
import torch

import w4a8_quantized_linear_gb300 as cider

pytestmark = pytest.mark.gpu


def layers(gen, k, f, block, n):
    make = lambda rows, cols: cider.cider_quantize_fp4(cols ** -0.5 * torch.randn((rows, cols), generator=gen, device="cuda"), block)
    return [(make(f, k), make(f, k), make(k, f)) for _ in range(n)]


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("m,k,f", [(1, 2048, 6144), (1, 4096, 12288), (3, 1024, 4096), (16, 512, 1024), (16, 1024, 1056)])
def test_a_chain_of_blocks(m, k, f, block):
    """Blocks one behind the other, eager and in a replayed graph, against the block's parts with waits between them."""
    gen = torch.Generator(device="cuda").manual_seed(zlib.crc32(repr((m, k, f, block)).encode()))
    blocks = layers(gen, k, f, block, 4)

    def chain(x):
        outs = []
        for gate, up, down in blocks:
            x = cider.cider_w4a4_feed_forward(x, gate, up, down, block)
            outs.append(x)
        return outs

    def parts(x):
        outs = []
        for gate, up, down in blocks:
            h = cider.cider_w4a4_gated_linear(x, gate, up, block)
            torch.cuda.synchronize()
            x = cider.cider_w4a4_linear(h, down, block)
            torch.cuda.synchronize()
            outs.append(x)
        return outs

    xs = [2 * torch.randn((m, k), generator=gen, device="cuda").bfloat16() for _ in range(5)]
    want = [parts(x) for x in xs]
    assert all(bool(torch.isfinite(t).all()) and bool((t != 0).any()) for w in want for t in w)
    x = xs[0].clone()
    chain(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ys = chain(x)
    for turn in range(25):
        i = turn % len(xs)
        x.copy_(xs[i])
        graph.replay()
        eager = chain(xs[(i + 2) % len(xs)])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ys, want[i]))
        assert all(torch.equal(a, b) for a, b in zip(eager, want[(i + 2) % len(xs)]))
    assert cider.cider_check_device_error() == 0
