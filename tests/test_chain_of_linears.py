"""Launches of a call overlap: each reads the codes, scales and partial sums as the one before wrote them, call for call,
where the same scratch comes back with other contents."""
import zlib

import pytest
import torch

import w4a8_quantized_linear_gb300 as cider

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("m", [1, 4, 16, 200, 1100])
def test_a_chain_of_linears(m, int4, group):
    gen = torch.Generator(device="cuda").manual_seed(zlib.crc32(repr((m, int4, group)).encode()))
    call = cider.cider_w4a8_linear if int4 else cider.cider_w8a8_linear
    layers = []
    for n, k in ((512, 4096), (4096, 512), (512, 4096), (2560, 512)):
        w = torch.randint(-128, 128, (n, k // 2 if int4 else k), generator=gen, dtype=torch.int8, device="cuda")
        if not int4:
            w.clamp_(min=-127)
        s = (0.5 + torch.rand((n, k // group if group else 1), generator=gen, device="cuda")) / (k ** 0.5 * (4.6 if int4 else 74))
        layers.append((w.view(torch.uint8) if int4 else w, s))

    def chain(x, wait=False):
        outs = []
        for w, s in layers:
            x = call(x, w, s, group)
            outs.append(x)
            if wait:
                torch.cuda.synchronize()
        return outs

    # rows of very different size, so that another call's scales are far from right
    xs = [(torch.randn((m, 4096), generator=gen, device="cuda") * torch.exp2(torch.randint(-4, 5, (m, 1), generator=gen, device="cuda"))).half()
          for _ in range(5)]
    want = [chain(x, wait=True) for x in xs]
    assert all(bool(torch.isfinite(t).all()) and bool((t != 0).any()) for w in want for t in w)
    x = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ys = chain(x)
    for turn in range(25):
        i, j = turn % 5, (turn + 2) % 5
        x.copy_(xs[i])
        graph.replay()
        eager = chain(xs[j])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ys, want[i]))
        assert all(torch.equal(a, b) for a, b in zip(eager, want[j]))
    assert cider.cider_check_device_error() == 0
