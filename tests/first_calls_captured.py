"""Run by tests/test_first_call_in_capture.py in a process of its own: the first use of every kernel, and of the library's
scratch memory, is inside a stream capture.  Each graph is replayed and compared with the same call afterwards."""
import sys

import torch

import w4a8_quantized_linear_gb300 as cider


def fp4(rows, cols, block):
    """Any codes; scales of 1/32, and with block size 16 of rows: 1/32 as E4M3, and 1."""
    return (torch.randint(0, 256, (rows, cols // 2), dtype=torch.uint8, device="cuda"),
            torch.full((-(-rows // 128), -(-cols // (4 * block)), 512), 0x10 if block == 16 else 122, dtype=torch.uint8, device="cuda"),
            torch.ones(rows, device="cuda") if block == 16 else None)


def int8(n, k):
    return torch.randint(-127, 128, (n, k), dtype=torch.int8, device="cuda"), 0.01 * torch.rand((n, 1), device="cuda")


def calls():
    rows = lambda m, k: torch.randn((m, k), device="cuda").half()
    for block in (16, 32):
        w, g, d = fp4(1024, 512, block), fp4(1024, 512, block), fp4(512, 1024, block)
        for m in (1, 40, 5000):
            x = rows(m, 512)
            yield f"feed-forward {m} {block}", lambda: cider.cider_w4a4_feed_forward(x, w, g, d, block)
            yield f"gated {m} {block}", lambda: cider.cider_w4a4_gated_linear(x, w, g, block)
            yield f"linear {m} {block}", lambda: cider.cider_w4a4_linear(x, w, block)
        yield f"quantize {block}", lambda: cider.cider_dequantize_fp4(cider.cider_quantize_fp4(x, block), block)
    for n, k in ((512, 1024), (2048, 768)):
        (w, s), (p, _) = int8(n, k), int8(n, k // 2)
        for m in (1, 9, 300, 4096):
            x = rows(m, k)
            yield f"w8a8 {m} {n}", lambda: cider.cider_w8a8_linear(x, w, s)
            yield f"w4a8 {m} {n}", lambda: cider.cider_w4a8_linear(x, p.view(torch.uint8), s)
            sg = 0.01 * torch.rand((n, k // 128), device="cuda")
            yield f"w8a8 groups {m} {n}", lambda: cider.cider_w8a8_linear(x, w, sg, 128)
    yield "quantize_act", lambda: cider.cider_quantize_act(x)


def main(order):
    torch.manual_seed(1)
    done = 0
    for name, call in calls():
        if (order == "fp4") == name.startswith(("w8a8", "w4a8", "quantize_act")):
            continue
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = call()
        graph.replay()
        torch.cuda.synchronize()
        want = call()
        for a, b in zip(y if isinstance(y, tuple) else (y,), want if isinstance(want, tuple) else (want,)):
            assert torch.equal(a, b), name
        done += 1
    assert cider.cider_check_device_error() == 0
    print(done, "captured")


if __name__ == "__main__":
    main(sys.argv[1])
