"""Cases of microscaled 4-bit floating point and of the linears that run on it.

Four operators, as a server that keeps its weights in four bits uses them:

  quantize  a matrix becomes 4-bit floating point (E2M1) with a scale for every
            block of a row: 32 values with a power of two (E8M0), or 16 values
            with an E4M3 number and one fp32 scale for the row.  It is read back
            as the values that the codes stand for
  linear    y = x W^T: the rows of x are quantized, the product is taken in four
            bits on both sides, the sum in fp32
  gated     h = act(x G^T) (x U^T), the first half of a gated feed-forward block:
            both projections, the activation and the product, on one quantized x
  forward   y = h D^T of such an h, rounded to x's type and quantized again: the
            whole block

`own` False: plain torch operations in 32 bits.  `own` True: this repository's
entry points.
"""
import math

import torch

own = False

_TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
_LARGEST = 2 * 2 * 4096 * 12288 * 4096  # operations of the largest case


# --------------------------------------------------------------------- cases
def listed():
    """Layer shapes: 10240 x 2560 and its transpose, and the feed-forward blocks of
    hidden sizes 2048 (6144 wide) and 4096 (12288 wide), those of this
    repository's benchmark."""
    return [
        # one token's activations: the smallest call
        _quantize_case(name="quantize_token", rows=1, k=2560, dtype="fp16", block=16),
        # a prompt's activations, an odd number of rows, a last block row that is not full
        _quantize_case(name="quantize_ragged", rows=1333, k=2080, dtype="bf16", block=16),
        # a prompt of 4096 tokens
        _quantize_case(name="quantize_prompt", rows=4096, k=4096, dtype="bf16", block=32),
        # a layer's fp32 weights, as they are quantized once when a model is loaded
        _quantize_case(name="quantize_weight", rows=10240, k=2560, dtype="fp32", block=16),
        # decoding one token: the weights are read once
        _linear_case(name="linear_token", m=1, n=10240, k=2560, dtype="fp16", block=16),
        # a decoding batch of 16, few outputs of long rows
        _linear_case(name="linear_few", m=16, n=2560, k=10240, dtype="bf16", block=32),
        # odd sizes everywhere
        _linear_case(name="linear_ragged", m=333, n=1000, k=2080, dtype="fp16", block=16),
        # a prompt of 4096 tokens, the benchmark's shape
        _linear_case(name="linear_prompt", m=4096, n=10240, k=2560, dtype="fp16", block=16),
        # a feed-forward block while one token is decoded
        _gated_case(name="gated_token", m=1, f=6144, k=2048, dtype="bf16", block=32, act="silu"),
        # a prompt of 4096 tokens through the larger block: the largest
        _gated_case(name="gated_prompt", m=4096, f=12288, k=4096, dtype="bf16", block=32, act="silu"),
        # the whole block: a decoding batch, an odd number of tokens
        _forward_case(name="forward_batch", m=61, f=12288, k=4096, dtype="fp16", block=16, act="gelu"),
        # the tokens of an image through the smaller block
        _forward_case(name="forward_image", m=1334, f=6144, k=2048, dtype="bf16", block=32, act="silu"),
    ]


def _quantize_case(**kw):
    return {"op": "quantize", **kw}


def _linear_case(**kw):
    return {"op": "linear", **kw}


def _gated_case(**kw):
    return {"op": "gated", **kw}


def _forward_case(**kw):
    return {"op": "forward", **kw}


def _log(rng, lo, hi, step=1):
    """A multiple of step between lo and hi, spread over the logarithm; odd multiples more often than not."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step))
    v = max(1, v | 1 if rng.random() < 0.6 else v)
    return max(lo, min(hi, v * step))


def draw(rng):
    op = rng.choice(("quantize", "linear", "linear", "gated", "forward"))
    block = rng.choice((16, 32))
    if op == "quantize":
        dtype = rng.choice(("fp16", "bf16", "fp32"))
        k = _log(rng, 64, 12288, 32)
        return _quantize_case(rows=_log(rng, 1, max(1, 10240 * 2560 // k)), k=k, dtype=dtype, block=block)
    dtype = rng.choice(("fp16", "bf16"))
    k = _log(rng, 64, 10240, 32)
    n = _log(rng, 64, 12288, 32 if op == "forward" else 8)
    most = _LARGEST // (2 * n * k * {"linear": 1, "gated": 2, "forward": 3}[op])
    # outputs of at most what the largest case writes
    m = _log(rng, 1, max(1, min(8192, most, 4096 * 12288 // n)))
    if op == "linear":
        return _linear_case(m=m, n=n, k=k, dtype=dtype, block=block)
    return (_gated_case if op == "gated" else _forward_case)(m=m, f=n, k=k, dtype=dtype, block=block, act=rng.choice(("silu", "gelu")))


# ---------------------------------------------------------------- sizes of a case
def _held(rows, k, block):
    """Bytes of a quantized matrix: codes, block scales, row scales."""
    return rows * k // 2 + rows * (k // block) + (4 * rows if block == 16 else 0)


def work(case):
    block = case["block"]
    if case["op"] == "quantize":
        rows, k = case["rows"], case["k"]
        wide = rows * k * (4 if case["dtype"] == "fp32" else 2)
        return {"bytes": 2 * wide + 2 * _held(rows, k, block), "flops": 4 * rows * k}
    m, k = case["m"], case["k"]
    if case["op"] == "forward":
        # the hidden values need not leave the chip
        f = case["f"]
        return {"bytes": 2 * m * k + 2 * _held(f, k, block) + _held(k, f, block) + 2 * m * k, "flops": 6 * m * f * k}
    n, sides = (case["n"], 1) if case["op"] == "linear" else (case["f"], 2)
    return {"bytes": 2 * m * k + sides * _held(n, k, block) + 2 * m * n, "flops": 2 * sides * m * n * k}


# ------------------------------------------------------------------ the format
def _power(k):
    """2^k in fp32 for whole numbers k of -126 .. 127."""
    return ((k.clamp(-126, 127) + 127).to(torch.int32) << 23).view(torch.float32)


def _e2m1(q):
    """The codes 0 .. 7 of the values nearest to q >= 0, ties to the even code."""
    return (q > 0.25).int() + (q >= 0.75).int() + (q > 1.25).int() + (q >= 1.75).int() + (q > 2.5).int() + (q >= 3.5).int() + (q > 5.0).int()


def _encode(x, block):
    """x [rows, k] -> (codes int 0 .. 15 [rows, k], block scales' bytes [rows, k / block], row scales [rows] or None)."""
    rows, k = x.shape
    x = x.float()
    top = x.abs().view(rows, k // block, block).amax(-1)
    if block == 32:
        # the smallest power of two that keeps the block's largest value within 6
        part, e = torch.frexp(top)
        e = torch.where(top == 0, torch.zeros_like(e), e - 3 + (part > 0.75).int())
        q = x.view(rows, -1, block) / _power(e)[..., None]
        held, row = (e + 127).to(torch.uint8), None
    else:
        # the smallest power of two that keeps the row's largest value within 6 * 448
        largest = top.amax(-1)
        part, e = torch.frexp(largest)
        row = torch.where(largest == 0, torch.ones_like(largest), _power(e - 12 + (part > 0.65625).int()))
        scaled = top / row[:, None]
        b8 = (scaled / torch.full_like(scaled, 6.0)).to(torch.float8_e4m3fn)  # by a tensor: torch multiplies by the reciprocal of a number
        held, b = b8.view(torch.uint8), b8.float()
        q = (x / row[:, None]).view(rows, -1, block) / torch.where(b == 0, torch.full_like(b, math.inf), b)[..., None]
    q = q.reshape(rows, k)
    return _e2m1(q.abs()) + 8 * (q < 0).int(), held, row


def _values(codes, held, row, block):
    """fp32 values of codes 0 .. 15 [rows, k] with their scales."""
    rows, k = codes.shape
    size = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0] + [-0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device=codes.device)
    b = _power(held.int() - 127) if block == 32 else held.view(torch.float8_e4m3fn).float()
    v = (size[codes].view(rows, -1, block) * b[..., None]).view(rows, k)
    return v if row is None else v * row[:, None]


def _tiles(held):
    """Block scales [rows, n] as the product reads them: tiles of 128 rows x 4 blocks; byte 16 (r % 32) + 4 (r // 32) + j of a tile
    is row r's block j.  Zeros past the last row and block."""
    rows, n = held.shape
    held = torch.nn.functional.pad(held, (0, -n % 4, 0, -rows % 128))
    return held.view(held.shape[0] // 128, 4, 32, held.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).reshape(held.shape[0] // 128, -1, 512).contiguous()


def _untiled(tiles, rows, n):
    t, a, _ = tiles.shape
    return tiles.view(t, a, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(t * 128, a * 4)[:rows, :n].contiguous()


def _pack(codes):
    return (codes[:, 0::2] | codes[:, 1::2] << 4).to(torch.uint8)


def _unpack(packed):
    return torch.stack((packed & 15, packed >> 4), -1).flatten(1).long()


def _weight(w, block):
    """A quantized matrix as a program keeps it: packed codes, tiles of block scales, row scales."""
    codes, held, row = _encode(w, block)
    return _pack(codes), _tiles(held), row


def _plain(q, block):
    packed, tiles, row = q
    codes = _unpack(packed)
    return _values(codes, _untiled(tiles, codes.shape[0], codes.shape[1] // block), row, block)


# --------------------------------------------------------------------- inputs
def _activations(gen, rows, k, dtype):
    """Normal values with one channel in a hundred twenty times as large."""
    x = torch.randn((rows, k), generator=gen, device="cuda")
    wide = torch.randperm(k, generator=gen, device="cuda")[: max(1, k // 100)]
    x[:, wide] *= 20.0
    return x.to(dtype)


def _layer(gen, n, k, block):
    return _weight(0.02 * torch.randn((n, k), generator=gen, device="cuda"), block)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, block, k, dtype = case["op"], case["block"], case["k"], _TYPES[case["dtype"]]
    st = {"op": op, "block": block}
    if op == "quantize":
        if case["dtype"] == "fp32":
            st["x"] = 0.02 * torch.randn((case["rows"], k), generator=gen, device="cuda")
        else:
            st["x"] = _activations(gen, case["rows"], k, dtype)
        return st
    st["x"] = _activations(gen, case["m"], k, dtype)
    if op == "linear":
        st["w"] = _layer(gen, case["n"], k, block)
    else:
        # sums of a thousand products of such values are of size one: gates on both sides of zero
        st["gate"], st["up"], st["act"] = _layer(gen, case["f"], k, block), _layer(gen, case["f"], k, block), case["act"]
    if op == "forward":
        st["down"] = _layer(gen, k, case["f"], block)
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    return {"quantize": _quantize, "linear": _linear, "gated": _gated, "forward": _forward}[st["op"]](st)


def _quantize(st):
    x, block = st["x"], st["block"]
    if own:
        import w4a8_quantized_linear_gb300 as cider

        return cider.cider_dequantize_fp4(cider.cider_quantize_fp4(x, block), block, x.dtype)
    return _values(*_through(x, block), block).to(x.dtype)


def _through(x, block):
    codes, held, row = _encode(x, block)
    return codes.long(), held, row


def _linear(st):
    x, block = st["x"], st["block"]
    if own:
        import w4a8_quantized_linear_gb300 as cider

        return cider.cider_w4a4_linear(x, st["w"], block)
    return torch.matmul(_values(*_through(x, block), block), _plain(st["w"], block).T).to(x.dtype)


def _gated(st):
    x, block = st["x"], st["block"]
    if own:
        import w4a8_quantized_linear_gb300 as cider

        return cider.cider_w4a4_gated_linear(x, st["gate"], st["up"], block, st["act"])
    v = _values(*_through(x, block), block)
    g = torch.matmul(v, _plain(st["gate"], block).T)
    u = torch.matmul(v, _plain(st["up"], block).T)
    if st["act"] == "silu":
        a = g / (1.0 + torch.exp(-g))
    else:
        a = 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))
    return (a * u).to(x.dtype)


def _forward(st):
    if own:
        import w4a8_quantized_linear_gb300 as cider

        return cider.cider_w4a4_feed_forward(st["x"], st["gate"], st["up"], st["down"], st["block"], st["act"])
    h = _gated(st)
    return torch.matmul(_values(*_through(h, st["block"]), st["block"]), _plain(st["down"], st["block"]).T).to(h.dtype)


# ------------------------------------------------------------------ 64 bits
def _rounded(x, block):
    """The values that x is quantized to, in 64 bits.  The format takes its quotients to 24 bits; all else here is exact."""
    rows, k = x.shape
    v = x.double().view(rows, k // block, block)
    top = v.abs().amax(-1, keepdim=True)
    if block == 32:
        b = torch.exp2(torch.ceil(torch.log2(torch.where(top > 0, top / 6.0, torch.ones_like(top)))).clamp_min(-127.0))
        # the logarithm is rounded: one step down or up where it was
        b = torch.where(top <= 3.0 * b, torch.where(top > 0, b / 2, b), torch.where(top > 6.0 * b, 2 * b, b))
        row = 1.0
    else:
        most = top.amax(1, keepdim=True)
        row = torch.exp2(torch.ceil(torch.log2(torch.where(most > 0, most / 2688.0, torch.ones_like(most)))))
        row = torch.where(most <= 1344.0 * row, torch.where(most > 0, row / 2, row), torch.where(most > 2688.0 * row, 2 * row, row))
        t = (top / row / 6.0).float().double()
        # E4M3: three bits behind the leading one, whole multiples of 2^-9 at the low end
        step = torch.exp2(torch.floor(torch.log2(t.clamp_min(2.0**-6))) - 3.0)
        b = torch.round(t / step) * step
    q = torch.where(b > 0, v / row / torch.where(b > 0, b, torch.ones_like(b)), torch.zeros_like(v)).float().double()
    # E2M1: steps of 1/2 below 2, of 1 below 4, of 2 up to 6
    step = torch.where(q.abs() < 2, 0.5, torch.where(q.abs() < 4, 1.0, 2.0)).double()
    return ((torch.round(q / step) * step).clamp(-6.0, 6.0) * b * row).view(rows, k)


def _kept(q, block):
    """A quantized matrix in 64 bits, from its bytes."""
    packed, tiles, row = q
    rows, k = packed.shape[0], 2 * packed.shape[1]
    c = torch.empty((rows, k), dtype=torch.int64, device=packed.device)
    c[:, 0::2], c[:, 1::2] = (packed % 16).long(), (packed // 16).long()
    e, m = (c % 8) // 2, (c % 2).double()
    size = torch.where(e == 0, 0.5 * m, torch.exp2(e.double() - 1.0) * (1.0 + 0.5 * m))
    r = torch.arange(rows, device=packed.device)[:, None]
    j = torch.arange(k // block, device=packed.device)[None]
    held = tiles[r // 128, j // 4, 16 * (r % 32) + 4 * (r % 128 // 32) + j % 4].long()
    if block == 32:
        b = torch.exp2(held.double() - 127.0)
    else:
        be, bm = held // 8, (held % 8).double()
        b = torch.where(be == 0, bm * 2.0**-9, torch.exp2(be.double() - 7.0) * (1.0 + bm / 8.0))
    v = torch.where(c >= 8, -size, size).view(rows, -1, block) * b[..., None]
    return v.view(rows, k) if row is None else v.view(rows, k) * row.double()[:, None]


def exact(case, seed):
    st = prepare(case, seed)
    block = case["block"]
    v = _rounded(st["x"], block)
    if case["op"] == "quantize":
        return v
    if case["op"] == "linear":
        return v @ _kept(st["w"], block).T
    g, u = v @ _kept(st["gate"], block).T, v @ _kept(st["up"], block).T
    h = (g * torch.sigmoid(g) if case["act"] == "silu" else torch.nn.functional.gelu(g, approximate="tanh")) * u
    if case["op"] == "gated":
        return h
    return _rounded(h.to(st["x"].dtype), block) @ _kept(st["down"], block).T
