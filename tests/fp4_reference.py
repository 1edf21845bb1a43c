"""Microscaled 4-bit floating point in 64 bits, from the format's definition: what
the kernels' codes, scales and products are compared with."""
import torch

VALUES = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def power_at_least(a, top, low):
    """The smallest 2^k, k >= low, with a <= top 2^k (a > 0; both 64-bit)."""
    k = torch.full_like(a, float(low))
    # exact: a and top have few bits, 2^k is a power of two
    guess = torch.floor(torch.log2(torch.clamp_min(a, 1e-300) / top)) - 1
    for step in (0, 1, 2, 3):
        k = torch.where(a > top * torch.exp2(torch.maximum(guess + step - 1, torch.full_like(a, low))),
                        torch.maximum(guess + step, torch.full_like(a, low)), k)
    return k


def nearest(q, grid):
    """Index of the value of an increasing grid nearest to q >= 0, ties to the even index."""
    g = grid.to(q.device)
    mid = (g[1:] + g[:-1]) / 2
    lo = torch.searchsorted(mid, q.contiguous(), right=False)   # mid[lo - 1] < q <= mid[lo]
    hi = torch.searchsorted(mid, q.contiguous(), right=True)
    return torch.where(lo % 2 == 0, lo, hi)


def e4m3_grid():
    g = [m * 2.0 ** -9 for m in range(8)]
    g += [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
    return torch.tensor(g[:127], dtype=torch.float64)   # 0x7F is NaN


def quantize(x, block):
    """x [rows, cols] -> codes [rows, cols] (0..15), scale bytes [rows, cols / block], row scales or None."""
    rows, cols = x.shape
    v = x.double().view(rows, cols // block, block)
    finite = torch.isfinite(v)
    top = torch.where(finite, v.abs(), torch.zeros_like(v)).amax(-1)
    if block == 32:
        bad = ~finite.all(-1)
        k = torch.where(top > 0, power_at_least(top, 6.0, -127), torch.zeros_like(top))
        q = v / torch.exp2(k)[..., None]
        held = torch.where(bad, torch.full_like(k, 255), k + 127).long()
        row = None
        dead = bad[..., None].expand_as(v)
    else:
        bad = ~finite.flatten(1).all(-1)
        most = top.amax(-1)
        k = torch.where(most > 0, power_at_least(most, 2688.0, -126), torch.zeros_like(most))
        r = torch.exp2(k)
        t = (top / r[:, None] / 6.0).float().double()
        grid = e4m3_grid()
        held = nearest(t, grid)
        b = grid.to(x.device)[held]
        q = (v / r[:, None, None] / torch.where(b > 0, b, torch.full_like(b, torch.inf))[..., None]).float().double()
        held = torch.where(bad[:, None], torch.zeros_like(held), held)
        row = torch.where(bad, torch.full_like(r, torch.nan), r).float()
        dead = bad[:, None, None].expand_as(v) | (b == 0)[..., None].expand_as(v)
    codes = nearest(q.abs().nan_to_num(0.0), VALUES) + 8 * torch.signbit(v).long()
    codes = torch.where(dead, torch.zeros_like(codes), codes)
    return codes.view(rows, cols), held, row


def pack(codes):
    return (codes[:, 0::2] | codes[:, 1::2] << 4).to(torch.uint8)


def tiles(held):
    """Scale bytes [rows, blocks] in the layout of the header: tiles of 128 rows x 4 blocks, zeros behind the end."""
    rows, blocks = held.shape
    out = torch.zeros(((rows + 127) // 128, (blocks + 3) // 4, 512), dtype=torch.uint8, device=held.device)
    r = torch.arange(rows, device=held.device)[:, None]
    j = torch.arange(blocks, device=held.device)[None]
    out[r // 128, j // 4, 16 * (r % 32) + 4 * (r % 128 // 32) + j % 4] = held.to(torch.uint8)
    return out


def values(q, block):
    """64-bit values of (packed codes, tiles, row scales)."""
    packed, t, row = q
    rows, cols = packed.shape[0], 2 * packed.shape[1]
    codes = torch.stack((packed & 15, packed >> 4), -1).flatten(1).long()
    size = torch.cat((VALUES, -VALUES)).to(packed.device)[codes]
    r = torch.arange(rows, device=packed.device)[:, None]
    j = torch.arange(cols // block, device=packed.device)[None]
    held = t[r // 128, j // 4, 16 * (r % 32) + 4 * (r % 128 // 32) + j % 4].long()
    if block == 32:
        b = torch.where(held == 255, torch.full(held.shape, torch.nan, dtype=torch.float64, device=held.device),
                        torch.exp2(held.double() - 127))
    else:
        b = e4m3_grid().to(packed.device)[held.clamp_max(126)]
    v = (size.view(rows, -1, block) * b[..., None]).view(rows, cols)
    return v if row is None else v * row.double()[:, None]


def matrix(w, block):
    """A matrix quantized by the reference, as the library takes it."""
    codes, held, row = quantize(w, block)
    return pack(codes).contiguous(), tiles(held), row


def half_step(t, y):
    """Half a step of type t at |y|: what one rounding to it is off by at most."""
    info = torch.finfo(t)
    return torch.maximum(y.abs() * (info.eps / 2), torch.full_like(y, info.tiny * info.eps / 2))


def sum_bound(a, w):
    """What fp32 sums of the products may be off by: an MMA adds 64 of them to the running sum, and each of these
    K / 64 steps (and four for the two row scales and the sums over a cluster) is off by at most two units in the
    last place of the sum of the absolute products."""
    return (a.shape[1] / 64 + 4) * 2.0 ** -22 * (a.abs() @ w.abs().T)


def activate(g, act):
    if act == "silu":
        return g * torch.sigmoid(g)
    return 0.5 * g * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (g + 0.044715 * g ** 3)))
