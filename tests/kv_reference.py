"""Plain 64-bit reference of the quantized key/value cache, the attention over
it and the verification of drafted tokens (numpy), and makers of their inputs.
Shares no code with the library."""
import numpy as np
import torch


# ------------------------------------------------------------------- format
def encode(x, bits):
    """x fp32 [..., D] -> (codes int8 [..., D], scales fp32 [...])."""
    x = np.asarray(x, np.float32)
    top = np.float32(127 if bits == 8 else 7)
    s = (np.abs(x).max(-1) / top).astype(np.float32)
    s = np.where(s == 0, np.float32(1), s)
    q = np.rint((x / s[..., None]).astype(np.float32))
    return np.clip(q, -top, top).astype(np.int8), s


def pack(codes, bits):
    """Codes as the cache stores them."""
    if bits == 8:
        return codes
    u = codes.astype(np.uint8) & 15
    return u[..., 0::2] | (u[..., 1::2] << 4)


def unpack(stored, bits):
    if bits == 8:
        return stored.astype(np.int64)
    both = np.stack([stored & 15, stored >> 4], -1).astype(np.int64)
    both = both.reshape(*stored.shape[:-1], 2 * stored.shape[-1])
    return (both ^ 8) - 8


class Cache:
    """A cache on the host (numpy, as stored) and on the device."""

    def __init__(self, rng, layers, pages, heads, dim, page, bits, zero=False):
        self.bits, self.page, self.heads, self.dim = bits, page, heads, dim
        self.host = []
        for _ in range(2):
            x = rng.standard_normal((layers, pages, heads, page, dim)).astype(np.float32)
            x *= rng.uniform(0.2, 3.0, (layers, pages, heads, page, 1)).astype(np.float32)
            q, s = encode(x * (0.0 if zero else 1.0), bits)
            self.host += [pack(q, bits), s]

    def device(self):
        return tuple(torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in self.host)

    def values(self, which, layer, table_row, positions, head):
        """fp64 values [len, dim] of K (0) or V (1) at a request's positions."""
        p, r = table_row[positions // self.page], positions % self.page
        codes = unpack(self.host[2 * which][layer][p, head, r], self.bits).astype(np.float64)
        return codes * self.host[2 * which + 1][layer][p, head, r].astype(np.float64)[:, None]


def table_for(rng, lengths, page, spare=2, width=1):
    """(int32 table padded with -1, number of pages); pages in random order."""
    need = [-(-int(n) // page) for n in lengths]
    pages = sum(need) + spare
    order = rng.permutation(pages)[:sum(need)]
    table = np.full((len(lengths), max(need + [1]) + width), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pages


def offsets_of(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


# ---------------------------------------------------------------- attention
def attend(q, cache, table, lengths, offsets, tree, scale, layer=0):
    """fp64 (out, sum_j p_j |v_j|), both [tokens, q_heads, D].  tree: list of
    Python integers (masks), or None for chains."""
    n, hq, d = q.shape
    group = hq // cache.heads
    out, size = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    q = q.astype(np.float64)
    for b in range(len(lengths)):
        t_n = int(offsets[b + 1] - offsets[b])
        if t_n == 0:
            continue
        length = int(lengths[b])
        ctx = length - t_n
        pos = np.arange(length)
        for h in range(cache.heads):
            k = cache.values(0, layer, table[b], pos, h)
            v = cache.values(1, layer, table[b], pos, h)
            for t in range(t_n):
                i = int(offsets[b]) + t
                mask = tree[i] if tree is not None else (2 << t) - 1
                seen = np.ones(length, bool)
                seen[ctx:] = [(mask >> j) & 1 == 1 for j in range(t_n)]
                if not seen.any():
                    continue
                for g in range(h * group, (h + 1) * group):
                    s = scale * (k[seen] @ q[i, g])
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    out[i, g] = p @ v[seen]
                    size[i, g] = p @ np.abs(v[seen])
    return out, size


def random_tree(rng, t, children=3):
    """(parents, masks) of t nodes, each node's parent before it."""
    parents, used = [-1], [0] * t
    for _ in range(1, t):
        free = [j for j in range(len(parents)) if used[j] < children]
        p = free[int(rng.integers(max(0, len(free) - 5), len(free)))]
        used[p] += 1
        parents.append(p)
    masks = []
    for i, p in enumerate(parents):
        masks.append((masks[p] if p >= 0 else 0) | (1 << i))
    return parents, masks


def signed(masks):
    return np.array([m - (1 << 64) if m >> 63 else m for m in masks], np.int64)


# ------------------------------------------------------------- verification
def softmax64(x):
    x = np.asarray(x, np.float64)
    if np.isneginf(x.max()):
        return np.zeros_like(x)
    e = np.exp(x - x.max())
    return e / e.sum()


def verify(logits, tokens, parents, uniforms, noise, draft, temperature):
    """One request, in 64 bits -> (path, next, margin): margin is the smallest
    relative distance of a decision from its tie (a call with a margin above
    the kernel's rounding has to decide the same)."""
    n = len(tokens)
    greedy = temperature <= 0
    now, path, margin = 0, [0], np.inf

    def near(a, b):
        return abs(a - b) / max(abs(a), abs(b), 1e-300)

    while True:
        row = logits[now].astype(np.float64)
        hot = int(np.argmax(row))
        r = softmax64(row / (1.0 if greedy else temperature))
        mass, rest, q = 1.0, 1.0, None
        if draft is not None:
            q = draft[now].astype(np.float64).copy()
        took = None
        for i in range(now + 1, n):
            if parents[i] != now:
                continue
            x = int(tokens[i])
            if greedy:
                if x == hot:
                    took = i
                    break
                continue
            left, right = (uniforms[i] * mass, r[x]) if q is None else (
                uniforms[i] * q[x] * mass, r[x] * rest)
            if max(left, right) > 0:
                margin = min(margin, near(left, right))
            if left < right:
                took = i
                break
            if q is None:
                mass -= r[x]
                r[x] = 0.0
            else:
                new = np.maximum(r / mass - q / rest, 0.0)
                if new.sum() > 0:
                    r, mass = new, new.sum()
                rest -= q[x]
                q[x] = 0.0
        if took is not None:
            path.append(took)
            now = took
            continue
        if greedy:
            return path, hot, margin
        key = r / noise.astype(np.float64)
        best = int(np.argmax(key))
        others = np.delete(key, best)
        if len(others) and key[best] > 0:
            margin = min(margin, near(key[best], others.max()))
        return path, best, margin
