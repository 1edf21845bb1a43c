"""Cases of the quantized key/value cache and of speculative decoding over it.

Five operators, as one decoding step of a server uses them:

  append   keys and values are quantized (INT8 or INT4, one scale per token and
           head) as they are written into a paged cache; what is cached is then
           read back, as a chunked prompt does for its own attention
  read     a prefix of every request is read back as fp16 / bf16
  attend   attention of 1..64 new tokens per request (one token, a chain or a
           tree of drafted tokens) over the request's paged cache
  verify   the drafted tokens are accepted or rejected against the target's
           probabilities, from given random numbers
  compact  the accepted tokens' rows move up behind the context, in every layer

`own` False: plain torch operations in 32 bits.  `own` True: this repository's
entry points.
"""
import math
import random

import numpy as np
import torch

own = False

_TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# --------------------------------------------------------------------- cases
def listed():
    """Head counts: 16 query / 8 key-value heads of 128 (hidden size 2048) and
    32 / 8 (hidden size 4096), the layer shapes of this repository's benchmark."""
    return [
        # eight requests decode one token each: the smallest write
        _cache_case("append", name="append_decode", bits=8, dtype="fp16", requests=8, tokens=8, kv_heads=8, dim=128, page=16),
        # a prompt chunk of 32k tokens into an INT4 cache
        _cache_case("append", name="append_prompt", bits=4, dtype="bf16", requests=4, tokens=32768, kv_heads=8, dim=128, page=64),
        # the cached prefix of one request, an odd number of tokens
        _cache_case("read", name="read_prefix", bits=8, dtype="fp16", requests=1, tokens=1334, kv_heads=8, dim=128, page=16),
        # the prefixes of 32 requests, of many lengths
        _cache_case("read", name="read_batch", bits=4, dtype="bf16", requests=32, tokens=131072, kv_heads=8, dim=128, page=64),
        # one request, one token, a short context: latency
        _attend_case(name="decode_one", bits=8, dtype="fp16", requests=1, length=333, nodes=1, heads=16, kv_heads=8, dim=128, page=16),
        # a serving batch of 64 requests of many lengths, INT4 cache
        _attend_case(name="decode_batch", bits=4, dtype="bf16", requests=64, length=8192, nodes=1, heads=32, kv_heads=8, dim=128, page=64),
        # one long document: few rows, a long axis
        _attend_case(name="decode_long", bits=8, dtype="fp16", requests=1, length=131071, nodes=1, heads=32, kv_heads=8, dim=128, page=64),
        # trees of up to 32 drafted tokens for 32 requests: the largest
        _attend_case(name="tree_batch", bits=8, dtype="bf16", requests=32, length=16384, nodes=32, heads=32, kv_heads=8, dim=128, page=64),
        # chains of four sampled drafts for two requests, with the drafter's probabilities, an odd vocabulary
        _verify_case(name="verify_chain", dtype="fp16", requests=2, nodes=5, vocab=32003, children=1, sampled=True),
        # trees of up to 32 drafts for 48 requests, a large vocabulary
        _verify_case(name="verify_tree", dtype="bf16", requests=48, nodes=32, vocab=128000, children=4, sampled=False),
        # the accepted nodes of four requests in a small stack of layers
        _compact_case(name="compact_few", bits=8, dtype="fp16", layers=4, requests=4, nodes=5, length=500, kv_heads=8, dim=128, page=16),
        # 64 requests, trees of up to 32 nodes, 32 layers
        _compact_case(name="compact_stack", bits=4, dtype="bf16", layers=32, requests=64, nodes=32, length=500, kv_heads=8, dim=128, page=64),
    ]


def _cache_case(op, **kw):
    return {"op": op, **kw}


def _attend_case(**kw):
    return {"op": "attend", **kw}


def _verify_case(**kw):
    return {"op": "verify", **kw}


def _compact_case(**kw):
    return {"op": "compact", **kw}


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm, odd more often than not."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, v | 1 if rng.random() < 0.6 else v))


def draw(rng):
    op = rng.choice(("append", "read", "attend", "attend", "attend", "verify", "compact"))
    common = {"bits": rng.choice((8, 4)), "dtype": rng.choice(("fp16", "bf16")), "dim": rng.choice((64, 128, 128)), "page": rng.choice((16, 32, 64, 128))}
    if op in ("append", "read"):
        tokens = _log(rng, 8, 32768 if op == "append" else 131072)
        return _cache_case(op, requests=_log(rng, 1, min(tokens, 48)), tokens=tokens, kv_heads=rng.choice((1, 2, 4, 8)), **common)
    if op == "attend":
        heads, kv_heads = rng.choice(((16, 8), (32, 8), (8, 8), (24, 8), (16, 2), (12, 1)))
        nodes = 1 if rng.random() < 0.4 else _log(rng, 2, 64)
        requests = _log(rng, 1, 64)
        # at most the largest listed case's tokens and products
        most = min(131072, 32 * 16384 // requests, 32 * 16384 * 32 * 32 // (requests * max(nodes, 4) * heads))
        return _attend_case(requests=requests, length=_log(rng, 16 + nodes, max(most, 32 + nodes)), nodes=nodes, heads=heads, kv_heads=kv_heads, **common)
    if op == "verify":
        nodes = _log(rng, 2, 48)
        sampled = rng.random() < 0.5
        vocab = _log(rng, 1000, 128000)
        return _verify_case(dtype=common["dtype"], requests=_log(rng, 1, max(1, min(64, 48 * 32 // nodes // (2 if sampled else 1)))), nodes=nodes, vocab=vocab,
                            children=rng.choice((1, 2, 4)), sampled=sampled)
    layers = _log(rng, 2, 32)
    return _compact_case(layers=layers, requests=_log(rng, 1, 64), nodes=_log(rng, 2, 32), length=_log(rng, 16, 500), kv_heads=rng.choice((1, 2, 8)), **common)


# ------------------------------------------------------- sizes of a case
def _spread(total_or_most, n, low=0.25):
    """n whole numbers from low * most to most, evenly spaced (at least 1)."""
    return [max(1, int(round(total_or_most * (low + (1 - low) * (i + 1) / n)))) for i in range(n)]


def _shares(total, n):
    """n whole numbers that grow evenly and add up to total (at least 1 each)."""
    left = total - n
    w = [i + 1 for i in range(n)]
    got = [1 + left * x // sum(w) for x in w]
    got[-1] += total - sum(got)
    return got


def _lengths(case):
    return _spread(case["length"], case["requests"])


def _nodes(case):
    return [case["nodes"]] * case["requests"] if case["nodes"] < 8 else _spread(case["nodes"], case["requests"], 0.5)


def _depth_guess(case):
    """Rows of logits that a request's walk visits: the root's and about one more for every two levels."""
    return min(case["nodes"], 2)


def work(case):
    op = case["op"]
    if op == "verify":
        # what no request can do without: the rows of its walk (the root's and one accepted child's, say), the drafter's row at the root, the noise of its draw
        size = 2
        rows = case["requests"] * _depth_guess(case)
        b = rows * case["vocab"] * (size + (4 if case["sampled"] else 0)) + case["requests"] * case["vocab"] * 4
        return {"bytes": b, "flops": 6 * rows * case["vocab"]}
    row = 2 * (case["dim"] * case["bits"] // 8 + 4)  # a token's key and value of one head, with their scales
    wide = 2 * case["dim"] * 2
    if op == "append":
        n = case["tokens"] * case["kv_heads"]
        return {"bytes": n * (wide + row) + n * (row + wide), "flops": 8 * n * case["dim"]}
    if op == "read":
        n = case["tokens"] * case["kv_heads"]
        return {"bytes": n * (row + wide), "flops": 2 * n * case["dim"]}
    if op == "compact":
        n = case["layers"] * case["kv_heads"]
        moved = n * case["requests"] * max(1, min(_kept(case), case["nodes"]))
        back = n * sum(_nodes(case))
        return {"bytes": moved * 2 * row + back * (row + wide), "flops": 2 * back * case["dim"]}
    lengths, nodes = _lengths(case), _nodes(case)
    tokens = sum(length + t for length, t in zip(lengths, nodes))
    rows = sum(nodes) * case["heads"] * case["dim"]
    products = sum(t * length + t * (t + 1) // 2 for length, t in zip(lengths, nodes))
    return {"bytes": tokens * case["kv_heads"] * row + rows * 2 * 2, "flops": 4 * case["heads"] * case["dim"] * products}


def _kept(case):
    return max(1, case["nodes"] // 4)


# --------------------------------------------------------------------- inputs
def _tree(rng, t, children):
    """Parents of t nodes, each before its children, at most `children` of one node: a chain for 1."""
    parent, free, used = [-1], [0], [0] * t
    for i in range(1, t):
        # the newest nodes and the root's neighbourhood both grow, as beams do
        p = free[int(rng.integers(max(0, len(free) - 6), len(free)))] if children > 1 else i - 1
        used[p] += 1
        if used[p] == children and children > 1:
            free.remove(p)
        parent.append(p)
        free.append(i)
    return parent


def _masks(parents):
    """Each node's ancestors and itself, one bit per node, as signed 64-bit numbers."""
    m = []
    for i, p in enumerate(parents):
        m.append((m[p] if p >= 0 else 0) | 1 << i)
    return [x - (1 << 64) if x >> 63 else x for x in m]


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _offsets(counts):
    return _ints([0] + list(np.cumsum(counts)))


def _table(gen, lengths, page):
    """A table of pages for requests of these lengths, in random order, -1 where a row has no page, and how many pages there are."""
    need = [-(-n // page) for n in lengths]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=gen, device="cuda")[: sum(need)].to(torch.int32)
    table = torch.full((len(lengths), max(need) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at : at + n]
        at += n
    return table, pages


def _values(gen, shape, dtype):
    """Keys or values: channels of unlike size, and a few outliers."""
    d = shape[-1]
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    x *= 0.5 + 1.5 * torch.rand(shape[-2:], generator=gen, device="cuda")
    x[..., d // 3] *= 6.0
    return x.to(dtype)


def _encode(x, bits):
    """Codes and scales of x [..., d], as the cache holds them."""
    x = x.float()
    top = 127.0 if bits == 8 else 7.0
    s = x.abs().amax(-1)
    s = s / torch.full_like(s, top)  # by a tensor: torch multiplies by the reciprocal of a number
    s = torch.where(s == 0, torch.ones_like(s), s)
    q = torch.round(x / s[..., None]).clamp(-top, top).to(torch.int8)
    if bits == 4:
        q = (q[..., 0::2].to(torch.uint8) & 15) | (q[..., 1::2].to(torch.uint8) << 4)
    return q, s


def _cache(gen, case, layers, pages):
    """Two caches (keys, values) of [layers, pages, heads, page, dim] codes with their scales, full of quantized data."""
    got = []
    for _ in range(2):
        codes, scales = [], []
        for _ in range(layers):
            step = max(1, (1 << 26) // (case["kv_heads"] * case["page"] * case["dim"]))
            for p in range(0, pages, step):
                n = min(step, pages - p)
                q, s = _encode(_values(gen, (n, case["kv_heads"], case["page"], case["dim"]), torch.float32), case["bits"])
                codes.append(q)
                scales.append(s)
        shape = (layers, pages) + tuple(codes[0].shape[1:])
        got += [torch.cat(codes).view(shape), torch.cat(scales).view(shape[:-1])]
    return got


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, dtype = case["op"], _TYPES[case["dtype"]]
    if op == "verify":
        return _prepare_verify(case, rng, gen, dtype)
    page, heads, dim = case["page"], case["kv_heads"], case["dim"]
    if op in ("append", "read"):
        counts = _shares(case["tokens"], case["requests"])
        rng.shuffle(counts)
        starts = [int(rng.integers(0, 200)) for _ in counts]
        table, pages = _table(gen, [a + n for a, n in zip(starts, counts)], page)
        st = {"op": op, "cache": _cache(gen, case, 1, pages), "table": table, "starts": _ints(starts), "offsets": _offsets(counts), "tokens": case["tokens"], "dtype": dtype}
        if op == "append":
            # keys and values are slices of one projection's output, as a model has them
            both = _values(gen, (case["tokens"], 2 * heads, dim), dtype)
            st["k"], st["v"] = both[:, :heads], both[:, heads:]
            at = np.concatenate([a + np.arange(n) for a, n in zip(starts, counts)])
            who = np.repeat(np.arange(len(counts)), counts)
            at, who = _ints(at, torch.int64), _ints(who, torch.int64)
            st["slots"] = table[who, at // page].to(torch.int64) * page + at % page
        return st
    nodes = _nodes(case)
    rng.shuffle(nodes)
    lengths = _spread(case["length"], case["requests"]) if op == "compact" else _lengths(case)
    rng.shuffle(lengths)
    full = [n + t for n, t in zip(lengths, nodes)]
    table, pages = _table(gen, full, page)
    layers = case["layers"] if op == "compact" else 1
    st = {"op": op, "cache": _cache(gen, case, layers, pages), "table": table, "offsets": _offsets(nodes), "most": max(nodes), "dtype": dtype, "tokens": sum(nodes)}
    if op == "compact":
        # the accepted path of each request: the root and then ever later nodes
        kept = [int(rng.integers(1, max(2, min(2 * _kept(case), t)) + 1)) if t > 1 else 1 for t in nodes]
        kept = [min(k, t) for k, t in zip(kept, nodes)]
        path = np.full((case["requests"], max(nodes)), -1, np.int32)
        for b, (k, t) in enumerate(zip(kept, nodes)):
            path[b, :k] = [0] + sorted(1 + rng.choice(t - 1, k - 1, replace=False)) if k > 1 else [0]
        st.update(starts=_ints(lengths), path=torch.from_numpy(path).cuda(), kept=_ints(kept))
        return st
    st["q"] = torch.randn((sum(nodes), case["heads"], dim), generator=gen, device="cuda").to(dtype)
    st["lengths"] = _ints(full)
    st["tree"] = _ints([m for t in nodes for m in _masks(_tree(rng, t, 4))], torch.int64) if max(nodes) > 1 else None
    return st


def _prepare_verify(case, rng, gen, dtype):
    """Logits as sharp as a language model's, drafts from a drafter that is near them."""
    vocab, kids = case["vocab"], case["children"]
    nodes = _nodes(case)
    rng.shuffle(nodes)
    total = sum(nodes)
    logits = (7.0 * torch.randn((total, vocab), generator=gen, device="cuda")).to(dtype)
    draft = logits.float() + torch.randn((total, vocab), generator=gen, device="cuda")
    order = draft
    if case["sampled"]:  # children drawn without replacement from the drafter's distribution
        order = draft - torch.log(torch.empty_like(draft).exponential_(generator=gen).clamp_min(1e-20))
    best = order.topk(kids, dim=-1).indices.cpu().numpy()
    parents, tokens, base = [], [], 0
    for t in nodes:
        tree = _tree(rng, t, kids)
        seen = [0] * t
        for i, p in enumerate(tree):
            tokens.append(int(best[base + p, seen[p]]) if p >= 0 else 0)
            if p >= 0:
                seen[p] += 1
        parents += tree
        base += t
    temperature = [(1.0, 0.7, 0.0, 1.3)[int(rng.integers(0, 4))] for _ in nodes]
    return {
        "op": "verify", "logits": logits, "tokens": _ints(tokens), "parents": _ints(parents), "offsets": _offsets(nodes), "most": max(nodes),
        "uniforms": torch.rand(total, generator=gen, device="cuda"),
        "noise": torch.empty((len(nodes), vocab), device="cuda").exponential_(generator=gen).clamp_min(1e-10),
        "draft": torch.softmax(draft, -1) if case["sampled"] else None,
        "temperature": torch.tensor(temperature, dtype=torch.float32, device="cuda"),
    }


# ------------------------------------------------------------------ one pass
def run(st):
    return {"append": _append, "read": _read, "attend": _attend, "verify": _verify, "compact": _compact}[st["op"]](st)


def _append(st):
    if own:
        import w4a8_quantized_linear_gb300 as cider

        cider.cider_kv_append(st["k"], st["v"], st["slots"], st["cache"], layer=0)
        return cider.cider_kv_read(st["cache"], st["table"], st["starts"], st["offsets"], st["tokens"], st["dtype"], layer=0)
    page = st["cache"][0].shape[3]
    p, r = st["slots"] // page, st["slots"] % page
    _store(st["cache"], st["k"], st["v"], p, r)
    return _read(st)


def _store(cache, k, v, p, r):
    bits = 8 if cache[0].dtype == torch.int8 else 4
    (kq, ks), (vq, vs) = _encode(k, bits), _encode(v, bits)
    cache[0][0][p, :, r] = kq
    cache[1][0][p, :, r] = ks
    cache[2][0][p, :, r] = vq
    cache[3][0][p, :, r] = vs


def _decode(codes, scales):
    """fp32 values of codes [..., d or d / 2] with scales [...]."""
    if codes.dtype == torch.uint8:
        both = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
        codes = both.to(torch.int8) - 16 * (both > 7).to(torch.int8)
    return codes.float() * scales[..., None]


def _places(st):
    """The page and the row in it of every token that is read back, by the requests' starts."""
    page = st["cache"][0].shape[3]
    i = torch.arange(st["tokens"], device="cuda")
    b = torch.searchsorted(st["offsets"][1:].long(), i, right=True)
    at = st["starts"][b].long() + i - st["offsets"][b].long()
    return st["table"][b, at // page].long(), at % page


def _read(st, layer=0):
    if own:
        import w4a8_quantized_linear_gb300 as cider

        return cider.cider_kv_read(st["cache"], st["table"], st["starts"], st["offsets"], st["tokens"], st["dtype"], layer=layer)
    p, r = _places(st)
    kq, ks, vq, vs = st["cache"]
    if layer is None:
        # [layers, tokens, heads, dim]
        got = [_decode(c[:, p, :, r].transpose(0, 1), s[:, p, :, r].transpose(0, 1)) for c, s in ((kq, ks), (vq, vs))]
    else:
        got = [_decode(c[layer][p, :, r], s[layer][p, :, r]) for c, s in ((kq, ks), (vq, vs))]
    return tuple(x.to(st["dtype"]) for x in got)


def _compact(st):
    if own:
        import w4a8_quantized_linear_gb300 as cider

        cider.cider_kv_compact(st["cache"], st["table"], st["starts"], st["path"], st["kept"])
        return cider.cider_kv_read(st["cache"], st["table"], st["starts"], st["offsets"], st["tokens"], st["dtype"], layer=None)
    page = st["cache"][0].shape[3]
    i = torch.arange(st["path"].shape[1], device="cuda")[None]
    # a node beyond the kept ones moves nowhere: it is written where it is
    size = (st["offsets"][1:] - st["offsets"][:-1])[:, None].long()
    i = torch.minimum(i, size - 1)
    to = st["starts"][:, None].long() + i
    frm = st["starts"][:, None].long() + torch.where(i < st["kept"][:, None], st["path"].long().gather(1, i), i)
    pt, rt = st["table"].long().gather(1, to // page), to % page
    pf, rf = st["table"].long().gather(1, frm // page), frm % page
    for x in st["cache"]:
        x[:, pt, :, rt] = x[:, pf, :, rf]
    return _read(st, layer=None)


def _attend(st):
    if own:
        import w4a8_quantized_linear_gb300 as cider

        return cider.cider_tree_attention(st["q"], st["cache"], st["table"], st["lengths"], st["offsets"], st["most"], tree=st["tree"], layer=0)
    kq, ks, vq, vs = (x[0] for x in st["cache"])
    page, most = kq.shape[2], st["most"]
    n, heads, dim = st["q"].shape
    kv_heads = kq.shape[1]
    batch, longest = st["table"].shape[0], st["table"].shape[1] * page
    # every request's cache, padded to the table's width
    at = torch.arange(longest, device="cuda")
    p = st["table"].clamp_min(0).long()[:, at // page]
    r = (at % page).expand_as(p)
    k = _decode(kq[p, :, r], ks[p, :, r]).permute(0, 2, 3, 1)
    # queries [batch, kv head, node, group] x dim, padded to the most nodes
    first = st["offsets"][:-1].long()
    size = st["offsets"][1:].long() - first
    t = torch.arange(most, device="cuda")
    rows = torch.minimum(first[:, None] + t, torch.tensor(n - 1, device="cuda"))
    q = st["q"].float()[rows].view(batch, most, kv_heads, heads // kv_heads, dim).permute(0, 2, 1, 3, 4)
    s = torch.matmul(q.flatten(2, 3), k).view(batch, kv_heads, most, -1, longest) / math.sqrt(dim)
    del k
    # visible: the context, and the node's own ancestors among the last tokens
    context = (st["lengths"].long() - size)[:, None, None]
    ahead = at[None, None] - context
    mask = st["tree"][rows][:, :, None] if st["tree"] is not None else ((2 << t) - 1)[None, :, None]
    seen = (ahead < 0) | ((ahead < size[:, None, None]) & ((mask >> ahead.clamp(0, 63)) & 1 == 1))
    s = s.masked_fill(~seen[:, None, :, None], float("-inf"))
    top = s.amax(-1, keepdim=True)
    w = torch.exp(s - torch.where(top == float("-inf"), torch.zeros_like(top), top))
    del s
    total = w.sum(-1, keepdim=True)
    v = _decode(vq[p, :, r], vs[p, :, r]).transpose(1, 2)
    out = torch.matmul(w.flatten(2, 3), v).view(batch, kv_heads, most, -1, dim)
    out = torch.where(total > 0, out / total, torch.zeros_like(out)).permute(0, 2, 1, 3, 4).reshape(batch, most, heads, dim)
    # back to the rows that there are
    i = torch.arange(n, device="cuda")
    b = torch.searchsorted(st["offsets"][1:].long(), i, right=True)
    return out[b, i - first[b]].to(st["q"].dtype)


def _verify(st):
    if own:
        import w4a8_quantized_linear_gb300 as cider

        return cider.cider_verify_drafts(st["logits"], st["tokens"], st["parents"], st["offsets"], st["uniforms"], st["noise"], st["most"],
                                         draft_probs=st["draft"], temperature=st["temperature"])
    most = st["most"]
    first = st["offsets"][:-1].long()
    size = st["offsets"][1:].long() - first
    batch = first.shape[0]
    rows = torch.arange(batch, device="cuda")
    greedy = st["temperature"] == 0
    warm = torch.where(greedy, torch.ones_like(st["temperature"]), st["temperature"])

    def target(node):
        x = st["logits"][first + node].float()
        hot = (x == x.amax(-1, keepdim=True)).int().argmax(-1)
        x = x / warm[:, None]
        p = torch.exp(x - x.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
        return torch.where(greedy[:, None], torch.nn.functional.one_hot(hot, x.shape[1]).float(), p)

    now = torch.zeros(batch, dtype=torch.long, device="cuda")
    count = torch.ones(batch, dtype=torch.long, device="cuda")
    path = torch.full((batch, most + 1), -1, dtype=torch.long, device="cuda")
    path[:, 0] = 0
    left = target(now)
    mass = torch.ones(batch, device="cuda")
    q = st["draft"][first].clone() if st["draft"] is not None else None
    drawn = torch.ones(batch, device="cuda")
    # the walk is serial by its nature: each node asks whether its parent was the last accepted one
    for i in range(1, most):
        at = torch.minimum(first + i, first + size - 1)
        ask = (i < size) & (st["parents"][at] == now)
        x = st["tokens"][at].long()
        u = st["uniforms"][at]
        r = left[rows, x]
        if q is None:
            yes = ask & (u * mass < r)
            no = ask & ~yes
            left[rows, x] = torch.where(no, torch.zeros_like(r), r)
            mass = torch.where(no, mass - r, mass)
        else:
            qx = q[rows, x]
            yes = ask & torch.where(greedy, r > 0, u * qx * mass < r * drawn)
            no = ask & ~yes
            rest = (left / mass[:, None] - q / drawn[:, None]).clamp_min(0)
            some = rest.sum(-1)
            empty = some == 0
            rest = torch.where((empty | greedy)[:, None], left, rest)
            some = torch.where(empty | greedy, mass, some)
            left = torch.where(no[:, None], rest, left)
            mass = torch.where(no, some, mass)
            drawn = torch.where(no, drawn - qx, drawn)
            q[rows, x] = torch.where(no, torch.zeros_like(qx), qx)
        now = torch.where(yes, torch.full_like(now, i), now)
        path[rows, torch.where(yes, count, torch.full_like(count, most))] = torch.where(yes, now, torch.full_like(now, -1))
        count = count + yes
        left = torch.where(yes[:, None], target(now), left)
        mass = torch.where(yes, torch.ones_like(mass), mass)
        if q is not None:
            q = torch.where(yes[:, None], st["draft"][first + now], q)
            drawn = torch.where(yes, torch.ones_like(drawn), drawn)
    key = torch.where(greedy[:, None], left, left / st["noise"])
    key = (key == key.amax(-1, keepdim=True)).int()
    return count.int(), path[:, :most].int(), key.argmax(-1).int()


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    op = case["op"]
    if op == "verify":
        return None
    st = prepare(case, seed)
    cache = [x.clone() for x in st["cache"]]
    offsets = st["offsets"].tolist()
    table = st["table"].cpu().numpy()
    page = cache[0].shape[3]

    def value(codes, scales, layer, b, at):
        """Codes times scales of one request's positions `at`: [heads, len, dim]."""
        p = torch.from_numpy(table[b, at // page].astype(np.int64)).cuda()
        r = torch.from_numpy(at % page).cuda()
        c = codes[layer][p, :, r].to(torch.int64)
        if codes.dtype == torch.uint8:
            c = torch.stack([((c & 15) ^ 8) - 8, ((c >> 4) ^ 8) - 8], -1).reshape(*c.shape[:-1], -1)
        return (c.double() * scales[layer][p, :, r].double()[..., None]).transpose(0, 1)

    if op == "append":
        got = []
        for x in (st["k"], st["v"]):
            # the format rounds a scale, and the quotient that a code is the nearest whole number of, to 24 bits: a tie
            # goes by them. The value is the product, in 64 bits
            x = x.double()
            top = 127 if case["bits"] == 8 else 7
            step = (x.abs().amax(-1, keepdim=True) / top).float().double()
            step = torch.where(step == 0, torch.ones_like(step), step)
            got.append((x / step).float().round().clamp(-top, top).double() * step)
        return tuple(got)
    if op == "attend":
        out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
        group = case["heads"] // case["kv_heads"]
        for b, n in enumerate(st["lengths"].tolist()):
            rows = slice(offsets[b], offsets[b + 1])
            t = offsets[b + 1] - offsets[b]
            at = np.arange(n)
            k, v = (value(cache[j], cache[j + 1], 0, b, at) for j in (0, 2))
            allow = torch.ones((t, n), dtype=torch.bool, device="cuda")
            for i in range(t):
                m = int(st["tree"][offsets[b] + i]) if st["tree"] is not None else (2 << i) - 1
                allow[i, n - t :] = torch.tensor([bool(m >> j & 1) for j in range(t)], device="cuda")
            q = st["q"][rows].double().transpose(0, 1)
            for h in range(case["kv_heads"]):
                for g in range(group):
                    s = q[h * group + g] @ k[h].T * case["dim"] ** -0.5
                    s = s.masked_fill(~allow, -math.inf)
                    out[rows, h * group + g] = torch.softmax(s, -1) @ v[h]
        return out
    layers = range(case.get("layers", 1))
    got = [torch.empty((len(layers), st["tokens"], case["kv_heads"], case["dim"]), dtype=torch.float64, device="cuda") for _ in range(2)]
    for b, start in enumerate(st["starts"].tolist()):
        at = start + np.arange(offsets[b + 1] - offsets[b])
        if op == "compact":
            kept = int(st["kept"][b])
            at[:kept] = start + st["path"][b, :kept].cpu().numpy()
        for layer in layers:
            for j in range(2):
                got[j][layer, offsets[b] : offsets[b + 1]] = value(cache[2 * j], cache[2 * j + 1], layer, b, at).transpose(0, 1)
    return tuple(got) if op == "compact" else tuple(x[0] for x in got)
