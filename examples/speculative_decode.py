"""Speculative decoding with a quantized model and a quantized cache.

A small decoder with random weights: W8A8 linears, an INT8 or INT4 paged
key/value cache, trees of drafted tokens.  One step for a batch of requests:

  1. the drafts (here: what followed a token the last times) form a tree
  2. every layer writes the nodes' keys and values (cider_kv_append) and
     attends over the cache (cider_tree_attention)
  3. the logits accept a path of the tree (cider_verify_drafts)
  4. the accepted rows move up behind the context (cider_kv_compact)

    python examples/speculative_decode.py [--bits 4] [--tokens 64] [--requests 4]

prints how many tokens a step yields, and how likely they are when the text is
read in one pass.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import w4a8_quantized_linear_gb300 as cider  # noqa: E402

# the tree's shape: node 0 is the last certain token, three guesses for the
# next one, two after the first of them, one more after the first of those
PARENTS = [-1, 0, 0, 0, 1, 1, 4]
RANKS = [0, 0, 1, 2, 0, 1, 0]   # which of its parent's guesses a node is


def masks(parents):
    m = []
    for i, p in enumerate(parents):
        m.append((m[p] if p >= 0 else 0) | 1 << i)
    return m


class Decoder:
    def __init__(self, vocab=1000, hidden=256, heads=8, kv_heads=2, head_dim=64, layers=2, most=2048, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.vocab, self.hidden, self.heads, self.kv_heads, self.dim, self.layers = vocab, hidden, heads, kv_heads, head_dim, layers

        def linear(n, k):
            w = torch.randn(n, k, generator=gen, device="cuda") * k ** -0.5
            return cider.cider_quantize_weight_int8(w, 0)

        self.embed = torch.randn(vocab, hidden, generator=gen, device="cuda").half()
        self.place = (0.1 * torch.randn(most, hidden, generator=gen, device="cuda")).half()
        self.qkv = [linear((heads + 2 * kv_heads) * head_dim, hidden) for _ in range(layers)]
        self.out = [linear(hidden, heads * head_dim) for _ in range(layers)]
        self.up = [linear(4 * hidden, hidden) for _ in range(layers)]
        self.down = [linear(hidden, 4 * hidden) for _ in range(layers)]
        self.head = linear(vocab, hidden)

    @staticmethod
    def norm(x):
        f = x.float()
        return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)).half()

    def forward(self, tokens, positions, slots, cache, table, lengths, offsets, most, tree):
        """Logits of `tokens`, whose keys and values go to `slots`; lengths
        count them, tree says what each sees of its request's."""
        x = self.embed[tokens] + self.place[positions]
        for i in range(self.layers):
            qkv = cider.cider_w8a8_linear(self.norm(x), *self.qkv[i]).view(-1, self.heads + 2 * self.kv_heads, self.dim)
            q, k, v = qkv.split((self.heads, self.kv_heads, self.kv_heads), 1)
            cider.cider_kv_append(k, v, slots, cache, layer=i)
            a = cider.cider_tree_attention(q, cache, table, lengths, offsets, most, tree=tree, layer=i)
            x = x + cider.cider_w8a8_linear(a.view(a.shape[0], -1), *self.out[i])
            h = torch.nn.functional.silu(cider.cider_w8a8_linear(self.norm(x), *self.up[i]))
            x = x + cider.cider_w8a8_linear(h, *self.down[i])
        return cider.cider_w8a8_linear(self.norm(x), *self.head)


def gaps(model, prompts, text, bits=8, page=16):
    """How far below the largest logit each generated token's is when the whole
    text is read in one pass (0: it is the likeliest)."""
    both = torch.cat((prompts, text.to(prompts.device)), 1)
    requests, length = both.shape
    width = -(-length // page)
    cache = cider.cider_kv_cache(model.layers, requests * width, model.kv_heads, model.dim, page, bits)
    table = torch.arange(requests * width, device="cuda", dtype=torch.int32).view(requests, width)
    logits = torch.cat(read(model, both, cache, table), 1)[:, prompts.shape[1] - 1:-1].float()
    chosen = logits.gather(2, text.to(logits.device)[:, :, None])[:, :, 0]
    return logits.amax(-1) - chosen


def read(model, prompts, cache, table):
    """A prompt in chunks that the attention takes at once -> each chunk's logits."""
    requests, length = prompts.shape
    page = cache[0].shape[3]
    who, out = torch.arange(requests, device="cuda")[:, None], []
    for begin in range(0, length, 64):
        n = min(64, length - begin)
        at = (begin + torch.arange(n, device="cuda")).expand(requests, n)
        slots = table[who, at // page].long() * page + at % page
        lengths = torch.full((requests,), begin + n, dtype=torch.int32, device="cuda")
        offsets = torch.arange(0, requests * n + 1, n, dtype=torch.int32, device="cuda")
        out.append(model.forward(prompts[:, begin:begin + n].reshape(-1), at.reshape(-1), slots.reshape(-1), cache, table,
                                 lengths, offsets, n, None).view(requests, n, -1))
    return out


def generate(model, prompts, tokens, parents=PARENTS, ranks=RANKS, bits=8, page=16, temperature=0.0, seed=0):
    """Decodes at least `tokens` tokens for every prompt [requests, length].
    -> (tokens [requests, tokens], steps).  parents of [-1]: one at a time."""
    requests, length = prompts.shape
    nodes = len(parents)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    width = -(-(length + tokens + 2 * nodes) // page)
    cache = cider.cider_kv_cache(model.layers, requests * width, model.kv_heads, model.dim, page, bits)
    table = torch.arange(requests * width, device="cuda", dtype=torch.int32).view(requests, width)
    i32 = dict(dtype=torch.int32, device="cuda")
    who = torch.arange(requests, device="cuda")[:, None]

    def slots_of(at):   # [requests, n] positions -> slots
        return (table[who, at // page].long() * page + at % page).reshape(-1)

    last = read(model, prompts, cache, table)[-1][:, -1].float().argmax(-1)

    # what followed each token, three guesses, the newest first
    guess = torch.randint(model.vocab, (model.vocab, 3), generator=gen, device="cuda")
    parent = torch.tensor(parents * requests, **i32)
    offsets = torch.arange(0, requests * nodes + 1, nodes, **i32)
    tree = torch.tensor(masks(parents) * requests, dtype=torch.int64, device="cuda")
    depth = torch.tensor([bin(m).count("1") - 1 for m in masks(parents)], device="cuda")
    heat = torch.full((requests,), temperature, device="cuda")
    context = torch.full((requests,), length, **i32)
    got, steps = [[t] for t in last.tolist()], 0
    while min(len(g) for g in got) < tokens:
        node = last[:, None].repeat(1, nodes)
        for i in range(1, nodes):
            node[:, i] = guess[node[:, parents[i]], ranks[i]]
        at = context[:, None].long() + torch.arange(nodes, device="cuda")
        logits = model.forward(node.reshape(-1), (context[:, None].long() + depth).reshape(-1), slots_of(at), cache, table,
                               context + nodes, offsets, nodes, tree)
        uniforms = torch.rand(requests * nodes, generator=gen, device="cuda")
        noise = torch.empty(requests, model.vocab, device="cuda").exponential_(generator=gen).clamp_min(1e-10)
        count, path, nxt = cider.cider_verify_drafts(logits, node.reshape(-1).int(), parent, offsets, uniforms, noise, nodes,
                                                      temperature=heat)
        cider.cider_kv_compact(cache, table, context, path, count)
        # a request that has its tokens waits: its pages are counted for them
        open_ = torch.tensor([len(g) < tokens for g in got], device="cuda")
        count, nxt = torch.where(open_, count, 0), nxt.long()
        context = context + count
        last = torch.where(open_, nxt, last)
        steps += 1
        done = [[int(x) for x in node[b, path[b, 1:c].long()]] + [int(last[b])] for b, c in enumerate(count.tolist())]
        for b, new in enumerate(done):
            if not count[b]:
                continue
            chain = [got[b][-1]] + new
            got[b] += new
            for x, y in zip(chain, chain[1:]):
                if y not in guess[x].tolist():
                    guess[x] = torch.tensor([y] + guess[x, :2].tolist(), device="cuda")
    return torch.tensor([g[:tokens] for g in got]), steps


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--bits", type=int, default=8)
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--temperature", type=float, default=0.0)
    a = ap.parse_args()
    model = Decoder()
    prompts = torch.randint(model.vocab, (a.requests, 100), generator=torch.Generator().manual_seed(1)).cuda()
    text, steps = generate(model, prompts, a.tokens, bits=a.bits, temperature=a.temperature)
    print(f"{a.requests} requests x {a.tokens} tokens in {steps} steps: {a.tokens / steps:.2f} tokens a step at least")
    if a.temperature == 0:
        gap = gaps(model, prompts, text, a.bits)
        print(f"read in one pass, {(gap == 0).float().mean():.1%} of the tokens are the likeliest, "
              f"the others at most {gap.max():.3f} below")
    assert cider.cider_check_device_error() == cider.CIDER_OK


if __name__ == "__main__":
    main()
