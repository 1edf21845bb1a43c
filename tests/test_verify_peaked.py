"""Verification of sampled drafts whose drafter is nearly certain: the mass that
is left of q after its likeliest tokens is many orders below 1.

The walk is repeated in 64 bits, with Q as the sum of what is left of q, and
carries a bound of the kernel's error along: relative errors of 2e-5 of a
probability (the exponential of arguments below 100 in fp32), 2e-6 of a quotient
or sum; a difference keeps the absolute errors of its terms.  A decision that
the bound leaves open may fall either way, and the request is left out from
there; at most a tenth may be.  Whatever is decided, a token of logit -inf is
never returned."""
import numpy as np
import pytest
import torch

from tests import kv_reference as ref
from tests.parity_util import require_gpu

OK = 0


def draws(rng, q, kids, requests):
    """kids tokens for each request, drawn from q without replacement."""
    key = np.log(np.maximum(q.astype(np.float64), 1e-300)) + rng.gumbel(size=(requests, len(q)))
    return np.argsort(-key, -1)[:, :kids]


def walk(row, tokens, uniforms, noise, q):
    """The root's children asked in 64 bits -> (accepted child or None, next
    token or None when the root's draw is not reached, certain)."""
    p = ref.softmax64(row)
    r, er = p.copy(), 2e-5 * p
    z, ez, big_q = 1.0, 0.0, 1.0
    q = q.astype(np.float64).copy()
    for i, x in enumerate(tokens):
        if big_q < 2.0 ** -126:
            break   # nothing is left of q: no later child can have been drawn
        left, right = uniforms[i] * q[x] / big_q * z, r[x]
        slack = left * (4e-6 + ez / z) + er[x]
        if abs(left - right) <= slack:
            return None, None, False
        if left < right:
            return i, None, True
        new = np.maximum(r / z - q / big_q, 0.0)
        e = (er + r * ez / z) / z + 4e-6 * (r / z + q / big_q)
        e = np.where(r / z + e < q / big_q, 0.0, e)   # certainly 0
        total, et = new.sum(), e.sum() + 2e-6 * new.sum()
        if total > 0 and total <= 4 * et:
            return None, None, False
        if total > 0:
            r, er, z, ez = new, e, total, et
        q[x] = 0.0
        big_q = q.sum()
    key, ek = r / noise, (er + 2e-6 * r) / noise
    best = int(np.argmax(key))
    low = key[best] - ek[best]
    others = np.delete(key + ek, best)
    return None, best, bool(len(others) == 0 or others.max() < low)


def launch(cider, row, drafts, uniforms, noise, q_row):
    requests, kids = drafts.shape
    n = requests * (1 + kids)
    tokens = np.concatenate([np.zeros((requests, 1)), drafts], 1).astype(np.int32).reshape(-1)
    parents = np.tile(np.array([-1] + [0] * kids, np.int32), requests)
    offsets = (np.arange(requests + 1) * (1 + kids)).astype(np.int32)
    dev = [torch.from_numpy(a).cuda() for a in (tokens, parents, offsets, uniforms.reshape(-1), noise)]
    logits = torch.from_numpy(row).half().cuda().expand(n, -1).contiguous()
    draft = torch.from_numpy(q_row).cuda().expand(n, -1).contiguous()
    got = cider.cider_verify_drafts(logits, *dev, 1 + kids, draft_probs=draft)
    assert cider.cider_check_device_error() == OK
    return [g.cpu().numpy() for g in got]


@pytest.mark.gpu
@pytest.mark.parametrize("vocab", [1000, 1003, 40000])
@pytest.mark.parametrize("kids", [3, 4, 6])
@pytest.mark.parametrize("lead", [10.0, 17.0, 25.0, 40.0])
def test_a_drafter_with_one_lead(lead, kids, vocab):
    """The drafter's lead is a token that the target masks, as constrained
    decoding does, and a third of the other tokens are masked too."""
    cider = require_gpu()
    rng = np.random.default_rng(int(lead) * 100 + kids + vocab)
    requests = 200 if vocab < 10000 else 20
    row = rng.standard_normal(vocab).astype(np.float16).astype(np.float32)
    near = row + rng.standard_normal(vocab).astype(np.float32)
    top = int(rng.integers(vocab))
    near[top] += lead + 10
    row[rng.permutation(vocab)[:vocab // 3]] = -np.inf
    row[top] = -np.inf
    q_row = ref.softmax64(near).astype(np.float32)
    drafts = draws(rng, q_row, kids, requests)
    uniforms = rng.random((requests, 1 + kids)).astype(np.float32)
    noise = np.maximum(rng.exponential(size=(requests, vocab)), 1e-10).astype(np.float32)
    count, path, nxt = launch(cider, row, drafts, uniforms, noise, q_row)
    ends = np.where(count > 1, drafts[np.arange(requests), path[:, 1].clip(1) - 1], nxt)
    assert np.isfinite(row[ends]).all() and np.isfinite(row[nxt]).all()
    open_ = 0
    for b in range(requests):
        child, last, certain = walk(row, drafts[b], uniforms[b, 1:], noise[b].astype(np.float64), q_row)
        if not certain:
            open_ += 1
        elif child is not None:
            assert count[b] == 2 and path[b, 1] == 1 + child, b
        else:
            assert count[b] == 1 and nxt[b] == last, b
    assert open_ <= requests // 10


@pytest.mark.gpu
@pytest.mark.parametrize("logits", [[0.0, 16.1, -0.7, 0.4, -1.2, 0.6], [18.0, 18.5, 0.2, -0.5, 0.3, -0.1],
                                    [30.0, 0.5, 14.0, 0.1, -0.4, 0.2]])
@pytest.mark.parametrize("kids", [3, 5])
def test_the_first_token_follows_the_target(kids, logits):
    """Drafters at 1 - 1e-7, with two tokens that hold all but 1e-8, and with a
    lead beyond fp32's reach: 20000 requests over 6 tokens, each count within 5
    standard deviations (a chance of 4e-6 in all for a right kernel)."""
    cider = require_gpu()
    rng = np.random.default_rng(77 + kids)
    vocab, requests = 6, 20000
    row = np.array([0.3, -2.5, -1.0, 1.0, 0.2, 0.6], np.float16).astype(np.float32)
    q_row = ref.softmax64(np.array(logits)).astype(np.float32)
    drafts = draws(rng, q_row, kids, requests)
    uniforms = rng.random((requests, 1 + kids)).astype(np.float32)
    noise = np.maximum(rng.exponential(size=(requests, vocab)), 1e-10).astype(np.float32)
    count, path, nxt = launch(cider, row, drafts, uniforms, noise, q_row)
    # an accepted child has no children here: the token after it is not looked at
    first = np.where(count > 1, drafts[np.arange(requests), path[:, 1].clip(1) - 1], nxt)
    p = ref.softmax64(row)
    seen = np.bincount(first, minlength=vocab)
    assert (np.abs(seen - requests * p) < 5 * np.sqrt(requests * p * (1 - p))).all(), (seen, requests * p)


@pytest.mark.gpu
@pytest.mark.parametrize("vocab", [8, 1000])
def test_nothing_is_left_of_the_drafter(vocab):
    """q is a single token, which the target masks: once it is refused no later
    child can have been drawn, none is accepted, and the draw is the target's."""
    cider = require_gpu()
    rng = np.random.default_rng(vocab)
    requests, kids = 50, 4
    row = rng.standard_normal(vocab).astype(np.float16).astype(np.float32)
    row[3] = -np.inf
    q_row = np.zeros(vocab, np.float32)
    q_row[3] = 1.0
    drafts = np.tile(np.array([3, 1, 2, 5]), (requests, 1))
    uniforms = np.zeros((requests, 1 + kids), np.float32)
    noise = np.maximum(rng.exponential(size=(requests, vocab)), 1e-10).astype(np.float32)
    count, path, nxt = launch(cider, row, drafts, uniforms, noise, q_row)
    assert (count == 1).all() and (path[:, 1:] == -1).all()
    for b in range(requests):
        _, last, certain = walk(row, drafts[b], uniforms[b, 1:], noise[b].astype(np.float64), q_row)
        assert nxt[b] == last or not certain
