"""Verification of drafted tokens against a 64-bit walk of the same rules, the
distribution that it draws from, and its refusals.

The outputs are whole numbers.  The kernel's probabilities carry relative errors
below 2e-5 (fp32 sums of up to 2^17 terms, the exponential of arguments below
100), and r is a difference at worst a hundred times smaller than its terms
here, so a walk whose every decision is further than 2e-3 from its tie has to
come out equal; the few that are nearer (the reference says so) are left out,
and at most a tenth may be."""
import numpy as np
import pytest
import torch

from tests import kv_reference as ref
from tests.parity_util import require_gpu
from w4a8_quantized_linear_gb300 import _build

OK, INVALID, MISALIGNED, UNSUPPORTED, INDEX = 0, 1, 2, 3, 6
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
P = 0x10000


@pytest.fixture(scope="module")
def lib():
    _build.build()
    import w4a8_quantized_linear_gb300 as pkg
    return pkg.library()


def call(lib, logits=P, stride=1001, dtype=0, tokens=P, parents=P, offsets=P, requests=2, nodes=5,
         vocab=1001, most=4, uniforms=P, noise=P, draft=P, temperature=P, count=P, path=P, nxt=P):
    return lib.cider_verify_drafts(logits, stride, dtype, tokens, parents, offsets, requests, nodes,
                                   vocab, most, uniforms, noise, draft, temperature, count, path,
                                   nxt, None)


@pytest.mark.parametrize("kw", [
    dict(logits=0), dict(tokens=0), dict(parents=0), dict(offsets=0), dict(uniforms=0),
    dict(noise=0), dict(count=0), dict(path=0), dict(nxt=0), dict(dtype=2), dict(requests=-1),
    dict(nodes=-1), dict(vocab=0), dict(most=0), dict(most=65), dict(stride=1000)])
def test_refusals(lib, monkeypatch, kw):
    monkeypatch.setenv("CIDER_FORCE_UNSUPPORTED", "1")
    assert call(lib, **kw) == INVALID


def test_alignment_device_and_empty(lib, monkeypatch):
    monkeypatch.setenv("CIDER_FORCE_UNSUPPORTED", "1")
    assert call(lib, logits=P + 1) == MISALIGNED
    assert call(lib, noise=P + 2) == MISALIGNED
    assert call(lib, draft=P + 1) == MISALIGNED
    assert call(lib, path=P + 2) == MISALIGNED
    assert call(lib) == UNSUPPORTED
    assert call(lib, draft=None, temperature=None) == UNSUPPORTED
    assert call(lib, nodes=0, logits=None, tokens=None, parents=None, uniforms=None) == UNSUPPORTED
    assert call(lib, requests=0) == OK


def inputs(rng, nodes, vocab, children, sampled, dtype, sharp=3.0, temperature=None):
    total = sum(nodes)
    logits = torch.from_numpy((sharp * rng.standard_normal((total, vocab))).astype(np.float32)).to(DTYPES[dtype])
    lf = logits.float().numpy()
    near = lf + 0.7 * rng.standard_normal(lf.shape)
    order = near + (rng.gumbel(size=lf.shape) if sampled else 0)
    best = np.argsort(-order, -1)[:, :max(children, 1)]
    tokens, parents, base = [], [], 0
    for t in nodes:
        if not t:
            continue
        par, _ = ref.random_tree(rng, t, children)
        seen = [0] * t
        for p in par:
            tokens.append(int(best[base + p, seen[p] % best.shape[1]]) if p >= 0 else -5)
            if p >= 0:
                seen[p] += 1
        parents += par
        base += t
    draft = np.stack([ref.softmax64(r) for r in near]).astype(np.float32) if sampled else None
    noise = np.maximum(rng.exponential(size=(len(nodes), vocab)), 1e-10).astype(np.float32)
    if temperature is None:
        temperature = rng.choice([0.0, 0.7, 1.0, 1.5], len(nodes))
    return dict(logits=logits, tokens=np.array(tokens, np.int32), parents=np.array(parents, np.int32),
                offsets=ref.offsets_of(nodes), uniforms=rng.random(total).astype(np.float32),
                noise=noise, draft=draft, temperature=np.asarray(temperature, np.float32))


def launch(cider, d, most, logits=None):
    dev = {k: torch.from_numpy(v).cuda() for k, v in d.items() if isinstance(v, np.ndarray)}
    logits = d["logits"].cuda() if logits is None else logits
    got = cider.cider_verify_drafts(logits, dev["tokens"], dev["parents"], dev["offsets"],
                                    dev["uniforms"], dev["noise"], most,
                                    draft_probs=dev.get("draft"), temperature=dev["temperature"])
    return [g.cpu().numpy() for g in got]


def compare(cider, d, nodes, most, logits=None):
    count, path, nxt = launch(cider, d, most, logits)
    assert cider.cider_check_device_error() == OK
    close = 0
    for b, t in enumerate(nodes):
        if t == 0:
            assert count[b] == 0 and nxt[b] == -1 and (path[b] == -1).all()
            continue
        s = slice(d["offsets"][b], d["offsets"][b + 1])
        want, last, margin = ref.verify(d["logits"][s].float().numpy(), d["tokens"][s], d["parents"][s],
                                        d["uniforms"][s], d["noise"][b],
                                        d["draft"][s] if d["draft"] is not None else None,
                                        float(d["temperature"][b]))
        if margin < 2e-3:
            close += 1
            continue
        assert list(path[b, :count[b]]) == want, b
        assert (path[b, count[b]:] == -1).all()
        assert nxt[b] == last, b
    assert close <= max(1, len(nodes) // 10)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("sampled", [False, True])
@pytest.mark.parametrize("children", [1, 4])
@pytest.mark.parametrize("vocab", [1, 7, 513, 2000, 32003])
def test_against_the_walk(vocab, children, sampled, dtype):
    cider = require_gpu()
    rng = np.random.default_rng(vocab + children)
    nodes = [1, 2, 9, 0, 30, 5, 5, 12, 64, 3, 8, 4]
    d = inputs(rng, nodes, vocab, min(children, vocab), sampled, dtype)
    compare(cider, d, nodes, 64)


@pytest.mark.gpu
@pytest.mark.parametrize("requests", [1, 40, 200])
def test_batch_sizes_and_a_large_vocabulary(requests):
    cider = require_gpu()
    rng = np.random.default_rng(requests)
    nodes = [4] * requests
    vocab = 128003 if requests == 1 else 3001
    d = inputs(rng, nodes, vocab, 2, requests != 40, "bf16", sharp=5.0)
    compare(cider, d, nodes, 4)


@pytest.mark.gpu
def test_strided_rows_and_masked_tokens():
    """Rows of a wider matrix, tokens masked with -inf, a row of -inf alone."""
    cider = require_gpu()
    rng = np.random.default_rng(5)
    nodes = [6, 6, 6, 6]
    d = inputs(rng, nodes, 701, 2, False, "fp16", temperature=[1.0, 0.0, 0.8, 1.0])
    x = d["logits"]
    x[:, ::3] = -np.inf
    x[18] = -np.inf
    wide = torch.zeros(24, 1100, dtype=torch.float16, device="cuda")[:, 37:738]
    wide.copy_(x)
    count, path, nxt = launch(cider, d, 6, wide)
    for b in range(3):
        s = slice(6 * b, 6 * b + 6)
        want, last, margin = ref.verify(x[s].float().numpy(), d["tokens"][s], d["parents"][s],
                                        d["uniforms"][s], d["noise"][b], None,
                                        float(d["temperature"][b]))
        if margin > 2e-3:
            assert list(path[b, :count[b]]) == want and nxt[b] == last
    # no distribution at the root: nothing accepted, every key is 0, the lowest index
    assert count[3] == 1 and nxt[3] == 0
    assert cider.cider_check_device_error() == OK


@pytest.mark.gpu
def test_ties_go_to_the_lowest_index():
    cider = require_gpu()
    for vocab in (5, 4097, 40000):
        x = torch.zeros(2, vocab, dtype=torch.float16)
        x[:, vocab // 2:] = 3.0   # many equal maxima
        d = dict(logits=x, tokens=np.array([0, vocab // 2], np.int32), parents=np.array([-1, 0], np.int32),
                 offsets=np.array([0, 2], np.int32), uniforms=np.zeros(2, np.float32),
                 noise=np.ones((1, vocab), np.float32), draft=None, temperature=np.zeros(1, np.float32))
        count, path, nxt = launch(cider, d, 2)
        assert count[0] == 2 and nxt[0] == vocab // 2
        d["temperature"][:] = 1.0
        d["uniforms"][:] = 0.999999
        d["tokens"][1] = 0
        count, path, nxt = launch(cider, d, 2)
        assert count[0] == 1 and nxt[0] == vocab // 2


@pytest.mark.gpu
def test_certain_acceptance_and_rejection():
    """A drafter equal to the target is always accepted; a draft that the target
    gives no probability never is, and the residual is then the target's."""
    cider = require_gpu()
    rng = np.random.default_rng(8)
    vocab, nodes = 900, [8] * 6
    d = inputs(rng, nodes, vocab, 1, True, "fp16", temperature=[1.0] * 6)
    d["draft"] = np.stack([ref.softmax64(r) for r in d["logits"].float().numpy()]).astype(np.float32)
    d["uniforms"][:] = 0.999
    count, _, _ = launch(cider, d, 8)
    assert (count == 8).all()
    x = d["logits"]
    x[torch.arange(48)[:, None], torch.from_numpy(d["tokens"]).long().clamp(min=0)[torch.arange(48).add(1).clamp(max=47)][:, None]] = -np.inf
    d["uniforms"][:] = 0.0
    count, _, _ = launch(cider, d, 8)
    assert (count == 1).all()


@pytest.mark.gpu
@pytest.mark.parametrize("sampled", [False, True])
def test_the_next_token_follows_the_target(sampled):
    """The first token after the root (accepted or drawn) has the target's
    distribution.  20000 requests over 6 tokens: each count is within 5 standard
    deviations of its mean (a chance of 4e-6 in all for a right kernel)."""
    cider = require_gpu()
    rng = np.random.default_rng(21)
    vocab, requests, kids = 6, 20000, 2
    row = np.array([1.0, 0.2, -0.5, 0.8, -1.5, 0.0], np.float32)
    q_row = ref.softmax64(np.array([0.1, 0.9, -0.2, 0.4, -0.3, 0.3]))
    n = requests * (1 + kids)
    if sampled:
        gumbel = np.log(q_row) + rng.gumbel(size=(requests, vocab))
        drafts = np.argsort(-gumbel, -1)[:, :kids]
    else:
        drafts = np.tile(np.array([3, 1]), (requests, 1))
    tokens = np.concatenate([np.zeros((requests, 1)), drafts], 1).astype(np.int32).reshape(-1)
    parents = np.tile(np.array([-1, 0, 0], np.int32), requests)
    d = dict(logits=torch.from_numpy(np.tile(row, (n, 1))).half(), tokens=tokens, parents=parents,
             offsets=(np.arange(requests + 1) * (1 + kids)).astype(np.int32),
             uniforms=rng.random(n).astype(np.float32),
             noise=rng.exponential(size=(requests, vocab)).astype(np.float32),
             draft=np.tile(q_row.astype(np.float32), (n, 1)) if sampled else None,
             temperature=np.ones(requests, np.float32))
    count, path, nxt = launch(cider, d, 1 + kids)
    first = np.where(count > 1, tokens.reshape(requests, -1)[np.arange(requests), path[:, 1].clip(0)], nxt)
    p = ref.softmax64(torch.from_numpy(row).half().float().numpy())
    seen = np.bincount(first, minlength=vocab)
    assert (np.abs(seen - requests * p) < 5 * np.sqrt(requests * p * (1 - p))).all(), (seen, requests * p)


@pytest.mark.gpu
def test_bad_tokens_and_offsets_are_reported():
    cider = require_gpu()
    rng = np.random.default_rng(13)
    nodes = [3, 3, 3]
    d = inputs(rng, nodes, 50, 1, False, "fp16", temperature=[1.0] * 3)
    d["tokens"][[1, 4]] = [50, -1]
    d["uniforms"][:] = 0.0
    count, path, nxt = launch(cider, d, 3)
    assert cider.cider_check_device_error() == INDEX
    assert count[0] == 1 and count[1] == 1 and count[2] == 3
    assert ((nxt >= 0) & (nxt < 50)).all()
    d["tokens"][[1, 4]] = 0
    d["offsets"] = np.array([0, 3, 8, 9], np.int32)   # five nodes of one request, max_nodes 3
    count, path, nxt = launch(cider, d, 3)
    assert cider.cider_check_device_error() == INDEX
    assert count[0] >= 1 and count[1] == 0 and nxt[1] == -1
