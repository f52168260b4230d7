"""The operators of a step over 4-bit caches one after another, as the example loop calls them:
append, attention, logits, accept, log probabilities, pages."""
import os
import sys

import pytest
import torch

import speculative_decode_verification_w4_gb300 as vw4
from step_util import status

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
from verify_step import VerifyLoop  # noqa: E402

pytestmark = pytest.mark.gpu
PROMPTS = [[5, 17, 300, 42], [9, 9, 1234], [7]]
KW = [dict(), dict(Kd=4, Hq=24, Hkv=4, D=256, layers=1), dict(Kd=1, D=64, Hq=16, Hkv=1, window=5, sinks=2, V=1003),
      dict(Kd=0, page=8), dict(Kd=4, Hq=16, Hkv=2, D=128, page=8)]


def check_pages(loop):
    """Every page is held once or free, and the held ones cover the next rows."""
    held, count = loop.held.tolist(), int(loop.free_count)
    pages = loop.free[:count].tolist()
    for b, n in enumerate(held):
        assert n * loop.page >= int(loop.seq_lens[b]) > (n - 1) * loop.page
        pages += loop.table[b, :n].tolist()
    assert sorted(pages) == list(range(loop.table.numel()))
    assert torch.equal(loop.cached, loop.length - 1)
    assert torch.equal(loop.seq_lens, loop.length + loop.Kd)


@pytest.mark.parametrize("kw", KW)
def test_steps(kw):
    V = kw.get("V", 4000)
    allowed = torch.arange(1, V, 3)
    prompts = [[t % V for t in p] for p in PROMPTS]
    loops = [VerifyLoop(prompts, allowed=allowed, kv="nvfp4", **kw) for _ in range(2)]
    for _ in range(6):
        before = loops[0].length.clone()
        tokens, n = loops[0].step()
        again, n2 = loops[1].step()
        status()
        assert torch.equal(n, n2) and torch.equal(loops[0].length, before + n)
        for b in range(len(prompts)):
            run = tokens[b, :n[b]].tolist()
            assert set(run) <= set(allowed.tolist()) and run == again[b, :n[b]].tolist()
            # a greedy alternative is never below the token
            lp = loops[0].logprobs
            assert (lp.top_logprobs[b, :n[b], 0] >= lp.logprob[b, :n[b]]).all()
            assert ((lp.rank[b, :n[b]] == 1) == (lp.top_ids[b, :n[b], 0] == tokens[b, :n[b]])).all()
        check_pages(loops[0])


def test_logprobs_of_the_verified_logits():
    """Against 64 bits: a sum of V exponentials of differences of at most 2^7, each within 2^-19
    of itself with the rounding of the difference, and a logarithm of about 8: 2^-19 + 2^-20."""
    loop = VerifyLoop(PROMPTS, kv="nvfp4")
    drafts, draft_logits = loop.draft()
    logits, _ = loop.verify(drafts)
    want = torch.log_softmax(logits.double(), -1)
    tokens, n = loop.commit(drafts, draft_logits)
    status()
    for b in range(loop.B):
        for i in range(int(n[b])):
            w = want[b, i, int(tokens[b, i])].item()
            assert abs(loop.logprobs.logprob[b, i].item() - w) <= 2.0 ** -18 + abs(w) * 2.0 ** -23


def test_four_bits_against_bf16_attention():
    """The cache read back gives, as a bf16 cache, nearly the same attention: read_kv4 rounds each
    value to bf16, 2^-9 of it (K: of a score's terms; V: of the output's)."""
    loop = VerifyLoop(PROMPTS, kv="nvfp4", Kd=3, Hq=8, Hkv=2, D=128, page=16)
    for _ in range(4):
        loop.step()
    c, n = loop.caches[0], int(loop.seq_lens.max())
    k, v = vw4.read_kv4(c, loop.seq_lens, n, first=torch.zeros_like(loop.seq_lens))
    g = torch.Generator(device="cuda").manual_seed(2)
    q = torch.randn(loop.B, 4, 8, 128, device="cuda", generator=g).to(torch.bfloat16)
    out = vw4.verify_attn(q, c, loop.seq_lens)
    status()
    for b in range(loop.B):
        L = int(loop.seq_lens[b])
        kk, vv = (t[b, :L].double().repeat_interleave(4, 1) for t in (k, v))
        s = torch.einsum("ihd,jhd->hij", q[b].double(), kk) * 128 ** -0.5
        a = torch.einsum("ihd,jhd->hij", q[b].double().abs(), kk.abs()) * 128 ** -0.5
        pos = torch.arange(L - 4, L, device="cuda")
        s = s.masked_fill(torch.arange(L, device="cuda") > pos[:, None], float("-inf"))
        p = torch.softmax(s, -1)
        want = torch.einsum("hij,jhd->ihd", p, vv)
        # weights off by twice the largest score's error, the values by 2^-9, the output by 2^-9
        mag = torch.einsum("hij,jhd->ihd", p, vv.abs())
        tol = mag * (2 * a.amax().item() * 2.0 ** -9 + 2.0 ** -9 + 2.0 ** -11) + want.abs() * 2.0 ** -9
        assert ((out[b].double() - want).abs() <= tol * 1.01 + 1e-6).all()


@pytest.mark.parametrize("kw", KW)
def test_captured_step(kw):
    """One graph of a whole step, replayed over and over: the bits of the steps call by call."""
    V = kw.get("V", 4000)
    prompts = [[t % V for t in p] for p in PROMPTS]
    a, b = (VerifyLoop(prompts, kv="nvfp4", **kw) for _ in range(2))
    for loop in (a, b):
        loop.commit(*loop.draft())
    drafts, draft_logits = (t.clone() if t is not None else None for t in a.draft())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tokens_b, n_b = b.commit(drafts, draft_logits)
    logprobs_b = b.logprobs
    for _ in range(6):
        d, dl = a.draft()
        drafts.copy_(d)
        if dl is not None:
            draft_logits.copy_(dl)
        tokens, n = a.commit(d, dl)
        graph.replay()
        status()
        assert torch.equal(n, n_b)
        for s in range(a.B):
            k = int(n[s])
            assert torch.equal(tokens[s, :k], tokens_b[s, :k])
            for x, y in zip(a.logprobs, logprobs_b):
                assert torch.equal(x[s, :k], y[s, :k])
        for name in ("history", "length", "table", "held", "free_count", "cached", "seq_lens"):
            assert torch.equal(getattr(a, name), getattr(b, name)), name
        for x, y in zip(a.caches, b.caches):
            assert torch.equal(x.k, y.k) and torch.equal(x.v, y.v)
    check_pages(b)
