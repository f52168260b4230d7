"""The example loop: the operators of a verify step one after another."""
import os
import sys

import pytest
import torch

from step_util import status

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
from verify_step import VerifyLoop  # noqa: E402

pytestmark = pytest.mark.gpu
PROMPTS = [[5, 17, 300, 42], [9, 9, 1234], [7]]


@pytest.mark.parametrize("kw", [
    dict(kv=torch.bfloat16),
    dict(kv=torch.float8_e4m3fn, Kd=4, Hq=24, Hkv=4, D=256, layers=1),
    dict(kv=torch.bfloat16, Kd=1, D=64, Hq=16, Hkv=1, window=5, sinks=2, V=1003),
    dict(kv=torch.float8_e4m3fn, Kd=0, page=8),
])
def test_committed_tokens_follow_the_grammar(kw):
    V = kw.get("V", 4000)
    allowed = torch.arange(1, V, 3)
    prompts = [[t % V for t in p] for p in PROMPTS]
    loops = [VerifyLoop(prompts, allowed=allowed, **kw) for _ in range(2)]
    ok = set(allowed.tolist())
    for _ in range(5):
        before = loops[0].length.clone()
        tokens, n = loops[0].step()
        again, n2 = loops[1].step()
        status()
        assert torch.equal(n, n2)
        assert int(n.min()) >= 1 and int(n.max()) <= loops[0].R
        assert torch.equal(loops[0].length, before + n)
        for b in range(len(prompts)):
            run = tokens[b, :n[b]].tolist()
            assert set(run) <= ok
            assert run == again[b, :n[b]].tolist()
            assert run == loops[0].history[b, before[b]:before[b] + n[b]].tolist()


def test_rejected_drafts_leave_no_trace():
    loop = VerifyLoop(PROMPTS, allowed=torch.arange(0, 4000, 2), kv=torch.float8_e4m3fn)
    loop.step()
    g = torch.Generator().manual_seed(3)
    drafts = [torch.randint(0, loop.V, (loop.B, loop.Kd), generator=g).to(torch.int32).cuda()
              for _ in range(2)]
    first = [t.clone() for t in loop.verify(drafts[0])]
    loop.verify(drafts[1])
    for t, u in zip(first, loop.verify(drafts[0])):
        assert torch.equal(t, u)
    logits, bmax = first
    assert torch.isneginf(logits[..., 1::2]).all() and torch.isfinite(logits[..., ::2]).all()
    assert torch.equal(bmax, logits.view(loop.B, loop.R, -1, 16).amax(-1))
    status()
