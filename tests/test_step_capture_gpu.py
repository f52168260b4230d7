"""The example loop with its steps captured: the accept's random numbers are the step's, not
those of the step that was captured."""
import os
import sys

import pytest
import torch

from step_util import status

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
from verify_step import VerifyLoop  # noqa: E402

pytestmark = pytest.mark.gpu
PROMPTS = [[5, 17, 300, 42], [9, 9, 1234], [7]]


@pytest.mark.parametrize("kw", [dict(), dict(Kd=4, Hq=24, Hkv=4, D=256, layers=1), dict(Kd=0, page=8),
                                dict(Kd=2, kv=torch.bfloat16, window=9)])
def test_captured_steps_draw_their_own_numbers(kw):
    a, b = (VerifyLoop(PROMPTS, **dict(dict(kv="nvfp4"), **kw)) for _ in range(2))
    for loop in (a, b):
        loop.step()
    b.capture()
    for _ in range(8):
        tokens, n = a.step()
        again, n2 = b.step()
        status()
        assert a.steps == b.steps and torch.equal(n, n2)
        for s in range(a.B):
            k = int(n[s])
            assert torch.equal(tokens[s, :k], again[s, :k])
            for x, y in zip(a.logprobs, b.logprobs):
                assert torch.equal(x[s, :k], y[s, :k])
        for name in ("history", "length", "table", "held", "free_count", "cached", "seq_lens"):
            assert torch.equal(getattr(a, name), getattr(b, name)), name


def test_replayed_steps_sample_afresh():
    """The same state, step after step set back: replays draw different tokens, as steps do."""
    loop = VerifyLoop(PROMPTS, Kd=0)
    loop.step()
    loop.capture()
    names = ("history", "length", "table", "held", "free", "free_count", "cached", "seq_lens")
    kept = {k: getattr(loop, k).clone() for k in names}
    seen = set()
    for _ in range(12):
        tokens, n = loop.step()
        seen.add(tuple(tokens[:, 0].tolist()))
        for k, v in kept.items():
            getattr(loop, k).copy_(v)
    status()
    # (three tokens of flat distributions over 4000 entries)
    assert len(seen) > 6
