"""token_logprobs where the magnitude of the logits has nothing to do with what carries weight:
finite masks, common offsets, forced tokens, tokens next to certain.

Tolerance of ln Z, from the roundings.  c = scale log2 e holds two (2^-23), a difference x - m
and its product with c one of 2^-24 each: an exponent d is off by 2^-22 |d|, its weight by ln 2
times that and 2^-22 (ex2).  An entry's exponents add up to its distance D from the row's maximum
and twice the lag of a thread's reference (at most 8), over at most 20 moves here; the fp32
additions of a thread, its block and the parts add 2^-24 each, at most 16 + 40 + 20.  Weighed
by p, sum p ln 2 |D| is at most 12 here: 2^-22 (12 + 2 * 8 ln 2 + 20 + 76 / 4) < 2^-22 * 63 <
2^-16, whatever the logits' size.  The results round by 2^-24 of themselves and of (x - m)
scale.  The entropy weighs such errors by |D| (at most 12 on average here, 17 in squares' root)
and once more: below 40 of them."""
import math

import pytest
import torch

import speculative_decode_verification_w4_gb300 as vw4
from step_util import check_close, status

pytestmark = pytest.mark.gpu
TOL = 2.0 ** -16


def reference(x, t, scale, top):
    """x [V] in 64 bits -> logprob, lse, entropy, rank, ids, lps.  (The log probabilities from
    the distance to the maximum: y - lse would round at the size of y.)"""
    y = x * scale
    m = y.max()
    lnz = (y - m).exp().sum().log()
    logp = (y - m) - lnz
    p = logp.exp()
    h = -torch.where(p > 0, p * logp, 0.0).sum().item()
    order = torch.sort(-x, stable=True).indices
    ids = torch.where(torch.isneginf(x[order[:top]]), -1, order[:top])
    return logp[t].item(), (m + lnz).item(), h, int((order == t).nonzero()) + 1, ids.tolist(), logp[order[:top]].tolist()


def check(rows, tokens, scale, top, whole):
    """rows [n, V]; whole: among so many rows that a block takes a whole one."""
    n, V = rows.shape
    B = 1300 if whole else n
    at = [(7 + 191 * k) % B if whole else k for k in range(n)]
    x = torch.zeros(B, 1, V, dtype=rows.dtype, device="cuda")
    tk, ln = torch.zeros(B, 1, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    for k, b in enumerate(at):
        x[b, 0], tk[b], ln[b] = rows[k].cuda(), tokens[k], 1
    r = vw4.token_logprobs(x, tk.cuda(), ln.cuda(), top=top, scale=scale)
    status()
    for k, b in enumerate(at):
        lp, lse, h, rank, ids, lps = reference(rows[k].double(), tokens[k], scale, top)
        got = {f: getattr(r, f)[b, 0].cpu() for f in r._fields if getattr(r, f) is not None}
        want = torch.tensor([lp, lse], dtype=torch.float64)
        near = TOL + 2.0 ** -23 * torch.where(torch.isfinite(want), want.abs(), 0.0)
        check_close(torch.stack([got["logprob"], got["lse"]]), want, near, f"row {k}")
        assert got["logprob"] <= 0 and abs(got["entropy"].item() - h) <= 40 * TOL, f"row {k}"
        assert got["rank"].item() == rank
        if top:
            assert got["top_ids"].tolist() == ids
            want = torch.tensor(lps, dtype=torch.float64)
            near = TOL + 2.0 ** -23 * torch.where(torch.isfinite(want), want.abs(), 0.0)
            check_close(got["top_logprobs"], want, near, f"alternatives of row {k}")
            assert (got["top_logprobs"] <= 0).all()


def normal(seed, V, gain=3.0):
    return torch.randn(V, generator=torch.Generator().manual_seed(seed)) * gain


@pytest.mark.parametrize("whole", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("scale,top", [(1.0, 5), (1.25, 0)])
@pytest.mark.parametrize("mask", [-1e4, -1e9, -1e10, -1e12, -1e30, -2e38])
def test_finite_masks(mask, scale, top, bf16, whole):
    """Most entries one large negative number, all of them, all but one, a first half of them."""
    V = 32000
    rows = torch.stack([normal(k, V) for k in range(4)])
    rows[0, torch.rand(V, generator=torch.Generator().manual_seed(9)) < 0.99] = mask
    rows[1] = mask
    rows[2], rows[2, V // 3] = mask, 2.0
    rows[3, :V // 2] = mask
    if bf16:
        rows = rows.to(torch.bfloat16)
    check(rows, [int(rows[0].float().argmax()), 5, V // 3, V - 7], scale, top, whole)
    check(rows, [3, V - 1, 0, 17], scale, top, whole)


@pytest.mark.parametrize("whole", [False, True])
@pytest.mark.parametrize("scale,top", [(1.0, 3), (1.25, 8)])
def test_common_offsets(scale, top, whole):
    """The same rows about any level: the log probabilities know nothing of it."""
    V = 9000
    rows = torch.stack([normal(20 + k, V) + off for k, off in
                        enumerate((1e3, -1e3, 1e4, -1e4, 1e6, -1e6, 3e7, -1e12))])
    check(rows, [11 * k for k in range(8)], scale, top, whole)


@pytest.mark.parametrize("whole", [False, True])
def test_forced_tokens(whole):
    """One entry far above the others, which are alike or not."""
    V = 5000
    rows = torch.stack([torch.zeros(V), normal(1, V), torch.zeros(V), torch.full((V,), 1e9)])
    rows[0, 77], rows[1, 4999], rows[2, 0], rows[3, 2500] = 1e9, 1e30, 50.0, 3e9
    check(rows, [77, 4999, 0, 2500], 1.0, 4, whole)
    check(rows, [78, 0, 4999, 2499], 1.25, 4, whole)


@pytest.mark.parametrize("scale", [1.0, 1.25])
@pytest.mark.parametrize("level", [30.0, 100.0, 1000.0, 10000.0])
def test_next_to_certain(level, scale):
    """A token that leaves the others less than 2^-20 together.  Its own weight is 1 without
    rounding, so the others' roundings and the logarithm's are all: 2^-22 at most, never above 0."""
    V, n = 20000, 40
    rows = torch.stack([normal(100 + k, V, 1.0) for k in range(n)])
    at = [(k * 499) % V for k in range(n)]
    for k in range(n):
        rows[k, at[k]] = level + 0.37 * k
    tokens = torch.tensor(at, dtype=torch.int32).view(n, 1).cuda()
    r = vw4.token_logprobs(rows[:, None].cuda(), tokens, top=2, scale=scale)
    status()
    want = torch.log_softmax(rows.double() * scale, -1).gather(1, torch.tensor(at)[:, None])[:, 0]
    for got in (r.logprob[:, 0].cpu(), r.top_logprobs[:, 0, 0].cpu()):
        assert (got <= 0).all(), f"{int((got > 0).sum())} above 0, {got.max().item():.3g}"
        assert (got.double() - want).abs().max() <= 2.0 ** -22
    # far from certain, and the rest of the row's mass beside an entry of nearly the same weight
    rows[:, 1] = level
    r = vw4.token_logprobs(rows[:, None].cuda(), tokens, top=2, scale=scale)
    status()
    want = torch.log_softmax(rows.double() * scale, -1).gather(1, torch.tensor(at)[:, None])[:, 0]
    assert (r.logprob[:, 0] <= 0).all()
    assert (r.logprob[:, 0].cpu().double() - want).abs().max() <= TOL


def test_masked_rows_in_many_parts():
    """One sequence's rows of the widest head, cut into 64 parts of which most hold masks alone."""
    V = 262144
    rows = torch.stack([normal(50 + k, V) for k in range(4)])
    for k, mask in enumerate((-1e9, -1e10, -1e30, -math.inf)):
        rows[k, 4096 * (k + 1):] = mask
    check(rows, [1, 2, 3, 4], 1.25, 20, False)
