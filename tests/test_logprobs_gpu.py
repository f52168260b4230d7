"""token_logprobs against its definition in 64 bits; ranks and the alternatives' ids exactly.

Tolerances, from the roundings: y = x scale log2(e) has two of 2^-24 (the factor, one product
in the reference m), so a difference y - m is off by 2^-23 of |y| + |m|; each weight by
2^-22 (ex2) and its exponent's share, and so a sum Z of them, whose fp32 additions add at
most (16 + V / 4096 / parts + 13) 2^-24: below 2^-18 for these sizes.  log2 Z adds 2^-18,
the results round to 2^-24 of themselves.  The entropy weighs errors of that size by up to
the largest |y - m| that has weight (60)."""
import math

import pytest
import torch

import speculative_decode_verification_w4_gb300 as vw4
from step_util import check_close, status

pytestmark = pytest.mark.gpu


def reference(x, t, scale, top):
    """x [V] in 64 bits (NaN as -infinity), one token -> logprob, lse, entropy, rank, ids, lps."""
    x = torch.where(torch.isnan(x), -math.inf, x)
    V = len(x)
    y = x * scale
    if torch.isposinf(y).any():
        w = torch.isposinf(y).double()
        lse, logp = math.inf, torch.where(w > 0, -math.log(w.sum()), -math.inf)
    elif torch.isneginf(y).all():
        lse, logp = -math.inf, y
    else:
        m = y.max()
        lse = (m + (y - m).exp().sum().log()).item()
        logp = y - lse
    p = logp.exp()
    h = -torch.where(p > 0, p * logp, 0.0).sum().item()
    order = torch.sort(-x, stable=True).indices
    ids, lps = order[:top].tolist(), []
    for k, v in enumerate(ids):
        if x[v] == -math.inf:
            ids[k] = -1
        lps.append(logp[v].item() if ids[k] >= 0 else -math.inf)
    ids += [-1] * (top - len(ids))
    lps += [-math.inf] * (top - len(lps))
    if not 0 <= t < V:
        return -math.inf, lse, h, 0, ids, lps
    return logp[t].item(), lse, h, int((order == t).nonzero()) + 1, ids, lps


def check(x, tokens, scale=1.0, top=5, length=None, bits=0, **kw):
    B, R, V = x.shape
    out = dict(logprob=torch.full((B, R), 9.0), lse=torch.full((B, R), 9.0),
               entropy=torch.full((B, R), 9.0), rank=torch.full((B, R), 9, dtype=torch.int32))
    if top:
        out.update(top_ids=torch.full((B, R, top), 9, dtype=torch.int32),
                   top_logprobs=torch.full((B, R, top), 9.0))
    out = {k: v.cuda() for k, v in out.items()}
    xd = x.cuda() if not x.is_cuda else x
    tk = torch.tensor(tokens, dtype=torch.int32).view(B, R)
    ln = None if length is None else torch.tensor(length, dtype=torch.int32, device="cuda")
    vw4.token_logprobs(xd, tk.cuda(), ln, top, scale, **out, **kw)
    status(bits)
    got = {k: v.cpu() for k, v in out.items()}
    for b in range(B):
        for i in range(R):
            g = {k: v[b, i] for k, v in got.items()}
            if length is not None and i >= length[b]:
                assert all((v == 9).all() for v in g.values()), "a row that is not read was written"
                continue
            row = x[b, i].double().cpu()
            lp, lse, h, rank, ids, lps = reference(row, int(tk[b, i]), scale, top)
            fin = row[torch.isfinite(row)].abs()
            big = float(fin.max()) * scale if len(fin) else 0.0
            tol = 2.0 ** -18 + 2.0 ** -22 * big
            want = torch.tensor([lp, lse], dtype=torch.float64)
            check_close(torch.stack([g["logprob"], g["lse"]]), want,
                        torch.full((2,), tol, dtype=torch.float64) + want.abs() * 2.0 ** -23, f"row {b} {i}")
            assert abs(g["entropy"].item() - h) <= 60 * tol, f"entropy {b} {i}"
            assert g["rank"].item() == rank
            if top:
                assert g["top_ids"].tolist() == ids, f"row {b} {i}"
                want = torch.tensor(lps, dtype=torch.float64)
                fin = torch.where(torch.isfinite(want), want.abs(), 0.0)
                check_close(g["top_logprobs"], want, tol + fin * 2.0 ** -23, f"alternatives {b} {i}")


def logits(seed, B, R, V, gain=3.0, bf16=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, R, V, generator=g) * gain
    return (x.to(torch.bfloat16) if bf16 else x), torch.randint(0, V, (B * R,), generator=g).tolist()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("top", [0, 1, 5, 20, 32])
@pytest.mark.parametrize("V", [1, 2, 31, 257, 4095, 4097, 32003, 151936])
def test_shapes(V, top, bf16):
    x, t = logits(V + top, 2, 3, V, bf16=bf16)
    check(x, t, 1 / 0.7, top)


@pytest.mark.parametrize("B,R,V", [(1, 8, 262144), (200, 7, 5003), (60, 9, 40000)])
def test_batches(B, R, V):
    """Rows in many parts, in a few, in one."""
    x, t = logits(B, B, R, V)
    ln = [(b * 5) % (R + 1) for b in range(B)]
    if B == 1:
        ln = None
    check(x, t, 1.0, 20, ln)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("shift", [1, 2, 3, 5])
def test_unaligned_rows(shift, bf16):
    """Rows that begin anywhere, spaced apart by an odd stride; what lies between is not read
    as a logit."""
    x, t = logits(shift, 2, 2, 5000, bf16=bf16)
    flat = torch.full((4 * 5003 + 9,), float("inf")).to(x.dtype).cuda()
    view = flat.as_strided((2, 2, 5000), (2 * 5003, 5003, 1), shift)
    view.copy_(x)
    check(view, t, 1.0, 7)


@pytest.mark.parametrize("order", ["up", "down", "flat", "blocks"])
def test_orders(order):
    """Ascending rows (every chunk of a row holds larger entries), descending ones, equal
    entries (the lowest indexes come first), -0 beside 0."""
    V = 50000
    x = {"up": torch.linspace(-20, 20, V), "down": torch.linspace(20, -20, V),
         "flat": torch.zeros(V), "blocks": (torch.arange(V) % 97).float() / 8}[order]
    if order == "flat":
        x[::3] = -0.0
    check(torch.stack([x, x.flip(0)])[:, None], [V // 2, 3], 1.0, 32)
    many = x[None, None].expand(1300, 1, V)[:, :, :9000].contiguous()
    lens = [1 if b in (0, 7, 1299) else 0 for b in range(1300)]
    check(many, [5] * 1300, 1.0, 32, lens)


@pytest.mark.parametrize("V", [40, 9000, 100000])
def test_masked_and_not_finite(V):
    g = torch.Generator().manual_seed(V)
    x = torch.randn(8, 1, V, generator=g)
    few = torch.randint(0, V, (3,), generator=g)
    x[0] = -math.inf                                    # nothing is allowed
    x[1] = -math.inf
    x[1, 0, few] = torch.tensor([0.5, -2.0, 1.0])       # fewer than `top`
    x[2, 0, ::2] = -math.inf
    x[3, 0, 5] = math.inf
    x[4, 0, [3, V - 1, V // 2]] = math.inf
    x[5, 0, ::3] = math.nan
    x[6] = math.nan
    x[7] = torch.finfo(torch.float32).min               # the type's lowest value, and one other
    x[7, 0, V // 3] = 1.0
    check(x, [1, int(few[0]), 2, 5, 4, 3, 0, V // 3], 1.0, 10)
    check(x, [1, 7, 3, 6, 3, 4, V - 1, 0], 1.0, 10)


def test_large_and_small_logits():
    x, t = logits(1, 3, 2, 3000, gain=1.0)
    check(x * 3e4, t, 1.0, 8)
    check(x * 1e-4, t, 1.0, 8)
    check(x, t, 50.0, 8)


def test_tokens_out_of_range():
    x, _ = logits(2, 1, 3, 1000)
    check(x, [-1, 5, -1], 1.0, 3)
    check(x, [7, 1000, -2], 1.0, 3, bits=vw4.DEV_BAD_LIST_ID)


def test_parts_of_the_outputs():
    x, t = logits(3, 2, 2, 6000)
    out = vw4.token_logprobs(x.cuda(), top=4)
    status()
    assert out.logprob is None and out.rank is None
    both = vw4.token_logprobs(x.cuda(), torch.tensor(t, dtype=torch.int32).view(2, 2).cuda(), top=0)
    status()
    assert both.top_ids is None and torch.equal(both.lse, out.lse)


def test_same_bits_every_time():
    x, t = logits(4, 3, 5, 70000)
    xd, td = x.cuda(), torch.tensor(t, dtype=torch.int32).view(3, 5).cuda()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    want = vw4.token_logprobs(xd, td, top=20)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call = vw4.PreparedLogprobs(xd, td, top=20)
        with torch.cuda.graph(graph, stream=side):
            call()
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(20):
        graph.replay()
        again = vw4.token_logprobs(xd, td, top=20)
        for a, b, c in zip(want, again, call.out):
            assert torch.equal(a, b) and torch.equal(a, c)
    status()
