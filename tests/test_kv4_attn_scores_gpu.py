"""verify_attn over the 4-bit cache with scores up to 2^26: their common part is large, what
tells them apart is not.

Dimension 0 gives every score of a row the same part, dimension 16 adds one of a few steps that
fp32 still holds beside it.  Scores are exact then, a difference of two of them too, the factor of
the exponents is off by 2^-23 of itself, and the exponents of the weights share whatever the
reference's rounding is.  Off by half a step of bf16 of the output,
and of the weights (sum p |v|) by half a step of f16 and 2^-21 of the exponent's step (up to 56):
2^-11 + 2^-16."""
import math

import pytest
import torch

import speculative_decode_verification_w4_gb300 as vw4
from kv4_util import make_cache4
from step_util import check_close, status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("order", ["rising", "falling", "mixed"])
@pytest.mark.parametrize("big", [0, 10, 20, 22, 23, 24, 25])
@pytest.mark.parametrize("R,Hq,D", [(1, 3, 64), (1, 8, 128), (2, 8, 64), (2, 8, 128), (3, 8, 128), (4, 8, 256),
                                    (4, 6, 256), (6, 8, 128), (16, 8, 128), (16, 8, 256), (9, 8, 64)])
def test_large_common_part(R, Hq, D, big, order):
    n, page, g = 1500, 16, torch.Generator().manual_seed(R * D + big)
    step = max(1.0, 2.0 ** (big - 23))         # what fp32 holds next to 2^big and 4 steps above
    c, _, v64 = make_cache4(11, [n], page, 1, D)
    for t in (c.k_scale, c.k_blocks):
        t.copy_(torch.ones(t.shape))
    level = torch.randint(0, 4, (n,), generator=g)           # 0, 1, 2 or 4 steps
    if order != "mixed":
        level = level.sort(descending=order == "falling").values
    c.k.zero_()
    codes = torch.tensor([0, 2, 4, 6], dtype=torch.uint8)[level]
    for j in range(n):
        row = c.k[c.block_table[0, j // page], j % page, 0]
        row[0], row[8] = 6, codes[j].item()                  # dimensions 0: 4, and 16
    q = torch.zeros(1, R, Hq, D)
    # (every row a common part of its own, of bf16's eight bits)
    part = 2.0 ** big * (1 + (torch.arange(R * Hq) * 37 % 64).view(R, Hq) / 128)
    q[0, ..., 0], q[..., 16] = part / 4, step
    add = torch.tensor([0.0, 1.0, 2.0, 4.0], dtype=torch.float64)[level] * step
    # so many sequences over the same pages that a thread block takes several tiles of one
    B = 160
    many = vw4.KVCache4(c.k, c.v, c.k_blocks, c.v_blocks, c.block_table.repeat(B, 1), c.k_scale, c.v_scale)
    q, lens = q.to(torch.bfloat16).cuda().repeat(B, 1, 1, 1), torch.full((B,), n, dtype=torch.int32, device="cuda")
    for factor in (1.0, 0.93, 1.1, 1.37, 1.73):              # (each rounds the reference differently)
        scale = torch.tensor(factor * math.log(2.0)).item()
        lse = torch.zeros(B, R, Hq, device="cuda")
        out = vw4.verify_attn(q, many, lens, scale=scale, lse=lse).cpu()
        status()
        lse = lse.cpu().double()
        for i in range(R):
            m = n - R + i + 1
            w = ((add[:m] - add[:m].max()) * scale).exp()
            p = w / w.sum()
            want = (p @ v64[0][:m, 0]).expand(B, Hq, D)
            tol = 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2.0 ** -16) * (p @ v64[0][:m, 0].abs()) + 1e-30
            check_close(out[:, i], want, tol, f"factor {factor}, row {i}")
            true = (part[i].double() + add[:m].max()) * scale + w.sum().log()
            assert ((lse[:, i] - true).abs() <= 2.0 ** -22 * true.abs() + 2.0 ** -11).all()
