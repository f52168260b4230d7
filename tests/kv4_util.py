"""Caches in 4 bits and their 64-bit values, for the tests of their operators."""
import torch

import speculative_decode_verification_w4_gb300 as vw4

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
E4M3 = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()


def values64(codes, blocks):
    """What nibbles u8 [..., D / 2] under block scales e4m3 [..., D / 16] stand for."""
    nib = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    v = torch.where(nib >= 8, -E2M1[nib & 7], E2M1[nib & 7])
    return v * blocks.float().double().repeat_interleave(16, -1)


def nearest(x, grid):
    """The nearest value of a grid that begins at 0, ties to the even index; x >= 0."""
    mid = (grid[1:] + grid[:-1]) / 2
    lo, hi = torch.searchsorted(mid, x, right=False), torch.searchsorted(mid, x, right=True)
    return grid[torch.where(lo % 2 == 0, lo, hi)]


def quantised64(t):
    """t [..., D] (over the head's scale) as a 4-bit cache holds it."""
    b = t.clamp(-2688, 2688).unflatten(-1, (-1, 16))
    s = nearest(b.abs().amax(-1, keepdim=True) / 6, E4M3)
    v = torch.where(s > 0, nearest(b.abs() / torch.where(s > 0, s, 1.0), E2M1) * s, 0.0)
    return torch.where(b < 0, -v, v).flatten(-2)


def make_cache4(seed, lens, page, Hkv, D, order="nhd", cols=None):
    """Pages in a random order; tokens beyond a length and unused pages hold any codes under
    NaN scales.  -> (KVCache4, k64, v64): the values of every sequence's tokens in 64 bits
    ([len, Hkv, D] each)."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    per = [-(-max(0, n) // page) for n in lens]
    cols = cols or max(1, max(per))
    total = sum(per) + 2
    ids = torch.randperm(total, generator=g).tolist()
    table = torch.full((B, cols), -7, dtype=torch.int32)
    rows = []
    live = torch.zeros(total, page, dtype=torch.bool)
    for b, n in enumerate(lens):
        row = [ids.pop() for _ in range(per[b])]
        table[b, :per[b]] = torch.tensor(row, dtype=torch.int32)
        rows.append(row)
        for j0 in range(0, max(0, n), page):
            live[row[j0 // page], :min(page, n - j0)] = True
    codes, blocks, head, vals = [], [], [], []
    for _ in range(2):
        c = torch.randint(0, 256, (total, Hkv, page, D // 2), generator=g, dtype=torch.uint8)
        s = torch.exp2(torch.randn(total, Hkv, page, D // 16, generator=g) * 0.7)
        s = torch.where(live[:, None, :, None], s, float("nan")).to(torch.float8_e4m3fn)
        h = (torch.rand(Hkv, generator=g) / 4 + 0.1) * (1 - 2 * torch.randint(0, 2, (Hkv,), generator=g))
        v = values64(c, s).transpose(1, 2) * h.double()[:, None]
        vals.append([torch.cat([v[p] for p in row])[:n] if row else v[0, :0]
                     for row, n in zip(rows, lens)])
        c = c.transpose(1, 2)
        codes.append(c.contiguous().cuda() if order == "nhd" else c.transpose(1, 2).cuda().transpose(1, 2))
        blocks.append(s.cuda())
        head.append(h.cuda())
    cache = vw4.KVCache4(*codes, *blocks, table.cuda(), *head)
    return cache, vals[0], vals[1]
