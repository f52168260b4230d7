"""The bytes that the 4-bit append stores, codes and block scales, against the 64-bit formula:
blocks whose rotation partners are far larger than themselves, zeros of either sign under head
scales of either sign, products that leave the range of 32 bits, sums of squares that do.

A code is the magnitude's index with a sign bit where t < 0, and 0 where the block's scale is 0
or t is; a NaN in a block makes its scale NaN, and its codes mean nothing.  There is no
tolerance."""
import pytest
import torch

import speculative_decode_verification_w4_gb300 as vw4
from kv4_util import E2M1, E4M3, make_cache4
from step_util import status
from test_append_gpu import norm64, rotate64

pytestmark = pytest.mark.gpu


def index_of(x, grid):
    """The index of the nearest value of a grid that begins at 0, ties to the even one; x >= 0."""
    mid = (grid[1:] + grid[:-1]) / 2
    lo, hi = torch.searchsorted(mid, x, right=False), torch.searchsorted(mid, x, right=True)
    return torch.where(lo % 2 == 0, lo, hi)


def bytes64(t):
    """t [..., D] (over the head's scale) -> codes u8 [..., D], scales u8 [..., D / 16]."""
    b = t.unflatten(-1, (-1, 16))
    bad = torch.isnan(b).any(-1)
    b = torch.nan_to_num(b, nan=0.0, posinf=2688.0, neginf=-2688.0).clamp(-2688, 2688)
    s = index_of((b.abs().amax(-1) / 6).contiguous(), E4M3)
    v = E4M3[s][..., None]
    c = torch.where(v > 0, index_of((b.abs() / torch.where(v > 0, v, 1.0)).contiguous(), E2M1), 0)
    c = torch.where((v > 0) & (b < 0), c + 8, c)
    return c.to(torch.uint8).flatten(-2), torch.where(bad, 0x7F, s).to(torch.uint8)


def run(x, lens, R, Hkv, D, scales, rot=0, adjacent=False, k_norm=None, eps=1e-6, page=16):
    """Rows x [B * R, (Hkv + 2 Hkv) D] into a cache, and every stored byte compared."""
    B, Hq, eps = len(lens), Hkv, torch.tensor(eps).item()  # (what fp32 has of it)
    c, _, _ = make_cache4(5, lens, page, Hkv, D)
    for t in (c.k_scale, c.v_scale):
        t.copy_(torch.tensor(scales))
    inv = 1e4 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / max(1, rot))
    vw4.verify_rope_append(x.cuda(), c, torch.tensor(lens, dtype=torch.int32, device="cuda"), R, Hq,
                           inv_freq=inv.cuda() if rot else None, adjacent=adjacent,
                           k_norm=None if k_norm is None else k_norm.cuda(), eps=eps)
    status()
    xs = x.double().view(B * R, 3 * Hkv, D)
    pos = (torch.tensor(lens)[:, None] - R + torch.arange(R)).flatten()
    k = rotate64(norm64(xs[:, Hkv:2 * Hkv], k_norm, eps), pos, inv, rot, adjacent)
    for what, got, blocks, w in (("keys", c.k, c.k_blocks, k), ("values", c.v, c.v_blocks, xs[:, 2 * Hkv:])):
        g = torch.tensor(scales).double()[:, None]
        w = torch.where(g == 0, 0.0, w / torch.where(g == 0, 1.0, g))
        codes, bl = bytes64(w)
        got, blocks = got.cpu(), blocks.cpu().view(torch.uint8)
        for r in range(B * R):
            p = int(pos[r])
            if p < 0:
                continue
            pg, at = int(c.block_table[r // R, p // page]), p % page
            have = torch.stack([got[pg, at] & 15, got[pg, at] >> 4], -1).flatten(-2)
            assert torch.equal(blocks[pg, :, at] & 0x7F, bl[r] & 0x7F), f"{what}: scales of row {r}"
            assert ((blocks[pg, :, at] == bl[r]) | (bl[r] == 0x7F)).all(), f"{what}: a scale's sign, row {r}"
            ok = (bl[r] != 0x7F).repeat_interleave(16, -1)
            assert torch.equal(have[ok], codes[r][ok]), f"{what}: codes of row {r}"


def heads(B, R, Hkv, D, seed=0, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(B * R, 3 * Hkv, D, generator=g) * gain


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("small,partner", [(0.0, 1.0), (0.0, 200.0), (1e-4, 200.0), (-1e-4, 200.0), (1e-7, 1.0),
                                           (0.0, 1e6)])
def test_blocks_far_below_their_partners(small, partner, adjacent, D):
    """At position 0, where nothing turns, and behind it: a block of zeros or next to them whose
    partners in the rotation are large, so that the bound of a key's error exceeds the block."""
    Hkv, R = 2, 3
    x = heads(2, R, Hkv, D, gain=1e-3)
    k = x[:, Hkv:2 * Hkv]
    if adjacent:
        k[..., 0::2], k[..., 1::2] = small, partner
    else:
        k[..., :D // 2], k[..., D // 2:] = small, partner
    x[:, Hkv + 1] = x[:, Hkv + 1].flip(-1)
    run(x.flatten(1), [R, 40], R, Hkv, D, [1 / 32, -1 / 32], rot=D, adjacent=adjacent)


@pytest.mark.parametrize("rot,norm", [(0, False), (64, False), (64, True), (6, False)])
@pytest.mark.parametrize("scales", [[1.0, -1.0], [0.03, -0.07], [0.0, -0.0]])
def test_zeros_of_either_sign(scales, rot, norm):
    """Zeros among others and blocks of nothing else, and blocks below half of the least scale."""
    D, Hkv, R = 64, 2, 4
    x = heads(1, R, Hkv, D)
    x[0, :, ::2], x[0, :, 1::4] = 0.0, -0.0
    x[1] = -0.0
    x[2, :, :16], x[2, :, 16:32], x[2, :, 32:48] = 0.0, -0.0, -1e-9
    x[3] *= 1e-8
    w = torch.linspace(0.5, 2.0, D) if norm else None
    run(x.flatten(1), [R], R, Hkv, D, scales, rot=rot, k_norm=w)


@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("rot,norm", [(0, False), (64, False), (64, True)])
@pytest.mark.parametrize("gain,g", [(1e19, 1e-20), (1e10, 1e-29), (1.0, 3e-30), (1e25, 1e-10), (1e29, 1e-29),
                                    (1e-20, 1e-25), (1e-25, 1e20)])
def test_quotients_beyond_32_bits(gain, g, rot, norm, D):
    """Values and head scales that are ordinary numbers, and quotients that are not."""
    Hkv, R = 2, 2
    x = heads(2, R, Hkv, D, 1, gain)
    x[0, Hkv, :16] = 0.0
    w = torch.linspace(0.5, 2.0, D) if norm else None
    run(x.flatten(1), [R, 77], R, Hkv, D, [g, -g], rot=rot, k_norm=w)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rot,adjacent", [(0, False), (64, False), (64, True), (10, False)])
@pytest.mark.parametrize("gain,eps", [(3e18, 1e-6), (1e19, 1e-6), (1e24, 1e-6), (1e37, 1e-6), (1e-19, 0.0),
                                      (1e-22, 0.0), (1e-30, 0.0), (1e-19, 1e-38), (0.0, 0.0)])
def test_sums_of_squares_beyond_32_bits(gain, eps, rot, adjacent, D):
    """Heads whose norm is an ordinary number in 64 bits alone."""
    Hkv, R = 2, 2
    x = heads(2, R, Hkv, D, 2)
    x[:, Hkv:2 * Hkv] *= gain
    run(x.flatten(1), [R, 1000], R, Hkv, D, [0.02, -0.02], rot=rot, adjacent=adjacent,
        k_norm=torch.linspace(-1.0, 2.0, D), eps=eps)


@pytest.mark.parametrize("rot,norm", [(0, False), (64, False), (64, True), (32, True)])
def test_not_finite(rot, norm):
    """NaN and infinities in keys and values, beside partners and heads that are finite."""
    D, Hkv, R = 128, 2, 6
    x = heads(1, R, Hkv, D, 3)
    for r, v in enumerate((float("nan"), float("inf"), float("-inf"))):
        x[2 * r, :, 3] = v
        x[2 * r + 1, :, 100] = v
    w = torch.linspace(0.5, 2.0, D) if norm else None
    run(x.flatten(1), [40], R, Hkv, D, [0.5, -0.25], rot=rot, k_norm=w)
