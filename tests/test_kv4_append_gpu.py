"""verify_rope_append into the 4-bit cache, and read_kv4, against their formulas in 64 bits:
the codes and block scales exactly, queries within half a step of bf16 and the fp32 work
before it (test_append_gpu)."""
import pytest
import torch

import speculative_decode_verification_w4_gb300 as vw4
from kv4_util import make_cache4, quantised64, values64
from step_util import check_close, status
from test_append_gpu import norm64, rotate64

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def run_case(seed, lens, R, Hq, Hkv, D, page, order, rot, adjacent, norm, bf16, gain=1.0, scales=None,
             x=None, far=1.0):
    g = torch.Generator().manual_seed(seed)
    c, _, _ = make_cache4(seed, lens, page, Hkv, D, order)
    if scales is not None:
        c.k_scale.copy_(torch.tensor(scales))
        c.v_scale.copy_(torch.tensor(scales))
    old = [t.cpu() for t in (c.k, c.v, c.k_blocks.view(torch.uint8), c.v_blocks.view(torch.uint8))]
    B, heads = len(lens), Hq + 2 * Hkv
    if x is None:
        x = torch.randn(B * R, heads * D, generator=g) * gain
    if bf16:
        x = x.to(torch.bfloat16)
    inv = 1e4 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / max(1, rot)) * far
    qn = kn = None
    eps = 2.0 ** -16
    if norm:
        qn, kn = torch.randn(D, generator=g) + 1, torch.randn(D, generator=g) + 1
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    q = vw4.verify_rope_append(x.cuda(), c, ints(lens), R, Hq, inv_freq=inv.cuda() if rot else None,
                               adjacent=adjacent, q_norm=dev(qn), k_norm=dev(kn), eps=eps)
    status()
    xs = x.double().view(B * R, heads, D)
    pos = (torch.tensor(lens)[:, None] - R + torch.arange(R)).flatten()
    wq = rotate64(norm64(xs[:, :Hq], qn, eps), pos, inv, rot, adjacent)
    wk = rotate64(norm64(xs[:, Hq:Hq + Hkv], kn, eps), pos, inv, rot, adjacent)
    wv = xs[:, Hq + Hkv:]
    tol = 2 ** -8 * wq.abs() + D * 2.0 ** -24 * wq.abs().amax(-1, keepdim=True) * 2
    check_close(q.view(B * R, Hq, D), wq, tol, "queries")
    for what, t, bl, w, o, ob, sc in (
            ("keys", c.k, c.k_blocks, wk, old[0], old[2], c.k_scale),
            ("values", c.v, c.v_blocks, wv, old[1], old[3], c.v_scale)):
        sc = sc.cpu().double()[:, None]
        got, bl = t.cpu(), bl.cpu()
        written = torch.zeros(got.shape[:2], dtype=torch.bool)
        for r in range(B * R):
            b, p = r // R, int(pos[r])
            if p < 0:
                continue
            pg, at = int(c.block_table[b, p // page]), p % page
            written[pg, at] = True
            want = quantised64(torch.where(sc == 0, 0.0, w[r] / torch.where(sc == 0, 1.0, sc)))
            have = values64(got[pg, at], bl[pg, :, at])
            assert torch.equal(have, want), f"{what} row {r}: {int((have != want).sum())} values differ"
        assert torch.equal(got[~written], o[~written]), f"{what}: another slot was written"
        keep = ~written[:, None, :].expand(bl.shape[:3])
        assert torch.equal(bl.view(torch.uint8)[keep], ob[keep]), f"{what}: another scale was written"
    return c


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("part,norm,bf16", [(1, True, False), (2, False, True), (4, True, True),
                                            (0, True, False), (0, False, False), (0, False, True)])
def test_shapes(part, norm, bf16, adjacent, D):
    rot = D // part if part else 0
    run_case(1, [1, 3, 65, 200], 4, 6, 2, D, 16, "nhd" if part else "hnd", rot, adjacent, norm, bf16)


@pytest.mark.parametrize("rot", [2, 6, 34, 126])
def test_odd_rotations(rot):
    run_case(2, [9, 40], 3, 4, 1, 128, 8, "hnd", rot, False, True, False)


@pytest.mark.parametrize("R,Hq,Hkv,B", [(1, 24, 4, 1), (16, 32, 4, 2), (9, 24, 4, 100), (1, 1, 1, 5)])
def test_batches(R, Hq, Hkv, B):
    """Half a million keys among them: some lie so near a border that 32 bits cannot tell."""
    run_case(3, [16 + 5 * b for b in range(B)], R, Hq, Hkv, 256, 16, "nhd", 256, False, True, False)


def test_far_positions():
    run_case(4, [131071], 2, 2, 1, 64, 512, "nhd", 64, False, False, False)


@pytest.mark.parametrize("gain", [1e-6, 1e-3, 30.0, 3000.0, 1e6])
def test_magnitudes(gain):
    """Blocks below the smallest scale, and beyond the largest."""
    run_case(5, [50], 4, 2, 2, 64, 16, "nhd", 64, False, False, False, gain=gain, scales=[1.0, -0.03])


def test_head_scale_of_zero():
    run_case(6, [50], 4, 2, 2, 64, 16, "nhd", 64, False, True, False, scales=[0.0, 1.0])


@pytest.mark.parametrize("bf16", [False, True])
def test_ties(bf16):
    """Values on the borders between codes, and maxima on those between scales."""
    D, R, Hkv = 64, 8, 2
    steps = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.5, 1.0, -0.25, -2.5, -5.0, 0.0, 5.5, 4.5])
    rows = []
    for k in range(R):
        head = torch.cat([steps * 2.0 ** (k - 3) * m for m in (1.0, 1.125, 17 / 16, 19 / 16)])
        rows.append(head.repeat(2 + 2 * Hkv))
    x = torch.stack(rows)
    run_case(7, [40], R, 2, Hkv, D, 16, "nhd", 0, False, False, bf16, scales=[1.0, 0.25], x=x)


def test_not_finite():
    """A NaN makes its block NaN; an infinity is the largest value of its block."""
    D, lens = 64, [20]
    c, _, _ = make_cache4(8, lens, 16, 1, D)
    c.v_scale.fill_(0.5)
    x = torch.ones(1, 3 * D)
    x[0, 2 * D + 3] = float("nan")
    x[0, 2 * D + 17] = float("-inf")
    vw4.verify_rope_append(x.cuda(), c, ints(lens), 1, 1)
    status()
    _, v = vw4.read_kv4(c, ints(lens), 1, dtype=torch.float32)
    v = v.cpu().flatten()
    assert torch.isnan(v[:16]).all()
    assert v[17] == -2688 * 0.5 and (v[16:32] == 0).sum() == 15
    # (a quotient of 2 is a third of the block's largest: scale 1/3 in e4m3, 0.34375, times 6)
    assert (v[32:] == 6 * 0.34375 * 0.5).all()


def test_bad_pages():
    D, lens = 64, [40, 49]  # 49: beyond the table's 48
    c, _, _ = make_cache4(9, [40, 40], 16, 1, D)
    before = c.k.clone()
    c.block_table[0, 2] = c.k.shape[0] + 3
    vw4.verify_rope_append(torch.randn(4, 3 * D, device="cuda"), c, ints(lens), 2, 1)
    status(vw4.DEV_BAD_PAGE)
    assert int((before != c.k).any(-1).sum()) == 1  # position 47 of the second sequence


@pytest.mark.parametrize("order", ["nhd", "hnd"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,page", [(1, 8), (77, 16), (700, 64)])
def test_read(n, page, dtype, D, order):
    lens = [1, 0, 63, 300, 699]
    c, k64, v64 = make_cache4(30 + n, lens, page, 3, D, order)
    for first in (None, [0, 0, 5, 290, -3]):
        k, v = vw4.read_kv4(c, ints(lens), n, None if first is None else ints(first), dtype)
        status()
        for got, want in ((k, k64), (v, v64)):
            for b, length in enumerate(lens):
                p = (length - n if first is None else first[b]) + torch.arange(n)
                live = (p >= 0) & (p < length)
                w = torch.zeros(n, 3, D, dtype=torch.float64)
                w[live] = want[b][p[live]]
                # a product by the head's scale: half a step of fp32, then of bf16
                step = 2.0 ** -24 if dtype == torch.float32 else 2.0 ** -8
                check_close(got[b], w, w.abs() * step * (1 + 2.0 ** -15), f"sequence {b}")


def test_read_bad_pages():
    c, k64, _ = make_cache4(31, [100], 16, 2, 64)
    c.block_table[0, 1] = 1 << 20
    k, _ = vw4.read_kv4(c, ints([100]), 100, dtype=torch.float32)
    status(vw4.DEV_BAD_PAGE)
    assert (k[0, 16:32] == 0).all()
    check_close(k[0, :16], k64[0][:16], k64[0][:16].abs() * 2.0 ** -23, "keys")
    vw4.read_kv4(c, ints([200]), 5)  # beyond the table
    status(vw4.DEV_BAD_PAGE)
