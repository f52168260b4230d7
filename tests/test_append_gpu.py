"""verify_rope_append against its formulas in 64 bits.

Tolerances count the roundings: half a step of the stored type (bf16 2^-8,
e4m3 2^-4 relative, 2^-10 of a unit of the scale below e4m3's normal range),
and for the fp32 work before it D 2^-24 relative of the head's largest rotated
pair (norm, sine and cosine, two products)."""
import pytest
import torch

import speculative_decode_verification_w4_gb300 as vw4
from step_util import check_close, make_cache, status

pytestmark = pytest.mark.gpu


def rotate64(t, pos, inv_freq, rot, adjacent):
    """t [n, heads, D] in 64 bits, pos [n]."""
    if rot == 0:
        return t
    a = pos.double()[:, None, None] * inv_freq
    c, s = a.cos(), a.sin()
    u = t.clone()
    if adjacent:
        x, y = t[..., 0:rot:2], t[..., 1:rot:2]
        u[..., 0:rot:2], u[..., 1:rot:2] = x * c - y * s, y * c + x * s
    else:
        h = rot // 2
        x, y = t[..., :h], t[..., h:rot]
        u[..., :h], u[..., h:rot] = x * c - y * s, y * c + x * s
    return u


def norm64(t, w, eps):
    return t if w is None else t / ((t * t).mean(-1, keepdim=True) + eps).sqrt() * w.double()


def run_case(seed, lens, R, Hq, Hkv, D, page, kv, order, rot, adjacent, norm, bf16, far=1.0,
             gain=1.0):
    g = torch.Generator().manual_seed(seed)
    c, _, _ = make_cache(seed, lens, page, Hkv, D, kv, order)
    old = [t.cpu().float() for t in (c.k, c.v)]
    B, heads = len(lens), Hq + 2 * Hkv
    x = torch.randn(B * R, heads * D, generator=g) * gain
    if bf16:
        x = x.to(torch.bfloat16)
    inv = 1e4 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / max(1, rot)) * far
    qn = kn = None
    eps = 1e-5
    if norm:
        qn, kn = torch.randn(D, generator=g) + 1, torch.randn(D, generator=g) + 1
    n = torch.tensor(lens, dtype=torch.int32)
    q = torch.full((B, R, Hq, D), 5.0, dtype=torch.bfloat16, device="cuda")
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    vw4.verify_rope_append(x.cuda(), c, n.cuda(), R, Hq, inv_freq=inv.cuda() if rot else None,
                           adjacent=adjacent, q_norm=dev(qn), k_norm=dev(kn), eps=eps, q_out=q)
    status()
    xs = x.double().view(B * R, heads, D)
    pos = (n[:, None] - R + torch.arange(R)).flatten()
    wq = rotate64(norm64(xs[:, :Hq], qn, eps), pos, inv, rot, adjacent)
    wk = rotate64(norm64(xs[:, Hq:Hq + Hkv], kn, eps), pos, inv, rot, adjacent)
    wv = xs[:, Hq + Hkv:]

    def fp32(t):
        return D * 2.0 ** -24 * t.abs().amax(-1, keepdim=True) * 2
    wq_t = 2 ** -8 * wq.abs() + fp32(wq)
    check_close(q.view(B * R, Hq, D), wq, wq_t, "queries")
    for what, t, w, o, sc in (("keys", c.k, wk, old[0], c.k_scale), ("values", c.v, wv, old[1], c.v_scale)):
        got = t.cpu().float()
        written = torch.zeros(got.shape[:2], dtype=torch.bool)
        for r in range(B * R):
            b, p = r // R, int(pos[r])
            if p < 0:
                continue
            pg = int(c.block_table[b, p // page])
            written[pg, p % page] = True
            want = w[r]
            if sc is None:
                tol = 2 ** -8 * want.abs() + fp32(want)
            else:
                want = (want / sc.cpu().double()[:, None])
                t32 = fp32(want)
                want = want.clamp(-448, 448)
                tol = 2 ** -4 * want.abs() + 2 ** -10 + t32
            check_close(got[pg, p % page], want, tol, f"{what} row {r}")
        same = (got == o) | (torch.isnan(got) & torch.isnan(o))
        assert same[~written].all(), f"{what}: another slot was written"


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("part,norm,bf16", [(1, True, False), (2, False, True), (4, True, True),
                                            (0, True, False), (0, False, False)])
def test_shapes(part, norm, bf16, adjacent, D, kv):
    rot = D // part if part else 0
    run_case(1, [1, 3, 65, 200], 4, 6, 2, D, 16, kv, "nhd" if part else "hnd", rot, adjacent, norm,
             bf16)


@pytest.mark.parametrize("rot", [2, 6, 34, 126])
def test_odd_rotations(rot):
    run_case(2, [9, 40], 3, 4, 1, 128, 8, "bf16", "hnd", rot, False, True, False)


@pytest.mark.parametrize("R,Hq,Hkv,B", [(1, 24, 4, 1), (16, 32, 4, 2), (9, 24, 4, 40), (1, 1, 1, 5)])
def test_batches(R, Hq, Hkv, B):
    run_case(3, [16 + 5 * b for b in range(B)], R, Hq, Hkv, 256, 16, "e4m3", "nhd", 256, False, True,
             False)


def test_far_positions_and_saturation():
    """Positions near 2^17 at full frequency (a 32-bit angle would be off by
    2^-7), and values beyond 448 scales."""
    run_case(4, [131071], 2, 2, 1, 64, 512, "bf16", "nhd", 64, False, False, False)
    run_case(5, [50], 4, 2, 1, 64, 16, "e4m3", "nhd", 64, False, False, False, gain=500.0)


def test_bad_pages():
    c, _, _ = make_cache(6, [40, 40], 16, 1, 64, "bf16")
    before = c.k.clone()
    c.block_table[0, 2] = c.k.shape[0] + 3
    n = torch.tensor([40, 49], dtype=torch.int32, device="cuda")   # 49: beyond the table's 48
    x = torch.randn(4, 3 * 64, device="cuda")
    q = vw4.verify_rope_append(x, c, n, 2, 1)
    status(vw4.DEV_BAD_PAGE)
    check_close(q.view(4, 64), x[:, :64].double().cpu(), 2 ** -8 * x[:, :64].double().abs().cpu(), "q")
    same = (before == c.k) | (torch.isnan(before) & torch.isnan(c.k))
    assert int((~same.flatten(2).all(-1)).sum()) == 1  # position 47 of the second sequence


def test_argument_checks():
    c, _, _ = make_cache(7, [40], 16, 1, 64, "bf16")
    n = torch.tensor([40], dtype=torch.int32, device="cuda")
    x = torch.randn(2, 3 * 64, device="cuda")
    with pytest.raises(ValueError):
        vw4.verify_rope_append(x.half(), c, n, 2, 1)
    with pytest.raises(ValueError):
        vw4.verify_rope_append(x, c, n.long(), 2, 1)
    with pytest.raises(ValueError):
        vw4.verify_rope_append(x, c, n, 2, 1, inv_freq=torch.ones(4, device="cuda"))
    with pytest.raises(vw4.VW4Error):
        vw4.verify_rope_append(x, c, n, 2, 1, inv_freq=torch.ones(33, dtype=torch.float64,
                                                                  device="cuda"))
    with pytest.raises(ValueError):
        vw4.verify_attn(torch.zeros(1, 2, 1, 64, device="cuda"), c, n)
    with pytest.raises(vw4.VW4Error):
        vw4.verify_attn(torch.zeros(1, 2, 1, 64, device="cuda", dtype=torch.bfloat16), c, n, sinks=3)
    with pytest.raises(ValueError):
        vw4.KVCache(c.k, c.v[:, :8], c.block_table)
    with pytest.raises(vw4.VW4Error):
        vw4.verify_attn(torch.zeros(1, 2, 1, 64, device="cuda", dtype=torch.bfloat16), c, n,
                        workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
