"""process_logits against its definition in 64 bits.

Tolerance: the fp32 operations after one another (a product or quotient, the
count's product, two or three sums), each half a step (2^-24) of the largest
magnitude on the way."""
import numpy as np
import pytest
import torch

import speculative_decode_verification_w4_gb300 as vw4
from step_util import check_close, status

pytestmark = pytest.mark.gpu
NINF = float("-inf")


def definition(x, drafts, hist, hl, pl, rep, pre, fre, bids, bvals, bl, mask):
    """x fp32 [B, R, V] (numpy, 64 bits inside) -> out, tolerance."""
    B, R, V = x.shape
    out = x.astype(np.float64)
    mag = np.abs(np.where(np.isfinite(out), out, 0))
    for b in range(B):
        for i in range(R):
            ids = [int(t) for t in hist[b, :hl[b]]]
            made = ids[pl[b]:] + [int(t) for t in drafts[b, :i]]
            known = set(t for t in ids + made if 0 <= t < V)
            r = float(rep[b])
            for t in known:
                out[b, i, t] = out[b, i, t] / r if out[b, i, t] > 0 else out[b, i, t] * r
                if np.isfinite(out[b, i, t]):
                    mag[b, i, t] = max(mag[b, i, t], abs(out[b, i, t]))
            for t in set(made):
                if 0 <= t < V:
                    n = made.count(t)
                    out[b, i, t] -= float(fre[b]) * n + float(pre[b])
                    mag[b, i, t] += abs(float(fre[b])) * n + abs(float(pre[b]))
            last = {}
            for t in range(bl[b]):
                if 0 <= bids[b, t] < V:
                    last[int(bids[b, t])] = float(bvals[b, t])
            for t, v in last.items():
                out[b, i, t] += v
                mag[b, i, t] += abs(v) if np.isfinite(v) else 0
            if mask is not None and mask[b][i] is not None:
                out[b, i, ~mask[b][i]] = NINF
    return out, 8 * 2.0 ** -24 * mag


def pack(bits):
    V = len(bits)
    w = np.zeros((V + 31) // 32 * 32, np.uint8)
    w[:V] = bits
    return np.packbits(w, bitorder="little").view(np.int32)


def run_case(seed, B, R, V, H, nb, p_mask=None, ldx=0, inplace=False, index=False, special=False):
    g = np.random.default_rng(seed)
    x = (g.standard_normal((B, R, V)) * 3).astype(np.float32)
    if special:
        x[:, :, 0], x[:, :, 1], x[:, :, 2] = np.inf, -np.inf, np.nan
        x[:, :, V // 2] = 0.0
        x[:, :, V // 2 + 1] = -0.0
    zipf = lambda *s: np.minimum((np.exp(g.random(s) * np.log(V)) - 1).astype(np.int32), V - 1)  # noqa: E731
    drafts, hist = zipf(B, R - 1), zipf(B, H)
    hl = g.integers(0, H + 1, B).astype(np.int32)
    hl[-1] = H
    pl = (hl * g.random(B)).astype(np.int32)
    rep = (1 + g.random(B)).astype(np.float32)
    pre, fre = g.random((2, B)).astype(np.float32)
    bids = zipf(B, nb)
    bvals = (g.standard_normal((B, nb)) * 5).astype(np.float32)
    if nb > 3:
        bvals[:, 0] = NINF
    bl = g.integers(0, nb + 1, B).astype(np.int32)
    mask = words = idx = None
    if p_mask is not None:
        rows = [[g.random(V) < p_mask for _ in range(R)] for _ in range(B)]
        rows[0][0][:] = False  # nothing allowed
        mask = rows
        words = np.stack([np.stack([pack(m) for m in r]) for r in rows])
        if index:  # some rows without a mask, the others' masks in another order
            order = g.permutation(B * R)
            flat = words.reshape(B * R, -1)
            table = np.empty_like(flat)
            table[order] = flat
            idx = order.astype(np.int32).reshape(B, R).copy()
            words = table
            idx[-1, -1] = -1
            mask[-1][-1] = None
    dev = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    wide = torch.full((B, R, V + ldx), 9.0, device="cuda")
    wide[:, :, :V] = dev(x)
    lx = wide[:, :, :V]
    ow = wide if inplace else torch.full((B, R, V + ldx), 9.0, device="cuda")
    bm = torch.full((B, R, (V + 15) // 16), 9.0, device="cuda")
    vw4.process_logits(lx, dev(drafts), history=dev(hist), hist_len=dev(hl), prompt_len=dev(pl),
                       repetition=dev(rep), presence=dev(pre), frequency=dev(fre),
                       bias_ids=dev(bids) if nb else None, bias_vals=dev(bvals) if nb else None,
                       bias_len=dev(bl) if nb else None, mask=dev(words), mask_index=dev(idx),
                       out=ow[:, :, :V], block_max=bm)
    status()
    if not nb:
        bl[:] = 0
    want, tol = definition(x, drafts, hist, hl, pl, rep, pre, fre, bids, bvals, bl, mask)
    got = ow[:, :, :V].cpu().numpy()
    assert (ow[:, :, V:] == 9.0).all()
    nan = np.isnan(want)
    assert np.array_equal(nan, np.isnan(got))
    w = torch.from_numpy(np.where(nan, 0, want))
    check_close(torch.from_numpy(np.where(nan, 0, got)), w, torch.from_numpy(tol), "logits")
    pad = np.full((B, R, -V % 16), NINF, np.float32)
    ref = np.where(np.isnan(got), NINF, got)
    ref = np.concatenate([ref, pad], -1).reshape(B, R, -1, 16).max(-1)
    assert np.array_equal(bm.cpu().numpy(), ref), "block maxima"


@pytest.mark.parametrize("B,R,V", [(1, 1, 1), (1, 1, 31), (2, 3, 33), (3, 2, 4096), (2, 4, 4097),
                                   (1, 16, 5000), (5, 3, 32003), (2, 9, 12288), (300, 2, 100)])
@pytest.mark.parametrize("p_mask", [None, 0.5])
def test_shapes(B, R, V, p_mask):
    run_case(B + R + V, B, R, V, 200, 5, p_mask)


@pytest.mark.parametrize("ldx", [0, 1, 4])
@pytest.mark.parametrize("inplace", [False, True])
def test_strides_and_in_place(ldx, inplace):
    run_case(1, 3, 4, 6000, 50, 4, 0.3, ldx, inplace, index=True)


@pytest.mark.parametrize("H,nb", [(0, 0), (1, 0), (0, 6), (3000, 40)])
def test_lists(H, nb):
    run_case(2, 2, 5, 9000, H, nb)


@pytest.mark.parametrize("p_mask", [None, 0.0, 0.02, 0.9])
def test_special_values(p_mask):
    run_case(3, 2, 3, 5000, 400, 6, p_mask, special=True)


def test_bad_ids():
    x = torch.randn(1, 3, 100, device="cuda")
    d = torch.tensor([[100, -1]], dtype=torch.int32, device="cuda")
    out = vw4.process_logits(x, d, repetition=torch.full((1,), 2.0, device="cuda"))
    status(vw4.DEV_BAD_DRAFT_ID)
    assert torch.equal(out, x)
    h = torch.tensor([[5, 100, -3, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    b = torch.tensor([[200, 7]], dtype=torch.int32, device="cuda")
    one = torch.ones(1, device="cuda")
    out = vw4.process_logits(x[:, :1], history=h, presence=one, bias_ids=b,
                             bias_vals=torch.tensor([[1.0, 2.0]], device="cuda"))
    status(vw4.DEV_BAD_LIST_ID)
    want = x[:, :1].clone()
    want[0, 0, 5] -= 1
    want[0, 0, 7] += 2
    assert torch.equal(out, want)


def test_feeds_the_sampled_accept():
    """The processed logits and their block maxima commit what accept_rejection
    commits on the processed logits alone."""
    import synth
    B, Kd, V = 3, 4, 5000
    target, draft, drafts = synth.stochastic_case(9, B, Kd, V)
    t, d = torch.from_numpy(target).cuda(), torch.from_numpy(draft).cuda()
    dr = torch.from_numpy(drafts).cuda()
    hist = dr.repeat(1, 3).contiguous()
    kw = dict(repetition=torch.full((B,), 1.2, device="cuda"),
              frequency=torch.full((B,), 0.3, device="cuda"), history=hist)
    bt, bd = (torch.empty(B, n, (V + 15) // 16, device="cuda") for n in (Kd + 1, Kd))
    pt = vw4.process_logits(t, dr, block_max=bt, **kw)
    pd = vw4.process_logits(d, dr[:, :Kd - 1].contiguous(), block_max=bd, **kw)
    a = vw4.accept_rejection(pt, pd, dr, 0.6, 0.95, 11)
    b = vw4.accept_rejection_blockmax(pt, bt, pd, bd, dr, 0.6, 0.95, 11)
    status()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_argument_checks():
    x = torch.randn(2, 3, 100, device="cuda")
    d = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        vw4.process_logits(x)
    with pytest.raises(ValueError):
        vw4.process_logits(x, d.long())
    with pytest.raises(ValueError):
        vw4.process_logits(x, d, mask=torch.zeros(2, 3, 3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        vw4.process_logits(x, d, bias_ids=d)
    with pytest.raises(ValueError):
        vw4.process_logits(x.half(), d)
    with pytest.raises(ValueError):
        vw4.process_logits(x, d, out=torch.empty(2, 3, 99, device="cuda"))
