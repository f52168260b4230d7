"""Caches and 64-bit definitions for the tests of the operators between the
verify GEMMs (attention, cache append, logits processing)."""
import numpy as np
import torch

import speculative_decode_verification_w4_gb300 as vw4


def status(expect=0):
    torch.cuda.synchronize()
    st = vw4.vw4_get_device_status()
    assert st == expect, f"device status {st:#x}, expected {expect:#x}"


def make_cache(seed, lens, page, Hkv, D, kv, order="nhd", cols=None, fill=True):
    """Pages in a random order; tokens beyond a length and unused pages hold NaN.
    -> (KVCache, k64, v64): the cache, and the values of every sequence's tokens
    in 64 bits ([len, Hkv, D] each)."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    per = [-(-max(0, n) // page) for n in lens]
    cols = cols or max(1, max(per))
    total = sum(per) + 2
    ids = torch.randperm(total, generator=g).tolist()
    table = torch.full((B, cols), -7, dtype=torch.int32)
    shape = (total, page, Hkv, D)
    nan = float("nan")
    ks = vs = None
    if kv == "e4m3":
        ks, vs = torch.rand(Hkv, generator=g) / 16 + 0.01, torch.rand(Hkv, generator=g) / 16 + 0.01
    dt = torch.bfloat16 if kv == "bf16" else torch.float8_e4m3fn
    store, vals = [], []
    for sc in (ks, vs):
        t = torch.full(shape, nan)
        store.append(t)
    seqs = []
    for b, n in enumerate(lens):
        row = [ids.pop() for _ in range(per[b])]
        table[b, :per[b]] = torch.tensor(row, dtype=torch.int32)
        if fill:
            for t in store:
                x = torch.randn(max(0, n), Hkv, D, generator=g) * (24 if kv == "e4m3" else 1)
                for j0 in range(0, max(0, n), page):
                    m = min(page, n - j0)
                    t[row[j0 // page], :m] = x[j0:j0 + m]
        seqs.append(row)
    out = []
    for t in store:
        t = t.to(dt)
        t = t if order == "nhd" else t.transpose(1, 2).contiguous().transpose(1, 2)
        out.append(t)
    for t, sc in zip(out, (ks, vs)):
        x = t.float().double()
        if sc is not None:
            x = x * sc.double()[:, None]
        vals.append([torch.cat([x[p] for p in row])[:n] if row else x[:0].reshape(0, Hkv, D)
                     for row, n in zip(seqs, lens)])

    def dev(t):
        if t is None:
            return None
        return t.cuda() if order == "nhd" or t.dim() < 4 else t.transpose(1, 2).cuda().transpose(1, 2)
    cache = vw4.KVCache(dev(out[0]), dev(out[1]), table.cuda(), dev(ks), dev(vs))
    return cache, vals[0], vals[1]


def seen(n, R, window, sinks):
    """bool [R, n]: which token of the cache each verify row sees."""
    p = (n - R + torch.arange(R))[:, None]
    j = torch.arange(n)[None, :]
    s = j <= p
    if window:
        s = s & ((j > p - window) | (j < sinks))
    return s


def attention64(q, k, v, n, scale, window, sinks, kv):
    """One sequence: q [R, Hq, D], k / v [n, Hkv, D] in 64 bits -> out, lse, and
    how far a kernel may be from them.

    The tolerance counts the roundings: half a step of bf16 on the output; the
    weights' half step on sum(p |v|): bf16 2^-8; e4m3 caches f16, 2^-11, and
    2^-25 below its normal range; the scores' fp32 error delta = 2 D 2^-24 scale
    sum|q k|, plus 2^-22 of the exponent, on every weight; e4m3 caches with more
    than 16 rows a key head: the queries' two e4m3 terms, 2^-17 of the row's
    largest, on every score."""
    R, Hq, D = q.shape
    Hkv = k.shape[1] if n else 1
    out = torch.zeros(R, Hq, D, dtype=torch.float64)
    lse = torch.full((R, Hq), float("-inf"), dtype=torch.float64)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    if n <= 0:
        return out, lse, tol, tol_lse
    G = Hq // Hkv
    vis = seen(n, R, window, sinks)
    terms = kv == "e4m3" and R * G > 16
    wp, tiny = (2 ** -8, 0.0) if kv == "bf16" else (2 ** -11, 2 ** -25)
    for i in range(R):
        sel = torch.nonzero(vis[i])[:, 0]
        if len(sel) == 0:
            continue
        ki, vi = k[sel], v[sel]

        def heads(x, y, eq):  # per key head, its G query heads
            return torch.einsum(eq, x.reshape(Hkv, G, -1), y).reshape(Hq, -1)
        s = heads(q[i], ki, "kgd,tkd->kgt") * scale
        mag = heads(q[i].abs(), ki.abs(), "kgd,tkd->kgt").amax(1) * scale
        m = s.amax(1, keepdim=True)
        p = (s - m).exp()
        z = p.sum(1, keepdim=True)
        o = heads(p / z, vi, "kgt,tkd->kgd")
        a = heads(p / z, vi.abs(), "kgt,tkd->kgd")
        delta = 2 * D * 2.0 ** -24 * mag + 2.0 ** -22 * (2 * s.abs().amax(1) + 1)
        if terms:
            k1 = ki.abs().sum(2).amax(0).repeat_interleave(G)  # largest sum|k| of the key head
            delta = delta + 2.0 ** -17 * q[i].abs().amax(1) * k1 * scale
        out[i], lse[i] = o, (m + z.log())[:, 0]
        tol[i] = (2 ** -8 * o.abs() + wp * a + 2 * delta[:, None] * a
                  + tiny * vi.abs().sum(0).repeat_interleave(G, 0) / z + 1e-30)
        tol_lse[i] = delta + 2.0 ** -22 * (1 + lse[i].abs())
    return out, lse, tol, tol_lse


def check_close(got, want, tol, what):
    got = got.double().cpu()
    assert torch.isfinite(got).all() or not torch.isfinite(want).all(), f"{what}: not finite"
    fin = torch.isfinite(want)
    assert torch.equal(got[~fin], want[~fin]), f"{what}: infinities differ"
    err = (got[fin] - want[fin]).abs()
    bad = ~(err <= tol[fin])
    if bad.any():
        k = int(torch.nonzero(bad)[0, 0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; first "
                             f"{got[fin][k].item()} for {want[fin][k].item()} +- {tol[fin][k].item()}")


def as_numpy(t):
    return np.asarray(t.cpu())
