"""verify_attn at the edges of what it takes: many short sequences, scales of any sign,
outputs spread far apart, weights over many powers of two, infinities and NaN in values
(tolerances: step_util.attention64)."""
import pytest
import torch

import speculative_decode_verification_w4_gb300 as vw4
from step_util import attention64, check_close, make_cache, status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("R,G", [(5, 4), (9, 4), (16, 7)])
def test_many_parts_of_one_tile(R, G, D, kv):
    """A thread block takes dozens of items of one tile each: no warp of it falls behind
    by more parts than its barriers can tell apart, and no wait runs out."""
    B, Hkv = 1500, 4
    lens = [16 + (29 * b) % 100 for b in range(B)]
    c, k64, v64 = make_cache(90 + R, lens, 16, Hkv, D, kv)
    g = torch.Generator().manual_seed(R)
    q = torch.randn(B, R, Hkv * G, D, generator=g).to(torch.bfloat16)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    call = vw4.PreparedAttn(q.cuda(), c, n)
    call()
    status()
    first = call.out.clone()
    for _ in range(20):
        call()
    status()
    assert torch.equal(first.view(torch.int16), call.out.view(torch.int16))
    for b in range(0, B, 113):
        o, _, t, _ = attention64(q[b].double(), k64[b], v64[b], lens[b], D ** -0.5, 0, 0, kv)
        check_close(first[b], o, t, f"sequence {b}")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("R,G", [(1, 6), (3, 2), (8, 6), (16, 8)])
@pytest.mark.parametrize("window", [0, 50])
def test_scales_of_any_sign(window, R, G, D):
    """A key head of scale 0 weighs its keys alike; a negative scale turns the scores
    round; a scale may be as small as fp32 has them."""
    lens, scales = [1, 200, 3, 5000], [0.03, 0.0, -0.05, 1e-42, -0.0]
    c, k64, v64 = make_cache(95, lens, 16, len(scales), D, "e4m3")
    new = torch.tensor(scales)
    old = c.k_scale.cpu().double()
    k64 = [k / old[:, None] * new.double()[:, None] for k in k64]
    c.k_scale.copy_(new)
    vs = torch.tensor([0.02, -0.04, 0.0, 0.03, 0.01])
    v64 = [v / c.v_scale.cpu().double()[:, None] * vs.double()[:, None] for v in v64]
    c.v_scale.copy_(vs)
    g = torch.Generator().manual_seed(D)
    q = (torch.randn(len(lens), R, G * len(scales), D, generator=g) * 3).to(torch.bfloat16)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    lse = torch.empty(q.shape[:3], device="cuda")
    out = vw4.verify_attn(q.cuda(), c, n, window=window, lse=lse)
    status()
    for b in range(len(lens)):
        o, l, t, tl = attention64(q[b].double(), k64[b], v64[b], lens[b], D ** -0.5, window, 0, "e4m3")
        check_close(out[b], o, t, f"sequence {b} out")
        check_close(lse[b], l, tl, f"sequence {b} lse")


@pytest.mark.parametrize("R,G,D,kv", [(2, 16, 64, "e4m3"), (2, 4, 128, "bf16")])
def test_output_rows_far_apart(R, G, D, kv):
    """Output rows 2 GiB apart, over more than 64 GiB in all: the bits of a compact output."""
    B, ldo = 34 // R + 1, 1 << 30
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 76 GiB of device memory")
    lens = [9000] + [20 + 3 * b for b in range(B - 1)]
    c, _, _ = make_cache(96, lens, 16, 1, D, kv)
    g = torch.Generator().manual_seed(D)
    q = torch.randn(B, R, G, D, generator=g).to(torch.bfloat16).cuda()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    want = vw4.verify_attn(q, c, n)
    flat = torch.empty((B * R - 1) * ldo + G * D, dtype=torch.bfloat16, device="cuda")
    out = flat.as_strided((B, R, G, D), (R * ldo, ldo, D, 1))
    out.fill_(7.0)
    vw4.verify_attn(q, c, n, out=out)
    status()
    same = torch.equal(out.view(torch.int16), want.view(torch.int16))
    del flat, out
    torch.cuda.empty_cache()
    assert same


@pytest.mark.parametrize("at", [53, 990])
@pytest.mark.parametrize("R,Hq,D", [(1, 4, 64), (2, 8, 128), (1, 3, 256), (8, 6, 64), (4, 6, 128),
                                    (16, 8, 128), (8, 6, 256)])
def test_tail_far_below_one_weight(R, Hq, D, at):
    """A token of weight near 1 and value zero over a thousand of weight 2^-26: the output is
    the tail's alone.  e4m3 caches, items inside one thread block (sequences of the same
    pages).  Off by half a step of bf16, half a step of f16 of every weight and 2^-31 of
    the largest, and the scores' error (delta of step_util.attention64)."""
    B, n, page = 640, 1000, 8
    c, k64, v64 = make_cache(97, [n], page, 1, D, "e4m3")
    one = torch.ones(1, device="cuda")
    c.k.copy_(torch.zeros(c.k.shape, device="cuda").to(c.k.dtype))
    c.v.copy_((torch.rand(c.v.shape, device="cuda") * 100 + 100).to(c.v.dtype))
    row = c.block_table[0].cpu().tolist()
    c.k[row[at // page], at % page, 0] = torch.full((D,), 18 / (0.25 * D ** 0.5) / 0.05,
                                                    device="cuda").to(c.k.dtype)
    c.v[row[at // page], at % page, 0] = (one * 0).to(c.v.dtype)
    c.k_scale.copy_(one * 0.05)
    k = c.k.float().cpu().double()[row].reshape(-1, 1, D)[:n] * float(c.k_scale[0])
    v = c.v.float().cpu().double()[row].reshape(-1, 1, D)[:n] * float(c.v_scale[0])
    cache = vw4.KVCache(c.k, c.v, c.block_table.repeat(B, 1), c.k_scale, c.v_scale)
    q = torch.full((B, R, Hq, D), 0.25, dtype=torch.bfloat16, device="cuda")
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    lse = torch.empty(B, R, Hq, device="cuda")
    out = vw4.verify_attn(q, cache, lens, lse=lse)
    status()
    want, l, _, tl = attention64(q[0].double().cpu(), k, v, n, D ** -0.5, 0, 0, "e4m3")
    score = float(0.25 * k[at].sum() * D ** -0.5)
    assert 17 < score < 20 and 0 < float(want[-1].max()) < 1e-3  # (earlier rows may not see it)
    delta = 2 * D * 2.0 ** -24 * score + 2.0 ** -22 * (2 * score + 1)
    if R * Hq > 16:
        delta += 2.0 ** -17 * 0.25 * float(k[at].sum()) * D ** -0.5
    tol = (2 ** -8 + 2 ** -11 + 2 * delta) * want + n * 2.0 ** -31 * float(v.max())
    check_close(out, want.expand(B, -1, -1, -1), tol.expand(B, -1, -1, -1), "out")
    check_close(lse, l.expand(B, -1, -1), tl.expand(B, -1, -1), "lse")


@pytest.mark.parametrize("kv,D", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("e4m3", 64),
                                  ("e4m3", 128), ("e4m3", 256)])
@pytest.mark.parametrize("R,Hq", [(5, 2), (16, 1), (16, 8), (8, 3), (4, 16)])
@pytest.mark.parametrize("n,window,sinks", [(203, 40, 0), (203, 40, 5), (130, 0, 0), (7000, 3000, 4),
                                            (9000, 0, 0)])
def test_infinite_values_where_they_are_seen(n, window, sinks, R, Hq, kv, D):
    """Infinities and NaN in the values alone: the rows that see one have it, in its
    dimensions and no others; other rows have none.  Short ones, and ones whose parts
    are joined."""
    c, k64, v64 = make_cache(98, [n], 16, 1, D, kv)
    inf, nan = float("inf"), float("nan")
    p0 = n - R
    bad = {n - 1: (1, inf), n - 2: (2, -inf), n - R // 2: (3, nan), n // 2: (4, inf),
           p0 + 1: (5, -inf)}
    if window:  # seen by the first row alone, by the rows up to the third, by none
        bad[p0 - window + 1] = (6, inf)
        bad[p0 - window + 3] = (7, -inf)
        bad[p0 - window] = (8, inf)
    if sinks:
        bad[sinks - 1], bad[sinks] = (9, inf), (10, inf)
    clean, dirty = v64[0].clone(), v64[0].clone()
    for j, (d, x) in bad.items():
        dims = [d, D // 2 + d, D - 20]
        x = nan if kv == "e4m3" else x
        pg = int(c.block_table[0, j // 16])
        for e in dims:
            c.v[pg, j % 16, 0, e] = torch.tensor(x, device="cuda").to(c.v.dtype)
            clean[j, 0, e], dirty[j, 0, e] = 0.0, x
    g = torch.Generator().manual_seed(n)
    q = torch.randn(1, R, Hq, D, generator=g).to(torch.bfloat16)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    lse = torch.empty(1, R, Hq, device="cuda")
    out = vw4.verify_attn(q.cuda(), c, lens, window=window, sinks=sinks, lse=lse)
    status()
    args = (n, D ** -0.5, window, sinks, kv)
    want, l, t, tl = attention64(q[0].double(), k64[0], clean, *args)
    special = attention64(q[0].double(), k64[0], dirty, *args)[0]
    fin = torch.isfinite(special)
    assert not fin[-1].all() and fin.any()
    got = out[0].double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(special))
    assert torch.equal(got[torch.isinf(special)], special[torch.isinf(special)])
    check_close(got[fin], want[fin], t[fin], "finite outputs")
    check_close(lse[0], l, tl, "lse")


def test_many_caches_in_turn():
    """Ninety layers' caches of one shape, and one that takes another's memory over: every
    call reads its own."""
    lens, D = [40], 64
    g = torch.Generator().manual_seed(1)
    q = torch.randn(1, 2, 2, D, generator=g).to(torch.bfloat16)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    caches = [make_cache(200 + i, lens, 16, 1, D, "bf16") for i in range(90)]
    calls = [vw4.PreparedAttn(q.cuda(), c, n) for c, _, _ in caches]
    for _ in range(2):
        for call in calls:
            call()
    status()
    for call, (_, k64, v64) in zip(calls, caches):
        o, _, t, _ = attention64(q[0].double(), k64[0], v64[0], lens[0], D ** -0.5, 0, 0, "bf16")
        check_close(call.out[0], o, t, "out")
    c, k64, v64 = caches[0]
    half = vw4.KVCache(c.k[:, :8], c.v[:, :8], c.block_table.repeat_interleave(2, 1))
    out = vw4.verify_attn(q.cuda(), half, n)  # the same memory as pages of 8, each read twice
    status()
    at = torch.tensor([j // 16 * 16 + j % 8 for j in range(lens[0])])
    k, v = (torch.nan_to_num(x[0][at.clamp(max=lens[0] - 1)]) for x in (k64, v64))
    o, _, t, _ = attention64(q[0].double(), k, v, lens[0], D ** -0.5, 0, 0, "bf16")
    check_close(out[0], o, t, "out")


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("R,G", [(1, 4), (8, 6)])
def test_nothing_in_any_cache(R, G, kv):
    """Every length zero, below zero or shorter than the rows: zeros and minus infinity."""
    c, _, v64 = make_cache(99, [16, 16, 16], 16, 2, 128, kv)
    q = torch.randn(3, R, 2 * G, 128, device="cuda").to(torch.bfloat16)
    for lens in ([0, 0, 0], [-5, 0, -2 ** 31], [0, 1, 0]):
        lse = torch.zeros(3, R, 2 * G, device="cuda")
        out = torch.full_like(q, 7.0)
        vw4.verify_attn(q, c, torch.tensor(lens, dtype=torch.int32, device="cuda"), out=out, lse=lse)
        status()
        seen = torch.zeros(3, R, dtype=torch.bool)
        seen[1, R - 1] = lens[1] == 1  # the last row of the second sequence sees its one token
        assert (out[~seen] == 0).all() and (lse[~seen] == float("-inf")).all()
        if lens[1] == 1:
            want = v64[1][0].repeat_interleave(G, 0)
            check_close(out[1, -1], want, 2.0 ** -7 * want.abs(), "one token")


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("order", ["nhd", "hnd"])
@pytest.mark.parametrize("R,G", [(2, 4), (8, 3)])
def test_cache_beyond_32_bits(R, G, order, kv):
    """Pages of a cache of more than 2^32 elements: the append writes its last ones, and the
    attention reads them."""
    page, Hkv, D, B, n = 64, 8, 128, 2, 150
    pages = (1 << 32) // (page * Hkv * D) + 100
    dt = torch.bfloat16 if kv == "bf16" else torch.float8_e4m3fn
    shape = (pages, page, Hkv, D) if order == "nhd" else (pages, Hkv, page, D)
    k, v = (torch.empty(shape, dtype=dt, device="cuda") for _ in range(2))
    if order == "hnd":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    table = torch.tensor([[pages - 1, pages - 7, 3], [pages - 3, 0, pages - 2]], dtype=torch.int32)
    scale = None if kv == "bf16" else torch.full((Hkv,), 1 / 32, device="cuda")
    c = vw4.KVCache(k, v, table.cuda(), scale, scale)
    g = torch.Generator().manual_seed(R)
    Hq, keys, values = Hkv * G, [], []
    for at in range(0, n, 10):  # (no rotation: what is stored is what is given)
        x = torch.randn(B * 10, (Hq + 2 * Hkv) * D, generator=g).to(torch.bfloat16)
        vw4.verify_rope_append(x.cuda(), c, torch.full((B,), at + 10, dtype=torch.int32, device="cuda"),
                               10, Hq)
        rows = x.view(B, 10, Hq + 2 * Hkv, D)
        keys.append(rows[:, :, Hq:Hq + Hkv])
        values.append(rows[:, :, Hq + Hkv:])
    stored = [torch.cat(t, 1) for t in (keys, values)]
    if kv == "e4m3":
        stored = [(t.float() * 32).clamp(-448, 448).to(dt).float() / 32 for t in stored]
    q = torch.randn(B, R, Hq, D, generator=g).to(torch.bfloat16)
    out = vw4.verify_attn(q.cuda(), c, torch.full((B,), n, dtype=torch.int32, device="cuda"))
    status()
    for b in range(B):
        o, _, t, _ = attention64(q[b].double(), stored[0][b].double(), stored[1][b].double(), n,
                                 D ** -0.5, 0, 0, kv)
        check_close(out[b], o, t, f"sequence {b}")
