"""The calls between the verify GEMMs together: on a stream of their own, in one
captured graph, inside guarded buffers; and sizes at the borders of their
kernels' variants."""
import pytest
import torch

import speculative_decode_verification_w4_gb300 as vw4
from step_util import attention64, check_close, make_cache, status
from test_logits_gpu import run_case

pytestmark = pytest.mark.gpu


def guarded(shape, dtype, fill):
    n = 1
    for d in shape:
        n *= d
    flat = torch.full((n + 512,), fill, dtype=dtype, device="cuda")
    return flat, flat[256:-256].view(shape)


@pytest.mark.parametrize("kv,R,Hq,Hkv,D", [("bf16", 3, 8, 2, 128), ("e4m3", 5, 24, 4, 256),
                                           ("e4m3", 1, 6, 2, 64)])
def test_stream_graph_and_guards(kv, R, Hq, Hkv, D):
    """A captured append, attention and logits call on another stream, replayed on new
    inputs, against the same calls made one by one: the same bits."""
    B, V, lens = 3, 1003, [70, 5, 200]
    g = torch.Generator().manual_seed(D)
    c, _, _ = make_cache(60, [256] * B, 16, Hkv, D, kv)
    cache2, _, _ = make_cache(60, [256] * B, 16, Hkv, D, kv)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    x = torch.randn(B * R, (Hq + 2 * Hkv) * D, generator=g).cuda()
    inv = (1e4 ** (-torch.arange(D // 2, dtype=torch.float64) * 2 / D)).cuda()
    logits = torch.randn(B, R, V, generator=g).cuda()
    ids = torch.randint(0, V, (B, R - 1 + 40), generator=g).to(torch.int32).cuda()
    drafts, hist = ids[:, :R - 1].contiguous(), ids[:, R - 1:].contiguous()
    hl = torch.tensor([40, 0, 7], dtype=torch.int32, device="cuda")
    rep = torch.full((B,), 1.3, device="cuda")
    fq, q = guarded((B, R, Hq, D), torch.bfloat16, -3.0)
    fo, out = guarded((B, R, Hq, D), torch.bfloat16, -3.0)
    fl, y = guarded((B, R, V), torch.float32, -3.0)
    fb, bmax = guarded((B, R, (V + 15) // 16), torch.float32, -3.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    calls = [vw4.PreparedAppend(x, c, n, R, Hq, inv_freq=inv, q_out=q, stream=s),
             vw4.PreparedAttn(q, c, n, out=out, workspace=vw4.Workspace(), stream=s),
             vw4.PreparedLogits(logits, drafts, history=hist, hist_len=hl, repetition=rep,
                                presence=rep, out=y, block_max=bmax, stream=s)]
    with torch.cuda.stream(s):
        for call in calls:
            call()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        for call in calls:
            call()
    for new in ([71, 6, 201], [1, 255, 33]):
        x.copy_(torch.randn(x.shape, generator=g))
        logits.copy_(torch.randn(logits.shape, generator=g))
        n.copy_(torch.tensor(new, dtype=torch.int32))
        cache2.k.view(torch.uint8).copy_(c.k.view(torch.uint8))
        cache2.v.view(torch.uint8).copy_(c.v.view(torch.uint8))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        q2 = vw4.verify_rope_append(x, cache2, n, R, Hq, inv_freq=inv)
        out2 = vw4.verify_attn(q2, cache2, n)
        y2 = vw4.process_logits(logits, drafts, history=hist, hist_len=hl, repetition=rep, presence=rep)
        status()
        for a, b in ((q, q2), (out, out2), (c.k, cache2.k), (c.v, cache2.v)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        assert torch.equal(y, y2)
        wide = torch.nn.functional.pad(y2, (0, -V % 16), value=float("-inf"))
        assert torch.equal(bmax, wide.view(B, R, -1, 16).amax(-1))
    for f in (fq, fo, fl, fb):
        assert (f[:256] == -3).all() and (f[-256:] == -3).all()


@pytest.mark.parametrize("B,R,V", [(1, 2, 1023), (1, 2, 1024), (1, 2, 1028), (4, 3, 2049),
                                   (40, 9, 4092), (40, 9, 4101), (152, 2, 4096), (153, 2, 4096)])
def test_logits_at_chunk_borders(B, R, V):
    run_case(V + B, B, R, V, 60, 4, 0.5)


@pytest.mark.parametrize("D,kv", [(64, "bf16"), (64, "e4m3"), (128, "e4m3"), (256, "bf16")])
@pytest.mark.parametrize("R,Hq", [(5, 4), (16, 4)])
def test_growing_maxima(D, kv, R, Hq):
    """Keys that grow by powers of two (exact in either type), now in one half of a tile
    and now in the other, so that the running maximum moves far at every step."""
    n, page = 900, 32
    c, _, v64 = make_cache(70, [n], page, 1, D, kv)
    at = torch.arange(n)
    e = torch.where(at // 64 % 3 == 1, at // 128, 0).clamp(max=6) - 4
    gain = torch.pow(2.0, e.double())
    if kv == "e4m3":  # (the stored values stay in e4m3's normal range)
        gain = torch.pow(2.0, (e.clamp(max=0) // 2).double())
    table = c.block_table[0].cpu()
    store = c.k.float().cpu()
    for j0 in range(0, n, page):
        m = min(page, n - j0)
        store[table[j0 // page], :m] *= gain[j0:j0 + m, None, None].float()
    c.k.copy_(store.to(c.k.dtype))
    ks = 1.0 if c.k_scale is None else float(c.k_scale[0])
    k = torch.cat([c.k.float().cpu()[table[j0 // page], :min(page, n - j0)].double() * ks
                   for j0 in range(0, n, page)])
    g = torch.Generator().manual_seed(5)
    q = (torch.randn(1, R, Hq, D, generator=g) * 4).to(torch.bfloat16)
    length = torch.tensor([n], dtype=torch.int32, device="cuda")
    lse = torch.empty(1, R, Hq, device="cuda")
    out = vw4.verify_attn(q.cuda(), c, length, lse=lse)
    status()
    o, want, t, tl = attention64(q[0].double(), k, v64[0], n, D ** -0.5, 0, 0, kv)
    check_close(out[0], o, t, "output")
    check_close(lse[0], want, tl, "log-sum-exp")


@pytest.mark.parametrize("D,page", [(64, 8), (64, 16), (128, 8), (128, 16), (128, 64), (256, 16)])
def test_first_call_on_a_cold_cache(D, page):
    """Pages scattered over memory that was not read before: loads land late and out of
    order.  The first call gives the bits of the ones after it."""
    B, Hkv, n = 32, 8, 4000
    cols = -(-n // page)
    g = torch.Generator().manual_seed(page + D)
    total = B * cols * 2
    table = torch.randperm(total, generator=g)[:B * cols].view(B, cols).to(torch.int32).cuda()
    k, v = ((torch.randn(total // 64 + 1, 64, page, Hkv, D, device="cuda", dtype=torch.bfloat16) * 20)
            .to(torch.float8_e4m3fn).view(-1, page, Hkv, D)[:total] for _ in range(2))
    sc = torch.full((Hkv,), 1 / 20, device="cuda")
    cache = vw4.KVCache(k, v, table, sc, sc)
    lens = torch.randint(n // 2, n, (B,), generator=g).to(torch.int32).cuda()
    q = torch.randn(B, 8, 4 * Hkv, D, generator=g).to(torch.bfloat16).cuda()
    status()
    first = vw4.verify_attn(q, cache, lens)
    for _ in range(3):
        again = vw4.verify_attn(q, cache, lens)
        status()
        assert torch.equal(first.view(torch.int16), again.view(torch.int16))


@pytest.mark.parametrize("R,G", [(1, 3), (4, 6), (16, 8)])
@pytest.mark.parametrize("B,Hkv,n", [(1, 1, 9000), (1, 8, 3000), (4, 8, 1500), (8, 8, 700), (20, 8, 300)])
def test_items_in_many_and_few_parts(B, Hkv, n, R, G):
    """One item over every CTA down to many items each inside one: every way of joining."""
    D, kv = 128, "e4m3" if R == 4 else "bf16"
    lens = [n - 7 * b for b in range(B)]
    c, k64, v64 = make_cache(80 + B, lens, 64, Hkv, D, kv)
    g = torch.Generator().manual_seed(B)
    q = (torch.randn(B, R, Hkv * G, D, generator=g) * 2).to(torch.bfloat16)
    length = torch.tensor(lens, dtype=torch.int32, device="cuda")
    lse = torch.empty(B, R, Hkv * G, device="cuda")
    out = vw4.verify_attn(q.cuda(), c, length, lse=lse)
    status()
    for b in {0, B // 2, B - 1}:
        o, want, t, tl = attention64(q[b].double(), k64[b], v64[b], lens[b], D ** -0.5, 0, 0, kv)
        check_close(out[b], o, t, f"sequence {b} output")
        check_close(lse[b], want, tl, f"sequence {b} log-sum-exp")
