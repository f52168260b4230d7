"""verify_attn against its definition in 64 bits (tolerances: step_util.attention64)."""
import pytest
import torch

import speculative_decode_verification_w4_gb300 as vw4
from step_util import attention64, check_close, make_cache, status

pytestmark = pytest.mark.gpu


def run_case(seed, lens, R, Hq, Hkv, D, page, kv, order="nhd", window=0, sinks=0, scale=None,
             gain=2.0, cache=None, q=None, **kw):
    cache = cache or make_cache(seed, lens, page, Hkv, D, kv, order)
    c, k64, v64 = cache
    g = torch.Generator().manual_seed(seed + 1)
    if q is None:
        q = (torch.randn(len(lens), R, Hq, D, generator=g) * gain).to(torch.bfloat16)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    lse = torch.full((len(lens), R, Hq), 7.0, device="cuda")
    out = torch.full((len(lens), R, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    vw4.verify_attn(q.cuda(), c, n, scale=scale, window=window, sinks=sinks, out=out, lse=lse, **kw)
    status()
    for b in range(len(lens)):
        o, l, t, tl = attention64(q[b].double(), k64[b], v64[b], lens[b], scale or D ** -0.5, window,
                                  sinks, kv)
        check_close(out[b], o, t, f"sequence {b} out")
        check_close(lse[b], l, tl, f"sequence {b} lse")
    return out, lse


LENGTHS = [1, 2, 63, 64, 65, 127, 129, 200]


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("R,Hq,Hkv", [(1, 8, 2), (8, 8, 4), (4, 6, 1), (5, 24, 4), (16, 8, 1),
                                      (9, 12, 1), (16, 32, 2)])
def test_shapes(R, Hq, Hkv, D, kv):
    """Every row layout (16, 32, 64, 128 rows and several blocks of rows), one
    to a few tiles, lengths on both sides of a tile, rows before the cache."""
    run_case(10 + R, LENGTHS, R, Hq, Hkv, D, 16, kv)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("order", ["nhd", "hnd"])
@pytest.mark.parametrize("page", [8, 32, 128, 512])
def test_pages(page, order, kv):
    run_case(page, [5, 300, 1025], 3, 8, 4, 128, page, kv, order)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page,order", [(8, "nhd"), (8, "hnd"), (128, "hnd"), (256, "nhd")])
def test_pages_many_rows(page, order, D, kv):
    run_case(page + 1, [5, 300, 1025], 9, 8, 4, D, page, kv, order)


@pytest.mark.parametrize("R", [2, 9])
@pytest.mark.parametrize("D,kv", [(64, "e4m3"), (128, "bf16"), (256, "bf16"), (256, "e4m3")])
def test_head_stride_of_its_own(D, kv, R):
    """Heads spaced apart by neither a head nor whole groups of tokens."""
    lens, page, Hkv = [200, 77], 16, 3
    c, k64, v64 = make_cache(33, lens, page, Hkv, D, kv)
    stores = []
    for t in (c.k, c.v):
        wide = torch.zeros(t.shape[0], page, Hkv, D + 32, device="cuda").to(t.dtype)
        wide[..., :D] = t
        stores.append(wide[..., :D])
    cache = vw4.KVCache(stores[0], stores[1], c.block_table, c.k_scale, c.v_scale)
    run_case(33, lens, R, 6, Hkv, D, page, kv, cache=(cache, k64, v64))


@pytest.mark.parametrize("D,kv", [(64, "bf16"), (128, "e4m3"), (256, "bf16"), (256, "e4m3")])
@pytest.mark.parametrize("R", [1, 8])
def test_long_split(R, D, kv):
    """One sequence over many CTAs, joined; beside a short and an empty one."""
    run_case(3, [9000], R, 4, 2, D, 64, kv)
    run_case(4, [0, 7001, 3, 0, 130], R, 4, 2, D, 64, kv)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 4), (7, 0), (64, 4), (100, 33), (130, 200),
                                          (5000, 3)])
@pytest.mark.parametrize("R", [1, 6])
def test_window_and_sinks(R, window, sinks, kv):
    run_case(window, [1, 4, 65, 199, 700, 1500], R, 6, 2, 128, 16, kv, window=window, sinks=sinks)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("R,G,D,page", [(8, 6, 256, 64), (16, 8, 256, 16), (16, 8, 128, 32),
                                        (4, 6, 128, 128), (9, 3, 64, 8), (16, 8, 64, 256),
                                        (1, 4, 256, 16), (2, 8, 64, 64)])
def test_many_tiles_per_block(R, G, D, page, kv):
    """Several tiles of one item in every thread block, and several items in one."""
    run_case(60, [41000], R, G, 1, D, page, kv)
    run_case(61, [300 + 37 * b for b in range(40)], R, 2 * G, 2, D, page, kv)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("R,G,D", [(4, 6, 256), (16, 6, 128), (7, 3, 64), (1, 6, 128)])
def test_many_windows_per_block(R, G, D, kv):
    run_case(62, [700 + 61 * b for b in range(40)], R, 2 * G, 2, D, 16, kv, window=500, sinks=5)


@pytest.mark.parametrize("D,R,G,kv", [(128, 16, 8, "bf16"), (256, 8, 6, "bf16"), (256, 4, 6, "e4m3"),
                                      (64, 9, 8, "e4m3"), (128, 1, 4, "e4m3")])
def test_calls_one_after_another(D, R, G, kv):
    """Two calls in turn, 300 times with nothing waiting between: the same bits as
    alone, and no wait ran out."""
    calls, outs, alone = [], [], []
    for k, lens in enumerate(([9000 + 77 * b for b in range(8)], [500 + 7 * b for b in range(30)])):
        c, _, _ = make_cache(70 + k, lens, 32, 2, D, kv)
        g = torch.Generator().manual_seed(k)
        q = torch.randn(len(lens), R, 2 * G, D, generator=g).to(torch.bfloat16).cuda()
        out = torch.empty_like(q)
        calls.append(vw4.PreparedAttn(q, c, torch.tensor(lens, dtype=torch.int32, device="cuda"), out=out))
        calls[-1]()
        torch.cuda.synchronize()
        outs.append(out)
        alone.append(out.clone())
    for _ in range(300):
        for c in calls:
            c()
    status()
    for a, b in zip(outs, alone):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_many_sequences():
    lens = [(37 * b) % 301 for b in range(300)]
    run_case(5, lens, 2, 4, 2, 64, 16, "bf16")


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("R,Hq,D", [(1, 4, 128), (8, 6, 256), (16, 4, 64)])
def test_long_tail_under_one_large_weight(R, Hq, D, kv):
    """One token takes most of the weight, and thousands of small ones the rest."""
    n = 6000
    c, k64, v64 = make_cache(25, [n], 16, 1, D, kv)
    q = torch.full((1, R, Hq, D), 0.25, dtype=torch.bfloat16)
    big = 9.0 / (0.25 * D * D ** -0.5)          # score 9: weight e^9 over 6000 of about 1
    unit = 1.0 if kv == "bf16" else float(c.k_scale[0])
    c.k[int(c.block_table[0, 3]), 5, 0] = torch.full((D,), big / unit, device="cuda").to(c.k.dtype)
    k64[0][53, 0] = (torch.full((D,), big / unit).to(c.k.dtype).float().double() * unit)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    out = vw4.verify_attn(q.cuda(), c, lens)
    status()
    o, _, t, _ = attention64(q[0].double(), k64[0], v64[0], n, D ** -0.5, 0, 0, kv)
    check_close(out[0], o, t, "out")


def test_small_and_large_scores():
    run_case(6, [500], 4, 4, 1, 128, 16, "bf16", gain=40.0)
    run_case(7, [500], 4, 4, 1, 128, 16, "e4m3", gain=1e-6)
    run_case(8, [500], 4, 4, 1, 128, 16, "bf16", scale=3.0)


@pytest.mark.parametrize("kv,D", [("bf16", 128), ("bf16", 256), ("e4m3", 64), ("e4m3", 256)])
@pytest.mark.parametrize("R,Hq", [(5, 2), (16, 8), (8, 3)])
def test_unseen_infinities(R, Hq, kv, D):
    """NaN and infinities in keys and values that only later rows see (and in
    what lies before the window) leave the earlier rows as they are."""
    n, window = 203, 40
    c, k64, v64 = make_cache(20, [n], 16, 1, D, kv)
    inf = torch.tensor(float("nan") if kv == "e4m3" else float("inf"), device="cuda")
    bad = [n - 1, n - 2, n - R - window - 3]
    for j in bad:
        pg = int(c.block_table[0, j // 16])
        c.k[pg, j % 16, 0, :7] = inf.to(c.k.dtype)
        c.v[pg, j % 16, 0, 1:9] = inf.to(c.v.dtype)
    q = torch.randn(1, R, Hq, D, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    lse = torch.empty(1, R, Hq, device="cuda")
    out = vw4.verify_attn(q.cuda(), c, lens, window=window, lse=lse)
    status()
    o, l, t, tl = attention64(q[0].double(), k64[0], v64[0], n, D ** -0.5, window, 0, kv)
    keep = R - 2  # rows that see neither of the last two tokens
    check_close(out[0, :keep], o[:keep], t[:keep], "out")
    check_close(lse[0, :keep], l[:keep], tl[:keep], "lse")
    assert torch.isnan(out[0, keep + 1]).any()


def test_strides_stream_and_graph():
    """Queries and outputs inside wider rows, K and V in one tensor, another
    stream, and a captured call replayed on new inputs and lengths."""
    B, R, Hq, Hkv, D, page = 3, 4, 8, 2, 128, 16
    lens = [100, 40, 333]
    c, k64, v64 = make_cache(30, lens, page, Hkv, D, "bf16")
    both = torch.stack([c.k, c.v], 1)  # [pages, 2, page, Hkv, D]
    cache = vw4.KVCache(both[:, 0], both[:, 1], c.block_table)
    g = torch.Generator().manual_seed(31)
    wide = torch.randn(B, R, Hq + 2 * Hkv, D, generator=g).to(torch.bfloat16).cuda()
    q = wide[:, :, :Hq]
    outw = torch.full((B, R, Hq + 1, D), 3.0, dtype=torch.bfloat16, device="cuda")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = vw4.Workspace()
    call = vw4.PreparedAttn(q, cache, n, out=outw[:, :, :Hq], workspace=ws, stream=s)
    with torch.cuda.stream(s):
        call()
    s.synchronize()

    def verify(lens):
        status()
        for b in range(B):
            o, _, t, _ = attention64(q[b].double().cpu(), k64[b][:lens[b]], v64[b][:lens[b]], lens[b],
                                     D ** -0.5, 0, 0, "bf16")
            check_close(outw[b, :, :Hq], o, t, f"sequence {b}")
        assert (outw[:, :, Hq] == 3.0).all()
    verify(lens)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call()
    wide.copy_(torch.randn(wide.shape, generator=g).to(torch.bfloat16))
    n.copy_(torch.tensor([99, 4, 17], dtype=torch.int32))
    graph.replay()
    verify([99, 4, 17])


def test_bad_pages_and_lengths():
    """A page id outside the cache reads as zero keys and values and sets
    VW4_DEV_BAD_PAGE; so does a length beyond the table (it is cut to it)."""
    lens, D = [200, 70], 64
    c, k64, v64 = make_cache(40, lens, 16, 2, D, "bf16")
    c.block_table[0, 3] = c.k.shape[0]
    c.block_table[1, 1] = -1
    k64[0][48:64] = 0
    v64[0][48:64] = 0
    k64[1][16:32] = 0
    v64[1][16:32] = 0
    q = torch.randn(2, 2, 4, D, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = vw4.verify_attn(q.cuda(), c, n)
    status(vw4.DEV_BAD_PAGE)
    for b in range(2):
        o, _, t, _ = attention64(q[b].double(), k64[b], v64[b], lens[b], D ** -0.5, 0, 0, "bf16")
        check_close(out[b], o, t, f"sequence {b}")
    c, k64, v64 = make_cache(41, [64], 16, 2, D, "bf16")
    n = torch.tensor([1000], dtype=torch.int32, device="cuda")
    out = vw4.verify_attn(q[:1].cuda(), c, n)
    status(vw4.DEV_BAD_PAGE)
    o, _, t, _ = attention64(q[0].double(), k64[0], v64[0], 64, D ** -0.5, 0, 0, "bf16")
    check_close(out[0], o, t, "cut length")


@pytest.mark.parametrize("D,kv,R,Hq", [(64, "bf16", 1, 4), (128, "e4m3", 8, 4), (256, "bf16", 16, 4),
                                       (128, "bf16", 16, 8)])
def test_canaries(D, kv, R, Hq):
    """Nothing is written beyond the outputs and the workspace, which needs no
    initialization; the same call again gives the same bits."""
    lens = [700, 1, 65]
    c, _, _ = make_cache(50, lens, 16, 1, D, kv)
    k0, v0 = c.k.view(torch.uint8).clone(), c.v.view(torch.uint8).clone()
    q = torch.randn(3, R, Hq, D, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    need = vw4.vw4_workspace_bytes(vw4.OP_ATTN, 3, R * Hq, D)
    ref = None
    for _ in range(2):
        ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        flat = torch.full((3 * R * Hq * D + 2048,), -3.0, dtype=torch.bfloat16, device="cuda")
        fl = torch.full((3 * R * Hq + 512,), -3.0, device="cuda")
        out = flat[1024:-1024].view(3, R, Hq, D)
        lse = fl[256:-256].view(3, R, Hq)
        vw4.verify_attn(q, c, n, out=out, lse=lse, workspace=ws[:need])
        status()
        assert (flat[:1024] == -3).all() and (flat[-1024:] == -3).all()
        assert (fl[:256] == -3).all() and (fl[-256:] == -3).all()
        assert (ws[need:] == 0xA5).all()
        if ref is not None:
            assert torch.equal(ref[0].view(torch.int16), out.view(torch.int16))
            assert torch.equal(ref[1], lse)
        ref = (out.clone(), lse.clone())
    assert torch.equal(k0, c.k.view(torch.uint8)) and torch.equal(v0, c.v.view(torch.uint8))
