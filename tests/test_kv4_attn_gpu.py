"""verify_attn over the 4-bit cache against its definition in 64 bits (tolerances:
step_util.attention64, with the f16 weights that verify_attn_kv4 documents)."""
import pytest
import torch

import speculative_decode_verification_w4_gb300 as vw4
from kv4_util import make_cache4
from step_util import attention64, check_close, status

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def queries(seed, B, R, Hq, D, gain=2.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(B, R, Hq, D, generator=g) * gain).to(torch.bfloat16)


def run_case(seed, lens, R, Hq, Hkv, D, page, order="nhd", window=0, sinks=0, scale=None, gain=2.0,
             cache=None, only=None):
    c, k64, v64 = cache or make_cache4(seed, lens, page, Hkv, D, order)
    q = queries(seed + 1, len(lens), R, Hq, D, gain)
    lse = torch.full((len(lens), R, Hq), 7.0, device="cuda")
    out = torch.full((len(lens), R, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    vw4.verify_attn(q.cuda(), c, ints(lens), scale=scale, window=window, sinks=sinks, out=out, lse=lse)
    status()
    for b in only if only is not None else range(len(lens)):
        o, l, t, tl = attention64(q[b].double(), k64[b], v64[b], lens[b], scale or D ** -0.5, window,
                                  sinks, "nvfp4")
        check_close(out[b], o, t, f"sequence {b} out")
        check_close(lse[b], l, tl, f"sequence {b} lse")
    return out, lse


LENGTHS = [1, 2, 63, 64, 65, 127, 129, 200]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("R,Hq,Hkv", [(1, 8, 2), (1, 12, 1), (4, 6, 1), (5, 24, 4), (8, 8, 2),
                                      (8, 6, 1), (16, 8, 2), (16, 32, 2), (13, 7, 1), (3, 256, 1)])
def test_shapes(R, Hq, Hkv, D):
    """Every number of row tiles and several blocks of rows, one to a few tiles, lengths on
    both sides of a tile, rows before the cache."""
    run_case(10 + R, LENGTHS, R, Hq, Hkv, D, 16)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("R,G", [(16, 2), (3, 11), (16, 4), (5, 13), (16, 8), (3, 43), (1, 129),
                                 (10, 13), (4, 33), (3, 48), (2, 200)])
def test_numbers_of_rows(R, G, D):
    """32 and 33, 64 and 65, 128 and 129 rows of a key head, and cuts of more into blocks by
    verify indexes and by heads; beside full tiles, with a window that ends inside some."""
    Hkv = 2 if G <= 128 else 1
    run_case(40 + R, [R, 150, 600, 1111], R, Hkv * G, Hkv, D, 16)
    run_case(41 + R, [333, 901], R, G, 1, D, 8, window=200, sinks=17)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("order", ["nhd", "hnd"])
@pytest.mark.parametrize("page", [8, 32, 128, 512])
def test_pages(page, order, D):
    run_case(page, [5, 300, 1025], 3, 8, 4, D, page, order)


@pytest.mark.parametrize("R", [1, 9])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_head_stride_of_its_own(D, R):
    """Heads spaced apart by neither a head nor whole groups of tokens; scales too."""
    lens, page, Hkv = [200, 77], 16, 3
    c, k64, v64 = make_cache4(33, lens, page, Hkv, D)
    wide = []
    for t in (c.k, c.v):
        w = torch.zeros(t.shape[0], page, Hkv, D // 2 + 32, dtype=torch.uint8, device="cuda")
        w[..., :D // 2] = t
        wide.append(w[..., :D // 2])
    for t in (c.k_blocks, c.v_blocks):
        w = torch.zeros(t.shape[0], Hkv + 1, page + 4, D // 16, device="cuda").to(t.dtype)
        w[:, :Hkv, :page] = t
        wide.append(w[:, :Hkv, :page])
    cache = vw4.KVCache4(*wide, c.block_table, c.k_scale, c.v_scale)
    run_case(33, lens, R, 6, Hkv, D, page, cache=(cache, k64, v64))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("R,G", [(1, 2), (8, 2), (8, 6)])
def test_long_split(R, G, D):
    """One sequence over many CTAs, joined; beside a short and an empty one."""
    run_case(3, [9000], R, 2 * G, 2, D, 64)
    run_case(4, [0, 7001, 3, 0, 130], R, 2 * G, 2, D, 64)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 4), (7, 0), (64, 4), (100, 33), (130, 200),
                                          (5000, 3)])
@pytest.mark.parametrize("R,Hq", [(1, 6), (6, 6), (9, 16)])
def test_window_and_sinks(R, Hq, window, sinks):
    run_case(window, [1, 4, 65, 199, 700, 1500], R, Hq, 2, 128, 16, window=window, sinks=sinks)


@pytest.mark.parametrize("R,G,D,page", [(8, 6, 256, 64), (16, 8, 128, 32), (4, 6, 128, 128),
                                        (9, 3, 64, 8), (1, 4, 256, 16), (2, 8, 64, 64),
                                        (4, 6, 256, 16)])
def test_many_tiles_per_block(R, G, D, page):
    """Several tiles of one item in every thread block, and several items in one."""
    run_case(60, [41000], R, G, 1, D, page)
    run_case(61, [300 + 37 * b for b in range(40)], R, 2 * G, 2, D, page, only=range(0, 40, 7))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("R,G,page,order,window,sinks", [(1, 4, 8, "nhd", 0, 0), (1, 8, 64, "hnd", 0, 0),
                                                         (2, 3, 512, "nhd", 700, 9), (1, 1, 16, "hnd", 257, 300),
                                                         (4, 2, 32, "nhd", 64, 1)])
def test_tables_for_every_sm(R, G, page, order, window, sinks, D):
    """Few rows over tables that hold a large tile for every SM; lengths on both sides of one."""
    lens = [0, 1, 63, 128, 129, 255, 256, 257, 511, 513, 1000, 4099] + [300 + 71 * b for b in range(28)]
    run_case(80 + R, lens, R, 2 * G, 2, D, page, order, window=window, sinks=sinks)


@pytest.mark.parametrize("R,G,D", [(5, 4, 64), (9, 4, 128), (16, 7, 256), (1, 3, 128)])
def test_many_parts_of_one_tile(R, G, D):
    B, Hkv = 1500, 4
    lens = [16 + (29 * b) % 100 for b in range(B)]
    out, _ = run_case(90 + R, lens, R, Hkv * G, Hkv, D, 16, only=range(0, B, 113))


@pytest.mark.parametrize("R,G,D", [(4, 6, 256), (16, 6, 128), (7, 3, 64), (1, 6, 128)])
def test_many_windows_per_block(R, G, D):
    run_case(62, [700 + 61 * b for b in range(40)], R, 2 * G, 2, D, 16, window=500, sinks=5,
             only=range(0, 40, 5))


@pytest.mark.parametrize("D,R,G", [(128, 16, 8), (256, 8, 6), (64, 9, 8), (128, 1, 4)])
def test_calls_one_after_another(D, R, G):
    """Two calls in turn, 300 times with nothing waiting between: the same bits as alone, and
    no wait ran out."""
    calls, outs, alone = [], [], []
    for k, lens in enumerate(([3000 + 77 * b for b in range(8)], [500 + 7 * b for b in range(30)])):
        c, _, _ = make_cache4(70 + k, lens, 32, 2, D)
        q = queries(k, len(lens), R, 2 * G, D).cuda()
        out = torch.empty_like(q)
        calls.append(vw4.PreparedAttn(q, c, ints(lens), out=out))
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


@pytest.mark.parametrize("R,Hq,D", [(1, 4, 128), (8, 6, 256), (16, 4, 64), (3, 5, 128)])
def test_growing_scores(R, Hq, D):
    """Keys whose scores rise along the sequence by far more than the reference may lag
    (every tile moves it), and fall: one token takes nearly all of the weight."""
    n, page = 3000, 16
    for order in (1, -1):
        c, k64, v64 = make_cache4(25, [n], page, 1, D)
        s = torch.exp2(torch.linspace(-8 * order, 7 * order, n) + (0 if order > 0 else -1))  # block scales of the tokens
        for j in range(n):
            c.k_blocks[c.block_table[0, j // page], 0, j % page] = s[j].item()
        c.k.fill_(0x22)  # ones
        got = s.to(torch.float8_e4m3fn).double() * c.k_scale.cpu().double()
        k64 = [got[:, None, None].expand(n, 1, D)]
        run_case(26, [n], R, Hq, 1, D, page, gain=0.3, cache=(c, k64, v64))


@pytest.mark.parametrize("R,Hq,D", [(1, 4, 64), (2, 8, 128), (1, 3, 256), (8, 6, 64)])
def test_tail_far_below_one_weight(R, Hq, D):
    """A token of weight near 1 and value zero over a thousand of weight 2^-24: the output is
    the tail's alone.  Off by half a step of bf16 and of f16 of every weight, 2^-34 of the
    largest, and the scores' error."""
    n, page = 1000, 8
    c, k64, v64 = make_cache4(97, [n], page, 1, D)
    c.k.zero_()
    c.v.fill_(0x66)  # fours
    c.k_scale.fill_(1.0)
    c.v_scale.fill_(1.0)
    c.v_blocks.copy_(torch.ones(c.v_blocks.shape))
    c.k_blocks.copy_(torch.ones(c.k_blocks.shape))
    at = 53
    page_id = int(c.block_table[0, at // page])
    c.k[page_id, at % page] = 0x22
    c.v[page_id, at % page] = 0
    q = torch.ones(1, R, Hq, D, dtype=torch.bfloat16)
    scale = 24 * 0.6931471805599453 / D
    out = vw4.verify_attn(q.cuda(), c, ints([n]), scale=scale)
    status()
    seen = n - R + torch.arange(R) + 1  # keys of the rows
    w = 2.0 ** -24
    want = (4.0 * (seen - 1) * w / (1 + (seen - 1) * w)).double()[:, None, None].expand(R, Hq, D)
    tol = want * (2 ** -8 + 2 ** -11) + 4.0 * n * 2.0 ** -34 + want * 2 * (2 * D * 2.0 ** -24 * 17 + 2.0 ** -22 * 49)
    check_close(out[0], want, tol, "out")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("R,G", [(1, 6), (3, 2), (8, 6), (16, 8)])
@pytest.mark.parametrize("window", [0, 50])
def test_scales_of_any_sign(window, R, G, D):
    """A key head of scale 0 weighs its keys alike; a negative scale turns the scores round;
    a scale may be as small as fp32 has them."""
    lens, scales = [1, 200, 3, 2000], [0.03, 0.0, -0.05, 1e-42, -0.0]
    c, k64, v64 = make_cache4(95, lens, 16, len(scales), D)
    new, vs = torch.tensor(scales), torch.tensor([0.02, -0.04, 0.0, 0.03, 0.01])
    k64 = [k / c.k_scale.cpu().double()[:, None] * new.double()[:, None] for k in k64]
    v64 = [v / c.v_scale.cpu().double()[:, None] * vs.double()[:, None] for v in v64]
    c.k_scale.copy_(new)
    c.v_scale.copy_(vs)
    run_case(95, lens, R, G * len(scales), len(scales), D, 16, window=window, gain=3.0,
             cache=(c, k64, v64))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("R,Hq", [(1, 2), (6, 2), (9, 6)])
@pytest.mark.parametrize("window", [0, 40])
def test_nan_scales(window, R, Hq, D):
    """A NaN block of a key takes the rows that see it, a NaN block of a value those rows'
    16 dimensions; no others."""
    n, page = 300, 16
    for at in (n - 3, n - 1, 250, 100, 0):
        for which in ("k", "v"):
            c, k64, v64 = make_cache4(44, [n], page, 1, D)
            clean = attention64(queries(45, 1, R, Hq, D)[0].double(), k64[0], v64[0], n, D ** -0.5,
                                window, 0, "nvfp4")
            blocks = c.k_blocks if which == "k" else c.v_blocks
            blocks[c.block_table[0, at // page], 0, at % page, 1] = float("nan")
            out = vw4.verify_attn(queries(45, 1, R, Hq, D).cuda(), c, ints([n]), window=window)
            status()
            got = out[0].double().cpu()
            for i in range(R):
                p = n - R + i
                hit = at <= p and (window == 0 or at > p - window)
                bad = torch.zeros(D, dtype=torch.bool)
                if hit:
                    bad[slice(0, D) if which == "k" else slice(16, 32)] = True
                assert torch.isnan(got[i][:, bad]).all(), (at, which, i)
                o, t = clean[0][i][:, ~bad], clean[2][i][:, ~bad]
                check_close(got[i][:, ~bad], o, t, f"{which} at {at}, row {i}")


def test_bad_pages_read_as_zeros():
    lens, page, D = [300, 200, 90], 16, 128
    c, k64, v64 = make_cache4(46, lens, page, 2, D)
    c.block_table[0, 3] = c.k.shape[0] + 5
    c.block_table[1, 0] = -1
    for t in (k64, v64):
        t[0][48:64] = 0
        t[1][:16] = 0
    q = queries(47, 3, 4, 6, D)
    out = vw4.verify_attn(q.cuda(), c, ints(lens))
    status(vw4.DEV_BAD_PAGE)
    for b in range(3):
        o, _, t, _ = attention64(q[b].double(), k64[b], v64[b], lens[b], D ** -0.5, 0, 0, "nvfp4")
        check_close(out[b], o, t, f"sequence {b}")
    # a length beyond the table is cut to it
    out = vw4.verify_attn(q.cuda(), c, ints([300, 200, 5000]))
    status(vw4.DEV_BAD_PAGE)


def test_graph_and_streams():
    """A captured call, replayed with other inputs, and calls on two streams: the bits of the
    calls alone."""
    lens = [700, 3, 5000]
    c, _, _ = make_cache4(48, lens, 32, 2, 128)
    q, n = queries(49, 3, 4, 8, 128).cuda(), ints(lens)
    want = vw4.verify_attn(q, c, n).clone()
    q2, n2 = queries(50, 3, 4, 8, 128).cuda(), ints([650, 2, 1])
    want2 = vw4.verify_attn(q2, c, n2).clone()
    call = vw4.PreparedAttn(q, c, n)
    call()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call = vw4.PreparedAttn(q, c, n)
        with torch.cuda.graph(graph, stream=side):
            call()
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        graph.replay()
    status()
    assert torch.equal(call.out.view(torch.int16), want.view(torch.int16))
    q.copy_(q2)
    n.copy_(n2)
    graph.replay()
    status()
    assert torch.equal(call.out.view(torch.int16), want2.view(torch.int16))
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    torch.cuda.synchronize()
    for _ in range(5):
        for s in streams:
            outs.append(vw4.verify_attn(q2, c, n2, stream=s))
    status()
    for o in outs:
        assert torch.equal(o.view(torch.int16), want2.view(torch.int16))
