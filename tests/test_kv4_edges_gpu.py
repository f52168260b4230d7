"""Calls of the 4-bit cache, the pages and the log probabilities that lie at the ends of what
they allow: several streams at once, captured and replayed, empty batches, shared pages,
strides, offsets beyond 32 bits, the widest and the most rows."""
import math

import pytest
import torch

import speculative_decode_verification_w4_gb300 as vw4
from kv4_util import make_cache4
from step_util import status

pytestmark = pytest.mark.gpu
KINDS = [(64, 16, 4), (128, 1, 4), (128, 8, 6), (256, 4, 3), (256, 8, 6), (256, 16, 8)]


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def bits(t):
    return t.view(torch.int16 if t.element_size() == 2 else torch.int32)


def queries(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * 2).to(torch.bfloat16).cuda()


def test_all_kinds_on_three_streams():
    """Every kernel of the attention, the read-back, the pages and the log probabilities at
    once on three streams: the bits of the calls alone, and no wait ran out."""
    calls = []
    for k, (D, R, G) in enumerate(KINDS):
        lens = [1 + (997 * b * (k + 1)) % 3000 for b in range(9)]
        c, _, _ = make_cache4(k, lens, 16, 2, D)
        q, n = queries(k, 9, R, 2 * G, D), ints(lens)
        calls.append(lambda s, c=c, q=q, n=n: [vw4.verify_attn(q, c, n, window=700, sinks=3, stream=s)])
        calls.append(lambda s, c=c, n=n: list(vw4.read_kv4(c, n, 65, stream=s)))
    x = torch.randn(30, 4, 40001, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    tok = torch.arange(120, dtype=torch.int32, device="cuda").view(30, 4) * 300
    calls.append(lambda s: list(vw4.token_logprobs(x, tok, top=7, stream=s)))

    def pages(s):
        with torch.cuda.stream(s):
            table, free = torch.full((5000, 8), -1, dtype=torch.int32, device="cuda"), torch.arange(40000, device="cuda").int()
            zero = torch.zeros(5000, dtype=torch.int32, device="cuda")
            grow = torch.arange(5000, device="cuda").int() % 60
            count = torch.full((1,), 40000, dtype=torch.int32, device="cuda")
        p = vw4.advance_pages(table, 16, zero, zero, free, count, rows_max=200000, grow=grow, stream=s)
        return [table, p.held, p.row_start, p.free_count]
    calls.append(pages)
    main = torch.cuda.current_stream()
    alone = []
    for f in calls:
        alone.append([t.clone() for t in f(main)])
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for turn in range(6):
        for k in range(len(calls)):
            f = (k + turn) % len(calls)
            outs.append((f, calls[f](streams[(k * 7 + turn) % 3])))
    status()
    for f, got in outs:
        for a, b in zip(alone[f], got):
            if a.is_floating_point():
                a, b = bits(a), bits(b)
            assert torch.equal(a, b), f


@pytest.mark.parametrize("D,R,G", KINDS)
def test_two_graphs_of_one_workspace(D, R, G):
    """Two captured calls over one workspace, replayed in turn on one stream with lengths that
    change between them, down to none at all."""
    lens = [900, 17, 2500, 64]
    c, _, _ = make_cache4(9, lens, 32, 2, D)
    ws = vw4.Workspace(torch.device("cuda", torch.cuda.current_device()))
    n = [ints(lens), ints(lens)]
    q = [queries(k, 4, R, 2 * G, D) for k in range(2)]
    calls = [vw4.PreparedAttn(q[k], c, n[k], workspace=ws) for k in range(2)]
    for call in calls:
        call()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    prepared = []
    with torch.cuda.stream(side):
        for k in range(2):
            call = vw4.PreparedAttn(q[k], c, n[k], workspace=ws)
            with torch.cuda.graph(graphs[k], stream=side):
                call()
            prepared.append(call)
    torch.cuda.synchronize()
    for cut in ([900, 17, 2500, 64], [0, 0, 0, 0], [5, 0, 1, 33], [899, 16, 64, 0]):
        for k in range(2):
            n[k].copy_(ints([v - k if v else 0 for v in cut]))
        for _ in range(2):
            for g in graphs:
                g.replay()
        status()
        for k in range(2):
            want = vw4.verify_attn(q[k], c, n[k])
            status()
            assert torch.equal(bits(prepared[k].out), bits(want))
            for b, v in enumerate(n[k].tolist()):
                if v == 0:
                    assert (want[b] == 0).all()


@pytest.mark.parametrize("D,R,G", KINDS)
def test_shared_pages_and_strides(D, R, G):
    """A sequence's pages twice in a batch give the same rows twice, whatever lies between;
    queries and outputs as slices of wider tensors."""
    lens = [700, 300]
    c, _, _ = make_cache4(3, lens, 16, 2, D)
    table = c.block_table[[0, 1, 0, 0, 1]].contiguous()
    c2 = vw4.KVCache4(c.k, c.v, c.k_blocks, c.v_blocks, table, c.k_scale, c.v_scale)
    Hq = 2 * G
    wide = queries(5, 5, R, Hq + 3, D)
    wide[2:4], wide[4] = wide[0], wide[1]
    q = wide[:, :, :Hq]
    room = torch.full((5, R, Hq + 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(5, R, Hq, device="cuda")
    out = vw4.verify_attn(q, c2, ints([700, 300, 700, 700, 300]), out=room[:, :, :Hq], lse=lse)
    status()
    alone = vw4.verify_attn(q[:2].contiguous(), c, ints(lens))
    status()
    for b, a in enumerate([0, 1, 0, 0, 1]):
        # (where an item is cut into parts depends on the batch: a rounding of the sums)
        assert (out[b].float() - alone[a].float()).abs().max() <= 2.0 ** -7 * alone[a].float().abs().max()
        assert torch.equal(lse[b] > 0, lse[a] > 0)
    assert (room[:, :, Hq:] == 7).all(), "beyond the heads"


@pytest.mark.parametrize("D,R,G", [(64, 1, 2), (128, 3, 4), (256, 1, 3), (64, 4, 12), (128, 5, 8)])
def test_four_million_tokens(D, R, G):
    """A table that names 16 pages over and over: the rows of 2^22 tokens see each of them
    equally often, so the outputs are those of one round, and the log-sum-exp is larger by the
    logarithm of the rounds.  Only the verify rows' own ends differ: R - 1 of 2^22 tokens."""
    page, rounds = 64, 4096
    lens = [16 * page]
    c, _, _ = make_cache4(21, lens, page, 1, D)
    q = queries(8, 1, R, G, D) * 0.25
    # one round as each row sees it: the cache cut at the row's own position
    long = vw4.KVCache4(c.k, c.v, c.k_blocks, c.v_blocks, c.block_table[:, :16].repeat(1, rounds).contiguous(),
                        c.k_scale, c.v_scale)
    n = 16 * page * rounds
    lse = torch.empty(1, R, G, device="cuda")
    out = vw4.verify_attn(q, long, ints([n + 0]), lse=lse)
    status()
    one, one_lse = torch.empty_like(out), torch.empty_like(lse)
    for i in range(R):
        one_row = torch.empty(1, 1, G, device="cuda")
        one[:, i] = vw4.verify_attn(q[:, i:i + 1].contiguous(), c, ints(lens), lse=one_row)[:, 0]
        one_lse[:, i] = one_row[:, 0]
    status()
    # two bf16 roundings, f16 weights, R - 1 missing tokens of weight at most 2^10 times a mean's
    tol = 2 * 2.0 ** -9 + 2 * 2.0 ** -11 + 2.0 ** -10 + R * 2.0 ** -12
    assert (out.double() - one.double()).abs().max() <= tol * one.double().abs().max()
    assert (lse.double() - one_lse.double() - math.log(rounds)).abs().max() <= 2.0 ** -11


def test_offsets_beyond_32_bits():
    """A cache of 5 GB of codes: rows appended, read back and attended in its last pages, as in a
    small one."""
    D, Hkv, page, Hq, R = 256, 8, 64, 16, 4
    pages = 5 * 2 ** 30 // (page * Hkv * D // 2)
    lens = [70, 3, 128]
    cols = 2
    g = torch.Generator().manual_seed(4)
    rows = (torch.randn(3 * R, (Hq + 2 * Hkv) * D, generator=g)).cuda()
    inv = 1e4 ** (-torch.arange(0, 64, 2, dtype=torch.float64, device="cuda") / 64)

    def run(n_pages, ids):
        k, v = (torch.zeros(n_pages, page, Hkv, D // 2, dtype=torch.uint8, device="cuda") for _ in range(2))
        kb, vb = (torch.zeros(n_pages, Hkv, page, D // 16, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
                  for _ in range(2))
        c = vw4.KVCache4(k, v, kb, vb, ints(ids).view(3, cols))
        n = ints(lens)
        q = vw4.verify_rope_append(rows, c, n, R, Hq, inv_freq=inv)
        out = vw4.verify_attn(q, c, n)
        more = vw4.verify_attn(q.repeat(1, 1, 4, 1).contiguous(), c, n)  # (32 rows a key head: 8 x 4)
        back = vw4.read_kv4(c, n, 9)
        status()
        return [q, out, more, *back]
    small = run(6, [5, 2, 0, 1, 3, 4])
    large = run(pages, [pages - 1, 7, pages - 2, pages - 3, pages // 2, pages - 5])
    for a, b in zip(small, large):
        assert torch.equal(bits(a), bits(b))


@pytest.mark.parametrize("bf16", [False, True])
def test_widest_row(bf16):
    """2^24 entries: the sum in 64 bits within its fp32 additions, ids exactly."""
    V = 2 ** 24
    g = torch.Generator("cuda").manual_seed(6)
    x = torch.randn(1, 1, V, device="cuda", generator=g)
    if bf16:
        x = x.to(torch.bfloat16)
    t = V - 3
    r = vw4.token_logprobs(x, ints([[t]]), top=32)
    status()
    row = x[0, 0].double()
    lse = torch.logsumexp(row, 0)
    # chunks of a part (64) and its threads, 64 parts: (16 + 64 + 13 + 64) 2^-24, each term 2^-22
    tol = 2.0 ** -16
    assert abs(r.lse.item() - lse.item()) <= tol + lse.item() * 2.0 ** -23
    assert abs(r.logprob.item() - (row[t] - lse).item()) <= tol + 20 * 2.0 ** -22
    order = torch.sort(-row, stable=True).indices[:32]
    assert torch.equal(r.top_ids[0, 0].long(), order)
    before = (row > row[t]).sum() + (row[:t] == row[t]).sum()
    assert r.rank.item() == before.item() + 1


def test_most_rows():
    """262144 rows of 5 entries, more alternatives asked for than there are."""
    x = torch.randn(16384, 16, 5, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    tok = torch.randint(0, 5, (16384, 16), device="cuda", dtype=torch.int32)
    r = vw4.token_logprobs(x, tok, top=8)
    status()
    want = torch.log_softmax(x.double(), -1)
    got = want.gather(-1, tok.long()[..., None])[..., 0]
    assert (r.logprob.double() - got).abs().max() <= 2.0 ** -17
    assert torch.equal(r.top_ids[..., :5].long(), torch.sort(-x, dim=-1, stable=True).indices)
    assert (r.top_ids[..., 5:] == -1).all() and torch.isneginf(r.top_logprobs[..., 5:]).all()


def test_slowly_rising_rows():
    """Rows whose entries rise by less than a thread's reference lags, chunk after chunk, and
    by more: the sums stay those of 64 bits."""
    for step in (0.0007, 0.002, 0.03):
        V = 60000
        x = (torch.arange(V, dtype=torch.float64) * step).float().view(1, 1, V)
        for y in (x, -x, x - 30000 * step):
            r = vw4.token_logprobs(y.cuda(), ints([[V - 1]]), top=3)
            status()
            row = y[0, 0].double()
            lse = torch.logsumexp(row, 0).item()
            p = torch.softmax(row, 0)
            big = float(row.abs().max())
            tol = 2.0 ** -18 + 2.0 ** -22 * big + abs(lse) * 2.0 ** -23
            assert abs(r.lse.item() - lse) <= tol
            h = -(p * torch.log_softmax(row, 0)).sum().item()
            assert abs(r.entropy.item() - h) <= 60 * tol


def test_pages_shared_by_sequences_return_twice():
    """Two ended sequences that name the same pages give them back twice: what the table says;
    more than the list holds is refused with the status."""
    table = ints([[4, 5, -1], [4, 5, 6]])
    free = ints([0, 1, 2, 9, 9, 9, 9, 9])
    p = vw4.advance_pages(table, 8, ints([10, 20]), ints([2, 3]), free, ints([3]), R=1, ended=ints([1, 1]))
    status()
    assert p.lens.tolist() == [0, 0] and p.held.tolist() == [1, 1]
    assert free[:8].tolist() == [0, 1, 2, 4, 5, 4, 5, 6] and p.free_count.tolist() == [6]
    assert table[:, 0].tolist() == [6, 5]
