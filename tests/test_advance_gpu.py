"""advance_pages against the same steps taken one after another on the host: exact."""
import pytest
import torch

import speculative_decode_verification_w4_gb300 as vw4
from step_util import status

pytestmark = pytest.mark.gpu


def reference(t, page, lens, held, free, count, rows_max, R, accepted, ended, grow, pages):
    """The rule, a sequence at a time.  t, free are changed in place."""
    B, cols = len(lens), len(t[0])
    status_bits = 0
    lens = [0 if ended[b] else max(0, lens[b]) + max(0, accepted[b]) for b in range(B)]
    held = [min(max(h, 0), cols) for h in held]
    for b in range(B):
        if ended[b]:
            for p in t[b][:held[b]]:
                if count < pages:
                    free[count] = p
                    count += 1
                else:
                    status_bits |= vw4.DEV_NO_ROOM
            held[b] = 0
    left, start, seq, slots = count, [0], [], []
    taken = 0
    for b in range(B):
        g = max(0, grow[b])
        want = -(-(lens[b] + g) // page)
        need = max(0, want - held[b])
        ok = want <= cols
        if ok and need:
            ok = need <= left
            left -= need  # counted whether or not it fits
        if not ok:
            status_bits |= vw4.DEV_NO_ROOM
            g = 0
        else:
            for _ in range(need):
                t[b][held[b]] = free[count - 1 - taken]
                taken += 1
                held[b] += 1
        seq.append(lens[b] + g if g else 0)
        for j in range(lens[b], lens[b] + g):
            p = t[b][j // page]
            if 0 <= p < pages:
                slots.append(p * page + j % page)
            else:
                slots.append(-1)
                status_bits |= vw4.DEV_BAD_PAGE
        start.append(start[-1] + g)
    if len(slots) > rows_max:
        status_bits |= vw4.DEV_NO_ROOM
    return lens, held, count - taken, seq, start, slots[:rows_max], status_bits


def make(seed, B, page, cols, spare, hi, used=None):
    g = torch.Generator().manual_seed(seed)
    lens = torch.randint(0, hi + 1, (B,), generator=g)
    held = (lens + page - 1) // page
    total = int(held.sum()) + spare
    ids = torch.randperm(total, generator=g).tolist()
    table = torch.full((B, cols), -1, dtype=torch.int32)
    for b in range(B):
        for k in range(int(held[b])):
            table[b, k] = ids.pop()
    free = torch.full((total,), -5, dtype=torch.int32)
    free[:len(ids)] = torch.tensor(ids, dtype=torch.int32)
    return lens.int(), held.int(), table, free, len(ids), total, g


def check(seed, B, page, cols, spare, hi, R=8, accepted=True, ended=0.2, grow=None, rows_max=None,
          in_place=False, break_input=None, shift=0):
    lens, held, table, free, count, total, g = make(seed, B, page, cols, spare, hi)
    acc = torch.randint(0, 3, (B,), generator=g).int() if accepted else torch.zeros(B, dtype=torch.int32)
    end = (torch.rand(B, generator=g) < ended).int()
    gr = torch.full((B,), R).int() if grow is None else torch.randint(0, grow + 1, (B,), generator=g).int()
    if break_input:
        break_input(lens, held, table, acc, gr)
    t, f = table.tolist(), free.tolist()
    rows = rows_max if rows_max is not None else int(gr.clamp(min=0).sum())
    want = reference(t, page, lens.tolist(), held.tolist(), f, count, rows, R, acc.tolist(),
                     end.tolist(), gr.tolist(), total)
    def put(x):  # on the device, `shift` elements behind an allocation's start
        d = torch.empty(x.numel() + shift, dtype=x.dtype, device="cuda")[shift:]
        return d.copy_(x)
    dl, dh, dc = put(lens), put(held), torch.tensor([count], dtype=torch.int32, device="cuda")
    dt, df = table.cuda(), free.cuda()
    kw = dict(lens_out=dl, held_out=dh, free_count_out=dc) if in_place else {}
    slots = torch.full((rows + 7,), -9, dtype=torch.int64, device="cuda")
    p = vw4.advance_pages(dt, page, dl, dh, df, dc, rows, R, accepted=put(acc) if accepted else None,
                          ended=put(end) if ended else None,
                          grow=None if grow is None and not break_input else put(gr), slots=slots, **kw)
    status(want[6])
    assert p.lens.tolist() == want[0]
    assert p.held.tolist() == want[1]
    assert p.free_count.tolist() == [want[2]]
    assert p.seq_lens.tolist() == want[3]
    assert p.row_start.tolist() == want[4]
    n = len(want[5])
    assert slots[:n].tolist() == want[5]
    assert (slots[n:] == -9).all(), "slots behind the last row were written"
    assert dt.tolist() == t
    assert df.tolist() == f
    if not in_place:
        assert dl.tolist() == lens.tolist() and dh.tolist() == held.tolist() and int(dc) == count


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("B,spare", [(4096, 9000), (4097, 50), (9001, 3000), (16384, 30000), (16383, 400)])
def test_many_sequences(B, spare, shift, in_place):
    """One and several groups of sequences a thread, with pages for all of them and for some,
    arrays that lie on 16 bytes or not."""
    check(B, B, 8, 6, spare, 24, 3, grow=9, in_place=in_place, shift=shift)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,page,hi,R", [(1, 16, 100, 1), (1, 8, 0, 9), (5, 16, 60, 8), (33, 64, 500, 3),
                                         (300, 16, 300, 9), (1025, 8, 90, 16), (3000, 32, 200, 1)])
def test_steps(B, page, hi, R, in_place):
    check(B, B, page, (hi + 2 * R + 2) // page + 2, 4 * B + 9, hi, R, in_place=in_place)


@pytest.mark.parametrize("B,page,grow", [(1, 16, 5000), (7, 8, 3000), (200, 16, 400), (1500, 64, 300)])
def test_prompts(B, page, grow):
    """Ragged growth, ended places taken over by new sequences in the same call."""
    check(100 + B, B, page, (200 + grow) // page + 2, B * (grow // page + 2), 190, grow=grow, ended=0.5)


@pytest.mark.parametrize("B", [6, 700])
@pytest.mark.parametrize("spare", [0, 3, 40])
def test_free_list_runs_out(B, spare):
    check(200 + spare, B, 16, 20, spare, 100, R=16, ended=0.0)
    check(201 + spare, B, 16, 20, spare, 100, grow=60, ended=0.1)


def test_table_too_short():
    """The sequence that does not fit gets nothing; those behind it are served."""
    check(300, 40, 16, 8, 200, 100, grow=60)


def test_rows_beyond_the_slots():
    check(301, 20, 16, 20, 100, 100, R=8, rows_max=50)
    check(302, 20, 16, 20, 100, 100, R=8, rows_max=0)


def test_no_optional_inputs():
    check(303, 20, 16, 20, 100, 100, R=8, accepted=False, ended=0.0)


def test_inputs_out_of_range():
    """Negative counts read as 0, page counts beyond the table as the table's; a page id that is
    none gives the slot -1."""
    def spoil(lens, held, table, acc, gr):
        lens[0], acc[1], gr[2] = -5, -3, -1
        held[3] = 99
        lens[5], held[5], acc[5] = 20, 2, 0
        table[5, 1] = 1 << 20
    check(304, 20, 16, 20, 200, 100, ended=0.0, break_input=spoil)
    check(305, 4000, 16, 20, 20000, 100, ended=0.0, break_input=spoil)


def test_more_pages_returned_than_the_list_holds():
    """A page in two rows of the table: what does not fit the free list is dropped."""
    B, page = 4, 16
    table = torch.tensor([[0, 1], [2, 3], [0, 1], [2, 3]], dtype=torch.int32, device="cuda")
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    free = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    p = vw4.advance_pages(table, page, i(0, 0, 0, 0), i(2, 2, 2, 2), free, i(0), ended=i(1, 1, 1, 1),
                          grow=i(0, 0, 0, 0))
    status(vw4.DEV_NO_ROOM)
    assert free.tolist() == [0, 1, 2, 3] and p.free_count.tolist() == [4]


def test_graph_replays():
    """In place, captured: each replay is the next step."""
    B, page, cols, R = 6, 16, 40, 8
    lens, held, table, free, count, total, g = make(7, B, page, cols, 300, 60)
    dl, dh, dt, df = lens.cuda(), held.cuda(), table.cuda(), free.cuda()
    dc = torch.tensor([count], dtype=torch.int32, device="cuda")
    acc = torch.zeros(B, dtype=torch.int32, device="cuda")
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call = vw4.PreparedAdvance(dt, page, dl, dh, df, dc, B * R, R, accepted=acc, lens_out=dl,
                                   held_out=dh, free_count_out=dc)
        with torch.cuda.graph(graph, stream=side):
            call()
    torch.cuda.current_stream().wait_stream(side)
    t, f, ln, hd = table.tolist(), free.tolist(), lens.tolist(), held.tolist()
    for step in range(12):
        kept = [(step + b) % R + 1 if step else 0 for b in range(B)]
        acc.copy_(torch.tensor(kept, dtype=torch.int32))
        graph.replay()
        ln, hd, count, seq, start, slots, bits = reference(t, page, ln, hd, f, count, B * R, R, kept,
                                                           [0] * B, [R] * B, total)
        assert bits == 0
        status()
        assert dl.tolist() == ln and dh.tolist() == hd and dc.tolist() == [count]
        assert dt.tolist() == t and df.tolist() == f
        assert call.seq_lens.tolist() == seq and call.slots.tolist() == slots
