"""Default scratch of calls that are captured into graphs: the graph's own, not the buffer that
later calls replace (host part, without a GPU), and graphs replayed after larger calls."""
import pytest
import torch

import speculative_decode_verification_w4_gb300 as vw4
from kv4_util import make_cache4
from step_util import status


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


def test_captured_calls_leave_the_default_workspace_alone(monkeypatch):
    cpu, s = torch.device("cpu"), Stream(0x70011)
    cached = vw4._workspace(None, 1000, cpu, s)
    before = dict(vw4._default_ws)
    monkeypatch.setattr(vw4, "_capturing", lambda device, stream: True)
    a = vw4._workspace(None, 500, cpu, s)
    b = vw4._workspace(None, 5000, cpu, s)
    assert a.numel() >= 500 and b.numel() >= 5000
    assert len({a.data_ptr(), b.data_ptr(), cached.data_ptr()}) == 3
    assert vw4._default_ws == before
    ws = vw4.Workspace("cpu")
    assert vw4._workspace(ws, 700, cpu, s).data_ptr() == ws.buf.data_ptr()
    monkeypatch.undo()
    assert vw4._workspace(None, 1000, cpu, s).data_ptr() == cached.data_ptr()


@pytest.mark.gpu
@pytest.mark.parametrize("D,R,G", [(128, 1, 4), (128, 8, 6), (256, 16, 8)])
def test_graphs_outlive_larger_calls(D, R, G):
    """A small call's graph, then a larger call's on the same stream, then eager ones; the cache
    of the allocator is emptied between.  Replays give the bits of the calls alone."""
    def inputs(seed, lens, Hkv):
        c, _, _ = make_cache4(seed, lens, 16, Hkv, D)
        g = torch.Generator().manual_seed(seed)
        q = torch.randn(len(lens), R, Hkv * G, D, generator=g).to(torch.bfloat16).cuda()
        return q, c, torch.tensor(lens, dtype=torch.int32, device="cuda")
    small, large = inputs(1, [900, 3], 1), inputs(2, [2000 + 300 * b for b in range(12)], 4)
    x = torch.randn(40, 4, 30000, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    want = [vw4.verify_attn(*small), vw4.verify_attn(*large), vw4.token_logprobs(x, top=9).lse]
    torch.cuda.synchronize()
    kept, graphs, outs = dict(vw4._default_ws), [], []
    for f in (lambda: vw4.verify_attn(*small), lambda: vw4.verify_attn(*large),
              lambda: vw4.token_logprobs(x, top=9).lse):
        torch.cuda.empty_cache()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(f())
        graphs.append(graph)
    assert vw4._default_ws == kept
    for _ in range(3):
        torch.cuda.empty_cache()
        for g in graphs:
            g.replay()
        vw4.verify_attn(*large)
        status()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_captured_on_another_stream_than_the_current():
    """A call whose stream is captured while another one is current, and the other way round."""
    c, _, _ = make_cache4(3, [300], 16, 1, 128)
    q = torch.randn(1, 2, 4, 128, device="cuda").to(torch.bfloat16)
    n = torch.tensor([300], dtype=torch.int32, device="cuda")
    want = vw4.verify_attn(q, c, n)
    side, current = torch.cuda.Stream(), torch.cuda.current_stream()
    torch.cuda.synchronize()
    assert not vw4._capturing(q.device, None) and not vw4._capturing(q.device, side)
    kept, graph = dict(vw4._default_ws), torch.cuda.CUDAGraph()
    out = torch.empty_like(want)
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        assert vw4._capturing(q.device, None) and vw4._capturing(q.device, main)
        assert not vw4._capturing(q.device, side)
        side.wait_stream(main)
        assert vw4._capturing(q.device, side) and torch.cuda.current_stream() == main
        vw4.verify_attn(q, c, n, out=out, stream=side)
        main.wait_stream(side)
    assert vw4._default_ws == kept and torch.cuda.current_stream() == current
    graph.replay()
    status()
    assert torch.equal(out, want)
