"""Scratch and results of calls on streams of their own: which memory a call gets (host
part, without a GPU), and calls on two streams of one thread against the same calls
made alone."""
import pytest
import torch

import speculative_decode_verification_w4_gb300 as vw4
from step_util import make_cache, status


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


def test_default_workspace_is_one_a_stream():
    cpu, a, b = torch.device("cpu"), Stream(0x70001), Stream(0x70002)
    wa, wb = (vw4._workspace(None, 1000, cpu, s) for s in (a, b))
    assert wa.data_ptr() != wb.data_ptr()
    assert vw4._workspace(None, 500, cpu, a).data_ptr() == wa.data_ptr()
    assert vw4._workspace(None, 4000, cpu, a).numel() >= 4000
    assert vw4._workspace(None, 1000, cpu, b).data_ptr() == wb.data_ptr()


def test_workspace_is_not_filled(monkeypatch):
    """A fill would be queued on the current stream, not on the call's."""
    def fill(*a, **kw):
        raise AssertionError("a workspace was filled")
    monkeypatch.setattr(torch, "zeros", fill)
    assert vw4.Workspace("cpu").get(1000).numel() >= 1000


def attn_inputs(seed, lens, R=8, G=6, Hkv=2, D=128):
    c, _, _ = make_cache(seed, lens, 32, Hkv, D, "bf16")
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(len(lens), R, Hkv * G, D, generator=g).to(torch.bfloat16).cuda()
    return q, c, torch.tensor(lens, dtype=torch.int32, device="cuda")


@pytest.mark.gpu
def test_two_streams_of_one_thread():
    """Calls that overlap, on the default workspace: the bits of the calls alone."""
    cases = [attn_inputs(1, [9000, 77, 5001]), attn_inputs(2, [300 + 70 * b for b in range(40)]),
             attn_inputs(3, [20000])]
    alone = [vw4.verify_attn(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    outs = [torch.empty_like(a) for a in alone]
    for _ in range(50):
        for c, s, o in zip(cases, streams, outs):
            vw4.verify_attn(*c, out=o, stream=s)
    status()
    for a, o in zip(alone, outs):
        assert torch.equal(a.view(torch.int16), o.view(torch.int16))


@pytest.mark.gpu
def test_workspace_made_while_the_current_stream_is_busy():
    """What is queued on the current stream when a call on another one is made does not
    reach the call's workspace."""
    case = attn_inputs(4, [9000, 77, 5001])
    alone = vw4.verify_attn(*case)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        out = torch.empty_like(alone)
        torch.cuda._sleep(2_000_000)  # about a millisecond
        call = vw4.PreparedAttn(*case, out=out, stream=s)
        for _ in range(60):
            call()
        status()
        assert torch.equal(alone.view(torch.int16), out.view(torch.int16))


@pytest.mark.gpu
@pytest.mark.parametrize("call", ["attention", "append", "logits"])
def test_results_made_while_the_current_stream_is_busy(call):
    """A result is not made of memory that the current stream still has to write to."""
    B, R, Hq, Hkv, D, V = 3, 8, 12, 2, 128, 50001
    q, c, n = attn_inputs(4, [9000, 77, 5001])
    x = torch.randn(B * R, (Hq + 2 * Hkv) * D, device="cuda")
    logits = torch.randn(B, 1, V, device="cuda")
    run = {"attention": lambda **kw: vw4.verify_attn(q, c, n, **kw),
           "append": lambda **kw: vw4.verify_rope_append(x, c, n, R, Hq, **kw),
           "logits": lambda **kw: vw4.process_logits(logits, **kw)}[call]
    alone = run()
    s = torch.cuda.Stream()
    run(stream=s)  # (its workspace is there)
    status()
    for _ in range(3):
        old = torch.empty_like(alone)
        torch.cuda._sleep(20_000_000)  # about ten milliseconds
        old.fill_(7.0)
        del old
        out = run(stream=s)
        status()
        assert torch.equal(alone.view(torch.int16), out.view(torch.int16))
