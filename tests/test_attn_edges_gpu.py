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
