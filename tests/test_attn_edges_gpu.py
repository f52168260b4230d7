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
