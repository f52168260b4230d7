"""verify_rope_append: scales of zero and below."""
import pytest
import torch

import speculative_decode_verification_w4_gb300 as vw4
from step_util import make_cache, status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128, 256])
def test_scales_of_any_sign(D):
    """value / scale for a negative scale; zeros for a head of scale 0, whose every byte
    reads back as 0 unless it is NaN."""
    lens, Hkv, R = [40, 7], 3, 4
    c, _, _ = make_cache(11, lens, 16, Hkv, D, "e4m3")
    c.k_scale.copy_(torch.tensor([0.0, -0.5, 0.5]))
    c.v_scale.copy_(torch.tensor([-0.25, 0.25, 0.0]))
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    x = torch.randn(len(lens) * R, 3 * Hkv * D, device="cuda")
    x[0] = 0.0
    vw4.verify_rope_append(x, c, n, R, Hkv)
    status()
    rows = x.view(len(lens) * R, 3 * Hkv, D)
    for r in range(len(lens) * R):
        b, p = r // R, lens[r // R] - R + r % R
        pg = int(c.block_table[b, p // 16])
        k, v = (t[pg, p % 16].float() for t in (c.k, c.v))
        assert (k[0] == 0).all() and (v[2] == 0).all()
        # a power of two scales exactly, so the bytes are those of the rounded quotient
        assert torch.equal(k[1], (rows[r, 4] / -0.5).to(torch.float8_e4m3fn).float())
        assert torch.equal(k[2], (rows[r, 5] / 0.5).to(torch.float8_e4m3fn).float())
        assert torch.equal(v[0], (rows[r, 6] / -0.25).to(torch.float8_e4m3fn).float())
        assert torch.equal(v[1], (rows[r, 7] / 0.25).to(torch.float8_e4m3fn).float())
