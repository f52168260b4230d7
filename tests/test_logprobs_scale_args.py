"""token_logprobs' range of scales, at the C ABI (fake device addresses, no launch)."""
import ctypes

import pytest

import speculative_decode_verification_w4_gb300 as vw4
from speculative_decode_verification_w4_gb300 import build as vbuild


@pytest.mark.parametrize("scale", [2.0 ** 126 * (1 + 2.0 ** -23), 2.0 ** 127, 3.4e38])
def test_scales_whose_base_2_form_overflows(scale):
    vbuild.build()
    lib = vw4.load_library()
    a = vw4.LogprobsArgs(x_dev=0x1000, tokens_dev=0x2000, logprob_dev=0x3000, ldx=100, B=2, R=3, V=100,
                         scale=scale)
    assert lib.token_logprobs(ctypes.byref(a), 0x100000, 1 << 20, None) == 1
