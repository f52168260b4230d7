"""What the Python binding of the calls between the verify GEMMs refuses before it looks at
the device (host tensors: a later check would refuse those too, with another message)."""
import ctypes

import pytest
import torch

import speculative_decode_verification_w4_gb300 as vw4


def pages():
    return torch.zeros(10, 16, 2, 64, dtype=torch.bfloat16)


@pytest.mark.parametrize("table", [
    torch.zeros(1, 4, dtype=torch.int32).expand(3, 4),
    torch.zeros(64, dtype=torch.int32).as_strided((3, 4), (2, 1)),
])
def test_block_table_of_overlapping_rows(table):
    """Its rows are not max_blocks apart, and the descriptor's stride is at least that: the
    kernels would read past them."""
    with pytest.raises(ValueError, match="overlap"):
        vw4.KVCache(pages(), pages(), table)


@pytest.mark.parametrize("table", [
    torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, 9, dtype=torch.int32)[:, :4],
    torch.zeros(4, dtype=torch.int32).as_strided((1, 4), (0, 1)),
    torch.zeros(3, 1, dtype=torch.int32),
])
def test_block_table_rows_that_are_taken(table):
    with pytest.raises(ValueError, match="CUDA"):
        vw4.KVCache(pages(), pages(), table)


def test_workspace_tensors():
    """A tensor as a workspace: on the call's device, without gaps, counted in bytes
    (the calls hand its address and size on as they are)."""
    gpu, cpu = torch.device("cuda", 0), torch.device("cpu")
    with pytest.raises(ValueError, match="cuda:0"):
        vw4._workspace(torch.empty(4096, dtype=torch.uint8), 4096, gpu, None)
    with pytest.raises(ValueError, match="contiguous"):
        vw4._workspace(torch.empty(8192, dtype=torch.uint8)[::2], 4096, cpu, None)
    with pytest.raises(vw4.VW4Error):
        vw4._workspace(torch.empty(1023), 4096, cpu, None)
    ws = torch.empty(32, 32)
    got = vw4._workspace(ws, 4096, cpu, None)
    assert got.data_ptr() == ws.data_ptr() and got.numel() == 4096


def test_output_rows_too_far_apart():
    """verify_attn addresses a sequence's output rows by 32-bit offsets in 16 bytes."""
    from speculative_decode_verification_w4_gb300 import build
    build.build()
    kv = vw4.KVDesc(vw4.KV_BF16, 16, 10, 2, 128, 4, 16 * 256, 256, 128, 4, 0x10000, 0x20000,
                    0x30000, None, None)

    def call(ldo):  # (a workspace of one byte is refused next)
        a = vw4.AttnArgs(kv, 0x1000, 0x2000, None, 0x3000, 1024, ldo, 2, 3, 8, 0, 0, 0.1)
        return vw4.load_library().verify_attn(ctypes.byref(a), 0x100000, 1, None)
    assert call(1024) == 6 and call(1 << 31) == 6
    assert call((1 << 31) + 8) == 1
