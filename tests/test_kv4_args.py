"""Refusals of the 4-bit cache's entry points, of advance_pages and token_logprobs, on the
host: at the C ABI (fake device addresses, no launch) and in the binding (host tensors)."""
import ctypes
import math

import pytest
import torch

import speculative_decode_verification_w4_gb300 as vw4
from speculative_decode_verification_w4_gb300 import build as vbuild


@pytest.fixture(scope="module")
def lib():
    vbuild.build()
    return vw4.load_library()


CACHE = dict(page_size=16, num_pages=10, Hkv=2, D=128, max_blocks=4, reserved=0,
             page_stride=16 * 128, token_stride=128, head_stride=64, blocks_page_stride=256,
             blocks_head_stride=128, table_stride=4, k_dev=0x10000, v_dev=0x20000,
             k_blocks_dev=0x30000, v_blocks_dev=0x40000, block_table_dev=0x50000,
             k_scale_dev=None, v_scale_dev=None)


def fields(cls, d, kw):
    names = {f[0] for f in cls._fields_}
    d = dict(d)
    if "kv" in names:
        d["kv"] = vw4.KV4Desc(**dict(CACHE, **{k: v for k, v in kw.items() if k in CACHE}))
    d.update({k: v for k, v in kw.items() if k in names})
    return cls(**d)


BAD_CACHE = [
    (dict(k_dev=None), 1), (dict(v_dev=None), 1), (dict(k_blocks_dev=None), 1),
    (dict(v_blocks_dev=None), 1), (dict(block_table_dev=None), 1), (dict(reserved=1), 1),
    (dict(num_pages=0), 1), (dict(max_blocks=0), 1), (dict(table_stride=3), 1), (dict(Hkv=0), 1),
    (dict(Hkv=257), 1), (dict(page_size=0), 1), (dict(page_size=12), 2), (dict(page_size=4), 2),
    (dict(page_size=1 << 17), 2), (dict(D=96), 2), (dict(D=32), 2), (dict(page_stride=-16), 1),
    (dict(page_stride=0), 1), (dict(token_stride=0), 1), (dict(head_stride=0), 1),
    (dict(blocks_page_stride=0), 1), (dict(blocks_head_stride=0), 1), (dict(blocks_head_stride=-16), 1),
    (dict(page_size=65536, max_blocks=1 << 20, table_stride=1 << 20), 1),
    (dict(k_dev=0x10008), 3), (dict(v_blocks_dev=0x40004), 3), (dict(token_stride=136), 3),
    (dict(page_stride=2052), 3), (dict(head_stride=72), 3), (dict(blocks_page_stride=264), 3),
    (dict(blocks_head_stride=136), 3), (dict(block_table_dev=0x50002), 3),
    (dict(k_scale_dev=0x102), 3), (dict(v_scale_dev=0x101), 3), (dict(B=0), 1), (dict(B=20000), 1),
]
BAD_ROWS = [(dict(R=0), 1), (dict(R=17), 1), (dict(Hq=7), 1), (dict(Hq=0), 1), (dict(Hq=258), 1),
            (dict(Hkv=3), 1)]


@pytest.mark.parametrize("kw,code", BAD_CACHE + BAD_ROWS + [
    (dict(q_dev=None), 1), (dict(out_dev=None), 1), (dict(seq_lens_dev=None), 1),
    (dict(ldq=1000), 1), (dict(ldo=1000), 1), (dict(ldo=1 << 32), 1), (dict(window=-1), 1),
    (dict(sinks=-1), 1), (dict(sinks=4), 1), (dict(scale=0.0), 1), (dict(scale=math.nan), 1),
    (dict(scale=math.inf), 1), (dict(scale=-1.0), 1), (dict(q_dev=0x1008), 3),
    (dict(out_dev=0x1002), 3), (dict(lse_dev=0x1002), 3), (dict(ldq=1028), 3), (dict(ldo=1028), 3),
    (dict(ws=None), 6), (dict(ws_bytes=1000), 6), (dict(ws=0x1010), 3),
])
def test_attention(lib, kw, code):
    a = fields(vw4.AttnKV4Args, dict(q_dev=0x1000, out_dev=0x2000, lse_dev=None, seq_lens_dev=0x3000,
                                     ldq=1024, ldo=1024, B=2, R=3, Hq=8, window=0, sinks=0,
                                     scale=0.1), kw)
    assert lib.verify_attn_kv4(ctypes.byref(a), kw.get("ws", 0x100000),
                               kw.get("ws_bytes", 1 << 30), None) == code
    assert lib.verify_attn_kv4(None, 0x100000, 1 << 30, None) == 1


@pytest.mark.parametrize("kw,code", BAD_CACHE + BAD_ROWS + [
    (dict(x_dev=None), 1), (dict(q_dev=None), 1), (dict(seq_lens_dev=None), 1),
    (dict(inv_freq_dev=None), 1), (dict(rot=130), 1), (dict(rot=63), 1), (dict(rot=-2), 1),
    (dict(adjacent=2), 1), (dict(x_bf16=2), 1), (dict(eps=-1.0), 1), (dict(eps=math.nan), 1),
    (dict(ldx=1528), 1), (dict(ldq=1016), 1), (dict(x_dev=0x1004), 3), (dict(q_dev=0x2004), 3),
    (dict(q_norm_dev=0x2004), 3), (dict(k_norm_dev=0x2004), 3), (dict(inv_freq_dev=0x2004), 3),
    (dict(ldx=1538), 3), (dict(x_bf16=1, ldx=1540), 3), (dict(ldq=1028), 3),
])
def test_append(lib, kw, code):
    a = fields(vw4.AppendKV4Args, dict(x_dev=0x1000, inv_freq_dev=0x4000, q_norm_dev=None,
                                       k_norm_dev=None, q_dev=0x2000, seq_lens_dev=0x3000, ldx=1536,
                                       ldq=1024, x_bf16=0, B=2, R=3, Hq=8, rot=128, adjacent=0,
                                       eps=1e-6), kw)
    assert lib.verify_rope_append_kv4(ctypes.byref(a), None) == code
    assert lib.verify_rope_append_kv4(None, None) == 1


@pytest.mark.parametrize("kw,code", BAD_CACHE + [
    (dict(seq_lens_dev=None), 1), (dict(k_out_dev=None), 1), (dict(v_out_dev=None), 1),
    (dict(n=0), 1), (dict(n=(1 << 24) + 1), 1), (dict(out_f32=2), 1), (dict(k_out_dev=0x1008), 3),
    (dict(v_out_dev=0x1004), 3), (dict(first_dev=0x1002), 3), (dict(seq_lens_dev=0x1001), 3),
])
def test_read(lib, kw, code):
    a = fields(vw4.ReadKV4Args, dict(seq_lens_dev=0x1000, first_dev=None, k_out_dev=0x2000,
                                     v_out_dev=0x3000, B=2, n=5, out_f32=0), kw)
    assert lib.read_kv4(ctypes.byref(a), None) == code
    assert lib.read_kv4(None, None) == 1


ADVANCE = dict(block_table_dev=0x1000, lens_dev=0x2000, accepted_dev=None, ended_dev=None,
               grow_dev=None, held_dev=0x3000, free_dev=0x4000, free_count_dev=0x5000,
               lens_out_dev=0x6000, held_out_dev=0x7000, free_count_out_dev=0x8000,
               seq_lens_dev=0x9000, row_start_dev=0xa000, slots_dev=0xb000, table_stride=10,
               rows_max=100, B=4, R=8, page_size=16, num_pages=50, max_blocks=10)


@pytest.mark.parametrize("kw,code", [
    *[({k: None}, 1) for k, v in ADVANCE.items() if k.endswith("_dev") and v and k != "slots_dev"],
    (dict(B=0), 1), (dict(B=16385), 1), (dict(R=-1), 1), (dict(R=1 << 21), 1), (dict(num_pages=0), 1),
    (dict(max_blocks=0), 1), (dict(table_stride=9), 1), (dict(page_size=0), 1), (dict(page_size=24), 2),
    (dict(page_size=1 << 17), 2), (dict(rows_max=-1), 1), (dict(rows_max=1 << 31), 1),
    (dict(page_size=65536, max_blocks=1 << 20, table_stride=1 << 20), 1),
    (dict(lens_dev=0x2002), 3), (dict(accepted_dev=0x2001), 3), (dict(slots_dev=0xb004), 3),
    (dict(ws=None), 6), (dict(ws_bytes=8), 6), (dict(ws=0x1010), 3),
])
def test_advance(lib, kw, code):
    a = fields(vw4.AdvanceArgs, ADVANCE, kw)
    assert lib.advance_pages(ctypes.byref(a), kw.get("ws", 0x100000), kw.get("ws_bytes", 1 << 20),
                             None) == code
    assert lib.advance_pages(None, 0x100000, 1 << 20, None) == 1


@pytest.mark.parametrize("kw,code", [
    (dict(x_dev=None), 1), (dict(B=0), 1), (dict(B=16385), 1), (dict(R=0), 1), (dict(R=17), 1),
    (dict(V=0), 1), (dict(V=(1 << 24) + 1, ldx=1 << 25), 1), (dict(ldx=99), 1), (dict(top=-1), 1),
    (dict(top=33), 1), (dict(top=0), 1), (dict(x_bf16=2), 1), (dict(scale=0.0), 1),
    (dict(scale=math.inf), 1), (dict(scale=math.nan), 1), (dict(tokens_dev=None), 1),
    (dict(top_ids_dev=None), 1), (dict(top_logprobs_dev=None), 1), (dict(x_dev=0x1002), 3),
    (dict(x_dev=0x1001, x_bf16=1), 3), (dict(lse_dev=0x1002), 3), (dict(len_dev=0x1002), 3),
    (dict(ws=None), 6), (dict(ws_bytes=8), 6), (dict(ws=0x1010), 3),
])
def test_logprobs(lib, kw, code):
    a = fields(vw4.LogprobsArgs, dict(x_dev=0x1000, tokens_dev=0x2000, len_dev=None, logprob_dev=0x3000,
                                      lse_dev=0x4000, entropy_dev=0x5000, rank_dev=0x6000,
                                      top_ids_dev=0x7000, top_logprobs_dev=0x8000, ldx=100, B=2, R=3,
                                      V=100, top=5, x_bf16=0, scale=1.0), kw)
    assert lib.token_logprobs(ctypes.byref(a), kw.get("ws", 0x100000), kw.get("ws_bytes", 1 << 20),
                              None) == code
    assert lib.token_logprobs(None, 0x100000, 1 << 20, None) == 1


def test_workspace_sizes(lib):
    size = vw4.vw4_workspace_bytes
    for D in (64, 128, 256):
        assert 0 < size(vw4.OP_ATTN_KV4, 1, 1, D) <= size(vw4.OP_ATTN_KV4, 1, 64, D)
        # a key head with more rows is cut into blocks: no more room
        assert size(vw4.OP_ATTN_KV4, 1, 128, D) == size(vw4.OP_ATTN_KV4, 1, 4096, D)
    assert size(vw4.OP_ATTN_KV4, 1, 0, 64) == size(vw4.OP_ATTN_KV4, 1, 1, 96) == 0
    assert size(vw4.OP_ADVANCE, 16384, 0, 0) >= 2 * 8 * 16385
    assert size(vw4.OP_ADVANCE, 0, 0, 0) == size(vw4.OP_ADVANCE, 16385, 0, 0) == 0
    assert size(vw4.OP_LOGPROBS, 8, 262144, 20) > 8 * 20 * 8
    assert size(vw4.OP_LOGPROBS, 8, 262144, 33) == size(vw4.OP_LOGPROBS, 0, 10, 1) == 0


def cache_tensors(**kw):
    d = dict(k=torch.zeros(10, 16, 2, 32, dtype=torch.uint8), v=torch.zeros(10, 16, 2, 32, dtype=torch.uint8),
             k_blocks=torch.zeros(10, 2, 16, 4).to(torch.float8_e4m3fn),
             v_blocks=torch.zeros(10, 2, 16, 4).to(torch.float8_e4m3fn),
             block_table=torch.zeros(3, 4, dtype=torch.int32), k_scale=None, v_scale=None)
    d.update(kw)
    return d


@pytest.mark.parametrize("kw,match", [
    (dict(k=torch.zeros(10, 16, 2, 32)), "uint8"),
    (dict(v=torch.zeros(10, 16, 2, 16, dtype=torch.uint8)), "equal strides"),
    (dict(v=torch.zeros(10, 2, 16, 32, dtype=torch.uint8).transpose(1, 2)), "equal strides"),
    (dict(k_blocks=torch.zeros(10, 2, 16, 4)), "k_blocks"),
    (dict(v_blocks=torch.zeros(10, 16, 2, 4).to(torch.float8_e4m3fn)), "v_blocks"),
    (dict(k_blocks=torch.zeros(10, 16, 2, 4).to(torch.float8_e4m3fn).transpose(1, 2)), "k_blocks"),
    (dict(v_blocks=torch.zeros(10, 3, 16, 4).to(torch.float8_e4m3fn)[:, :2]), "v_blocks"),
    (dict(block_table=torch.zeros(1, 4, dtype=torch.int32).expand(3, 4)), "overlap"),
    (dict(block_table=torch.zeros(3, 4)), "block_table"),
    (dict(k_scale=torch.ones(3)), "k_scale"),
    (dict(v_scale=torch.ones(2, dtype=torch.float64)), "v_scale"),
    (dict(), "CUDA"),
])
def test_cache_tensors(kw, match):
    with pytest.raises(ValueError, match=match):
        vw4.KVCache4(**cache_tensors(**kw))


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


@pytest.mark.parametrize("kw,match", [
    (dict(lens=torch.zeros(4)), "lens"), (dict(held=i32(5)), "held"), (dict(grow=i32(8)[::2]), "grow"),
    (dict(free_count=i32(2)), "free_count"), (dict(free=torch.zeros(9)), "free"),
    (dict(row_start=i32(4)), "row_start"), (dict(slots=i32(9)), "slots"),
    (dict(slots=torch.zeros(9, dtype=torch.int64), rows_max=10), "rows_max"),
    (dict(block_table=i32(4)), "block_table"), (dict(), "CUDA"),
])
def test_advance_tensors(kw, match):
    d = dict(block_table=i32(4, 6), page_size=16, lens=i32(4), held=i32(4), free=i32(9),
             free_count=i32(1), R=2)
    with pytest.raises(ValueError, match=match):
        vw4.PreparedAdvance(**dict(d, **kw))


@pytest.mark.parametrize("kw,match", [
    (dict(logits=torch.zeros(2, 3)), "logits"), (dict(logits=torch.zeros(2, 3, 9).double()), "logits"),
    (dict(logits=torch.zeros(2, 9, 3).transpose(1, 2)), "logits"), (dict(tokens=i32(2, 2)), "tokens"),
    (dict(tokens=torch.zeros(2, 3, dtype=torch.int64)), "tokens"), (dict(length=i32(3)), "length"),
    (dict(top=33), "top"), (dict(logprob=torch.zeros(2, 3), tokens=None), "tokens"),
    (dict(top_ids=i32(2, 3, 0)), "top"), (dict(top=4, top_ids=i32(2, 3, 5)), "top_ids"),
    (dict(lse=torch.zeros(2, 3).half()), "lse"), (dict(), "CUDA"),
])
def test_logprobs_tensors(kw, match):
    d = dict(logits=torch.zeros(2, 3, 9), tokens=i32(2, 3))
    with pytest.raises(ValueError, match=match):
        vw4.PreparedLogprobs(**dict(d, **kw))
