"""Refusals of the entry points between the verify GEMMs, on the host (fake
device addresses, no launch)."""
import ctypes
import math

import pytest

import speculative_decode_verification_w4_gb300 as vw4
from speculative_decode_verification_w4_gb300 import build as vbuild


@pytest.fixture(scope="module")
def lib():
    vbuild.build()
    return vw4.load_library()


def kv(**kw):
    d = dict(dtype=vw4.KV_BF16, page_size=16, num_pages=10, Hkv=2, D=128, max_blocks=4,
             page_stride=16 * 256, token_stride=256, head_stride=128, table_stride=4,
             k_dev=0x10000, v_dev=0x20000, block_table_dev=0x30000, k_scale_dev=None,
             v_scale_dev=None)
    d.update({k: v for k, v in kw.items() if k in d})
    return vw4.KVDesc(**d)


BAD_CACHE = [
    (dict(dtype=3), 1), (dict(k_dev=None), 1), (dict(v_dev=None), 1),
    (dict(block_table_dev=None), 1), (dict(num_pages=0), 1), (dict(max_blocks=0), 1),
    (dict(table_stride=3), 1), (dict(Hkv=3), 1), (dict(Hkv=0), 1), (dict(page_size=0), 1),
    (dict(page_size=12), 2), (dict(page_size=4), 2), (dict(page_size=1 << 17), 2), (dict(D=96), 2),
    (dict(page_stride=-8), 1), (dict(page_size=65536, max_blocks=1 << 20, table_stride=1 << 20), 1),
    (dict(k_scale_dev=0x100), 1),
    (dict(k_dev=0x10008), 3), (dict(token_stride=260), 3), (dict(page_stride=4100), 3),
    (dict(head_stride=4), 3), (dict(dtype=vw4.KV_E4M3, head_stride=136), 3),
    (dict(block_table_dev=0x30002), 3),
    (dict(B=0), 1), (dict(B=20000), 1), (dict(R=0), 1), (dict(R=17), 1), (dict(Hq=7), 1),
    (dict(Hq=0), 1), (dict(Hq=258), 1),
]


def fields(cls, d, kw):
    names = {f[0] for f in cls._fields_}
    d = dict(d, kv=kv(**kw))
    d.update({k: v for k, v in kw.items() if k in names})
    return cls(**d)


@pytest.mark.parametrize("kw,code", BAD_CACHE + [
    (dict(q_dev=None), 1), (dict(out_dev=None), 1), (dict(seq_lens_dev=None), 1),
    (dict(ldq=1000), 1), (dict(ldo=1000), 1), (dict(window=-1), 1), (dict(sinks=-1), 1),
    (dict(sinks=4), 1), (dict(scale=0.0), 1), (dict(scale=math.nan), 1), (dict(scale=math.inf), 1),
    (dict(scale=-1.0), 1), (dict(q_dev=0x1008), 3), (dict(out_dev=0x1002), 3),
    (dict(lse_dev=0x1002), 3), (dict(ldq=1028), 3), (dict(ldo=1028), 3),
    (dict(ws=None), 6), (dict(ws_bytes=1000), 6), (dict(ws=0x1010), 3),
])
def test_attention_refusals(lib, kw, code):
    a = fields(vw4.AttnArgs, dict(q_dev=0x1000, out_dev=0x2000, lse_dev=None, seq_lens_dev=0x3000,
                                  ldq=1024, ldo=1024, B=2, R=3, Hq=8, window=0, sinks=0,
                                  scale=0.1), kw)
    assert lib.verify_attn(ctypes.byref(a), kw.get("ws", 0x100000), kw.get("ws_bytes", 1 << 30),
                           None) == code
    assert lib.verify_attn(None, 0x100000, 1 << 30, None) == 1


@pytest.mark.parametrize("kw,code", BAD_CACHE + [
    (dict(x_dev=None), 1), (dict(q_dev=None), 1), (dict(seq_lens_dev=None), 1),
    (dict(inv_freq_dev=None), 1), (dict(rot=130), 1), (dict(rot=63), 1), (dict(rot=-2), 1),
    (dict(adjacent=2), 1), (dict(x_bf16=2), 1), (dict(eps=-1.0), 1), (dict(eps=math.nan), 1),
    (dict(ldx=1528), 1), (dict(ldq=1016), 1), (dict(x_dev=0x1004), 3), (dict(q_dev=0x2004), 3),
    (dict(q_norm_dev=0x2004), 3), (dict(k_norm_dev=0x2004), 3), (dict(inv_freq_dev=0x2004), 3),
    (dict(ldx=1538), 3), (dict(x_bf16=1, ldx=1540), 3), (dict(ldq=1028), 3),
])
def test_append_refusals(lib, kw, code):
    a = fields(vw4.AppendArgs, dict(x_dev=0x1000, inv_freq_dev=0x4000, q_norm_dev=None,
                                    k_norm_dev=None, q_dev=0x2000, seq_lens_dev=0x3000, ldx=1536,
                                    ldq=1024, x_bf16=0, B=2, R=3, Hq=8, rot=128, adjacent=0,
                                    eps=1e-6), kw)
    assert lib.verify_rope_append(ctypes.byref(a), None) == code
    assert lib.verify_rope_append(None, None) == 1


@pytest.mark.parametrize("kw,code", [
    (dict(x_dev=None), 1), (dict(out_dev=None), 1), (dict(B=0), 1), (dict(R=0), 1),
    (dict(R=17), 1), (dict(V=0), 1), (dict(V=(1 << 24) + 1, ldx=1 << 25, ldo=1 << 25), 1),
    (dict(B=16385), 1), (dict(ldx=99), 1), (dict(ldo=99), 1),
    (dict(out_dev=0x1000, ldo=104), 1), (dict(drafts_dev=None), 1), (dict(hist_max=11), 1),
    (dict(hist_max=-1), 1), (dict(bias_vals_dev=None), 1), (dict(bias_ids_dev=None), 1),
    (dict(bias_max=5), 1), (dict(mask_rows=0), 1), (dict(mask_stride=3), 1),
    (dict(x_dev=0x1002), 3), (dict(out_dev=0x2001), 3), (dict(block_max_dev=0x2001), 3),
    (dict(mask_dev=0x2002), 3), (dict(history_dev=0x2002), 3),
])
def test_logits_refusals(lib, kw, code):
    d = dict(x_dev=0x1000, out_dev=0x2000, block_max_dev=None, drafts_dev=0x3000,
             history_dev=0x4000, bias_ids_dev=0x5000, bias_vals_dev=0x6000, mask_dev=0x7000,
             ldx=100, ldo=100, hist_stride=10, bias_stride=4, mask_stride=4, B=2, R=3, V=100,
             hist_max=10, bias_max=4, mask_rows=6)
    d.update(kw)
    a = vw4.LogitsArgs(**d)
    assert lib.process_logits(ctypes.byref(a), None) == code
    assert lib.process_logits(None, None) == 1


def test_workspace_bytes(lib):
    w = vw4.vw4_workspace_bytes
    assert 0 < w(vw4.OP_ATTN, 1, 1, 64) < w(vw4.OP_ATTN, 1, 64, 64) <= w(vw4.OP_ATTN, 1, 128, 64)
    assert w(vw4.OP_ATTN, 4096, 8, 128) > w(vw4.OP_ATTN, 1, 8, 128)
    for bad in ((0, 8, 128), (1, 0, 128), (1, 8, 96), (20000, 8, 128), (1, 1 << 20, 128)):
        assert w(vw4.OP_ATTN, *bad) == 0
