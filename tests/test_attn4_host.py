"""Host checks and page arithmetic of the 4-bit cache (nothing is launched: the
device pointers are fake), and the definition that the GPU tests measure by."""
import numpy as np
import pytest
import torch

import gated_deltanet_state_gb300 as gdn
from gated_deltanet_state_gb300 import inputs
from gated_deltanet_state_gb300.inputs import F32, AttnShape

import attn4_harness as a4
from test_attn_host import C, append, decode, desc, gather, pool, prefill, tables

SH4 = AttnShape(8, 2, 128, 64, kv_bits=4)
CALLS = [tables, append, gather, decode, prefill]


@pytest.mark.parametrize("call", CALLS)
def test_bits_of_a_value(call):
    for bits in (-4, 1, 2, 3, 5, 16, 1 << 30):
        assert call(desc(reserved=bits)) == C["GDN_ERR_INVALID_ARG"], bits
    for d in (16, 48, 80, 112, 144, 240, 288):
        assert call(desc(reserved=4, head_dim=d)) == C["GDN_ERR_UNSUPPORTED_SHAPE"], d


@pytest.mark.parametrize("call", [append, gather, decode])
def test_pools_of_4_bits(call):
    """A pool whose pages hold 4 bits a value does not do for 8, and any smaller one for neither."""
    small = pool(page_bytes=SH4.page_bytes)
    assert call(desc(reserved=8), small) == C["GDN_ERR_INVALID_ARG"]
    assert call(desc(reserved=4), pool(page_bytes=SH4.page_bytes - 256)) == C["GDN_ERR_INVALID_ARG"]
    assert call(desc(reserved=4), pool(page_bytes=SH4.page_bytes + 8)) == C["GDN_ERR_INVALID_ARG"]


def test_arguments_and_empty_calls():
    four = desc(reserved=4)
    for call, bad in ((append, dict(k=None)), (append, dict(v_stride=260)), (append, dict(slot_map=None)), (gather, dict(k=0x10002)),
                      (gather, dict(cu_kv=None)), (decode, dict(max_q_len=33)), (decode, dict(q_stride=1000)), (decode, dict(o=0x10002)),
                      (decode, dict(dev_error=None))):
        assert call(four, pool(page_bytes=SH4.page_bytes), **bad) == C["GDN_ERR_INVALID_ARG"], bad
    p = pool(page_bytes=SH4.page_bytes)
    assert append(four, p, total_tokens=0) == 0 and gather(four, p, num_seqs=0) == 0 and decode(four, p, num_seqs=0) == 0
    need = gdn.gdn_attn_decode_workspace_size(SH4, 2, 2, 5000)
    assert decode(four, p, max_kv_len=5000, size=need - 1) == C["GDN_ERR_WORKSPACE"]


def test_page_bytes():
    for sh in (SH4, AttnShape(24, 4, 256, 896, kv_bits=4), AttnShape(1, 1, 32, 16, dtype=F32, kv_bits=4), AttnShape(3, 3, 96, 48, kv_bits=4)):
        per = sh.head_dim + sh.head_dim // 32 + 1                    # a token and head: codes, K scales, V scale
        assert gdn.gdn_kv_page_bytes(sh) == sh.page_bytes == -(-sh.num_kv_heads * sh.page_tokens * per // 256) * 256
    # 0.517 of the 8-bit page at d = 256
    assert inputs.with_(inputs.ATTN27B, kv_bits=4).page_bytes / inputs.ATTN27B.page_bytes < 0.52
    assert gdn.gdn_kv_page_bytes(AttnShape(4, 2, 80, 16, kv_bits=4)) == -1


def test_views_of_a_pool():
    sh = AttnShape(4, 2, 64, 32, kv_bits=4)
    pool = gdn.KVPool(sh, 3, device="cpu", fill=0)
    assert pool.k_codes().shape == (3, 2, 2, 2, 16, 16) and pool.v_codes().shape == (3, 2, 2, 64, 8)
    assert pool.k_scales().shape == (3, 2, 2, 2, 16) and pool.v_scales().shape == (3, 2, 2, 16)
    for i, x in enumerate((pool.k_codes(), pool.v_codes(), pool.k_scales(), pool.v_scales())):
        x.fill_(i + 1)
    n = sh.codes_bytes
    assert [int((pool.buf == i).sum()) for i in range(1, 5)] == [3 * n, 3 * n, 3 * sh.scales_bytes[0], 3 * sh.scales_bytes[1]]


def test_the_definition():
    """Codes are the nearest values of the least scale that reaches the largest one."""
    x = np.random.default_rng(3).standard_normal((50, 32)) * 3
    n, b = a4.quantise(x)
    val = a4.scale_values()
    assert (n.min(), n.max()) == (1, 15) and np.all(np.abs(x).max(1) <= 7 * val[b]) and np.all(np.abs(x).max(1) > 7 * val[b - 1])
    assert np.all(np.abs(x - (n - 8) * val[b][:, None]) <= val[b][:, None] / 2)
    n, b = a4.quantise(np.array([[0.5, -0.5, 1.5, 7.0], [0, 0, 0, 0], [np.nan, 1, 2, 3], [np.inf, 1, -np.inf, 0]]))
    assert n[0].tolist() == [9, 7, 10, 15] and val[b[0]] == 1 and b.tolist()[1:3] == [0, 255]
    assert n[1].tolist() == n[2].tolist() == [8] * 4 and n[3].tolist() == [15, 14, 1, 8]   # 1 / 0.15625 = 6.4
    # every value is exact in bf16
    v = torch.tensor((np.arange(1, 16)[:, None] - 8) * val[None, :255])
    assert torch.equal(v.to(torch.bfloat16).double(), v)
