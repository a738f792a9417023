"""Host checks of the attention layers' entry points: refused before any
launch (the device pointers are fake and never dereferenced)."""
import math

import pytest
import torch

import gated_deltanet_state_gb300 as gdn
from gated_deltanet_state_gb300 import attention as A
from gated_deltanet_state_gb300 import inputs
from gated_deltanet_state_gb300.inputs import F32, AttnShape

F = 0x10000
C = gdn.STATUS_CODE
SH = AttnShape(8, 2, 128, 64)


def desc(**kw):
    v = dict(num_q_heads=8, num_kv_heads=2, head_dim=128, page_tokens=64, dtype=1, scale=0.1, reserved=0)
    v.update(kw)
    return A._AttnDesc(*v.values())


def pool(**kw):
    v = dict(base=0x100000, page_bytes=SH.page_bytes, num_pages=4, reserved=0)
    v.update(kw)
    return gdn._Pool(*v.values())


def args(cls, **kw):
    """Fake pointers everywhere, small counts."""
    v = {f: (F if t is A._P else 0) for f, t in cls._fields_}
    v.update(kw)
    return cls(*v.values())


def tables(d=None, **kw):
    v = dict(num_seqs=2, max_pages=3, num_free=4, num_pages=9, total_tokens=5, kv_len_out=2 * F)
    v.update(kw)
    return gdn.load_library().gdn_kv_tables(d or desc(), args(A._KvTablesArgs, **v), None)


def append(d=None, p=None, **kw):
    v = dict(total_tokens=3, k_stride=256, v_stride=256)
    v.update(kw)
    return gdn.load_library().gdn_kv_append(d or desc(), p or pool(), args(A._KvAppendArgs, **v), None)


def gather(d=None, p=None, **kw):
    v = dict(num_seqs=2, max_pages=3, total_tokens=5)
    v.update(kw)
    return gdn.load_library().gdn_kv_gather(d or desc(), p or pool(), args(A._KvGatherArgs, **v), None)


def decode(d=None, p=None, ws=F, size=1 << 40, **kw):
    v = dict(num_seqs=2, max_pages=3, max_q_len=1, max_kv_len=1000, total_tokens=2, q_stride=1024)
    v.update(kw)
    return gdn.load_library().gdn_attn_decode(d or desc(), p or pool(), args(A._AttnDecodeArgs, **v), ws, size, None)


def prefill(d=None, **kw):
    v = dict(num_seqs=2, total_q=5, total_kv=7, q_stride=1024, k_stride=256, v_stride=256)
    v.update(kw)
    return gdn.load_library().gdn_attn_prefill(d or desc(), args(A._AttnPrefillArgs, **v), None)


CALLS = [tables, append, gather, decode, prefill]


@pytest.mark.parametrize("call", CALLS)
def test_malformed_and_unsupported_layers(call):
    for bad in (dict(num_q_heads=0), dict(num_kv_heads=-1), dict(head_dim=0), dict(page_tokens=0), dict(dtype=2),
                dict(scale=0.0), dict(scale=math.nan), dict(scale=math.inf), dict(reserved=1)):
        assert call(desc(**bad)) == C["GDN_ERR_INVALID_ARG"], bad
    for bad in (dict(num_q_heads=7), dict(head_dim=24), dict(head_dim=272), dict(page_tokens=40), dict(num_q_heads=2048)):
        assert call(desc(**bad)) == C["GDN_ERR_UNSUPPORTED_SHAPE"], bad


@pytest.mark.parametrize("call", [append, gather, decode])
def test_pools(call):
    for bad in (dict(base=None), dict(base=0x100010), dict(page_bytes=SH.page_bytes - 256), dict(page_bytes=SH.page_bytes + 8),
                dict(num_pages=0)):
        assert call(p=pool(**bad)) == C["GDN_ERR_INVALID_ARG"], bad


@pytest.mark.parametrize("call,bad", [
    (tables, dict(num_seqs=-1)), (tables, dict(num_seqs=1 << 17)), (tables, dict(total_tokens=-1)), (tables, dict(kv_len=None)),
    (tables, dict(new_len=None)), (tables, dict(free_pages=None)), (tables, dict(block_table=None)), (tables, dict(cu_kv=None)),
    (tables, dict(kv_len_out=F)), (tables, dict(slot_map=None)), (tables, dict(dev_error=None)), (tables, dict(num_pages=0)),
    (append, dict(total_tokens=-1)), (append, dict(k=None)), (append, dict(v=F + 8)), (append, dict(k_stride=255)),
    (append, dict(v_stride=260)), (append, dict(slot_map=None)), (append, dict(dev_error=None)),
    (gather, dict(num_seqs=-1)), (gather, dict(cu_kv=None)), (gather, dict(block_table=None)), (gather, dict(k=F + 2)),
    (gather, dict(v=None)), (gather, dict(dev_error=None)),
    (decode, dict(max_q_len=0)), (decode, dict(max_q_len=33)), (decode, dict(max_kv_len=-1)), (decode, dict(q=None)),
    (decode, dict(q=F + 4)), (decode, dict(q_stride=1000)), (decode, dict(o=None)), (decode, dict(kv_len=None)),
    (decode, dict(cu_seqlens=None)), (decode, dict(dev_error=None)), (decode, dict(total_tokens=-5)),
    (prefill, dict(total_q=-1)), (prefill, dict(q=None)), (prefill, dict(k=None)), (prefill, dict(v=F + 2)),
    (prefill, dict(k_stride=128)), (prefill, dict(q_stride=1028)), (prefill, dict(o=F + 2)), (prefill, dict(cu_kv=None)),
    (prefill, dict(dev_error=None)), (prefill, dict(reserved=3)), (prefill, dict(max_q_len=-1))])
def test_bad_arguments(call, bad):
    assert call(**bad) == C["GDN_ERR_INVALID_ARG"]


def test_decode_needs_its_workspace():
    need = gdn.gdn_attn_decode_workspace_size(SH, 2, 2, 1000)
    assert need >= 4 * 2 * 8 * (128 * 4 + 8)                     # four pieces of 256 keys
    assert decode(size=need - 1) == C["GDN_ERR_WORKSPACE"]
    assert decode(ws=None, size=0) == C["GDN_ERR_WORKSPACE"]
    assert gdn.gdn_attn_decode_workspace_size(SH, 2, 2, 256) == 256


def test_empty_calls_are_no_ops():
    assert tables(num_seqs=0) == 0 and append(total_tokens=0) == 0 and gather(num_seqs=0) == 0
    assert gather(total_tokens=0) == 0 and decode(num_seqs=0) == 0 and prefill(total_q=0) == 0 and prefill(num_seqs=0) == 0


def test_page_bytes():
    for sh in (inputs.ATTN27B, inputs.ATTN4B, inputs.ATTN_TINY, AttnShape(3, 3, 16, 16, dtype=F32)):
        assert gdn.gdn_kv_page_bytes(sh) == sh.page_bytes
    # 16 tokens of a head: 16 d code bytes and a 4-byte scale, K and V
    assert gdn.gdn_kv_page_bytes(inputs.ATTN27B) == 4 * 56 * 2 * (16 * 256 + 4)
    assert gdn.gdn_kv_page_bytes(AttnShape(8, 3, 128, 40)) == -1


def test_binding_checks_tensors():
    t = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gdn_attn_prefill(SH, q=t, k=t, v=t, cu_seqlens=torch.zeros(2), cu_kv=t, o=t, dev_error=t)
    with pytest.raises(ValueError, match="buf"):
        gdn.KVPool(SH, 4, buf=torch.zeros(5, dtype=torch.uint8))
