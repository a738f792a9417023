"""Attention over the 8-bit cache and over packed prompts against 64 bits
(attn_harness.py states the bounds)."""
import math

import numpy as np
import pytest
import torch

import gated_deltanet_state_gb300 as gdn
from gated_deltanet_state_gb300 import inputs
from gated_deltanet_state_gb300.inputs import BF16, F32, AttnShape

from attn_harness import assert_attention, attention64, err_word, fill_cache, sequence_rows, table_for

pytestmark = pytest.mark.gpu

INVALID = gdn.STATUS_CODE["GDN_ERR_INVALID_ARG"]
PAGE_RANGE = gdn.STATUS_CODE["GDN_ERR_PAGE_RANGE"]

# heads and sizes: (Hq, Hkv, d, dtype)
LAYERS = [(24, 4, 256, BF16), (8, 8, 128, BF16), (16, 2, 128, BF16), (6, 2, 64, BF16), (5, 1, 32, BF16), (4, 2, 80, BF16),
          (4, 2, 32, F32), (6, 1, 256, F32), (3, 3, 16, F32), (40, 1, 128, BF16)]


def rows_of(n, heads, d, dtype, seed, extra=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, heads * d + extra, generator=g).to(dtype).cuda()
    return x[:, :heads * d].unflatten(1, (heads, d))


def cu_of(lens):
    return torch.tensor([0] + np.cumsum(lens).tolist(), dtype=torch.int32).cuda()


# ------------------------------------------------------------------ decode

def run_decode(sh, pool, q, news, lens, table, **kw):
    o = torch.full((sum(news), sh.num_q_heads, sh.head_dim), 7.0, dtype=sh.torch_dtype(), device="cuda")
    lse = torch.full((sum(news), sh.num_q_heads), 7.0, device="cuda")
    err = err_word()
    gdn.gdn_attn_decode(sh, pool, q=q, cu_seqlens=cu_of(news), kv_len=torch.tensor(lens, dtype=torch.int32).cuda(),
                        block_table=table.cuda(), o=o, lse=lse, max_q_len=max(max(news), 1), dev_error=err, **kw)
    return o, lse, err.item()


def decode_case(sh, lens, news, seed, extra=8, fill=0xFF, **kw):
    P = sh.page_tokens
    pages = sum(-(-n // P) for n in lens) + 1
    pool = gdn.KVPool(sh, pages, fill=fill)
    table = table_for(lens, P, pages, seed)
    fill_cache(pool, table, lens, seed)
    q = rows_of(sum(news), sh.num_q_heads, sh.head_dim, sh.torch_dtype(), seed + 5, extra)
    o, lse, err = run_decode(sh, pool, q, news, lens, table, **kw)
    assert err == 0
    r0 = 0
    for s, (n, L) in enumerate(zip(news, lens)):
        k, v = sequence_rows(pool, table[s], L)
        assert_attention(o[r0:r0 + n], lse[r0:r0 + n], attention64(q[r0:r0 + n], k, v, sh.softmax_scale), sh.dtype)
        r0 += n
    return pool, table, q, o, lse


@pytest.mark.parametrize("Hq,Hkv,d,dt", LAYERS)
def test_decode_single_tokens(Hq, Hkv, d, dt):
    """Ragged contexts, lengths of zero and one among them; what was never written is NaN."""
    decode_case(AttnShape(Hq, Hkv, d, 48, dtype=dt), [1, 300, 16, 0, 17, 127, 128, 129, 2500], [1] * 9, seed=d + Hq)


@pytest.mark.parametrize("Hq,Hkv,d,dt", LAYERS)
def test_decode_draft_rows(Hq, Hkv, d, dt):
    """1 to 32 rows a request, more rows than keys (the first see none), and requests with no row."""
    decode_case(AttnShape(Hq, Hkv, d, 64, dtype=dt), [40, 700, 3, 16, 900, 20], [16, 32, 9, 0, 5, 20], seed=d + Hq + 1)


@pytest.mark.parametrize("page", [16, 112, 640, 784, 896])
def test_decode_page_sizes(page):
    decode_case(AttnShape(12, 2, 128, page), [1700, 5000, 33], [1, 4, 2], seed=page)


def test_decode_pieces_of_long_contexts():
    decode_case(AttnShape(2, 1, 64, 512), [2048, 2049, 38912, 45001], [1, 1, 1, 2], seed=4)


def test_decode_row_stride_dense_and_own_scale():
    decode_case(AttnShape(6, 1, 128, 64, scale=0.3), [333, 90], [1, 1], seed=8, extra=0)


def test_decode_bits_do_not_depend_on_the_batch():
    sh = AttnShape(24, 4, 256, 64)
    lens, news = [5000, 31, 700, 2049, 1], [3, 1, 16, 1, 1]
    pool, table, q, o, lse = decode_case(sh, lens, news, seed=12)
    r0 = 0
    for s, n in enumerate(news):
        o1, l1, err = run_decode(sh, pool, q[r0:r0 + n], [n], [lens[s]], table[s:s + 1])
        assert err == 0 and torch.equal(o1, o[r0:r0 + n]) and torch.equal(l1, lse[r0:r0 + n])
        r0 += n


def test_decode_ignores_what_a_row_may_not_see():
    """The second draft row's K and V are NaN: the first row's bits stay."""
    sh = AttnShape(4, 1, 128, 64)
    pool, table, q, o, lse = decode_case(sh, [77], [2], seed=3)
    bad = torch.full((1, 1, 128), math.nan).bfloat16().cuda()
    gdn.gdn_kv_append(sh, pool, k=bad, v=bad, slot_map=torch.tensor([int(table[0, 1]) * 64 + 12]).cuda(), dev_error=err_word())
    o2, l2, err = run_decode(sh, pool, q, [2], [77], table)
    assert torch.equal(o2[0], o[0]) and torch.equal(l2[0], lse[0]) and torch.isnan(o2[1].float()).all()


def test_decode_refuses_on_the_device():
    sh = AttnShape(4, 2, 64, 32)
    pool, table, q, o, _ = decode_case(sh, [100, 40], [1, 1], seed=2)
    far = table.clone()
    far[0, 1] = 999
    _, _, err = run_decode(sh, pool, q, [1, 1], [100, 40], far)
    assert err == PAGE_RANGE
    o2, _, err = run_decode(sh, pool, q, [1, 1], [100, 40], table, max_kv_len=64)     # a context beyond the bound
    assert err == INVALID and bool((o2[0] == 7).all()) and torch.equal(o2[1], o[1])


def test_decode_on_another_stream_and_in_a_graph():
    sh = AttnShape(8, 2, 128, 64)
    pool, table, q, o, lse = decode_case(sh, [900, 64], [1, 1], seed=6)
    cu, kv, bt = cu_of([1, 1]), torch.tensor([900, 64], dtype=torch.int32).cuda(), table.cuda()
    o2, err = torch.zeros_like(o), err_word()
    ws = gdn.workspace_for(gdn.gdn_attn_decode_workspace_size(sh, 2, 2, 1024))
    call = lambda: gdn.gdn_attn_decode(sh, pool, q=q, cu_seqlens=cu, kv_len=kv, block_table=bt, o=o2, max_kv_len=1024,  # noqa: E731
                                       workspace=ws, dev_error=err)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        call()
    st.synchronize()
    assert torch.equal(o2, o)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    o2.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o2, o) and err.item() == 0


# ------------------------------------------------------------------ prefill

def run_prefill(sh, q, k, v, news, lens, lse=True, **kw):
    o = torch.full((sum(news), sh.num_q_heads, sh.head_dim), 7.0, dtype=sh.torch_dtype(), device="cuda")
    ls = torch.full((sum(news), sh.num_q_heads), 7.0, device="cuda") if lse else None
    err = err_word()
    gdn.gdn_attn_prefill(sh, q=q, k=k, v=v, cu_seqlens=cu_of(news), cu_kv=cu_of(lens), o=o, lse=ls, dev_error=err, **kw)
    return o, ls, err.item()


def prefill_case(sh, news, lens, seed, extra=8, **kw):
    dt = sh.torch_dtype()
    q = rows_of(sum(news), sh.num_q_heads, sh.head_dim, dt, seed, extra)
    k = rows_of(sum(lens), sh.num_kv_heads, sh.head_dim, dt, seed + 1, extra)
    v = rows_of(sum(lens), sh.num_kv_heads, sh.head_dim, dt, seed + 2, extra)
    o, lse, err = run_prefill(sh, q, k, v, news, lens, **kw)
    assert err == 0
    a = b = 0
    for n, L in zip(news, lens):
        assert_attention(o[a:a + n], lse[a:a + n], attention64(q[a:a + n], k[b:b + L], v[b:b + L], sh.softmax_scale), sh.dtype)
        a, b = a + n, b + L
    return q, k, v, o, lse


@pytest.mark.parametrize("Hq,Hkv,d,dt", LAYERS)
def test_prefill_whole_prompts(Hq, Hkv, d, dt):
    lens = [1, 130, 17, 0, 64, 257, 33]
    prefill_case(AttnShape(Hq, Hkv, d, 16, dtype=dt), lens, lens, seed=d + Hq)


@pytest.mark.parametrize("Hq,Hkv,d,dt", LAYERS)
def test_prefill_after_a_prefix(Hq, Hkv, d, dt):
    """Chunks after cached prefixes, no rows, no keys, and more rows than keys (the first see none)."""
    prefill_case(AttnShape(Hq, Hkv, d, 16, dtype=dt), [5, 70, 0, 40, 12, 1], [300, 129, 50, 7, 0, 555], seed=d + Hq + 2,
                 max_q_len=70, max_kv_len=555)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prefill_long(d):
    prefill_case(AttnShape(4, 2, d, 16), [1500], [2111], seed=d, extra=0)


@pytest.mark.parametrize("d", [64, 128, 256, 96])
def test_prefill_bits_do_not_depend_on_batch_or_chunks(d):
    """A prompt alone, in a batch and cut into chunks (each over the keys so far) gives the same bits."""
    sh = AttnShape(6, 2, d, 16)
    lens = [700, 301]
    q, k, v, o, lse = prefill_case(sh, lens, lens, seed=d)
    o1, l1, _ = run_prefill(sh, q[:700], k[:700], v[:700], [700], [700])
    assert torch.equal(o1, o[:700]) and torch.equal(l1, lse[:700])
    for a, b in ((0, 33), (33, 448), (448, 449), (449, 700)):
        o2, l2, _ = run_prefill(sh, q[a:b], k[:b], v[:b], [b - a], [b])
        assert torch.equal(o2, o[a:b]) and torch.equal(l2, lse[a:b])


@pytest.mark.parametrize("Hq,Hkv,d,dt", [(4, 2, 128, BF16), (4, 2, 256, BF16), (2, 1, 64, BF16), (4, 2, 96, BF16), (2, 1, 32, F32)])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_prefill_ignores_what_a_row_may_not_see(Hq, Hkv, d, dt, bad):
    """A bad key and value at position 200 of one prompt: the rows before it and the other prompts keep their bits."""
    sh = AttnShape(Hq, Hkv, d, 16, dtype=dt)
    lens = [90, 300, 50]
    q, k, v, o, lse = prefill_case(sh, lens, lens, seed=d + 3)
    k, v = k.clone(), v.clone()
    k[90 + 200], v[90 + 200] = bad, bad
    o2, l2, err = run_prefill(sh, q, k, v, lens, lens)
    keep = torch.ones(440, dtype=torch.bool)
    keep[90 + 200:390] = False
    assert err == 0 and torch.equal(o2[keep], o[keep]) and torch.equal(l2[keep], lse[keep])
    assert torch.isnan(o2[~keep].float()).all()


def test_prefill_value_infinity_reaches_its_rows():
    """One infinite value: its element is infinite in the rows that see it, and nothing else moves."""
    sh = AttnShape(2, 2, 128, 16)
    q, k, v, o, lse = prefill_case(sh, [200], [200], seed=5)
    v = v.clone()
    v[150, 0, 7], v[160, 1, 9] = math.inf, -math.inf
    o2, l2, _ = run_prefill(sh, q, k, v, [200], [200])
    want = o.clone()
    want[150:, 0, 7], want[160:, 1, 9] = math.inf, -math.inf
    assert torch.equal(o2, want) and torch.equal(l2, lse)


def test_prefill_without_lse_and_beyond_the_bound():
    sh = AttnShape(4, 2, 128, 16)
    q, k, v, o, _ = prefill_case(sh, [100, 40], [100, 40], seed=1)
    o2, _, err = run_prefill(sh, q, k, v, [100, 40], [100, 40], lse=False)
    assert err == 0 and torch.equal(o2, o)
    o3, _, err = run_prefill(sh, q, k, v, [100, 40], [100, 40], max_q_len=64, max_kv_len=100)
    assert err == INVALID and bool((o3[:100] == 7).all()) and torch.equal(o3[100:], o[100:])


def test_chunks_through_the_cache_keep_the_bits():
    """Append, read back, attend: a prompt in one chunk and in two (cut on a block of 16) gives the same bits."""
    sh = AttnShape(6, 2, 128, 64)
    T, cut = 500, 320
    q, k, v = (rows_of(T, h, 128, torch.bfloat16, i) for i, h in ((1, 6), (2, 2), (3, 2)))
    outs = []
    for ends in ([T], [cut, T]):
        pool = gdn.KVPool(sh, 9, fill=0xFF)
        table = table_for([T], 64, 9, 2)
        a, parts = 0, []
        for b in ends:
            slot = torch.tensor([int(table[0, t // 64]) * 64 + t % 64 for t in range(a, b)]).cuda()
            err = err_word()
            gdn.gdn_kv_append(sh, pool, k=k[a:b], v=v[a:b], slot_map=slot, dev_error=err)
            kk, vv = (torch.empty(b, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
            gdn.gdn_kv_gather(sh, pool, cu_kv=cu_of([b]), block_table=table.cuda(), k=kk, v=vv, dev_error=err)
            parts.append(run_prefill(sh, q[a:b], kk, vv, [b - a], [b])[0])
            assert err.item() == 0
            a = b
        outs.append(torch.cat(parts))
    assert torch.equal(outs[0], outs[1])
