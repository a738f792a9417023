"""Attention over the 4-bit cache against 64 bits (bounds: attn_harness.py)."""
import math

import numpy as np
import pytest
import torch

import gated_deltanet_state_gb300 as gdn
from gated_deltanet_state_gb300.inputs import BF16, F32, AttnShape

from attn4_harness import sequence_rows
from attn_harness import assert_attention, attention64, err_word, fill_cache, table_for

pytestmark = pytest.mark.gpu

INVALID = gdn.STATUS_CODE["GDN_ERR_INVALID_ARG"]
PAGE_RANGE = gdn.STATUS_CODE["GDN_ERR_PAGE_RANGE"]

# heads and sizes: (Hq, Hkv, d, dtype)
LAYERS = [(24, 4, 256, BF16), (8, 8, 128, BF16), (16, 2, 128, BF16), (6, 2, 64, BF16), (5, 1, 32, BF16), (4, 2, 96, BF16),
          (3, 1, 160, BF16), (2, 2, 224, BF16), (4, 2, 32, F32), (6, 1, 256, F32), (3, 3, 96, F32), (40, 1, 128, BF16)]


def shape(Hq, Hkv, d, dt, page, **kw):
    return AttnShape(Hq, Hkv, d, page, dtype=dt, kv_bits=4, **kw)


def rows_of(n, heads, d, dtype, seed, extra=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, heads * d + extra, generator=g).to(dtype).cuda()
    return x[:, :heads * d].unflatten(1, (heads, d))


def largest_term(q, k, v, scale):
    """max over the keys of a row's normalised weight times the key's largest value, [n, Hq] in 64 bits."""
    q, k, v = (torch.as_tensor(x).double().cpu() for x in (q, k, v))
    n, Hq, L, G = q.shape[0], q.shape[1], k.shape[0], q.shape[1] // k.shape[1]
    s = torch.einsum("nhd,lhd->nhl", q, k.repeat_interleave(G, 1)) * scale
    s = s.masked_fill((torch.arange(L)[None] > torch.arange(L - n, L)[:, None])[:, None], -math.inf)
    w = torch.softmax(s, 2).nan_to_num(0.0)
    return (w * v.abs().amax(2).repeat_interleave(G, 1).T[None]).amax(2)


def cu_of(lens):
    return torch.tensor([0] + np.cumsum(lens).tolist(), dtype=torch.int32).cuda()


def run_decode(sh, pool, q, news, lens, table, **kw):
    o = torch.full((sum(news), sh.num_q_heads, sh.head_dim), 7.0, dtype=sh.torch_dtype(), device="cuda")
    lse = torch.full((sum(news), sh.num_q_heads), 7.0, device="cuda")
    err = err_word()
    gdn.gdn_attn_decode(sh, pool, q=q, cu_seqlens=cu_of(news), kv_len=torch.tensor(lens, dtype=torch.int32).cuda(),
                        block_table=table.cuda(), o=o, lse=lse, max_q_len=max(max(news), 1), dev_error=err, **kw)
    return o, lse, err.item()


def check(sh, pool, table, q, o, lse, news, lens):
    r0 = 0
    for s, (n, L) in enumerate(zip(news, lens)):
        k, v = sequence_rows(pool, table[s], L)
        assert_attention(o[r0:r0 + n], lse[r0:r0 + n], attention64(q[r0:r0 + n], k, v, sh.softmax_scale), sh.dtype)
        r0 += n


def decode_case(sh, lens, news, seed, extra=8, fill=0xFF, size=1.0, **kw):
    P = sh.page_tokens
    pages = sum(-(-n // P) for n in lens) + 1
    pool = gdn.KVPool(sh, pages, fill=fill)
    table = table_for(lens, P, pages, seed)
    fill_cache(pool, table, lens, seed, size)
    q = rows_of(sum(news), sh.num_q_heads, sh.head_dim, sh.torch_dtype(), seed + 5, extra)
    o, lse, err = run_decode(sh, pool, q, news, lens, table, **kw)
    assert err == 0
    check(sh, pool, table, q, o, lse, news, lens)
    return pool, table, q, o, lse


@pytest.mark.parametrize("Hq,Hkv,d,dt", LAYERS)
def test_decode4_single_tokens(Hq, Hkv, d, dt):
    """Ragged contexts, lengths of zero and one among them; what was never written is NaN."""
    decode_case(shape(Hq, Hkv, d, dt, 48), [1, 300, 16, 0, 17, 127, 128, 129, 2500], [1] * 9, seed=d + Hq)


@pytest.mark.parametrize("Hq,Hkv,d,dt", LAYERS)
def test_decode4_draft_rows(Hq, Hkv, d, dt):
    """1 to 32 rows a request, more rows than keys (the first see none), and requests with no row."""
    decode_case(shape(Hq, Hkv, d, dt, 64), [40, 700, 3, 16, 900, 20], [16, 32, 9, 0, 5, 20], seed=d + Hq + 1)


@pytest.mark.parametrize("page", [16, 112, 640, 784, 896])
def test_decode4_page_sizes(page):
    decode_case(shape(12, 2, 128, BF16, page), [1700, 5000, 33], [1, 4, 2], seed=page)


@pytest.mark.parametrize("n", [1, 2, 3, 5, 9, 17, 32])
def test_decode4_every_width_of_rows(n):
    """Rows that fill, pass and split the tiles of rows, at pieces' ends."""
    decode_case(shape(12, 2, 64, BF16, 128), [1024, 1025, 3000, n], [n] * 4, seed=n)


def test_decode4_pieces_of_long_contexts():
    decode_case(shape(2, 1, 64, BF16, 512), [2048, 2049, 38912, 45001], [1, 1, 1, 2], seed=4)


def test_decode4_row_stride_dense_and_own_scale():
    decode_case(shape(6, 1, 128, BF16, 64, scale=0.3), [333, 90], [1, 1], seed=8, extra=0)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("n", [1, 20])
def test_decode4_scores_of_hundreds(dt, n):
    """Large rows: scores far apart, the largest late in the sequence, most weights nothing."""
    sh = shape(8, 2, 128, dt, 64)
    lens, news = [1500, 260, 40], [n, n, n]
    pages = sum(-(-x // 64) for x in lens) + 1
    pool, table = gdn.KVPool(sh, pages, fill=0xFF), table_for(lens, 64, pages, 3)
    g = torch.Generator().manual_seed(7)
    T = sum(lens)
    k = torch.randn(T, 2, 128, generator=g) * torch.linspace(0.1, 30, T)[:, None, None]
    v = torch.randn(T, 2, 128, generator=g)
    from attn_harness import slots_for
    err = err_word()
    gdn.gdn_kv_append(sh, pool, k=k.to(sh.torch_dtype()).cuda(), v=v.to(sh.torch_dtype()).cuda(),
                      slot_map=slots_for(table, lens, lens, 64).cuda(), dev_error=err)
    q = rows_of(sum(news), 8, 128, sh.torch_dtype(), 1) * 4
    o, lse, e2 = run_decode(sh, pool, q, news, lens, table)
    assert err.item() == 0 and e2 == 0
    r0 = 0
    for s, (m, L) in enumerate(zip(news, lens)):
        kk, vv = sequence_rows(pool, table[s], L)
        ro, rl, A = attention64(q[r0:r0 + m], kk, vv, sh.softmax_scale)
        got, gl = o[r0:r0 + m].double().cpu(), lse[r0:r0 + m].double().cpu()
        # scores of up to S carry 2^-22 S each (d products in fp32, exponent and reference): weights e^that
        smax = float(rl[torch.isfinite(rl)].abs().max()) if torch.isfinite(rl).any() else 0.0
        rel = 2.0 ** -18 * max(smax, 1.0) + (2.0 ** -8 * (1 + 1 / 16) if dt == BF16 else 1e-6)
        # a weight times its V scale is an f16 of 2^-24 steps (2^-20 for every second pair of tokens), so off by
        # 2^-21 at most where the piece's largest is 2^10 (fp32: 2^12) or more; times 7 and V's scale, that is
        # at most 1.125 max|v| of its token: in all 2^-31 (2^-33) times the largest w max|v| for each key
        floor = 1.125 * 2.0 ** (-31 if dt == BF16 else -33) * L * largest_term(q[r0:r0 + m], kk, vv, sh.softmax_scale)
        tol = rel * A + 2.0 ** -8 * ro.abs() + floor[..., None] + 1e-30
        assert bool(((got - ro).abs() <= tol).all()), float(((got - ro).abs() / tol).max())
        fin = torch.isfinite(rl)
        assert torch.equal(fin, torch.isfinite(gl)) and bool(((gl - rl).abs()[fin] <= 1e-5 * (1 + smax)).all())
        r0 += m


def test_decode4_bits_do_not_depend_on_the_batch():
    sh = shape(24, 4, 256, BF16, 64)
    lens, news = [5000, 31, 700, 2049, 1], [3, 1, 16, 1, 1]
    pool, table, q, o, lse = decode_case(sh, lens, news, seed=12)
    r0 = 0
    for s, n in enumerate(news):
        o1, l1, err = run_decode(sh, pool, q[r0:r0 + n], [n], [lens[s]], table[s:s + 1])
        assert err == 0 and torch.equal(o1, o[r0:r0 + n]) and torch.equal(l1, lse[r0:r0 + n])
        r0 += n


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_decode4_ignores_what_a_row_may_not_see(bad):
    """The second draft row's K and V are no numbers: the first row's bits stay."""
    sh = shape(4, 1, 128, BF16, 64)
    pool, table, q, o, lse = decode_case(sh, [77], [2], seed=3)
    x = torch.full((1, 1, 128), bad).bfloat16().cuda()
    gdn.gdn_kv_append(sh, pool, k=x, v=x, slot_map=torch.tensor([int(table[0, 1]) * 64 + 12]).cuda(), dev_error=err_word())
    o2, l2, err = run_decode(sh, pool, q, [2], [77], table)
    assert err == 0 and torch.equal(o2[0], o[0]) and torch.equal(l2[0], lse[0])
    if math.isnan(bad):
        assert torch.isnan(o2[1].float()).all() and torch.isnan(l2[1]).all()


def test_decode4_nan_in_one_value_row():
    """A NaN in V reaches the rows that see its token and that head alone."""
    sh = shape(6, 2, 64, BF16, 32)
    pool, table, q, o, lse = decode_case(sh, [50, 90], [4, 1], seed=13)
    x = torch.zeros(1, 2, 64).bfloat16().cuda()
    y = torch.zeros(1, 2, 64).bfloat16().cuda()
    y[0, 1, 3] = math.nan
    gdn.gdn_kv_append(sh, pool, k=x, v=y, slot_map=torch.tensor([int(table[0, 1]) * 32 + 16]).cuda(), dev_error=err_word())   # token 48
    o2, _, err = run_decode(sh, pool, q, [4, 1], [50, 90], table)
    nan = torch.isnan(o2.float())
    assert err == 0 and nan[2:4, 3:].all() and not nan[:2].any() and not nan[2:4, :3].any() and torch.equal(o2[4], o[4])
    assert torch.equal(o2[:2], o[:2])


def test_decode4_refuses_on_the_device():
    sh = shape(4, 2, 64, BF16, 32)
    pool, table, q, o, _ = decode_case(sh, [100, 40], [1, 1], seed=2)
    far = table.clone()
    far[0, 1] = 999
    o2, _, err = run_decode(sh, pool, q, [1, 1], [100, 40], far)
    assert err == PAGE_RANGE and torch.equal(o2[1], o[1])
    k, v = sequence_rows(pool, table[0], 100)
    keep = np.r_[0:32, 64:100]                                       # that page's keys are left out
    ref = attention64(q[:1], k[keep], v[keep], sh.softmax_scale)
    assert float((o2[:1].double().cpu() - ref[0]).abs().max()) <= 2.0 ** -7 * float(ref[2].max())
    o2, _, err = run_decode(sh, pool, q, [1, 1], [100, 40], table, max_kv_len=64)     # a context beyond the bound
    assert err == INVALID and bool((o2[0] == 7).all()) and torch.equal(o2[1], o[1])


def test_decode4_on_another_stream_and_in_a_graph():
    sh = shape(8, 2, 128, BF16, 64)
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
