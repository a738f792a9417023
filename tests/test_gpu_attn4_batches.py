"""Attention over the 4-bit cache in large and mixed batches, where the softmax is
not flat, behind waits that run out, in pools past 4 GB, and the operators in a
serving run (bounds: attn_harness.py; the cache's values enter exactly)."""
import importlib.util
import math
import os

import numpy as np
import pytest
import torch

import gated_deltanet_state_gb300 as gdn
from gated_deltanet_state_gb300 import inputs
from gated_deltanet_state_gb300.inputs import BF16, F32, AttnShape

from attn4_harness import sequence_rows
from attn_harness import assert_attention, attention64, err_word, fill_cache, slots_for, table_for

pytestmark = pytest.mark.gpu

TIMEOUT = gdn.STATUS_CODE["GDN_ERR_TIMEOUT"]
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Batch:
    def __init__(self, sh, news, lens, seed, fill=0xFF):
        self.sh, self.news, self.lens = sh, news, lens
        P = sh.page_tokens
        pages = sum(-(-n // P) for n in lens) + 1
        self.pool = gdn.KVPool(sh, pages, fill=fill)
        self.table = table_for(lens, P, pages, seed)
        fill_cache(self.pool, self.table, lens, seed)
        g = torch.Generator().manual_seed(seed + 1)
        self.q = torch.randn(sum(news), sh.num_q_heads, sh.head_dim, generator=g).to(sh.torch_dtype()).cuda()
        self.at = np.concatenate([[0], np.cumsum(news)]).tolist()

    def rows(self, s):
        return slice(self.at[s], self.at[s + 1])

    def run(self, seqs, wait=0, err=None):
        i32 = dict(dtype=torch.int32, device="cuda")
        q = torch.cat([self.q[self.rows(s)] for s in seqs])
        news, lens = [self.news[s] for s in seqs], [self.lens[s] for s in seqs]
        o, lse, err = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda"), err_word() if err is None else err
        gdn.gdn_attn_decode(self.sh, self.pool, q=q, cu_seqlens=torch.tensor([0] + np.cumsum(news).tolist(), **i32),
                            kv_len=torch.tensor(lens, **i32), block_table=self.table[list(seqs)].cuda(), o=o, lse=lse,
                            max_q_len=max(max(news), 1), max_kv_len=max(lens), wait_cycles=wait, dev_error=err)
        return o, lse, err.item()

    def check(self, every):
        """Twice the same, and a sequence as it is alone (in the kernel that its own rows ask for)."""
        N = len(self.news)
        o, lse, err = self.run(range(N))
        assert err == 0
        o2, lse2, _ = self.run(range(N))
        assert torch.equal(o2, o) and torch.equal(lse2, lse)
        for s in range(N):
            r, L = self.rows(s), self.lens[s]
            if L == 0:
                assert not o[r].any() and bool((lse[r] == -math.inf).all())
            elif s % every == 0 and self.news[s]:
                o1, lse1, _ = self.run([s])
                assert torch.equal(o1, o[r]) and torch.equal(lse1, lse[r]), s
                k, v = sequence_rows(self.pool, self.table[s], L)
                assert_attention(o[r], lse[r], attention64(self.q[r], k, v, self.sh.softmax_scale), self.sh.dtype)


@pytest.mark.parametrize("Hq,Hkv,d,dt,page", [(6, 1, 64, BF16, 16), (12, 2, 128, BF16, 64), (4, 1, 256, BF16, 128), (4, 2, 32, F32, 32)])
def test_more_sequences_than_a_launch_takes(Hq, Hkv, d, dt, page):
    """Rows of none, few (one kernel's) and many (the other's), keys of none and pieces' ends between them."""
    r = np.random.default_rng(d)
    N = 300
    news = [int(x) for x in r.choice([0, 1, 1, 1, 2, 5, 16, 32], N)]
    lens = [int(x) for x in r.choice([0, 1, 15, 16, 17, 127, 128, 129, 300, 700], N)]
    lens[7], news[7], lens[290], news[290] = 5000, 1, 3000, 9
    Batch(AttnShape(Hq, Hkv, d, page, dtype=dt, kv_bits=4), news, lens, seed=d).check(every=23)


@pytest.mark.parametrize("d", [64, 256])
def test_one_row_each(d):
    r = np.random.default_rng(d + 1)
    lens = [int(x) for x in r.integers(0, 2600, 70)]
    Batch(AttnShape(16, 2, d, 16, kv_bits=4), [1] * 70, lens, seed=5).check(every=9)


@pytest.mark.parametrize("n,others", [(1, 0), (2, 3), (1, 170), (9, 2), (16, 90)])
def test_as_many_pieces_as_there_can_be(n, others):
    """A context of 1,016 tiles (113 pieces for a few rows, 64 for more), joined by itself and in a batch."""
    b = Batch(AttnShape(8, 1, 64, 512, kv_bits=4), [n] + [1] * others, [130000] + [40] * others, seed=n)
    b.check(every=64)
    o, lse, err = b.run([0], wait=-1)
    assert err == TIMEOUT and bool((o == 7).all()) and bool((lse == 7).all())


@pytest.mark.parametrize("G", [1, 2, 3, 5, 7, 8, 9, 16, 17, 33])
def test_group_sizes(G):
    """Pairs at and around the widths of the row tiles; rows of one sequence of every number."""
    Batch(AttnShape(G, 1, 96, 48, kv_bits=4), [1, 2, 3, 4, 8, 11], [700, 30, 1300, 129, 64, 2049], seed=G).check(every=1)


# ------------------------------------------------------------------ weights far apart

def peaked_case(d, G, n, L, weight, at, own=0.02, mean=0.0, dt=BF16):
    """n rows over L keys, key `at` with about `weight` of the softmax and small values of its own."""
    sh = AttnShape(G, 1, d, 64, dtype=dt, kv_bits=4)
    g = torch.Generator().manual_seed(L + n + int(1000 * weight))
    q, k, v = torch.randn(n, G, d, generator=g), torch.randn(L, 1, d, generator=g), torch.randn(L, 1, d, generator=g) + mean
    q[..., 0], k[..., 0], k[at] = 1.0, 0.0, 0.0
    # other keys' scores are about N(0, 1): their weights sum to about (L - 1) e^(1/2)
    k[at, 0, 0] = (math.log(weight / (1 - weight)) + math.log(L - 1) + 0.5) * d ** 0.5
    v[at] = own * torch.randn(d, generator=g)
    pages = -(-L // 64) + 1
    pool, table = gdn.KVPool(sh, pages, fill=0xFF), table_for([L], 64, pages, 1)
    err = err_word()
    gdn.gdn_kv_append(sh, pool, k=k.to(sh.torch_dtype()).cuda(), v=v.to(sh.torch_dtype()).cuda(),
                      slot_map=slots_for(table, [L], [L], 64).cuda(), dev_error=err)
    q = q.to(sh.torch_dtype()).cuda()
    o, lse = torch.empty_like(q), torch.empty(n, G, device="cuda")
    gdn.gdn_attn_decode(sh, pool, q=q, cu_seqlens=torch.tensor([0, n], dtype=torch.int32).cuda(),
                        kv_len=torch.tensor([L], dtype=torch.int32).cuda(), block_table=table.cuda(), o=o, lse=lse, max_q_len=n,
                        max_kv_len=L, dev_error=err)
    assert err.item() == 0
    kk, vv = sequence_rows(pool, table[0], L)
    s = (torch.as_tensor(kk[:, 0]) @ q[0, 0].double().cpu()) * sh.softmax_scale
    assert weight / 4 < float(torch.softmax(s, 0)[at])          # the case is what it says
    assert_attention(o, lse, attention64(q, kk, vv, sh.softmax_scale), dt)


@pytest.mark.parametrize("weight", [0.5, 0.9, 0.99, 0.999, 0.99999])
@pytest.mark.parametrize("n,L", [(1, 500), (1, 4096), (1, 32768), (2, 3000), (5, 900), (16, 2000), (16, 8320)])
def test_one_key_takes_most_of_the_weight(n, L, weight):
    for at in (0, L * 3 // 4):
        peaked_case(256, 6, n, L, weight, at)


@pytest.mark.parametrize("n,G,d,dt", [(1, 1, 64, BF16), (2, 8, 128, BF16), (2, 3, 32, BF16), (32, 8, 128, BF16), (1, 4, 128, F32)])
def test_one_key_takes_most_of_the_weight_other_layers(n, G, d, dt):
    for weight in (0.9, 0.999):
        peaked_case(d, G, n, 1500, weight, 700, dt=dt)
        peaked_case(d, G, n, 1500, weight, 3, own=1.0, mean=1.0, dt=dt)


@pytest.mark.parametrize("n", [1, 16])
@pytest.mark.parametrize("gap", [10, 17])
def test_query_elements_far_apart(n, gap):
    """Half of a row's elements 2^-gap of the other half's, against keys the other way round."""
    sh, L = AttnShape(6, 1, 128, 64, kv_bits=4), 900
    g = torch.Generator().manual_seed(gap)
    q, k, v = torch.randn(n, 6, 128, generator=g), torch.randn(L, 1, 128, generator=g), torch.randn(L, 1, 128, generator=g)
    q[..., 64:] *= 2.0 ** -gap
    k[..., :64] *= 2.0 ** -gap
    q *= 2.0 ** (gap / 2)                    # scores of a few units
    k *= 2.0 ** (gap / 2)
    pool, table, err = gdn.KVPool(sh, 16, fill=0xFF), table_for([L], 64, 16, 2), err_word()
    gdn.gdn_kv_append(sh, pool, k=k.bfloat16().cuda(), v=v.bfloat16().cuda(), slot_map=slots_for(table, [L], [L], 64).cuda(), dev_error=err)
    q = q.bfloat16().cuda()
    o, lse = torch.empty_like(q), torch.empty(n, 6, device="cuda")
    gdn.gdn_attn_decode(sh, pool, q=q, cu_seqlens=torch.tensor([0, n], dtype=torch.int32).cuda(),
                        kv_len=torch.tensor([L], dtype=torch.int32).cuda(), block_table=table.cuda(), o=o, lse=lse, max_q_len=n,
                        max_kv_len=L, dev_error=err)
    kk, vv = sequence_rows(pool, table[0], L)
    assert err.item() == 0
    assert_attention(o, lse, attention64(q, kk, vv, sh.softmax_scale), BF16)


@pytest.mark.parametrize("n", [1, 16])
@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_query_rows_that_are_no_numbers(n, bad):
    """Their own outputs are NaN; the other rows keep their bits."""
    b = Batch(AttnShape(4, 1, 128, 64, kv_bits=4), [n, n], [600, 90], seed=8)
    o, lse, _ = b.run([0, 1])
    b.q[0, 2, 5] = bad
    o2, lse2, err = b.run([0, 1])
    hit = torch.zeros(2 * n, 4, dtype=torch.bool, device="cuda")
    hit[0, 2] = True
    assert err == 0 and torch.isnan(o2[hit].float()).all() and torch.isnan(lse2[hit]).all()
    assert torch.equal(o2[~hit], o[~hit]) and torch.equal(lse2[~hit], lse[~hit])


# ------------------------------------------------------------------ waits

BATCHES = {
    "few rows, one piece": ([1, 1, 1], [100, 7, 0]),
    "few rows, pieces": ([1, 1, 1], [9000, 700, 31]),
    "drafts, one piece": ([16, 32], [200, 90]),
    "drafts, pieces": ([16, 24], [5000, 9000]),
    "some rows": ([2, 2, 5], [3000, 40, 4000]),
    "both": ([16, 1, 2, 32, 0, 1], [3000, 4000, 60, 700, 50, 9000]),
}


def layer(d, dt=BF16):
    return AttnShape(12, 2, d, 64, dtype=dt, kv_bits=4)


@pytest.mark.parametrize("batch", list(BATCHES))
@pytest.mark.parametrize("d,dt", [(64, BF16), (256, BF16), (128, F32)])
def test_waits_that_run_out_write_nothing(batch, d, dt):
    b = Batch(layer(d, dt), *BATCHES[batch], seed=3)
    all_ = range(len(b.news))
    want, want_lse, err = b.run(all_)
    assert err == 0
    o, lse, err = b.run(all_, wait=-1)
    assert err == TIMEOUT and bool((o == 7).all()) and bool((lse == 7).all())
    word = lambda code: torch.tensor([code], dtype=torch.int32, device="cuda")  # noqa: E731
    o, lse, err = b.run(all_, err=word(TIMEOUT))                                # an earlier call's code stops nothing
    assert err == TIMEOUT and torch.equal(o, want) and torch.equal(lse, want_lse)
    o, lse, err = b.run(all_, wait=-1, err=word(gdn.STATUS_CODE["GDN_ERR_PAGE_RANGE"]))
    assert err == TIMEOUT and bool((o == 7).all())


@pytest.mark.parametrize("batch", list(BATCHES))
@pytest.mark.parametrize("d", [64, 256])
def test_waits_that_run_out_midway(batch, d):
    """Whatever wait gives up first, the call returns and the context is intact."""
    b = Batch(layer(d), *BATCHES[batch], seed=4)
    all_ = range(len(b.news))
    want, want_lse, err = b.run(all_)
    assert err == 0
    for wait in (1, 1, 3000, 10000, 30000):
        o, lse, err = b.run(all_, wait=wait)
        assert err in (0, TIMEOUT)
        assert err == TIMEOUT or (torch.equal(o, want) and torch.equal(lse, want_lse))
    o, lse, err = b.run(all_)
    assert err == 0 and torch.equal(o, want) and torch.equal(lse, want_lse)


# ------------------------------------------------------------------ together

def test_pages_past_4_gb():
    """Pages whose bytes lie beyond 32 bits: append, gather and decode find them."""
    sh = AttnShape(8, 4, 256, 896, kv_bits=4)
    pages = (5 << 30) // sh.page_bytes
    pool = gdn.KVPool(sh, pages)
    lens = [2000, 500]
    table = torch.tensor([[pages - 1, 3, pages - 2], [pages // 2, -1, -1]], dtype=torch.int32)
    fill_cache(pool, table, lens, 6)
    k, v = (torch.empty(2500, 4, 256, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    err = err_word()
    gdn.gdn_kv_gather(sh, pool, cu_kv=torch.tensor([0, 2000, 2500], dtype=torch.int32).cuda(), block_table=table.cuda(), k=k, v=v, dev_error=err)
    q = torch.randn(2, 8, 256, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    o, lse = torch.empty_like(q), torch.empty(2, 8, device="cuda")
    gdn.gdn_attn_decode(sh, pool, q=q, cu_seqlens=torch.tensor([0, 1, 2], dtype=torch.int32).cuda(),
                        kv_len=torch.tensor(lens, dtype=torch.int32).cuda(), block_table=table.cuda(), o=o, lse=lse, dev_error=err)
    assert err.item() == 0
    for s, at in ((0, 0), (1, 2000)):
        kk, vv = sequence_rows(pool, table[s], lens[s])
        np.testing.assert_array_equal(k[at:at + lens[s]].double().cpu().numpy(), kk)
        np.testing.assert_array_equal(v[at:at + lens[s]].double().cpu().numpy(), vv)
        assert_attention(o[s:s + 1], lse[s:s + 1], attention64(q[s:s + 1], kk, vv, sh.softmax_scale), BF16)


def example():
    spec = importlib.util.spec_from_file_location("attention_layer", os.path.join(ROOT, "examples", "attention_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_example_serves_from_4_bits():
    """Unit normal rows: K is off by a step of its group of 32 (about 2.1 / 7, up to an eighth more) over sqrt(12), 0.095 at
    most, V by one of its row (2.7 / 7), 0.125; as for 8 bits the outputs move by both: 0.16.  Bound: 0.25."""
    m = example()
    errors = m.serve(AttnShape(12, 2, 128, page_tokens=128, kv_bits=4))
    assert set(errors) == {"prefill", "decode", "draft"} and all(e < 0.25 for e in errors.values()), errors


def test_serving_run_over_the_cache():
    """Tables, append, gather, prefill, decode and drafts over a pool shared with GDN state pages: every phase is
    attention over what the cache holds, and the GDN pages stay."""
    sh = AttnShape(24, 4, 256, page_tokens=896, kv_bits=4)
    gdn_shape = inputs.QWEN27B
    m = example()
    lay = m.Layer(sh, num_pages=12, max_seqs=2, max_pages=4)
    state = gdn.StatePool(gdn_shape, 14)                       # 3,670,016-byte pages
    lay.pool = gdn.KVPool(sh, 14, page_bytes=gdn_shape.page, buf=state.buf)
    state.buf.view(14, -1)[12:].fill_(0x3C)
    g = torch.Generator(device="cuda").manual_seed(2)
    width = (24 + 8) * 256
    for new in ([900, 33], [40, 0], [1, 1], [1, 1], [7, 5], [2, 0]):
        qkv = torch.randn(sum(new), width, generator=g, device="cuda").bfloat16()
        o = lay.step(new, qkv)
        at = 0
        for s in range(2):
            q = qkv[at:at + new[s], :24 * 256].unflatten(1, (24, 256))
            k, v = sequence_rows(lay.pool, lay.table[s].cpu(), lay.len_host[s])
            ro, _, A = attention64(q, k, v, sh.softmax_scale)
            tol = 2.0 ** -8 * ro.abs() + 2.0 ** -8 * (1 + 1 / 16) * A
            assert bool(((o[at:at + new[s]].double().cpu() - ro).abs() <= tol + 1e-30).all())
            at += new[s]
    assert lay.error.item() == 0 and bool((state.buf.view(14, -1)[12:] == 0x3C).all())


def test_two_calls_at_once_and_two_graphs_of_one_workspace():
    b = Batch(AttnShape(12, 2, 128, 64, kv_bits=4), [1, 1, 20], [3000, 70, 2500], seed=9)
    i32 = dict(dtype=torch.int32, device="cuda")
    calls = []
    ws = gdn.workspace_for(gdn.gdn_attn_decode_workspace_size(b.sh, 1, 20, 4096))
    for s in (0, 2):
        q = b.q[b.rows(s)].clone()
        o, err = torch.zeros_like(q), err_word()
        kw = dict(q=q, cu_seqlens=torch.tensor([0, b.news[s]], **i32), kv_len=torch.tensor([b.lens[s]], **i32),
                  block_table=b.table[s:s + 1].cuda(), o=o, max_q_len=b.news[s], max_kv_len=4096, dev_error=err)
        calls.append((s, kw))
    want = [b.run([s])[0] for s, _ in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(3):                               # at once, each on its own stream and workspace
        for (s, kw), st in zip(calls, streams):
            with torch.cuda.stream(st):
                gdn.gdn_attn_decode(b.sh, b.pool, **kw)
        torch.cuda.synchronize()
        assert all(torch.equal(kw["o"], x) for (_, kw), x in zip(calls, want))
    graphs = []
    for s, kw in calls:                              # one after another over one workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            gdn.gdn_attn_decode(b.sh, b.pool, workspace=ws, **kw)
        graphs.append(g)
    for (_, kw) in calls:
        kw["o"].zero_()
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(kw["o"], x) and kw["dev_error"].item() == 0 for (_, kw), x in zip(calls, want))
