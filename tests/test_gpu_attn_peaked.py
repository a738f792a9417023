"""Attention over the 8-bit cache where the softmax is not flat: one key of the
context takes most of the weight and its own values are small, as the first
tokens of real prompts do, so that the outputs come from weights far below the
largest; and query rows whose elements are far apart.  The bounds are the
harness's, which allow a weight one rounding to 8 significant bits whatever
its size (attn_harness.py)."""
import math

import pytest
import torch

import gated_deltanet_state_gb300 as gdn
from gated_deltanet_state_gb300 import inputs
from gated_deltanet_state_gb300.inputs import AttnShape

from attn_harness import assert_attention, attention64, err_word, sequence_rows, slots_for, table_for

pytestmark = pytest.mark.gpu

ONES = 6   # elements of a query that are 1: the peaked key's score is put together from these


def e4m3_parts(x: float, n: int) -> list[float]:
    """x as a sum of n values of 4 significant bits (a power-of-two scale keeps them)."""
    out = []
    for _ in range(n):
        u = 2.0 ** (math.floor(math.log2(abs(x))) - 3) if x else 1.0
        out.append(math.trunc(x / u) * u)
        x -= out[-1]
    return out


def cache(sh, k, v, seed=1):
    """A pool that holds one sequence's rows; its table."""
    L, P = len(k), sh.page_tokens
    pages = -(-L // P) + 1
    pool = gdn.KVPool(sh, pages, fill=0xFF)
    table = table_for([L], P, pages, seed)
    err = err_word()
    gdn.gdn_kv_append(sh, pool, k=k.bfloat16().cuda(), v=v.bfloat16().cuda(), slot_map=slots_for(table, [L], [L], P).cuda(),
                      dev_error=err)
    assert err.item() == 0
    return pool, table


def attend(sh, pool, table, q, L):
    n = len(q)
    o, lse, err = torch.empty_like(q), torch.empty(n, sh.num_q_heads, device="cuda"), err_word()
    gdn.gdn_attn_decode(sh, pool, q=q, cu_seqlens=torch.tensor([0, n], dtype=torch.int32).cuda(),
                        kv_len=torch.tensor([L], dtype=torch.int32).cuda(), block_table=table.cuda(), o=o, lse=lse, max_q_len=n,
                        max_kv_len=L, dev_error=err)
    assert err.item() == 0
    return o, lse


def peaked_case(d, G, n, L, weight, at, mean=0.0, steps=False, own=0.02):
    """n rows over L keys, key `at` with about `weight` of the softmax."""
    sh = AttnShape(G, 1, d, 64, scale=d ** -0.5)
    g = torch.Generator().manual_seed(L + n + int(1000 * weight))
    q, k, v = torch.randn(n, G, d, generator=g), torch.randn(L, 1, d, generator=g), torch.randn(L, 1, d, generator=g) + mean
    q[..., :ONES], k[..., :ONES], k[at] = 1.0, 0.0, 0.0
    # other keys' scores are about N(0, 1): their weights sum to about (L - 1) e^(1/2)
    nats = math.log(weight / (1 - weight)) + math.log(L - 1) + 0.5
    k[at, 0, :ONES] = torch.tensor(e4m3_parts(nats * d ** 0.5, ONES))
    v[at] = own * torch.randn(d, generator=g)
    if steps:                      # every second block's values 2^8 smaller
        v *= torch.where(torch.arange(L) // 16 % 2 == at // 16 % 2, 1.0, 2.0 ** -8)[:, None, None]
    q = q.bfloat16().cuda()
    pool, table = cache(sh, k, v)
    o, lse = attend(sh, pool, table, q, L)
    kk, vv = sequence_rows(pool, table[0], L)
    s = (torch.as_tensor(kk[:, 0]) @ q[0, 0].double().cpu()) * sh.softmax_scale
    got = float(torch.softmax(s, 0)[at])
    assert weight / 2 < got < (1 + weight) / 2 + 1e-3, got      # the case is what it says
    assert_attention(o, lse, attention64(q, kk, vv, sh.softmax_scale), inputs.BF16)


@pytest.mark.parametrize("weight", [0.5, 0.9, 0.99, 0.999])
@pytest.mark.parametrize("n,L", [(1, 500), (1, 777), (1, 4096), (1, 32768), (16, 500), (16, 2000), (16, 8320), (16, 32768)])
def test_one_key_takes_most_of_the_weight(n, L, weight):
    """Few rows (6 pairs a kv head) and drafts (96 pairs); the key in the first piece and in a later one."""
    for at in (0, L * 3 // 4):
        peaked_case(256, 6, n, L, weight, at)


@pytest.mark.parametrize("n,G,d", [(1, 1, 64), (2, 8, 128), (2, 5, 32), (5, 6, 64), (32, 8, 128), (1, 40, 128)])
def test_one_key_takes_most_of_the_weight_other_layers(n, G, d):
    for weight in (0.9, 0.99):
        peaked_case(d, G, n, 1500, weight, 700)


@pytest.mark.parametrize("n,L", [(1, 777), (1, 8192), (16, 8320)])
@pytest.mark.parametrize("weight", [0.61, 0.82, 0.99])
def test_values_that_do_not_cancel(n, L, weight):
    """Values with a mean: what a lost weight takes away adds up instead of averaging out."""
    peaked_case(256, 6, n, L, weight, 0, mean=1.0, own=1.0)


@pytest.mark.parametrize("n,L", [(1, 777), (1, 8192), (16, 8320)])
@pytest.mark.parametrize("weight", [0.61, 0.99])
def test_value_scales_that_differ_between_blocks(n, L, weight):
    for own in (0.02, 1.0):
        peaked_case(256, 6, n, L, weight, 5, mean=1.0, steps=True, own=own)


@pytest.mark.parametrize("n", [1, 16])
@pytest.mark.parametrize("gap", [10, 13])
def test_query_elements_far_apart(n, gap):
    """Half of a row's elements 2^-gap of the other half's, against keys the
    other way round, so that both halves of a score count alike."""
    d, L = 256, 600
    sh = AttnShape(6, 1, d, 64, scale=2.0 ** 7 * d ** -0.5)
    g = torch.Generator().manual_seed(gap)
    q, k, v = torch.randn(n, 6, d, generator=g), torch.randn(L, 1, d, generator=g), torch.randn(L, 1, d, generator=g)
    q[..., d // 2:] *= 2.0 ** -gap
    k[..., :d // 2] *= 2.0 ** -7
    k[..., d // 2:] *= 2.0 ** (gap - 7)
    q = q.bfloat16().cuda()
    pool, table = cache(sh, k, v)
    o, lse = attend(sh, pool, table, q, L)
    kk, vv = sequence_rows(pool, table[0], L)
    assert_attention(o, lse, attention64(q, kk, vv, sh.softmax_scale), inputs.BF16)


@pytest.mark.parametrize("n", [1, 16])
def test_scores_that_keep_growing(n):
    """Each tile's scores lie 6 above the one's before, so that the reference of
    every row moves with every tile, and the last keys decide."""
    d, L = 128, 1000
    sh = AttnShape(6, 1, d, 64, scale=d ** -0.5)
    g = torch.Generator().manual_seed(n)
    q, k, v = torch.randn(n, 6, d, generator=g), torch.randn(L, 1, d, generator=g), torch.randn(L, 1, d, generator=g)
    q[..., 0] = 1.0
    k[:, 0, 0] = (torch.arange(L) // 128 * 6.0) * d ** 0.5
    q = q.bfloat16().cuda()
    pool, table = cache(sh, k, v)
    o, lse = attend(sh, pool, table, q, L)
    kk, vv = sequence_rows(pool, table[0], L)
    assert_attention(o, lse, attention64(q, kk, vv, sh.softmax_scale), inputs.BF16)


@pytest.mark.parametrize("d,G,dtype", [(64, 3, inputs.BF16), (128, 4, inputs.BF16), (256, 6, inputs.BF16), (96, 2, inputs.BF16),
                                       (32, 2, inputs.F32)])
@pytest.mark.parametrize("weight", [0.9, 0.999])
def test_prefill_one_key_takes_most_of_the_weight(d, G, dtype, weight):
    """The same over plain rows: every row of a prompt sees the first key, whose
    values are small."""
    T = 700
    sh = AttnShape(G, 1, d, 16, dtype=dtype)
    g = torch.Generator().manual_seed(d)
    q, k, v = (torch.randn(T, h, d, generator=g) for h in (G, 1, 1))
    q[..., 0], k[..., 0], k[0] = 1.0, 0.0, 0.0
    k[0, 0, 0] = (math.log(weight / (1 - weight)) + math.log(T - 1) + 0.5) * d ** 0.5
    v[0] *= 0.02
    q, k, v = (x.to(sh.torch_dtype()).cuda() for x in (q, k, v))
    cu = torch.tensor([0, T], dtype=torch.int32).cuda()
    o, lse, err = torch.empty_like(q), torch.empty(T, G, device="cuda"), err_word()
    gdn.gdn_attn_prefill(sh, q=q, k=k, v=v, cu_seqlens=cu, cu_kv=cu, o=o, lse=lse, dev_error=err)
    assert err.item() == 0
    assert_attention(o, lse, attention64(q, k, v, sh.softmax_scale), dtype)
