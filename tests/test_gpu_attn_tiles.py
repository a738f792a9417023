"""Attention over many more tiles than CTAs run at once, so that a CTA goes from
one to the next: row tiles of a prefill (some of them empty, some with values
that not every row may see), pieces of drafts' contexts."""
import math

import numpy as np
import pytest
import torch

import gated_deltanet_state_gb300 as gdn
from gated_deltanet_state_gb300 import inputs
from gated_deltanet_state_gb300.inputs import AttnShape

from attn_harness import assert_attention, attention64, err_word, table_for

pytestmark = pytest.mark.gpu


def rows_of(n, heads, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(n, heads, d, generator=g).to(dtype).cuda()


def cu_of(lens):
    return torch.tensor([0] + np.cumsum(lens).tolist(), dtype=torch.int32).cuda()


def prefill(sh, q, k, v, lens):
    o = torch.full((sum(lens), sh.num_q_heads, sh.head_dim), 7.0, dtype=sh.torch_dtype(), device="cuda")
    err = err_word()
    gdn.gdn_attn_prefill(sh, q=q, k=k, v=v, cu_seqlens=cu_of(lens), cu_kv=cu_of(lens), o=o, dev_error=err)
    assert err.item() == 0
    return o


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prefill_values_of_one_tile_do_not_reach_the_next(d):
    """NaN or an infinity near the end of some prompts: its element in the rows
    that see it, and not a bit of anything else, in whichever order tiles run."""
    sh = AttnShape(4, 4, d, 16)
    lens = [200 + 37 * s % 321 for s in range(48)]
    T = sum(lens)
    q, k, v = (rows_of(T, 4, d, torch.bfloat16, d + i) for i in range(3))
    want = prefill(sh, q, k, v, lens)
    v, a = v.clone(), 0
    for s, n in enumerate(lens):
        p, bad = a + n - 60 + s, (math.nan, math.inf, None, -math.inf)[s % 4]
        if bad is not None:
            v[p, s % 3, (5 * s) % d] = bad
            want[p:a + n, s % 3, (5 * s) % d] = bad
        a += n
    for _ in range(3):
        o = prefill(sh, q, k, v, lens)
        same = (o == want) | (torch.isnan(o) & torch.isnan(want))
        assert same.all(), int((~same).sum())


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prefill_with_mostly_empty_tiles(d):
    """One long prompt among many of one token and of none."""
    sh = AttnShape(6, 2, d, 16)
    lens = [1] * 30 + [1300] + [1, 0] * 25 + [300]
    T = sum(lens)
    q, k, v = (rows_of(T, h, d, torch.bfloat16, d + h) for h in (6, 2, 2))
    o, lse, err = torch.empty_like(q), torch.empty(T, 6, device="cuda"), err_word()
    gdn.gdn_attn_prefill(sh, q=q, k=k, v=v, cu_seqlens=cu_of(lens), cu_kv=cu_of(lens), o=o, lse=lse, dev_error=err)
    assert err.item() == 0
    a = 0
    for n in lens:
        r = slice(a, a + n)
        assert_attention(o[r], lse[r], attention64(q[r], k[r], v[r], sh.softmax_scale), inputs.BF16)
        a += n


@pytest.mark.parametrize("d,rows", [(256, 16), (128, 5), (64, 32)])
def test_drafts_in_many_pieces_keep_their_bits(d, rows):
    """Drafts over contexts of many pieces: in a batch as alone, time after time."""
    sh = AttnShape(24, 4, d, 128)
    lens = [900 + 613 * s % 7000 for s in range(24)]
    N, width = len(lens), 64
    pages = sum(-(-n // 128) for n in lens)
    pool = gdn.KVPool(sh, pages, fill=0xFF)
    table = table_for(lens, 128, pages, 3, width)
    T = sum(lens)
    k, v = (rows_of(T, 4, d, torch.bfloat16, i) for i in (1, 2))
    t = torch.cat([torch.arange(n) for n in lens])
    s = torch.repeat_interleave(torch.arange(N), torch.tensor(lens))
    slots = table[s, t // 128].long() * 128 + t % 128
    err = err_word()
    gdn.gdn_kv_append(sh, pool, k=k, v=v, slot_map=slots.cuda(), dev_error=err)
    q = rows_of(N * rows, 24, d, torch.bfloat16, 3)

    def decode(seqs, top):
        x = torch.cat([q[i * rows:(i + 1) * rows] for i in seqs]).contiguous()
        o = torch.full_like(x, 7.0)
        gdn.gdn_attn_decode(sh, pool, q=x, cu_seqlens=cu_of([rows] * len(seqs)),
                            kv_len=torch.tensor([lens[i] for i in seqs], dtype=torch.int32).cuda(),
                            block_table=table[list(seqs)].cuda(), o=o, max_q_len=rows, max_kv_len=top, dev_error=err)
        return o

    alone = torch.cat([decode([i], lens[i]) for i in range(N)])
    for _ in range(4):
        assert torch.equal(decode(range(N), max(lens)), alone)
    assert err.item() == 0
