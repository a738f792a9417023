"""Decode attention where the rows' total does not tell what each sequence has: a
sequence refused for its rows beside valid ones, and rows behind the last sequence
(a captured step's padding).  Every other row keeps the bits that it has alone."""
import numpy as np
import pytest
import torch

import gated_deltanet_state_gb300 as gdn
from gated_deltanet_state_gb300.inputs import AttnShape

import attn4_harness
import attn_harness
from attn_harness import assert_attention, attention64, err_word, fill_cache, table_for

pytestmark = pytest.mark.gpu

INVALID = gdn.STATUS_CODE["GDN_ERR_INVALID_ARG"]


class Step:
    def __init__(self, sh, news, lens, rows, seed):
        self.sh, self.news, self.lens = sh, news, lens
        P = sh.page_tokens
        pages = sum(-(-n // P) for n in lens) + 1
        self.pool, self.table = gdn.KVPool(sh, pages, fill=0xFF), table_for(lens, P, pages, seed)
        fill_cache(self.pool, self.table, lens, seed)
        g = torch.Generator().manual_seed(seed + 1)
        self.q = torch.randn(rows, sh.num_q_heads, sh.head_dim, generator=g).to(sh.torch_dtype()).cuda()
        self.at = np.concatenate([[0], np.cumsum(news)]).tolist()

    def rows(self, s):
        return slice(self.at[s], self.at[s + 1])

    def run(self, seqs, q, max_q):
        """What the workspace held before is no number."""
        i32 = dict(dtype=torch.int32, device="cuda")
        news, lens = [self.news[s] for s in seqs], [self.lens[s] for s in seqs]
        o, lse, err = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda"), err_word()
        ws = gdn.workspace_for(gdn.gdn_attn_decode_workspace_size(self.sh, len(seqs), q.shape[0], max(lens)))
        ws.view(torch.uint8).fill_(0xFF)
        gdn.gdn_attn_decode(self.sh, self.pool, q=q, cu_seqlens=torch.tensor([0] + np.cumsum(news).tolist(), **i32),
                            kv_len=torch.tensor(lens, **i32), block_table=self.table[list(seqs)].cuda(), o=o, lse=lse,
                            max_q_len=max_q, max_kv_len=max(lens), workspace=ws, dev_error=err)
        return o, lse, err.item()

    def check(self, s, o, lse):
        r, n = self.rows(s), self.news[s]
        o1, lse1, err = self.run([s], self.q[r], n)
        assert err == 0 and torch.equal(o[r], o1) and torch.equal(lse[r], lse1)
        rows = (attn4_harness if self.sh.kv_bits == 4 else attn_harness).sequence_rows
        k, v = rows(self.pool, self.table[s], self.lens[s])
        assert_attention(o[r], lse[r], attention64(self.q[r], k, v, self.sh.softmax_scale), self.sh.dtype)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("G,news,max_q", [(8, [1, 3], 2), (8, [1, 5], 3), (4, [1, 8, 3], 4), (1, [2, 18], 10)])
def test_a_neighbour_with_too_many_rows(bits, G, news, max_q):
    """As many rows in all as if each sequence had the most."""
    st = Step(AttnShape(G, 1, 64, 512, kv_bits=bits), news, [100000, 50, 700][:len(news)], sum(news), seed=G)
    assert sum(news) == len(news) * max_q
    o, lse, err = st.run(range(len(news)), st.q, max_q)
    assert err == INVALID
    for s, n in enumerate(news):
        if n > max_q:
            assert bool((o[st.rows(s)] == 7).all()) and bool((lse[st.rows(s)] == 7).all())
        else:
            st.check(s, o, lse)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("G,news,max_q,padded", [(8, [3, 1, 2], 3, 9), (8, [1, 1], 2, 4), (8, [0, 1, 0, 2], 4, 16), (4, [1, 1, 1], 5, 15),
                                                 (8, [1, 1], 1, 5), (24, [1, 2], 2, 4)])
def test_rows_behind_the_last_sequence(bits, G, news, max_q, padded):
    st = Step(AttnShape(G, 1, 64, 512, kv_bits=bits), news, [300, 90000, 20, 1500][:len(news)], padded, seed=G + padded)
    o, lse, err = st.run(range(len(news)), st.q, max_q)
    assert err == 0 and bool((o[sum(news):] == 7).all()) and bool((lse[sum(news):] == 7).all())
    for s, n in enumerate(news):
        if n:
            st.check(s, o, lse)
