"""Decode attention over large batches: sequences without keys or without rows
between others, more sequences than one launch takes, few rows and drafts in
one call.  A sequence gives the bits that it gives alone."""
import numpy as np
import pytest
import torch

import gated_deltanet_state_gb300 as gdn
from gated_deltanet_state_gb300 import inputs
from gated_deltanet_state_gb300.inputs import AttnShape

from attn_harness import assert_attention, attention64, err_word, fill_cache, sequence_rows, table_for

pytestmark = pytest.mark.gpu


class Batch:
    def __init__(self, sh, news, lens, seed):
        self.sh, self.news, self.lens = sh, news, lens
        P = sh.page_tokens
        pages = sum(-(-n // P) for n in lens) + 1
        self.pool = gdn.KVPool(sh, pages, fill=0xFF)
        self.table = table_for(lens, P, pages, seed)
        fill_cache(self.pool, self.table, lens, seed)
        g = torch.Generator().manual_seed(seed + 1)
        self.q = torch.randn(sum(news), sh.num_q_heads, sh.head_dim, generator=g).to(sh.torch_dtype()).cuda()
        self.at = np.concatenate([[0], np.cumsum(news)]).tolist()

    def rows(self, s):
        return slice(self.at[s], self.at[s + 1])

    def run(self, seqs):
        i32 = dict(dtype=torch.int32, device="cuda")
        q = torch.cat([self.q[self.rows(s)] for s in seqs])
        news, lens = [self.news[s] for s in seqs], [self.lens[s] for s in seqs]
        o, lse, err = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda"), err_word()
        gdn.gdn_attn_decode(self.sh, self.pool, q=q, cu_seqlens=torch.tensor([0] + np.cumsum(news).tolist(), **i32),
                            kv_len=torch.tensor(lens, **i32), block_table=self.table[list(seqs)].cuda(), o=o, lse=lse,
                            max_q_len=max(max(self.news), 1), max_kv_len=max(lens), dev_error=err)
        assert err.item() == 0
        return o, lse

    def check(self, every):
        N = len(self.news)
        o, lse = self.run(range(N))
        for _ in range(2):
            o2, lse2 = self.run(range(N))
            assert torch.equal(o2, o) and torch.equal(lse2, lse)
        for s in range(N):
            r, L = self.rows(s), self.lens[s]
            if L == 0:
                assert not o[r].any() and bool((lse[r] == -float("inf")).all())
            elif s % every == 0 and self.news[s]:
                o1, lse1 = self.run([s])
                assert torch.equal(o1, o[r]) and torch.equal(lse1, lse[r]), s
                k, v = sequence_rows(self.pool, self.table[s], L)
                ref = attention64(self.q[r], k, v, self.sh.softmax_scale)
                assert_attention(o[r], lse[r], ref, inputs.BF16)


@pytest.mark.parametrize("rows", [1, 2, 16])
def test_many_sequences_without_keys(rows):
    """Runs of them, so that a CTA has several in a row, between sequences with keys."""
    N = 500
    lens = [0 if s % 11 else 40 + 13 * s % 500 for s in range(N)]
    Batch(AttnShape(48, 8, 64, 64), [rows] * N, lens, seed=rows).check(every=33)


@pytest.mark.parametrize("rows", [1, 16])
def test_no_sequence_has_keys(rows):
    Batch(AttnShape(48, 8, 64, 64), [rows] * 400, [0] * 399 + [1], seed=rows).check(every=399)


@pytest.mark.parametrize("N", [257, 600])
def test_more_sequences_than_a_launch_takes(N):
    """0, 1 and 32 rows mixed: both kernels, each launched more than once."""
    news = [(0, 1, 32, 2, 1)[s * 7 % 5] for s in range(N)]
    lens = [(0, 700, 33, 1500, 128, 1)[s * 5 % 6] + s % 3 for s in range(N)]
    Batch(AttnShape(12, 2, 64, 64), news, lens, seed=N).check(every=29)


@pytest.mark.parametrize("G", [1, 16, 24])
def test_more_sequences_than_a_launch_takes_one_row_each(G):
    Batch(AttnShape(G, 1, 64, 64), [1] * 520, [s * 17 % 900 for s in range(520)], seed=G).check(every=37)
