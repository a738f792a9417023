"""Bounded waits of the attention kernels that run out: the call returns, says
so, and the next one is as always.  No fault is made: wait_cycles < 0 has every
wait report at once, and a bound of a few clocks ends waits that would have
been served a moment later."""
import numpy as np
import pytest
import torch

import gated_deltanet_state_gb300 as gdn
from gated_deltanet_state_gb300.inputs import AttnShape

from attn_harness import err_word, fill_cache, table_for

pytestmark = pytest.mark.gpu

TIMEOUT = gdn.STATUS_CODE["GDN_ERR_TIMEOUT"]

# (rows, keys) of each sequence: 6 (row, head) pairs a row and kv head
BATCHES = {
    "few rows, one piece": [(1, 100), (2, 7), (1, 0)],
    "few rows, pieces": [(1, 5000), (2, 700), (1, 31)],
    "drafts, one piece": [(16, 200), (32, 90)],
    "drafts, pieces": [(16, 5000), (24, 9000)],
    "both": [(16, 3000), (1, 4000), (2, 60), (32, 700), (0, 50), (1, 9000)],
}


class Decode:
    def __init__(self, batch, d=128):
        self.sh = AttnShape(12, 2, d, 64)
        news, lens = [n for n, _ in batch], [k for _, k in batch]
        pages = sum(-(-k // 64) for k in lens) + 1
        self.pool = gdn.KVPool(self.sh, pages, fill=0xFF)
        table = table_for(lens, 64, pages, 2)
        fill_cache(self.pool, table, lens, 3)
        self.q = torch.randn(sum(news), 12, d, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
        i32 = dict(dtype=torch.int32, device="cuda")
        self.cu, self.kv = torch.tensor([0] + np.cumsum(news).tolist(), **i32), torch.tensor(lens, **i32)
        self.table, self.top = table.cuda(), (max(news), max(lens))

    def __call__(self, wait=0, err=None):
        o, lse = torch.full_like(self.q, 7.0), torch.full(self.q.shape[:2], 7.0, device="cuda")
        err = err_word() if err is None else err
        gdn.gdn_attn_decode(self.sh, self.pool, q=self.q, cu_seqlens=self.cu, kv_len=self.kv, block_table=self.table, o=o,
                            lse=lse, max_q_len=self.top[0], max_kv_len=self.top[1], wait_cycles=wait, dev_error=err)
        return o, lse, err.item()


@pytest.mark.parametrize("batch", list(BATCHES))
def test_decode_waits_that_run_out_write_nothing(batch):
    call = Decode(BATCHES[batch])
    want, want_lse, err = call()
    assert err == 0
    o, lse, err = call(-1)
    assert err == TIMEOUT and bool((o == 7).all()) and bool((lse == 7).all())
    o, lse, err = call()
    assert err == 0 and torch.equal(o, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("batch", list(BATCHES))
def test_decode_waits_that_run_out_midway(batch):
    """Whatever wait gives up first, the call returns and the context is intact."""
    call = Decode(BATCHES[batch], d=256)
    want, want_lse, err = call()
    assert err == 0
    for wait in (1, 1, 3000, 10000, 30000):
        o, lse, err = call(wait)
        assert err in (0, TIMEOUT)
        assert err == TIMEOUT or (torch.equal(o, want) and torch.equal(lse, want_lse))
    o, lse, err = call()
    assert err == 0 and torch.equal(o, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("batch", list(BATCHES))
def test_decode_goes_by_its_own_run_outs(batch):
    """A code that dev_error holds from an earlier call neither stops this one
    nor hides that its waits have run out."""
    call = Decode(BATCHES[batch])
    want, want_lse, _ = call()
    word = lambda code: torch.tensor([code], dtype=torch.int32, device="cuda")  # noqa: E731
    o, lse, err = call(err=word(TIMEOUT))
    assert err == TIMEOUT and torch.equal(o, want) and torch.equal(lse, want_lse)
    o, lse, err = call(-1, err=word(gdn.STATUS_CODE["GDN_ERR_PAGE_RANGE"]))
    assert err == TIMEOUT and bool((o == 7).all()) and bool((lse == 7).all())


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prefill_reports_a_run_out_over_an_earlier_code(d):
    sh = AttnShape(4, 2, d, 16)
    g = torch.Generator().manual_seed(d)
    q, k, v = (torch.randn(300, h, d, generator=g).bfloat16().cuda() for h in (4, 2, 2))
    cu = torch.tensor([0, 300], dtype=torch.int32).cuda()
    o = torch.full((300, 4, d), 7.0, dtype=torch.bfloat16, device="cuda")
    err = torch.tensor([gdn.STATUS_CODE["GDN_ERR_PAGE_RANGE"]], dtype=torch.int32, device="cuda")
    gdn.gdn_attn_prefill(sh, q=q, k=k, v=v, cu_seqlens=cu, cu_kv=cu, o=o, dev_error=err, wait_cycles=-1)
    assert err.item() == TIMEOUT and bool((o == 7).all())


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prefill_waits_that_run_out_midway(d):
    """Several row tiles a CTA, alone and in pairs; whatever wait gives up
    first, the call returns and the context is intact."""
    sh = AttnShape(6, 2, d, 16)
    lens = [40 + 97 * s % 700 for s in range(30)]
    T = sum(lens)
    g = torch.Generator().manual_seed(d)
    q, k, v = (torch.randn(T, h, d, generator=g).bfloat16().cuda() for h in (6, 2, 2))
    cu = torch.tensor([0] + np.cumsum(lens).tolist(), dtype=torch.int32, device="cuda")

    def call(wait):
        o, err = torch.full_like(q, 7.0), err_word()
        gdn.gdn_attn_prefill(sh, q=q, k=k, v=v, cu_seqlens=cu, cu_kv=cu, o=o, dev_error=err, max_q_len=max(lens),
                             max_kv_len=max(lens), wait_cycles=wait)
        return o, err.item()

    want, err = call(0)
    assert err == 0
    for wait in (1, 1, 3000, 10000, 30000):
        o, err = call(wait)
        assert err in (0, TIMEOUT) and (err == TIMEOUT or torch.equal(o, want))
    o, err = call(0)
    assert err == 0 and torch.equal(o, want)
