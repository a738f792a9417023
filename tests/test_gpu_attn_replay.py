"""A decode step captured once, with rows for the most that its requests may add, and
replayed over other lengths: each replay is the eager call of those lengths, bit for
bit, and rows behind the last sequence stay."""
import numpy as np
import pytest
import torch

import gated_deltanet_state_gb300 as gdn
from gated_deltanet_state_gb300.inputs import BF16, F32, AttnShape

from attn_harness import err_word, fill_cache, table_for

pytestmark = pytest.mark.gpu

STEPS = [([4, 4, 4, 4], [700, 4000, 35, 129]), ([1, 0, 3, 2], [600, 90, 4096, 3]), ([1, 1, 1, 1], [1, 2049, 0, 512]), ([0, 0, 0, 4], [50, 60, 70, 3000])]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("Hq,d,dt", [(8, 64, BF16), (4, 256, BF16), (24, 128, BF16), (2, 96, F32)])
def test_replays_over_other_lengths(Hq, d, dt, bits):
    sh = AttnShape(Hq, 1, d, 64, dtype=dt, kv_bits=bits)
    N, most, full = 4, 4, [4096] * 4
    pool, table = gdn.KVPool(sh, 4 * 64 + 1, fill=0xFF), table_for(full, 64, 4 * 64 + 1, 1)
    fill_cache(pool, table, full, 2)
    q = torch.randn(N * most, Hq, d, generator=torch.Generator().manual_seed(5)).to(sh.torch_dtype()).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    cu, kv, bt = torch.zeros(N + 1, **i32), torch.zeros(N, **i32), table.cuda()
    o, lse, err = torch.empty_like(q), torch.empty(N * most, Hq, device="cuda"), err_word()
    ws = gdn.workspace_for(gdn.gdn_attn_decode_workspace_size(sh, N, N * most, 4096))

    def call(rows, o, lse, max_q):
        gdn.gdn_attn_decode(sh, pool, q=q[:rows], cu_seqlens=cu, kv_len=kv, block_table=bt, o=o, lse=lse, max_q_len=max_q, max_kv_len=4096,
                            workspace=ws, dev_error=err)

    call(N * most, o, lse, most)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(N * most, o, lse, most)
    for news, lens in STEPS + STEPS[:1]:
        cu.copy_(torch.tensor([0] + np.cumsum(news).tolist(), **i32))
        kv.copy_(torch.tensor(lens, **i32))
        o.fill_(7.0)
        lse.fill_(7.0)
        ws.view(torch.uint8).fill_(0xFF)
        g.replay()
        T = sum(news)
        o1, lse1 = torch.empty_like(o[:T]), torch.empty_like(lse[:T])
        call(T, o1, lse1, max(news))
        assert err.item() == 0 and torch.equal(o[:T], o1) and torch.equal(lse[:T], lse1) and not torch.isnan(o1.float()).any()
        assert bool((o[T:] == 7).all()) and bool((lse[T:] == 7).all())
