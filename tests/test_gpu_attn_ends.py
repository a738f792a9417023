"""Calls of the attention layers at the ends of their ranges: a step without
requests, scratch on another stream, the longest lengths, bounds left to the
call."""
import pytest
import torch

import gated_deltanet_state_gb300 as gdn
from gated_deltanet_state_gb300.inputs import AttnShape

from attn_harness import err_word

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("stream", ["current", "other", "handle"])
def test_tables_of_a_step_without_requests(stream):
    """Sums of 0, no pages taken, rows without slots: a caller that drops the
    first *pages_taken free pages drops none."""
    sh = AttnShape(2, 1, 16, 16)
    i32 = lambda *n: torch.full(n, 77, dtype=torch.int32, device="cuda")  # noqa: E731
    i64 = lambda n: torch.full((n,), 77, dtype=torch.int64, device="cuda")  # noqa: E731
    cu, cu_kv, taken, pos, slot, free, err = i32(1), i32(1), i32(1), i64(5), i64(5), i32(9), err_word()
    torch.cuda.synchronize()
    st = {"current": None, "other": torch.cuda.Stream()}.get(stream, torch.cuda.Stream().cuda_stream)
    gdn.gdn_kv_tables(sh, 20, kv_len=i32(0), new_len=i32(0), free_pages=free, block_table=i32(0, 3), cu_seqlens=cu, cu_kv=cu_kv,
                      kv_len_out=i32(0), positions=pos, slot_map=slot, pages_taken=taken, dev_error=err, stream=st)
    torch.cuda.synchronize()
    assert cu.tolist() == [0] and cu_kv.tolist() == [0] and taken.tolist() == [0] and err.item() == 0
    assert pos.tolist() == [0] * 5 and slot.tolist() == [-1] * 5 and free.tolist() == [77] * 9
