"""Calls of the attention layers at the ends of their ranges: a step without
requests, scratch on another stream, the longest lengths, bounds left to the
call."""
import pytest
import torch

import gated_deltanet_state_gb300 as gdn
from gated_deltanet_state_gb300.inputs import BF16, F32, AttnShape

from attn_harness import err_word, fill_cache, table_for

pytestmark = pytest.mark.gpu

INVALID, TIMEOUT = (gdn.STATUS_CODE[c] for c in ("GDN_ERR_INVALID_ARG", "GDN_ERR_TIMEOUT"))


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


@pytest.mark.parametrize("handle", [False, True])
def test_scratch_of_a_call_on_another_stream_is_its_own(handle):
    """A call on a stream that is still busy takes its scratch from the
    allocator; what the current stream allocates and writes meanwhile is other
    memory."""
    sh, L = AttnShape(24, 4, 128, 64), 9000
    pages = -(-L // 64)
    pool = gdn.KVPool(sh, pages, fill=0xFF)
    table = table_for([L], 64, pages, 1)
    fill_cache(pool, table, [L], 1)
    q = torch.randn(1, 24, 128, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    cu, kv, bt = (torch.tensor(x, dtype=torch.int32).cuda() for x in ([0, 1], [L], table.tolist()))
    err = err_word()
    size = gdn.gdn_attn_decode_workspace_size(sh, 1, 1, L)

    def call(stream):
        o = torch.zeros_like(q)
        gdn.gdn_attn_decode(sh, pool, q=q, cu_seqlens=cu, kv_len=kv, block_table=bt, o=o, max_kv_len=L, dev_error=err,
                            stream=stream)
        return o

    want = call(None)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(20_000_000)          # about 10 ms
    o = call(st.cuda_stream if handle else st)
    done = st.record_event()
    while not done.query():
        torch.full((size,), 0x7F, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert torch.equal(o, want) and err.item() == 0


@pytest.mark.parametrize("rows,dtype", [(1, BF16), (16, BF16), (1, F32)])
def test_decode_refuses_lengths_that_its_counts_do_not_hold(rows, dtype):
    """Contexts within a few tiles of 2^31 tokens; the others of the batch are as always."""
    sh = AttnShape(6, 1, 64, 64, dtype=dtype)
    pool = gdn.KVPool(sh, 3, fill=0xFF)
    table = torch.tensor([[0], [1], [2]], dtype=torch.int32)
    fill_cache(pool, table, [64, 64, 64], 2)
    q = torch.randn(3 * rows, 6, 64, generator=torch.Generator().manual_seed(2)).to(sh.torch_dtype()).cuda()
    cu = torch.arange(0, 3 * rows + 1, rows, dtype=torch.int32).cuda()

    def call(lens):
        o, err = torch.full_like(q, 7.0), err_word()
        gdn.gdn_attn_decode(sh, pool, q=q, cu_seqlens=cu, kv_len=torch.tensor(lens, dtype=torch.int32).cuda(),
                            block_table=table.cuda(), o=o, max_q_len=rows, max_kv_len=0x7fffffff, dev_error=err)
        return o.unflatten(0, (3, rows)), err.item()

    want, err = call([64, 64, 64])
    assert err == 0
    for far in (0x7fffffff, 0x7fffffff - 1022):
        o, err = call([64, far, 64])
        assert err == INVALID and bool((o[1] == 7).all()) and torch.equal(o[0], want[0]) and torch.equal(o[2], want[2])


def test_decode_shares_out_more_than_2_31_tiles():
    """256 requests of 64 kv heads over 20 million tokens: every row's pieces
    belong to some CTA.  With every wait run out nothing is computed, each CTA
    only marks the rows of its pieces, and no row is joined."""
    sh = AttnShape(64, 64, 32, 64)
    N, L = 256, 20_000_000
    pool = gdn.KVPool(sh, 1, fill=0)
    q = torch.zeros(N, 64, 32, dtype=torch.bfloat16, device="cuda")
    o, lse, err = torch.full_like(q, 7.0), torch.full((N, 64), 7.0, device="cuda"), err_word()
    ws = gdn.workspace_for(gdn.gdn_attn_decode_workspace_size(sh, N, N, L)).zero_()
    gdn.gdn_attn_decode(sh, pool, q=q, cu_seqlens=torch.arange(N + 1, dtype=torch.int32).cuda(),
                        kv_len=torch.full((N,), L, dtype=torch.int32).cuda(),
                        block_table=torch.full((N, 1), -1, dtype=torch.int32).cuda(), o=o, lse=lse, max_kv_len=L, workspace=ws,
                        wait_cycles=-1, dev_error=err)
    assert err.item() == TIMEOUT and bool((o == 7).all()) and bool((lse == 7).all())


def prefill(sh, q, k, v, lens, **kw):
    cu = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
    o, err = torch.full_like(q, 7.0), err_word()
    gdn.gdn_attn_prefill(sh, q=q, k=k, v=v, cu_seqlens=cu, cu_kv=cu, o=o, dev_error=err, **kw)
    return o, err.item()


def test_prefill_of_65535_prompts_without_a_bound():
    """One token each: every output is its own value row."""
    N, H, G, d = 65535, 4, 8, 16
    sh = AttnShape(H * G, H, d, 16, dtype=F32)
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(N, h, d, generator=g, device="cuda") for h in (H * G, H, H))
    o, err = prefill(sh, q, k, v, [1] * N)
    assert err == 0 and torch.equal(o, v.repeat_interleave(G, 1))


@pytest.mark.parametrize("H,G,d,dtype", [(2, 6, 256, BF16), (4, 4, 128, BF16), (1, 3, 64, BF16), (2, 2, 96, BF16), (2, 2, 32, F32),
                                         (1, 40, 64, BF16)])
@pytest.mark.parametrize("lens", [[37 * s % 201 for s in range(60)], [1] * 40 + [1500] + [0, 1] * 30, [3000], [1] * 300])
def test_prefill_gives_the_same_bits_whatever_bound_it_has(lens, H, G, d, dtype):
    """The longest prompt as the bound, the call's rows (0) and more than those."""
    sh = AttnShape(H * G, H, d, 16, dtype=dtype)
    g = torch.Generator(device="cuda").manual_seed(d)
    T = sum(lens)
    q, k, v = (torch.randn(T, h, d, generator=g, device="cuda").to(sh.torch_dtype()) for h in (H * G, H, H))
    want, err = prefill(sh, q, k, v, lens, max_q_len=max(lens), max_kv_len=max(lens))
    assert err == 0
    for s in (0, len(lens) // 2, len(lens) - 1):           # alone
        a, n = sum(lens[:s]), lens[s]
        if n:
            r = slice(a, a + n)
            o, err = prefill(sh, q[r], k[r], v[r], [n], max_q_len=n)
            assert err == 0 and torch.equal(o, want[r])
    for bound in (0, 50 * T):
        o, err = prefill(sh, q, k, v, lens, max_q_len=bound)
        assert err == 0 and torch.equal(o, want)
    if max(lens) > 1:
        o, err = prefill(sh, q, k, v, lens, max_q_len=max(lens) - 1)
        assert err == INVALID
