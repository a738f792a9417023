"""Query rows over the cache whose elements are far apart, or far from 1
(bounds: attn_harness.py; over 4 bits the cases' q and K enter exactly)."""
import pytest
import torch

import gated_deltanet_state_gb300 as gdn
from gated_deltanet_state_gb300.inputs import BF16, F32, AttnShape

import attn4_harness
import attn_harness
from attn_harness import assert_attention, attention64, err_word, slots_for, table_for

pytestmark = pytest.mark.gpu


def attend(sh, q, k, v):
    """One sequence of q's rows over k, v, cached; against 64 bits."""
    L, n = k.shape[0], q.shape[0]
    pages = -(-L // sh.page_tokens) + 1
    pool, table, err = gdn.KVPool(sh, pages, fill=0xFF), table_for([L], sh.page_tokens, pages, 2), err_word()
    dt = sh.torch_dtype()
    gdn.gdn_kv_append(sh, pool, k=k.to(dt).cuda(), v=v.to(dt).cuda(), slot_map=slots_for(table, [L], [L], sh.page_tokens).cuda(), dev_error=err)
    q = q.to(dt).cuda()
    o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    gdn.gdn_attn_decode(sh, pool, q=q, cu_seqlens=torch.tensor([0, n], dtype=torch.int32).cuda(),
                        kv_len=torch.tensor([L], dtype=torch.int32).cuda(), block_table=table.cuda(), o=o, lse=lse, max_q_len=n,
                        max_kv_len=L, dev_error=err)
    assert err.item() == 0
    kk, vv = (attn4_harness if sh.kv_bits == 4 else attn_harness).sequence_rows(pool, table[0], L)
    ref = attention64(q, kk, vv, sh.softmax_scale)
    assert bool(torch.isfinite(ref[1]).all())
    assert_attention(o, lse, ref, sh.dtype)
    return kk


@pytest.mark.parametrize("n", [1, 16])
@pytest.mark.parametrize("gap", [10, 14, 17, 22])
@pytest.mark.parametrize("residue", [0, 2, 5, 7])
def test_large_elements_beside_codes_of_zero(n, gap, residue):
    """Every eighth element of a row 2^gap of the others in the same groups of 32, where K is 0: a large
    element times 0 adds nothing, so scores are the small elements', and no error goes with the large ones."""
    L, d = 600, 128
    sh = AttnShape(6, 1, d, 64, kv_bits=4)
    g = torch.Generator().manual_seed(gap + residue)
    q, k, v = torch.randn(n, 6, d, generator=g), torch.randn(L, 1, d, generator=g), torch.randn(L, 1, d, generator=g)
    q[..., residue::8] = 2.0 ** gap * (1 + torch.rand(n, 6, d // 8, generator=g))
    k[..., residue::8] = 0
    kk = attend(sh, q, k, v)
    assert not kk[..., residue::8].any()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("n,dt", [(1, BF16), (4, BF16), (16, BF16), (2, F32)])
@pytest.mark.parametrize("power", [-112, -60, 60, 96, 110, 117, 123])
def test_rows_far_from_one(bits, n, dt, power):
    """q of about 2^power under a scale that brings the scores back to a few units: from the
    smallest to within 2^5 of the largest finite values, products and scores are fp32 numbers."""
    L, d = 300, 64
    g = torch.Generator().manual_seed(abs(power))
    q, k, v = torch.randn(n, 4, d, generator=g), torch.randn(L, 1, d, generator=g), torch.randn(L, 1, d, generator=g)
    # K small where q is large, so that the products are far from overflow; 2^-10 of 1 has scales of its own all the same
    size = 2.0 ** -10 if power > 0 else 1.0
    q.clamp_(-8, 8)
    attend(AttnShape(4, 1, d, 64, dtype=dt, kv_bits=bits, scale=d ** -0.5 * 2.0 ** -power / size), q * 2.0 ** power, k * size, v)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("n,dt", [(1, BF16), (16, BF16), (1, F32), (9, F32)])
def test_the_largest_finite_elements(bits, n, dt):
    """Half of a row's elements at or next to the largest number of the type."""
    L, d, most = 200, 64, torch.finfo(torch.bfloat16 if dt == BF16 else torch.float32).max
    g = torch.Generator().manual_seed(n)
    q, k, v = torch.randn(n, 4, d, generator=g), torch.randn(L, 1, d, generator=g), torch.randn(L, 1, d, generator=g)
    q = (q.double() * 2.0 ** 127.5).clamp(-most, most)
    attend(AttnShape(4, 1, d, 64, dtype=dt, kv_bits=bits, scale=2.0 ** -114), q, k * 2.0 ** -16, v)
