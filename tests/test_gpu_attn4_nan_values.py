"""A NaN in V and the log-sum-exp over the 4-bit cache: outputs of the rows that see it
are NaN, lse, which V is no part of, is what it is."""
import math

import pytest
import torch

import gated_deltanet_state_gb300 as gdn
from gated_deltanet_state_gb300.inputs import BF16, F32, AttnShape

from attn4_harness import sequence_rows
from attn_harness import attention64, err_word
from test_gpu_attn4 import decode_case, run_decode

pytestmark = pytest.mark.gpu


def nan_value(sh, pool, table, token, head, k=None):
    """Token `token` of the first sequence becomes k (or zeros) and zeros, but for a NaN in V of one head."""
    x, y = (torch.zeros(1, sh.num_kv_heads, sh.head_dim) for _ in range(2))
    if k is not None:
        x[0, head] = k
    y[0, head, 5] = math.nan
    slot = int(table[0, token // sh.page_tokens]) * sh.page_tokens + token % sh.page_tokens
    gdn.gdn_kv_append(sh, pool, k=x.to(sh.torch_dtype()).cuda(), v=y.to(sh.torch_dtype()).cuda(),
                      slot_map=torch.tensor([slot]).cuda(), dev_error=err_word())


def check_lse(got, q, k, v, sh):
    got, want = got.double().cpu(), attention64(q, k, v, sh.softmax_scale)[1]
    some = torch.isfinite(want)                      # (rows without keys: -inf)
    assert torch.equal(got[~some], want[~some])
    assert bool(((got - want).abs()[some] <= 1e-4 * (1 + want.abs()[some])).all()), (got, want)


@pytest.mark.parametrize("Hq,Hkv,d,dt", [(4, 2, 64, BF16), (16, 2, 128, BF16), (12, 2, 256, BF16), (4, 2, 96, F32)])
@pytest.mark.parametrize("n,L", [(1, 300), (2, 90), (9, 700), (20, 40), (1, 5000), (16, 5000), (32, 20)])
@pytest.mark.parametrize("back", [0, 1, 130])
def test_lse_beside_a_nan_in_v(Hq, Hkv, d, dt, n, L, back):
    token = max(L - 1 - back, 0)
    sh = AttnShape(Hq, Hkv, d, 64, dtype=dt, kv_bits=4)
    pool, table, q, o, lse = decode_case(sh, [L, 60], [n, 1], seed=n + L)
    nan_value(sh, pool, table, token, 1)
    o2, lse2, err = run_decode(sh, pool, q, [n, 1], [L, 60], table)
    assert err == 0
    k, v = sequence_rows(pool, table[0], L)
    check_lse(lse2[:n], q[:n], k, v, sh)
    G = Hq // Hkv
    sees = torch.arange(L - n, L) >= token
    assert torch.isnan(o2[:n][sees][:, G:].float()).all() and not torch.isnan(o2[:n][sees][:, :G].float()).any()
    assert torch.equal(o2[:n][~sees], o[:n][~sees]) and torch.equal(lse2[:n][~sees], lse[:n][~sees])
    assert torch.equal(o2[n:], o[n:]) and torch.equal(lse2[n:], lse[n:])


@pytest.mark.parametrize("n,dt", [(1, BF16), (16, BF16), (1, F32)])
def test_a_nan_in_v_with_no_weight(n, dt):
    """Its key's score is hundreds below the others': the weight is 0, and 0 times NaN is NaN."""
    sh = AttnShape(2, 1, 64, 64, dtype=dt, kv_bits=4)
    pool, table, q, o, lse = decode_case(sh, [200], [n], seed=3)
    q = q.abs() + 0.5
    nan_value(sh, pool, table, 70, 0, k=torch.full((64,), -100.0))
    o, lse, err = run_decode(sh, pool, q, [n], [200], table)
    k, v = sequence_rows(pool, table[0], 200)
    assert err == 0 and torch.isnan(o.float()).all()
    check_lse(lse, q, k, v, sh)


@pytest.mark.parametrize("n,dt", [(1, BF16), (16, BF16), (1, F32)])
def test_nothing_but_nan_in_v(n, dt):
    sh = AttnShape(2, 1, 64, 64, dtype=dt, kv_bits=4)
    pool, table, q, _, _ = decode_case(sh, [150], [n], seed=4)
    pool.v_scales().fill_(255)
    o, lse, err = run_decode(sh, pool, q, [n], [150], table)
    k, v = sequence_rows(pool, table[0], 150)
    assert err == 0 and torch.isnan(o.float()).all()
    check_lse(lse, q, k, v, sh)
