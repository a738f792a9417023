"""fp32 rows over the 4-bit cache, to fp32's own precision where the scores are next to 0."""
import pytest
import torch

from gated_deltanet_state_gb300.inputs import F32, AttnShape

from attn4_harness import sequence_rows
from attn_harness import attention64
from test_gpu_attn4 import decode_case, run_decode

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 32), (6, 1, 128), (2, 2, 256), (3, 1, 96)])
@pytest.mark.parametrize("n", [1, 4])
def test_weights_keep_their_bits(Hq, Hkv, d, n):
    """With a scale of 2^-12 a score is about 2^-8 at most, so d products' rounding (24 steps of 2^-23 of a sum of
    d / 1.5, times the scale: 2^-24) is no part of the error.  What is left of a weight, relative to it: exponent and
    offset below 16, rounded twice (2 * 2^-21 ln 2), log2 of V's scale 2^-22 ln 2, ex2 2^-22, the scale's inverse 2^-22,
    two f16 parts 2^-23: in all under 2^-19, in sums and weights 2^-18.  Sums of 300 keys, 16 a step in two parts: 40
    steps of 2^-23, under 2^-17.6.  Together 2^-16.7 A; the bound is 2^-16.5 A, a ninth of what the general one allows."""
    sh = AttnShape(Hq, Hkv, d, 64, dtype=F32, kv_bits=4, scale=2.0 ** -12)
    lens = [2, 5, 17, 300]
    pool, table, q, o, lse = decode_case(sh, lens, [n] * 4, seed=d + n)
    o, lse, err = run_decode(sh, pool, q, [n] * 4, lens, table)
    assert err == 0
    for s, L in enumerate(lens):
        r = slice(n * s, n * s + n)
        k, v = sequence_rows(pool, table[s], L)
        ro, rl, A = attention64(q[r], k, v, sh.softmax_scale)
        got = o[r].double().cpu()
        tol = 2.0 ** -24 * ro.abs() + 2.0 ** -16.5 * A + 1e-30
        assert bool(((got - ro).abs() <= tol).all()), float(((got - ro).abs() / tol).max())
