"""The joins of pieces over the 4-bit cache: the one of a few rows and the other give a
row the same bits, at every number of a head's channels and in either dtype."""
import pytest

from gated_deltanet_state_gb300.inputs import BF16, F32, AttnShape

from test_gpu_attn4_batches import Batch

pytestmark = pytest.mark.gpu

# rows a call has at most for the join of a few: 2,400 over heads and parts of 32 channels
@pytest.mark.parametrize("Hq,Hkv,d,dt,n,others", [(2, 1, 96, BF16, 1, 420), (2, 1, 256, BF16, 1, 160), (4, 1, 256, BF16, 2, 60),
                                                  (4, 2, 128, F32, 1, 160), (2, 1, 32, F32, 3, 420), (9, 1, 160, BF16, 1, 60)])
@pytest.mark.parametrize("L", [38000, 66000])
def test_either_join_gives_the_same_bits(Hq, Hkv, d, dt, n, others, L):
    """A context of 33 or 65 pieces, joined by itself and in a batch of many rows."""
    most = 2400 // (Hq * -(-d // 32) * n)
    assert 1 <= most < 1 + others
    Batch(AttnShape(Hq, Hkv, d, 512, dtype=dt, kv_bits=4), [n] + [1] * others, [L] + [17] * others, seed=d).check(every=1 + others // 2)
