"""Prefill over prompts of which every one has values that only some rows may
see and that are not finite, in elements of both CTAs of a pair: each row
tile's notes are cleared before the next one's are made, whichever CTA of the
pair is ahead."""
import math

import numpy as np
import pytest
import torch

import gated_deltanet_state_gb300 as gdn
from gated_deltanet_state_gb300.inputs import AttnShape

from attn_harness import err_word

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,G", [(64, 3), (128, 3), (256, 3), (256, 1), (128, 8)])
def test_notes_of_every_tile_stay_with_it(d, G):
    H = 2
    sh = AttnShape(H * G, H, d, 16)
    lens = [130 + 41 * s % 260 for s in range(150)]
    T = sum(lens)
    g = torch.Generator().manual_seed(d + G)
    q, k, v = (torch.randn(T, h, d, generator=g).bfloat16().cuda() for h in (H * G, H, H))
    cu = torch.tensor([0] + np.cumsum(lens).tolist(), dtype=torch.int32, device="cuda")

    def prefill(v):
        o, err = torch.full_like(q, 7.0), err_word()
        gdn.gdn_attn_prefill(sh, q=q, k=k, v=v, cu_seqlens=cu, cu_kv=cu, o=o, dev_error=err, max_q_len=max(lens),
                             max_kv_len=max(lens))
        assert err.item() == 0
        return o

    want = prefill(v)
    v, a = v.clone(), 0
    for s, n in enumerate(lens):
        for i, bad in enumerate((math.nan, math.inf, -math.inf)):
            p, h, e = a + n - 5 - 31 * i, (s + i) % H, (7 * s + i * d // 3) % d
            v[p, h, e] = bad
            want[p:a + n, h * G:(h + 1) * G, e] = bad
        a += n
    for _ in range(4):
        o = prefill(v)
        same = (o == want) | (torch.isnan(o) & torch.isnan(want))
        assert same.all(), int((~same).sum())
