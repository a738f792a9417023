"""The attention layer's operators together: the example's serving run, and a
prefill whose device waits run out."""
import importlib.util
import os

import pytest
import torch

import gated_deltanet_state_gb300 as gdn
from gated_deltanet_state_gb300.inputs import AttnShape

from attn_harness import err_word

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_example_serves():
    """Every phase within the cache's rounding: e4m3 keeps 4 significant bits, so
    an element is off by up to 2^-4 of itself and by 2.6 % in the root mean
    square.  Values move the outputs by that; keys move the scores of unit
    normal rows by about 0.026 and the weights, so the outputs, by as much.  The
    two together are 3.7 %; bound: 6 %."""
    spec = importlib.util.spec_from_file_location("attention_layer", os.path.join(ROOT, "examples", "attention_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    errors = m.serve()
    assert set(errors) == {"prefill", "decode", "draft"} and all(e < 0.06 for e in errors.values()), errors


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prefill_waits_that_run_out_write_nothing(d):
    """wait_cycles < 0: every device wait of the tensor-core path reports a
    timeout at once; nothing is written, and the next call is as always."""
    sh = AttnShape(4, 2, d, 16)
    g = torch.Generator().manual_seed(d)
    q, k, v = (torch.randn(300, h, d, generator=g).bfloat16().cuda() for h in (4, 2, 2))
    cu = torch.tensor([0, 300], dtype=torch.int32).cuda()

    def call(wait):
        o, err = torch.full((300, 4, d), 7.0, dtype=torch.bfloat16, device="cuda"), err_word()
        gdn.gdn_attn_prefill(sh, q=q, k=k, v=v, cu_seqlens=cu, cu_kv=cu, o=o, dev_error=err, wait_cycles=wait)
        return o, err.item()

    want, err = call(0)
    assert err == 0
    o, err = call(-1)
    assert err == gdn.STATUS_CODE["GDN_ERR_TIMEOUT"] and bool((o == 7).all())
    o, err = call(0)
    assert err == 0 and torch.equal(o, want)
