"""Calls from several host threads on streams of their own, whose shapes need different
amounts of shared memory in the same kernels: every launch goes through, with the
results of a call alone."""
import threading

import pytest
import torch

import gated_deltanet_state_gb300 as gdn
from gated_deltanet_state_gb300 import attention
from gated_deltanet_state_gb300.inputs import F32, AttnShape

from attn_harness import err_word, fill_cache, table_for

pytestmark = pytest.mark.gpu


def direct(call, name):
    """The C entry with the arguments that the binding's call gives it, on a stream: the interpreter's
    own work between two calls would leave the entries themselves one after another."""
    lib, got = gdn.load_library(), []

    class Note:
        def __getattr__(self, key):
            def take(*args):
                got.append(args)
                return 0
            return take if key == name else getattr(lib, key)

    real = attention.load_library
    attention.load_library = Note
    try:
        call()
    finally:
        attention.load_library = real
    args, entry = got[0], getattr(lib, name)

    def run(stream):
        st = entry(*args[:-1], stream.cuda_stream)
        if st:
            raise RuntimeError(f"{name}: {st}")
    run.keep = call              # (and with it the tensors)
    return run


def decode_call(sh, n, L):
    pages = -(-L // sh.page_tokens) + 1
    pool, table = gdn.KVPool(sh, pages, fill=0), table_for([L], sh.page_tokens, pages, 1)
    fill_cache(pool, table, [L], 2)
    q = torch.randn(n, sh.num_q_heads, sh.head_dim, generator=torch.Generator().manual_seed(3)).to(sh.torch_dtype()).cuda()
    o, err = torch.zeros_like(q), err_word()
    ws = gdn.workspace_for(gdn.gdn_attn_decode_workspace_size(sh, 1, n, L))
    kw = dict(q=q, cu_seqlens=torch.tensor([0, n], dtype=torch.int32).cuda(), kv_len=torch.tensor([L], dtype=torch.int32).cuda(),
              block_table=table.cuda(), o=o, max_q_len=n, max_kv_len=L, workspace=ws, dev_error=err)
    return direct(lambda: gdn.gdn_attn_decode(sh, pool, **kw), "gdn_attn_decode"), o


def prefill_call(sh, L):
    g = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn(L, h, sh.head_dim, generator=g).to(sh.torch_dtype()).cuda() for h in (sh.num_q_heads, sh.num_kv_heads, sh.num_kv_heads))
    o, cu = torch.zeros_like(q), torch.tensor([0, L], dtype=torch.int32).cuda()
    kw = dict(q=q, k=k, v=v, cu_seqlens=cu, cu_kv=cu, o=o, dev_error=err_word())
    return direct(lambda: gdn.gdn_attn_prefill(sh, **kw), "gdn_attn_prefill"), o


CASES = {
    "4 bits, few rows": [lambda d=d: decode_call(AttnShape(4, 1, d, 64, kv_bits=4), 1, 200) for d in (160, 256)],
    "4 bits": [lambda d=d: decode_call(AttnShape(4, 1, d, 64, kv_bits=4), 20, 200) for d in (32, 256)],
    "4 bits, fp32": [lambda d=d: decode_call(AttnShape(4, 1, d, 64, dtype=F32, kv_bits=4), 1, 200) for d in (32, 256)],
    "8 bits, few rows": [lambda d=d: decode_call(AttnShape(4, 1, d, 64), 1, 200) for d in (32, 256)],
    "8 bits": [lambda d=d: decode_call(AttnShape(20, 1, d, 64), 2, 200) for d in (32, 256)],
    "prefill, fp32": [lambda d=d: prefill_call(AttnShape(2, 1, d, 64, dtype=F32), 70) for d in (144, 256)],
}


@pytest.mark.parametrize("case", list(CASES))
def test_shapes_of_different_sizes_at_once(case):
    calls, errors = [make() for make in CASES[case] * 2], []
    for call, _ in calls:
        call(torch.cuda.current_stream())
    torch.cuda.synchronize()
    want = [o.clone() for _, o in calls]

    start = threading.Barrier(len(calls))

    def work(call):
        try:
            stream = torch.cuda.Stream()
            start.wait()
            for _ in range(6000):
                call(stream)
            stream.synchronize()
        except Exception as e:  # noqa: BLE001 - reported by the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(call,)) for call, _ in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors[0]
    assert all(torch.equal(o, x) for (_, o), x in zip(calls, want))
