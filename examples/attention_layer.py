"""One attention layer of a hybrid model through a short serving run.

Two prompts are prefilled in chunks (the second one starts from a cached
prefix: its first pages are the first prompt's), then both decode a few tokens,
then both verify a draft of several rows.  Every step is what a server does
for the layer, on the GPU from request lengths to outputs:

    gdn_kv_tables    block tables, slots and positions of the step
    gdn_kv_append    the step's K and V rows into the 8-bit cache
    gdn_kv_gather    (prefill) the keys so far back as rows
    gdn_attn_prefill / gdn_attn_decode

Run it with `python examples/attention_layer.py`; it prints how far each
phase's outputs are from attention in plain torch over unquantised keys.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gated_deltanet_state_gb300 as gdn  # noqa: E402
from gated_deltanet_state_gb300.inputs import AttnShape  # noqa: E402


class Layer:
    """Cache and tables of one layer, and what the host keeps of them."""

    def __init__(self, shape: AttnShape, num_pages: int, max_seqs: int, max_pages: int):
        i32 = dict(dtype=torch.int32, device="cuda")
        self.shape, self.num_pages = shape, num_pages
        self.pool = gdn.KVPool(shape, num_pages)
        self.free = torch.arange(num_pages, **i32)
        self.table = torch.full((max_seqs, max_pages), -1, **i32)
        self.kv_len = torch.zeros(max_seqs, **i32)
        self.len_host = [0] * max_seqs
        self.error = torch.zeros(1, **i32)

    def step(self, new: list[int], qkv: torch.Tensor) -> torch.Tensor:
        """New rows of every request (qkv: q heads | k heads | v heads) through the layer."""
        sh, n, T = self.shape, len(new), sum(new)
        i32 = dict(dtype=torch.int32, device="cuda")
        cu, cu_kv, out_len, taken = (torch.empty(k, **i32) for k in (n + 1, n + 1, n, 1))
        pos, slot = (torch.empty(T, dtype=torch.int64, device="cuda") for _ in range(2))
        gdn.gdn_kv_tables(sh, self.num_pages, kv_len=self.kv_len, new_len=torch.tensor(new, **i32), free_pages=self.free,
                          block_table=self.table, cu_seqlens=cu, cu_kv=cu_kv, kv_len_out=out_len, positions=pos,
                          slot_map=slot, pages_taken=taken, dev_error=self.error)
        lens = [a + b for a, b in zip(self.len_host, new)]
        P = sh.page_tokens
        took = sum(-(-b // P) - (-(-a // P)) for a, b in zip(self.len_host, lens))   # what `taken` says, known here too
        self.free, self.kv_len, self.len_host = self.free[took:].contiguous(), out_len, lens
        hq, hkv, d = sh.num_q_heads, sh.num_kv_heads, sh.head_dim
        q = qkv[:, :hq * d].unflatten(1, (hq, d))
        k, v = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)), qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
        gdn.gdn_kv_append(sh, self.pool, k=k, v=v, slot_map=slot, dev_error=self.error)
        o = torch.empty(T, hq, d, dtype=qkv.dtype, device="cuda")
        if max(new) <= gdn.ATTN_DECODE_ROWS:
            gdn.gdn_attn_decode(sh, self.pool, q=q, cu_seqlens=cu, kv_len=self.kv_len, block_table=self.table, o=o,
                                max_q_len=max(new), max_kv_len=max(lens), dev_error=self.error)
        else:
            kk, vv = (torch.empty(sum(lens), hkv, d, dtype=qkv.dtype, device="cuda") for _ in range(2))
            gdn.gdn_kv_gather(sh, self.pool, cu_kv=cu_kv, block_table=self.table, k=kk, v=vv, dev_error=self.error)
            gdn.gdn_attn_prefill(sh, q=q, k=kk, v=vv, cu_seqlens=cu, cu_kv=cu_kv, o=o, max_q_len=max(new),
                                 max_kv_len=max(lens), dev_error=self.error)
        return o

    def share_prefix(self, src: int, dst: int, tokens: int) -> None:
        """Request dst starts from the first `tokens` (whole pages) of src's cache."""
        pages = tokens // self.shape.page_tokens
        self.table[dst, :pages] = self.table[src, :pages]
        self.kv_len[dst] = tokens
        self.len_host[dst] = tokens


def plain(q, k, v, scale):
    """Causal attention of rows q [n, Hq, d] over keys [L, Hkv, d] in fp32."""
    n, L, g = q.shape[0], k.shape[0], q.shape[1] // k.shape[1]
    k, v = k.float().repeat_interleave(g, 1), v.float().repeat_interleave(g, 1)
    s = torch.einsum("nhd,lhd->hnl", q.float(), k) * scale
    s.masked_fill_(torch.arange(L, device=q.device)[None] > torch.arange(L - n, L, device=q.device)[:, None], float("-inf"))
    return torch.einsum("hnl,lhd->nhd", s.softmax(-1), v)


def serve(shape: AttnShape = AttnShape(12, 2, 128, page_tokens=128), seed: int = 0) -> dict:
    """The run; {phase: relative error of its outputs against plain attention}."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    hq, hkv, d = shape.num_q_heads, shape.num_kv_heads, shape.head_dim
    layer = Layer(shape, num_pages=64, max_seqs=2, max_pages=32)
    rows = [torch.empty(0, (hq + 2 * hkv) * d, device="cuda") for _ in range(2)]
    errors = {}

    def step(name, new):
        for s in range(2):
            rows[s] = torch.cat([rows[s], torch.randn(new[s], (hq + 2 * hkv) * d, generator=g, device="cuda").bfloat16().float()])
        o = layer.step(new, torch.cat([rows[s][len(rows[s]) - new[s]:] for s in range(2)]).to(shape.torch_dtype()))
        want = []
        for s in range(2):
            x = rows[s].unflatten(1, (hq + 2 * hkv, d))
            want.append(plain(x[len(x) - new[s]:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], shape.softmax_scale))
        want = torch.cat(want)
        errors[name] = max(errors.get(name, 0.0), float((o.float() - want).norm() / want.norm()))

    step("prefill", [700, 0])                       # the first prompt's first chunk
    layer.share_prefix(0, 1, 512)                   # a hit: four whole pages of it
    rows[1] = rows[0][:512]
    step("prefill", [333, 401])                     # the rest of both
    for _ in range(4):
        step("decode", [1, 1])
    step("draft", [8, 5])                           # rows to verify
    assert layer.error.item() == 0
    return errors


if __name__ == "__main__":
    for phase, e in serve().items():
        print(f"{phase:8s} relative error against unquantised attention {e:.4f}")
