"""The 4-bit cache of the attention layers from its definition, in 64 bits, for
the tests: scales by search over all of them, codes by the nearest value, pages
read by explicit indices.  The bounds on attention are attn_harness.py's: the
cache's values enter exactly (7 bits in bf16), so no more rounding is in it.
"""
from __future__ import annotations

import numpy as np
import torch

NAN = 255
GROUP = 32


def scale_values() -> np.ndarray:
    """The value of each scale byte."""
    out = np.array([(8 + b % 8) * 2.0 ** (b // 8 - 23) for b in range(256)])
    out[NAN] = np.nan
    return out


def quantise(x: np.ndarray):
    """Rows [..., m] under one scale each -> codes 1 .. 15 [..., m], bytes [...]."""
    x = np.asarray(x, dtype=np.float64)
    fin = np.isfinite(x)
    top = np.where(fin, np.abs(x), 0.0).max(-1)
    val = scale_values()[:NAN]
    b = np.minimum((7 * val[None] < top.reshape(-1, 1)).sum(1), NAN - 1).reshape(top.shape)
    s = val[b][..., None]
    with np.errstate(invalid="ignore"):
        n = np.minimum(np.floor(np.abs(x) / s + 0.5), 7) * np.sign(x)
    bad = np.isnan(x).any(-1)
    return np.where(bad[..., None], 8, np.nan_to_num(n) + 8).astype(int), np.where(bad, NAN, b)


def _place(sh, h, t):
    """Block index within a page of head h and token t, and the token in it."""
    return h * (sh.page_tokens // 16) + t // 16, t % 16


def addresses(sh):
    """For every (head, token, channel) of a page: byte and shift of K's and V's code, byte of the scales."""
    H, P, d = sh.num_kv_heads, sh.page_tokens, sh.head_dim
    h, t, e = np.meshgrid(np.arange(H), np.arange(P), np.arange(d), indexing="ij")
    blk, tt = _place(sh, h, t)
    codes = H * P * d // 2
    kw = ((blk * (d // 32) + e // 32) * 16 + tt) * 4 + e % 32 // 8          # the word of eight channels
    vw = codes // 4 + (blk * d + e) * 2 + tt // 8                            # the word of eight tokens
    bits = lambda i: 4 * (i // 2) + 16 * (i % 2)  # noqa: E731
    k_at, k_sh = kw * 4 + bits(e % 8) // 8, bits(e % 8) % 8
    v_at, v_sh = vw * 4 + bits(tt % 8) // 8, bits(tt % 8) % 8
    ks = 2 * codes + (blk * (d // 32) + e // 32) * 16 + tt
    vs = 2 * codes + H * P * (d // 32) + blk * 16 + tt
    return k_at, k_sh, v_at, v_sh, ks, vs


def cache_rows(pool, page: int):
    """K and V [page_tokens, Hkv, d] in 64 bits of one page."""
    raw, val = pool.buf[page].cpu().numpy(), scale_values()
    k_at, k_sh, v_at, v_sh, ks, vs = addresses(pool.shape)
    k = ((raw[k_at] >> k_sh & 15).astype(np.float64) - 8) * val[raw[ks]]
    v = ((raw[v_at] >> v_sh & 15).astype(np.float64) - 8) * val[raw[vs]]
    return k.transpose(1, 0, 2), v.transpose(1, 0, 2)


def sequence_rows(pool, table_row, length: int):
    """K and V [length, Hkv, d] of a sequence."""
    P = pool.shape.page_tokens
    parts = [cache_rows(pool, int(table_row[j])) for j in range(-(-length // P))]
    none = np.zeros((0, pool.shape.num_kv_heads, pool.shape.head_dim))
    return tuple(np.concatenate([x[i] for x in parts] + [none])[:length] for i in (0, 1))


def append_pages(pool_bytes: np.ndarray, sh, k: torch.Tensor, v: torch.Tensor, slots) -> np.ndarray:
    """A pool's bytes [pages, page_bytes] after the append of k, v [T, Hkv, d] at slots."""
    out = pool_bytes.copy()
    k_at, k_sh, v_at, v_sh, ks, vs = addresses(sh)
    H, d = sh.num_kv_heads, sh.head_dim
    for row, slot in enumerate(slots):
        if slot < 0:
            continue
        page, t = divmod(int(slot), sh.page_tokens)
        raw = out[page]
        nk, bk = quantise(k[row].double().cpu().numpy().reshape(H, d // GROUP, GROUP))
        nv, bv = quantise(v[row].double().cpu().numpy())
        for at, sft, n in ((k_at, k_sh, nk.reshape(H, d)), (v_at, v_sh, nv)):
            a, s = at[:, t].ravel(), sft[:, t].ravel()
            for half in (0, 4):          # a byte holds two codes: one after another
                m = s == half
                raw[a[m]] = raw[a[m]] & (0xF0 if half == 0 else 0x0F) | (n.ravel()[m] << half).astype(np.uint8)
        raw[ks[:, t, ::GROUP]] = bk
        raw[vs[:, t, 0]] = bv
    return out
