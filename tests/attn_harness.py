"""Shared helpers of the attention layers' tests: the cache read and written
from its definition, attention in 64 bits, and the bounds on the errors.

Bounds, per element, from the arithmetic (u = 2^-8: bf16's relative rounding
bound, A = sum_j p_j |v_j| / sum_j p_j in 64 bits):
  * bf16: the output's own rounding, u |o|, and one rounding of every weight
    to 8 significant bits, at most u A; the fp32 sums and the exponential are
    far below that: u A / 16 covers them;
  * fp32: scores of d products in fp32 carry an error of at most d 2^-24 times
    the products' sizes (about 10 for unit normal rows of d = 256 at scale
    1 / sqrt(d), 2e-4 in the worst case, sqrt(d) smaller for independent
    signs), weights the same relative error: 1e-4 A;
  * lse: the scores' error, 1e-4 (1 + |lse|).
"""
from __future__ import annotations

import math

import numpy as np
import torch

import gated_deltanet_state_gb300 as gdn
from gated_deltanet_state_gb300 import inputs

U = 2.0 ** -8


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 e4m3 codes, from the format's definition."""
    out = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        x = math.nan if e == 15 and m == 7 else (8 + m) * 2.0 ** (e - 10) if e else m * 2.0 ** -9
        out[c] = -x if s else x
    return out


def cache_rows(pool, page: int):
    """K and V [page_tokens, Hkv, d] in 64 bits of one page, by explicit indices."""
    sh = pool.shape
    raw = pool.buf[page].cpu().numpy()
    H, P, d = sh.num_kv_heads, sh.page_tokens, sh.head_dim
    val = e4m3_values()
    t = np.arange(P)
    h, tt, e = np.meshgrid(np.arange(H), t, np.arange(d), indexing="ij")
    blk = h * (P // 16) + tt // 16
    k_at = blk * 16 * d + (tt % 16 // 8) * (d // 16) * 128 + (e // 16) * 128 + (tt % 8) * 16 + e % 16
    v_at = sh.codes_bytes + blk * 16 * d + e * 16 + tt % 16
    scales = raw[2 * sh.codes_bytes:2 * sh.codes_bytes + 2 * 4 * H * (P // 16)].view(np.float32).astype(np.float64)
    ks, vs = scales[:H * (P // 16)], scales[H * (P // 16):]
    k, v = val[raw[k_at]] * ks[blk], val[raw[v_at]] * vs[blk]
    return k.transpose(1, 0, 2), v.transpose(1, 0, 2)


def sequence_rows(pool, table_row, length: int):
    """K and V [length, Hkv, d] of a sequence."""
    P = pool.shape.page_tokens
    parts = [cache_rows(pool, int(table_row[j])) for j in range(-(-length // P))]
    shape = (0, pool.shape.num_kv_heads, pool.shape.head_dim)
    k, v = (np.concatenate([x[i] for x in parts])[:length] if parts else np.zeros(shape) for i in (0, 1))
    return k, v


def attention64(q, k, v, scale):
    """(o, lse, A) of rows q [n, Hq, d] over keys [L, Hkv, d], causal at the end, in 64 bits."""
    q, k, v = (torch.as_tensor(x).double().cpu() for x in (q, k, v))
    n, Hq, d = q.shape
    L, Hkv = k.shape[0], k.shape[1]
    o, A = torch.zeros(n, Hq, d).double(), torch.zeros(n, Hq, d).double()
    lse = torch.full((n, Hq), -math.inf).double()
    if L == 0 or n == 0:
        return o, lse, A
    see = torch.arange(L)[None] <= torch.arange(L - n, L)[:, None]
    some = see.any(1)
    for h in range(Hq):
        g = h // (Hq // Hkv)
        s = torch.where(see, q[:, h] @ k[:, g].T * scale, torch.tensor(-math.inf).double())
        m = torch.where(some, s.amax(1), torch.tensor(0.0).double())
        p = torch.exp(s - m[:, None])
        l = p.sum(1)
        w = p / torch.where(some, l, torch.tensor(1.0).double())[:, None]
        o[:, h], A[:, h] = w @ v[:, g], w @ v[:, g].abs()
        lse[:, h] = torch.where(some, m + l.log(), torch.tensor(-math.inf).double())
    return o, lse, A


def assert_attention(o, lse, ref, dtype):
    ro, rl, A = ref
    o, lse = o.double().cpu(), lse.double().cpu()
    tol = U * ro.abs() + U * (1 + 1 / 16) * A if dtype == inputs.BF16 else 2.0 ** -24 * ro.abs() + 1e-4 * A
    bad = ((o - ro).abs() > tol + 1e-30) | ~torch.isfinite(o)
    assert not bad.any(), (int(bad.sum()), float(((o - ro).abs() / (tol + 1e-30)).max()))
    none = torch.isinf(rl)
    assert torch.equal(none, torch.isinf(lse) & (lse < 0))
    far = (lse - rl).abs()[~none] > 1e-4 * (1 + rl.abs()[~none])
    assert not far.any(), float((lse - rl).abs()[~none].max())


def table_for(lens, page_tokens, num_pages, seed, width=None):
    """Disjoint random pages for every sequence: int32 [N][width], -1 beyond its pages."""
    perm = inputs.permutation(num_pages, seed).tolist()
    need = [-(-n // page_tokens) for n in lens]
    width = width or max(1, max(need))
    rows, at = [], 0
    for n in need:
        rows.append(perm[at:at + n] + [-1] * (width - n))
        at += n
    assert at <= num_pages
    return torch.tensor(rows, dtype=torch.int32)


def slots_for(table, lens, news, page_tokens):
    """Slots of the last news[s] of lens[s] tokens of every sequence."""
    out = []
    for s, (n, m) in enumerate(zip(lens, news)):
        for t in range(n - m, n):
            out.append(int(table[s, t // page_tokens]) * page_tokens + t % page_tokens)
    return torch.tensor(out, dtype=torch.int64)


def err_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def fill_cache(pool, table, lens, seed, size=1.0):
    """Random K / V rows for every sequence, appended in one call; the cache around them stays as it was."""
    sh = pool.shape
    g = torch.Generator().manual_seed(seed)
    T = sum(lens)
    if T == 0:
        return
    k, v = (size * torch.randn(T, sh.num_kv_heads, sh.head_dim, generator=g) for _ in range(2))
    err = err_word()
    gdn.gdn_kv_append(sh, pool, k=k.to(sh.torch_dtype()).cuda(), v=v.to(sh.torch_dtype()).cuda(),
                      slot_map=slots_for(table, lens, lens, sh.page_tokens).cuda(), dev_error=err)
    assert err.item() == 0
