"""The attention layers' cache: a step's tables, the append of rows into 8-bit
blocks and the read-back, against plain restatements of include/gdn.h."""
import math

import numpy as np
import pytest
import torch

import gated_deltanet_state_gb300 as gdn
from gated_deltanet_state_gb300 import inputs
from gated_deltanet_state_gb300.inputs import AttnShape

from attn_harness import cache_rows, e4m3_values, err_word, fill_cache, sequence_rows, slots_for, table_for

pytestmark = pytest.mark.gpu

PAGE_RANGE = gdn.STATUS_CODE["GDN_ERR_PAGE_RANGE"]


# ------------------------------------------------------------------ tables

def tables_ref(P, num_pages, kv, new, free, table, T):
    table = [list(r) for r in table]
    cu, cukv, out, pos, slot, at, taken, ok_all = [0], [0], [], [], [], 0, 0, True
    for s, (k, a) in enumerate(zip(kv, new)):
        good = k >= 0 and a >= 0 and -(-(k + a) // P) <= len(table[s])
        k, a = max(k, 0), max(a, 0)
        have = -(-k // P)
        need = -(-(k + a) // P) - have if good else 0
        if good and need and at + need > len(free):
            good = False
        first, at = at, at + need
        if good:
            table[s][have:have + need] = free[first:first + need]
            taken += need
        ok_all &= good
        out.append(k + a if good else k)
        cu.append(cu[-1] + a)
        cukv.append(cukv[-1] + out[-1])
        for i in range(a):
            t = k + i
            page = table[s][t // P] if good else -1
            inside = 0 <= page < num_pages
            ok_all &= inside
            pos.append(t)
            slot.append(page * P + t % P if inside else -1)
    pos += [0] * (T - len(pos))
    slot += [-1] * (T - len(slot))
    return table, cu, cukv, out, pos[:T], slot[:T], taken, ok_all


def run_tables(P, num_pages, kv, new, free, table, T):
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    n = len(kv)
    bt = i32(table).reshape(n, -1)
    o32 = lambda k: torch.full((k,), -7, dtype=torch.int32, device="cuda")  # noqa: E731
    o64 = lambda: torch.full((T,), -7, dtype=torch.int64, device="cuda")  # noqa: E731
    cu, cukv, out, pos, slot, taken, err = o32(n + 1), o32(n + 1), o32(n), o64(), o64(), o32(1), err_word()
    sh = AttnShape(2, 1, 16, P)
    for _ in range(2):   # the same call again gives the same answer
        gdn.gdn_kv_tables(sh, num_pages, kv_len=i32(kv), new_len=i32(new), free_pages=i32(free), block_table=bt,
                          cu_seqlens=cu, cu_kv=cukv, kv_len_out=out, positions=pos, slot_map=slot, pages_taken=taken,
                          dev_error=err)
    return [x.tolist() for x in (bt, cu, cukv, out, pos, slot)] + [int(taken), int(err) == 0], int(err)


@pytest.mark.parametrize("n,P,lo,hi,extra", [(1, 16, 1, 1, 0), (3, 16, 0, 40, 5), (256, 896, 1, 1, 0),
                                             (300, 32, 0, 70, 0), (3000, 16, 0, 3, 17), (2, 128, 5000, 9000, 3)])
def test_tables(n, P, lo, hi, extra):
    r = np.random.RandomState(n + P)
    kv, new = r.randint(0, 5 * P, n).tolist(), r.randint(lo, hi + 1, n).tolist()
    width = max(-(-(k + a) // P) for k, a in zip(kv, new)) + 1
    total = sum(-(-(k + a) // P) for k, a in zip(kv, new)) + 4
    perm = r.permutation(total).tolist()
    table, at = [], 0
    for k in kv:
        have = -(-k // P)
        table.append(perm[at:at + have] + [-1] * (width - have))
        at += have
    T = sum(new) + extra
    want = tables_ref(P, total, kv, new, perm[at:], table, T)
    got, _ = run_tables(P, total, kv, new, perm[at:], table, T)
    assert got == list(want)


def test_tables_leave_out_what_does_not_fit():
    P = 16
    kv = [0, 15, -3, 16, 40, 7, 0]
    new = [33, 1, 5, 200, 1, -2, 17]          # too many pages for the row at 3, negative lengths at 2 and 5
    table = [[-1] * 4, [5, -1, -1, -1], [-1] * 4, [6, -1, -1, -1], [7, 8, 99, -1], [4, -1, -1, -1], [-1] * 4]
    want = tables_ref(P, 50, kv, new, [20, 21, 22, 23], table, 300)   # one page short at the last; page 99 outside
    got, err = run_tables(P, 50, kv, new, [20, 21, 22, 23], table, 300)
    assert got == list(want) and err == PAGE_RANGE and not want[-1]


# ------------------------------------------------------------------ append

def quantise(rows, before, old):
    """(codes as values, scale) of a block of one head: old values [off, d] under `before`, then rows [n, d]."""
    fin = np.abs(rows[np.isfinite(rows)])
    top = fin.max() if fin.size else 0.0
    e = -64
    while top / 2.0 ** e > 448 and e < 200:
        e += 1
    scale = max(2.0 ** e, before) if len(old) else 2.0 ** e
    grid = e4m3_values()
    grid = np.sort(grid[np.isfinite(grid)])

    def near(x):
        y = np.clip(x / scale, -448, 448)
        hi = np.searchsorted(grid, y).clip(1, len(grid) - 1)
        a, b = grid[hi - 1], grid[hi]
        step = np.where(np.abs(y) < 2.0 ** -6, 2.0 ** -9, 2.0 ** (np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6))) - 3))
        tie = np.abs((y - a) - (b - y)) == 0
        even = np.round(a / step) % 2 == 0
        r = np.where(tie, np.where(even, a, b), np.where(y - a < b - y, a, b))
        return np.where(np.isnan(y), np.nan, r) * scale

    with np.errstate(invalid="ignore"):
        return np.concatenate([near(old), near(rows)]) if len(old) else near(rows), scale


SHAPES = [(4, 256, inputs.BF16), (8, 128, inputs.BF16), (3, 64, inputs.BF16), (2, 80, inputs.BF16), (1, 16, inputs.F32),
          (2, 32, inputs.F32), (2, 256, inputs.F32), (2, 128, inputs.F32)]


def check_append(sh, lens, news, seed, wide=True, poke=None):
    """Old tokens in one call, the new ones in another; every block against its definition."""
    P = sh.page_tokens
    pages = sum(-(-n // P) for n in lens) + 2
    pool = gdn.KVPool(sh, pages, fill=0xFF)                 # NaN codes and scales all over
    table = table_for(lens, P, pages, seed)
    old = [a - b for a, b in zip(lens, news)]
    fill_cache(pool, table, old, seed, size=0.7)
    before = pool.buf.cpu().numpy().copy()
    held = [sequence_rows(pool, table[s], old[s]) for s in range(len(lens))]
    T, H, d = sum(news), sh.num_kv_heads, sh.head_dim
    g = torch.Generator().manual_seed(seed + 1)
    rows = torch.randn(T, 3 * H * d, generator=g) * torch.exp(torch.randn(T, 1, generator=g))
    if poke is not None:
        poke(rows)
    rows = rows.to(sh.torch_dtype()).cuda()
    k, v = rows[:, H * d:2 * H * d].unflatten(1, (H, d)), rows[:, 2 * H * d:].unflatten(1, (H, d))
    if not wide:
        k, v = k.contiguous(), v.contiguous()
    err = err_word()
    gdn.gdn_kv_append(sh, pool, k=k, v=v, slot_map=slots_for(table, lens, news, P).cuda(), dev_error=err)
    assert err.item() == 0
    sc = {0: pool.k_scales().cpu().numpy(), 1: pool.v_scales().cpu().numpy()}
    was = torch.from_numpy(before).view(torch.float32).numpy()[:, sh.codes_bytes // 2:][:, :2 * H * (P // 16)]
    was = was.reshape(pages, 2, H, P // 16)
    r0 = 0
    for s, n in enumerate(lens):
        now = sequence_rows(pool, table[s], n)
        for which, x in ((0, k), (1, v)):
            x64 = x[r0:r0 + news[s]].double().cpu().numpy()
            for b in range(old[s] // 16 if news[s] else 0, -(-n // 16) if news[s] else 0):
                lo, hi = max(16 * b, old[s]), min(16 * b + 16, n)
                page, j = int(table[s, 16 * b // P]), 16 * b % P // 16
                for h in range(H):
                    o = held[s][which][16 * b:lo, h]
                    want, scale = quantise(x64[lo - old[s]:hi - old[s], h], float(was[page, which, h, j]), o)
                    assert float(sc[which][page, h, j]) == scale
                    np.testing.assert_array_equal(now[which][16 * b:hi, h], want)
            full = old[s] // 16 * 16 if news[s] else old[s]
            np.testing.assert_array_equal(now[which][:full], held[s][which][:full])   # earlier blocks untouched
        r0 += news[s]
    # tokens past a sequence's end keep their bytes (a block's own scale may have moved)
    after = pool.buf.cpu().numpy()
    used = {int(p) for p in table.reshape(-1).tolist() if p >= 0}
    for p in range(pages):
        if p not in used:
            np.testing.assert_array_equal(after[p], before[p])


@pytest.mark.parametrize("H,d,dt", SHAPES)
def test_append(H, d, dt):
    check_append(AttnShape(2 * H, H, d, 48, dtype=dt), [1, 16, 17, 47, 100, 5, 33], [1, 16, 2, 30, 100, 0, 1], seed=H + d)


def test_append_long_prompts_take_the_wide_rows_kernel():
    check_append(AttnShape(2, 1, 32, 64), [4000, 1013], [3990, 513], seed=5, wide=False)


def test_append_infinities_nan_zero_and_tiny_rows():
    def poke(rows):
        rows[0, :] = 0.0
        rows[1, 40] = math.inf
        rows[2, 70] = -math.inf
        rows[3, 50] = math.nan
        rows[20, :] = 1e-38
        rows[21, :] = 3e38
        rows[30:46, :] = 0.0
    check_append(AttnShape(2, 1, 32, 32), [46, 64], [46, 20], seed=9, poke=poke)


def test_append_skips_and_refuses_slots():
    sh = AttnShape(2, 2, 32, 32)
    pool = gdn.KVPool(sh, 2, fill=0)
    k = torch.randn(4, 2, 32).bfloat16().cuda()
    err = err_word()
    gdn.gdn_kv_append(sh, pool, k=k, v=k, slot_map=torch.tensor([-1, 3, 64, -1]).cuda(), dev_error=err)
    assert err.item() == PAGE_RANGE
    kk, vv = cache_rows(pool, 0)
    assert np.abs(kk[3]).sum() > 0 and np.abs(kk[:3]).sum() == 0 and np.abs(kk[4:]).sum() == 0
    assert not pool.buf[1].any()


def test_append_beyond_four_gigabytes():
    sh = AttnShape(4, 4, 256, 896)
    pages = 2500                                            # 4.6 GB
    pool = gdn.KVPool(sh, pages)
    pool.buf[pages - 1].zero_()
    k = torch.randn(3, 4, 256).bfloat16().cuda()
    err = err_word()
    slot = torch.arange(3).cuda() + (pages - 1) * 896 + 893
    gdn.gdn_kv_append(sh, pool, k=k, v=-k, slot_map=slot, dev_error=err)
    kk, vv = cache_rows(pool, pages - 1)
    assert err.item() == 0
    assert np.abs(kk[893:] - k.double().cpu().numpy()).max() < 0.3
    np.testing.assert_array_equal(kk, -vv)


# ------------------------------------------------------------------ gather

@pytest.mark.parametrize("H,d,dt", SHAPES)
def test_gather(H, d, dt):
    sh = AttnShape(H, H, d, 48, dtype=dt)
    lens = [0, 1, 15, 16, 17, 48, 49, 200, 0, 3]
    pages = sum(-(-n // 48) for n in lens) + 1
    pool = gdn.KVPool(sh, pages, fill=0xFF)
    table = table_for(lens, 48, pages, 3)
    fill_cache(pool, table, lens, 4)
    cu = torch.tensor([0] + np.cumsum(lens).tolist(), dtype=torch.int32).cuda()
    k, v = (torch.full((sum(lens), H, d), 7.0, dtype=sh.torch_dtype()).cuda() for _ in range(2))
    err = err_word()
    gdn.gdn_kv_gather(sh, pool, cu_kv=cu, block_table=table.cuda(), k=k, v=v, dev_error=err)
    assert err.item() == 0
    rows = [sequence_rows(pool, table[s], n) for s, n in enumerate(lens)]
    np.testing.assert_array_equal(k.double().cpu().numpy(), np.concatenate([x[0] for x in rows]))
    np.testing.assert_array_equal(v.double().cpu().numpy(), np.concatenate([x[1] for x in rows]))


def test_gather_gives_zeros_for_pages_outside_the_pool():
    sh = AttnShape(1, 1, 32, 16)
    pool = gdn.KVPool(sh, 2, fill=0)
    table = torch.tensor([[0, 7], [-1, 1]], dtype=torch.int32)
    fill_cache(pool, torch.tensor([[0], [1]]), [16, 16], 1)
    k, v = (torch.full((64, 1, 32), 7.0).bfloat16().cuda() for _ in range(2))
    err = err_word()
    gdn.gdn_kv_gather(sh, pool, cu_kv=torch.tensor([0, 32, 64], dtype=torch.int32).cuda(), block_table=table.cuda(), k=k,
                      v=v, dev_error=err)
    assert err.item() == PAGE_RANGE
    assert not k[16:48].any() and not v[16:48].any()
    np.testing.assert_array_equal(k[:16].double().cpu().numpy(), cache_rows(pool, 0)[0])
    np.testing.assert_array_equal(v[48:].double().cpu().numpy(), cache_rows(pool, 1)[1])
