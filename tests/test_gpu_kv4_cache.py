"""The 4-bit cache: append and gather against their definitions, bit for bit
(every step of a code or a scale is exact, so nothing may differ)."""
import math

import numpy as np
import pytest
import torch

import gated_deltanet_state_gb300 as gdn
from gated_deltanet_state_gb300 import inputs
from gated_deltanet_state_gb300.inputs import BF16, F32, AttnShape

import attn4_harness as a4
from attn_harness import err_word, slots_for, table_for

pytestmark = pytest.mark.gpu

PAGE_RANGE = gdn.STATUS_CODE["GDN_ERR_PAGE_RANGE"]

# heads and sizes: (Hq, Hkv, d, dtype)
LAYERS = [(24, 4, 256, BF16), (8, 8, 128, BF16), (3, 3, 96, BF16), (4, 1, 64, BF16), (5, 5, 32, BF16), (2, 2, 224, BF16),
          (4, 2, 32, F32), (6, 3, 128, F32), (1, 1, 256, F32), (3, 3, 160, F32)]


def shape(Hq, Hkv, d, dt, page=48):
    return AttnShape(Hq, Hkv, d, page, dtype=dt, kv_bits=4)


def rows(sh, T, seed, extra=8):
    """K and V rows as slices of wider ones; tokens and channels of different sizes, values on halves among them."""
    g = torch.Generator().manual_seed(seed)
    H, d = sh.num_kv_heads, sh.head_dim
    x = torch.randn(T, 2 * H * d + extra, generator=g)
    x *= torch.exp(2 * torch.randn(T, 1, generator=g))
    x[:, ::7] *= 8
    x[::3] = (x[::3] * 2).round() / 2          # quotients of exactly a half
    x = x.to(sh.torch_dtype()).cuda()
    return x[:, :H * d].unflatten(1, (H, d)), x[:, H * d:2 * H * d].unflatten(1, (H, d))


def append(sh, pool, k, v, slots):
    err = err_word()
    gdn.gdn_kv_append(sh, pool, k=k, v=v, slot_map=torch.as_tensor(slots, dtype=torch.int64).cuda(), dev_error=err)
    return err.item()


def check_append(sh, T_slots, seed, fill=0x5A, change=None, pages=None):
    slots = torch.as_tensor(T_slots, dtype=torch.int64)
    pages = pages or int(slots.max()) // sh.page_tokens + 2
    pool = gdn.KVPool(sh, pages, fill=fill)
    k, v = rows(sh, len(slots), seed)
    if change is not None:
        change(k, v)
    before = pool.buf.cpu().numpy()
    assert append(sh, pool, k, v, slots) == 0
    want = a4.append_pages(before, sh, k, v, slots.tolist())
    got = pool.buf.cpu().numpy()
    assert np.array_equal(got, want), (int((got != want).sum()), np.argwhere(got != want)[:5].tolist())
    return pool


@pytest.mark.parametrize("Hq,Hkv,d,dt", LAYERS)
@pytest.mark.parametrize("lens,news", [([1, 17, 48, 100, 31], [1, 1, 1, 1, 1]), ([50, 130, 16, 9], [50, 90, 16, 9]),
                                       ([40, 45, 33, 7], [3, 2, 17, 5])])
def test_append_bytes(Hq, Hkv, d, dt, lens, news):
    """Single tokens, whole prompts and runs inside blocks; the bytes around them stay."""
    sh = shape(Hq, Hkv, d, dt)
    pages = sum(-(-n // sh.page_tokens) for n in lens) + 1
    table = table_for(lens, sh.page_tokens, pages, d)
    check_append(sh, slots_for(table, lens, news, sh.page_tokens), seed=d + Hq, pages=pages)


@pytest.mark.parametrize("dt", [BF16, F32])
def test_append_many_rows(dt):
    """More rows than a step's: sequences that begin and end inside windows of rows, slots left out."""
    sh = shape(2, 2, 64, dt, page=64)
    lens, news = [900, 700, 333, 450, 64, 5], [900, 601, 333, 450, 63, 5]
    pages = sum(-(-n // 64) for n in lens) + 1
    slots = slots_for(table_for(lens, 64, pages, 4), lens, news, 64)
    slots[1000:1003] = -1
    assert len(slots) > 2048
    check_append(sh, slots, seed=9, pages=pages)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("T", [5, 2100])
def test_append_values_that_are_no_numbers(dt, T):
    """Infinities saturate, a NaN takes the values that share its scale; sizes past every scale, zeros, subnormals."""
    sh = shape(4, 2, 96, dt, page=T // 16 * 16 + 16)

    def change(k, v):
        for x in (k, v):
            x[0, 0, 5], x[0, 1, 40] = math.inf, -math.inf
            x[1, 1, 70] = math.nan
            x[2, 0, 33] = 3e38
            x[2, 1] = 0.0
            x[3, 0] = 1e-39
            x[3, 1, :32] = math.inf
            x[4, 0, 10], x[4, 0, 11] = math.nan, math.inf
            x[4, 1] = 30000.0

    check_append(sh, list(range(3, 3 + T)), seed=3, change=change)


def test_append_every_scale_and_half():
    """Every scale's own limit, and every half between codes, from below and above (fp32)."""
    sh = AttnShape(1, 1, 32, 16, dtype=F32, kv_bits=4)
    val = a4.scale_values()
    rows_ = []
    for b in list(range(0, 255, 5)) + [1, 253, 254]:
        s = np.float32(val[b])
        x = np.array([(j + 0.5) * s for j in range(7)], dtype=np.float32)
        near = np.concatenate([x, np.nextafter(x, np.float32(0)), np.nextafter(x, np.float32(np.inf))])
        for top in (7 * s, np.nextafter(7 * s, np.float32(0)), np.nextafter(7 * s, np.float32(np.inf))):
            r = np.zeros(32, dtype=np.float32)
            r[:21] = near * np.where(np.arange(21) % 2, -1, 1)
            r[:21] = np.clip(r[:21], -top, top)
            r[31] = top
            rows_.append(r)
    x = torch.tensor(np.stack(rows_))[:, None].cuda()
    pool = gdn.KVPool(sh, len(x) // 16 + 1, fill=0)
    before = pool.buf.cpu().numpy()
    assert append(sh, pool, x, x, list(range(len(x)))) == 0
    assert np.array_equal(pool.buf.cpu().numpy(), a4.append_pages(before, sh, x, x, range(len(x))))


def test_append_is_the_same_in_parts():
    """A prompt's rows in one call, in chunks that split blocks, and token by token."""
    sh = shape(6, 3, 128, BF16, page=64)
    k, v = rows(sh, 150, 2)
    pools = [gdn.KVPool(sh, 4, fill=0x11) for _ in range(3)]
    for pool, cuts in zip(pools, ([0, 150], [0, 7, 16, 17, 64, 99, 150], list(range(151)))):
        for a, b in zip(cuts, cuts[1:]):
            assert append(sh, pool, k[a:b], v[a:b], list(range(20 + a, 20 + b))) == 0
    assert torch.equal(pools[0].buf, pools[1].buf) and torch.equal(pools[0].buf, pools[2].buf)


def test_append_pages_out_of_range_and_wide_pool_pages():
    sh = shape(2, 2, 64, BF16, page=32)
    page_bytes = sh.page_bytes + 512
    pool = gdn.KVPool(sh, 3, fill=7, page_bytes=page_bytes)
    k, v = rows(sh, 4, 1)
    before = pool.buf.cpu().numpy()
    assert append(sh, pool, k, v, [5, 40, 96, 1000]) == PAGE_RANGE
    want = a4.append_pages(before, sh, k, v, [5, 40, -1, -1])
    assert np.array_equal(pool.buf.cpu().numpy(), want)


# ------------------------------------------------------------------ gather

def gather(sh, pool, lens, table, T=None):
    T = sum(lens) if T is None else T
    k, v = (torch.full((T, sh.num_kv_heads, sh.head_dim), 7.0, dtype=sh.torch_dtype(), device="cuda") for _ in range(2))
    err = err_word()
    cu = torch.tensor([0] + np.cumsum(lens).tolist(), dtype=torch.int32).cuda()
    gdn.gdn_kv_gather(sh, pool, cu_kv=cu, block_table=table.cuda(), k=k, v=v, dev_error=err)
    return k, v, err.item()


def random_pool(sh, pages, seed):
    """A pool of random bytes: every code and scale, NaN among them."""
    pool = gdn.KVPool(sh, pages)
    g = torch.Generator().manual_seed(seed)
    pool.buf.copy_(torch.randint(0, 256, pool.buf.shape, generator=g, dtype=torch.uint8))
    return pool


@pytest.mark.parametrize("Hq,Hkv,d,dt", LAYERS)
def test_gather_every_byte(Hq, Hkv, d, dt):
    """All codes (0 among them) and scales, ragged lengths, empty sequences: exact in either dtype."""
    sh = shape(Hq, Hkv, d, dt)
    lens = [100, 0, 1, 16, 17, 47, 200, 3]
    pages = sum(-(-n // 48) for n in lens) + 1
    pool, table = random_pool(sh, pages, d), table_for(lens, 48, pages, d)
    k, v, err = gather(sh, pool, lens, table)
    assert err == 0
    want = [a4.sequence_rows(pool, table[s], n) for s, n in enumerate(lens)]
    for got, i in ((k, 0), (v, 1)):
        np.testing.assert_array_equal(got.double().cpu().numpy(), np.concatenate([w[i] for w in want]))


def test_gather_after_append_is_within_half_a_step():
    sh = shape(24, 4, 256, BF16, page=128)
    lens = [300, 77]
    pool, table = gdn.KVPool(sh, 6, fill=0xFF), table_for(lens, 128, 6, 1)
    k, v = rows(sh, 377, 6)
    assert append(sh, pool, k, v, slots_for(table, lens, lens, 128)) == 0
    kk, vv, err = gather(sh, pool, lens, table)
    assert err == 0
    for x, y, m in ((k, kk, 32), (v, vv, 256)):
        x, y = (t.double().unflatten(2, (-1, m)) for t in (x, y))
        # a step is the scale: an eighth above max / 7 at most, or the least scale there is
        step = (x.abs().amax(-1, keepdim=True) / 7 * 1.125).clamp(min=2.0 ** -20)
        assert bool(((x - y).abs() <= step / 2).all())


def test_gather_pages_out_of_range_give_zeros():
    sh = shape(2, 2, 64, BF16, page=32)
    pool, lens = random_pool(sh, 5, 3), [40, 33]
    table = torch.tensor([[1, 99], [-1, 2]], dtype=torch.int32)
    k, v, err = gather(sh, pool, lens, table)
    assert err == PAGE_RANGE
    assert bool((k[32:72] == 0).all()) and bool((v[32:72] == 0).all())
    np.testing.assert_array_equal(k[:32].double().cpu().numpy(), a4.cache_rows(pool, 1)[0])
    np.testing.assert_array_equal(v[72:].double().cpu().numpy(), a4.cache_rows(pool, 2)[1][:1])


def test_gather_leaves_rows_behind_the_last_sequence():
    sh = shape(1, 1, 32, F32, page=16)
    pool = random_pool(sh, 3, 5)
    k, v, err = gather(sh, pool, [20], torch.tensor([[0, 1]], dtype=torch.int32), T=40)
    assert err == 0 and bool((k[20:] == 7).all()) and bool((v[20:] == 7).all())
