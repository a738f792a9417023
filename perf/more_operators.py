"""The attention layers' cache in 4 bits: its operators' cases.

A cache of 4 bits a value holds twice the requests of the 8-bit one in the
same pages.  Three operators carry it, the 4-bit forms of the attention
layers' own:

  append   new K / V rows into the paged 4-bit cache
  gather   a cached prefix back as plain K / V rows
  decode   attention of 1 to 32 new rows a request over the 4-bit cache

`run` makes one pass of one of them; `own` picks the engine's kernels or the
plain form.

The cache: a value is (n - 8) * scale with n = 1 .. 15.  K has a scale for each
32 channels of a token and head (a few channels of K are much larger than the
others), V one for a token and head.  A scale is a byte b: (8 + b % 8) *
2^(b // 8 - 23); 255 stands for NaN.  It is the least with 7 * scale >= the
largest magnitude it covers.  A page holds `page` tokens of every kv head:

  K codes   [hkv][page/16][d/32][16 tokens][16 bytes: 32 channels]
  V codes   [hkv][page/16][d][8 bytes: 16 tokens]
  K scales  [hkv][page/16][d/32][16 tokens]
  V scales  [hkv][page/16][16 tokens]
  padding up to a multiple of 256 bytes

Eight codes of consecutive channels (K) or tokens (V) are a little-endian
32-bit word: element 2 i in bits 4 i .. 4 i + 3, element 2 i + 1 in bits
16 + 4 i .. 19 + 4 i.
"""
import math
import random

import torch

own = False

BLOCK = 16          # tokens of a block
GROUP = 32          # channels of K that share a scale
NAN = 255           # the scale byte of NaN


# ------------------------------------------------------------------ cases

def _case(name, op, **kw):
    c = dict(op=op, hq=24, hkv=4, d=256, page=896, f32=False, n=1, lo=1, hi=1, prefix_lo=0, prefix_hi=0, mix=1)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # the K / V rows of one decode step: single tokens into blocks that are partly filled
        _case("append_decode_256", "append", n=256, lo=1, hi=1, prefix_lo=0, prefix_hi=127, page=128, mix=21),
        # the rows of ragged prompts, some continuing inside a block
        _case("append_prompts_5", "append", n=5, lo=3000, hi=9000, prefix_lo=0, prefix_hi=500, mix=22),
        # a small fp32 model's prompts of odd lengths
        _case("append_f32_9", "append", n=9, lo=1, hi=1000, prefix_lo=0, prefix_hi=50, hq=4, hkv=2, d=32, page=64, f32=True, mix=23),
        # the cached prefix of two long requests, read back before their next chunk
        _case("gather_prefix_2", "gather", n=2, lo=57344, hi=114688, mix=24),
        # short prefixes of odd lengths in small pages, one of them empty, narrow heads
        _case("gather_ragged_19", "gather", n=19, lo=0, hi=4001, hq=32, hkv=8, d=128, page=16, mix=25),
        # one request's next token over a short context: latency
        _case("decode_1_short", "decode", n=1, lo=1, hi=1, prefix_lo=777, prefix_hi=777, mix=26),
        # one request's next token over the longest context: its keys spread over the card
        _case("decode_1_long", "decode", n=1, lo=1, hi=1, prefix_lo=229375, prefix_hi=229375, mix=27),
        # a full decode batch over ragged contexts
        _case("decode_256_ragged", "decode", n=256, lo=1, hi=1, prefix_lo=1024, prefix_hi=8192, mix=28),
        # a batch of a layer with narrow heads, some contexts short, small pages
        _case("decode_64_narrow", "decode", n=64, lo=1, hi=1, prefix_lo=1, prefix_hi=8192, hq=32, hkv=8, d=64, page=16, mix=29),
        # drafts of up to 16 rows verified over long contexts
        _case("decode_verify_16", "decode", n=16, lo=16, hi=16, prefix_lo=2048, prefix_hi=32768, mix=30),
        # drafts of a few rows, ragged
        _case("decode_verify_ragged", "decode", n=24, lo=1, hi=6, prefix_lo=0, prefix_hi=9001, hq=32, hkv=8, d=128, page=64, mix=31),
        # an fp32 layer's step
        _case("decode_f32_16", "decode", n=16, lo=1, hi=1, prefix_lo=100, prefix_hi=8192, hq=8, hkv=2, d=128, page=64, f32=True, mix=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    hkv, d = rng.choice([(4, 256), (4, 256), (8, 128), (4, 128), (2, 256), (8, 64), (2, 96), (1, 32)])
    return dict(hkv=hkv, d=d, hq=hkv * rng.choice([1, 2, 4, 5, 6, 8]))


def draw(rng):
    op = rng.choice(["append", "gather", "decode", "decode"])
    c = _case(None, op, mix=rng.randrange(1, 1 << 30), page=rng.choice([16, 64, 128, 640, 784, 896]), **_heads(rng))
    c["f32"] = rng.random() < 0.2
    if op == "append":
        if rng.random() < 0.5:
            c.update(n=_log(rng, 1, 256), prefix_hi=rng.randrange(0, 128), page=128)
        else:
            c.update(n=_log(rng, 1, 16), prefix_hi=rng.randrange(0, 500))
            c["hi"] = _log(rng, 2, 32768 // c["n"])
            if c["f32"]:
                c["hi"] = min(c["hi"], 12000 // c["n"])
    elif op == "gather":
        c["n"] = _log(rng, 1, 32)
        c["hi"] = _log(rng, 16, (80000 if c["f32"] else 160000) // c["n"])
        c["lo"] = rng.choice([0, 1, c["hi"] // 2])
    else:
        c["n"] = _log(rng, 1, 256)
        c["prefix_hi"] = _log(rng, 16, min(229376, 1000000 // c["n"]))
        c["hi"] = rng.choice([1, 1, 1, 4, 16, 32])
        if c["hi"] > 1:
            c["n"] = min(c["n"], 32)
            c["lo"] = rng.choice([1, c["hi"]])
        # rows times keys times channels of a batch of drafts: no more than the listed one's
        c["prefix_hi"] = max(16, min(c["prefix_hi"], int(1.0e11 / (4 * c["d"] * c["hq"] * c["hi"] * c["n"])) if c["hi"] > 1 else c["prefix_hi"]))
        if c["f32"]:
            c.update(n=min(c["n"], 16), prefix_hi=min(c["prefix_hi"], 8192), hi=min(c["hi"], 4), lo=1)
        c["prefix_lo"] = rng.choice([0, c["prefix_hi"] // 8, c["prefix_hi"]])
    return c


def _lens(c):
    """(rows new in this call, tokens cached before it) of every request."""
    r = random.Random(c["mix"])
    new = [r.randint(c["lo"], c["hi"]) for _ in range(c["n"])]
    old = [r.randint(c["prefix_lo"], c["prefix_hi"]) for _ in range(c["n"])]
    new[0] = max(new[0], 1)                          # a call has a row at least
    if c["op"] == "gather" and c["n"] > 4 and c["lo"] == 0:
        new[3] = 0                                   # a request without a prefix
    return new, old


def _pages(tokens, page):
    return -(-tokens // page)


def work(case):
    new, old = _lens(case)
    c, n = case, case["n"]
    e = 4 if c["f32"] else 2
    tok = c["hkv"] * (c["d"] + c["d"] / GROUP + 1)   # cache bytes of a token: codes and scales of K and V
    row = c["hkv"] * 2 * c["d"] * e                  # the same as plain rows
    T, ctx = sum(new), [a + b for a, b in zip(new, old)]
    if c["op"] == "append":
        return {"bytes": T * (row + tok + 8), "flops": 3 * T * c["hkv"] * 2 * c["d"]}
    if c["op"] == "gather":
        return {"bytes": T * (tok + row) + 4 * (n + 1) + 4 * sum(_pages(t, c["page"]) for t in new), "flops": T * c["hkv"] * 2 * c["d"]}
    pairs = sum(sum(max(0, k - a + 1 + i) for i in range(a)) for a, k in zip(new, ctx))
    io = T * c["hq"] * (2 * c["d"] * e + 4)          # q, o, lse
    return {"bytes": io + tok * sum(ctx) + 4 * sum(_pages(k, c["page"]) for k in ctx) + 8 * n,
            "flops": 4 * c["d"] * c["hq"] * pairs}


# ------------------------------------------------------------------ the cache's layout, in elementary operations

def _sizes(s):
    """Bytes of a page's K (or V) codes, of its K scales, of its V scales, and of the page."""
    codes = s["hkv"] * s["page"] * s["d"] // 2
    ks, vs = s["hkv"] * s["page"] * (s["d"] // GROUP), s["hkv"] * s["page"]
    return codes, ks, vs, -(-(2 * codes + ks + vs) // 256) * 256


def _parts(s):
    """K codes, V codes, K scales, V scales of every page, as views of the pool's bytes."""
    codes, nk, nv, _ = _sizes(s)
    b, g = s["buf"], s["d"] // GROUP
    hb = (s["hkv"], s["page"] // BLOCK)
    k = b[:, :codes].unflatten(1, hb + (g, BLOCK, 16))
    v = b[:, codes:2 * codes].unflatten(1, hb + (s["d"], 8))
    ks = b[:, 2 * codes:2 * codes + nk].unflatten(1, hb + (g, BLOCK))
    vs = b[:, 2 * codes + nk:2 * codes + nk + nv].unflatten(1, hb + (BLOCK,))
    return k, v, ks, vs


def _scale_table(dev, dtype=torch.float32):
    """The value of each scale byte."""
    b = torch.arange(256, device=dev)
    t = torch.ldexp((8 + b % 8).to(dtype), b // 8 - 23)
    t[NAN] = math.nan
    return t


_SHIFT = [4 * (i // 2) + 16 * (i % 2) for i in range(8)]     # of element i in its word


def _unpack(b):
    """[..., 4 m] bytes -> [..., 8 m] values n - 8 in fp32."""
    w = b.contiguous().view(torch.int32)
    return torch.stack([(w >> i & 15) - 8 for i in _SHIFT], -1).flatten(-2).float()


def _pack(n):
    """[..., 8 m] values n - 8 (whole numbers) -> [..., 4 m] bytes."""
    n = n.long().unflatten(-1, (-1, 8)) + 8
    w = sum(n[..., i] << _SHIFT[i] for i in range(8))
    return (w - ((w >> 31) << 32)).int().view(torch.uint8)


def _cached(s, table):
    """K and V [n, hkv, tokens, d] in fp32 of the pages in `table` [n, pages] (-1: any page)."""
    k, v, ks, vs = _parts(s)
    n, t, h, d = table.shape[0], table.shape[1] * s["page"], s["hkv"], s["d"]
    at, val = table.clamp(min=0).long(), _scale_table(table.device)
    kk = _unpack(k[at]) * val[ks[at].long()][..., None]          # [n, pages, hkv, blocks, d / 32, 16, 32]
    kk = kk.permute(0, 2, 1, 3, 5, 4, 6).reshape(n, h, t, d)
    vv = _unpack(v[at]) * val[vs[at].long()][..., None, :]       # [n, pages, hkv, blocks, d, 16]
    vv = vv.permute(0, 2, 1, 3, 5, 4).reshape(n, h, t, d)
    return kk, vv


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    s = dict(case)
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    dt = torch.float32 if s["f32"] else torch.bfloat16
    new, old = _lens(case)
    n, page, hq, hkv, d = s["n"], s["page"], s["hq"], s["hkv"], s["d"]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    run_up = lambda v: ints([sum(v[:i]) for i in range(len(v) + 1)])  # noqa: E731
    ctx = [a + b for a, b in zip(new, old)]
    s["T"], s["max_new"], s["max_ctx"] = sum(new), max(new), max(ctx)
    s["cu"], s["cu_kv"], s["new"], s["ctx"] = run_up(new), run_up(ctx), ints(new), ints(ctx)
    s["err"] = torch.zeros(1, dtype=torch.int32, device=dev)
    width = max(1, max(_pages(t, page) for t in ctx))
    if s["op"] == "append":                 # the pages that this call writes, and no others
        first = [o // page for o in old]
        count = [_pages(k, page) - f for k, f in zip(ctx, first)]
    else:
        first = [0] * n
        count = [_pages(k, page) for k in ctx]
    s["num_pages"] = sum(count) + 3
    held = torch.randperm(s["num_pages"], generator=g, device=dev).tolist()
    table = [[-1] * width for _ in range(n)]
    at = 0
    for i in range(n):
        for j in range(count[i]):
            table[i][first[i] + j] = held[at]
            at += 1
    s["table"] = ints(table)
    codes, _, _, size = _sizes(s)
    s["buf"] = torch.zeros(s["num_pages"], size, dtype=torch.uint8, device=dev)
    k, v, ks, vs = _parts(s)
    step = max(1, (1 << 27) // codes)
    for x in (k, v):                        # two codes a byte, spread over their range as after quantisation
        for i in range(0, s["num_pages"], step):
            y = (torch.randn((2,) + x[i:i + step].shape, generator=g, device=dev) * 2.5).round_().clamp_(-7, 7).to(torch.uint8) + 8
            x[i:i + step] = y[0] | y[1] << 4
    for x in (ks, vs):                      # scales of 0.1 to 0.4: values of about 0.6 in size
        x.copy_(torch.randint(134, 150, x.shape, generator=g, device=dev))
    if s["op"] == "gather":
        s["k_out"], s["v_out"] = (torch.empty(s["T"], hkv, d, dtype=dt, device=dev) for _ in range(2))
        return s
    # rows as a fused projection leaves them: q heads, k heads, v heads
    qkv = torch.randn(s["T"], (hq + 2 * hkv) * d, generator=g, device=dev).to(dt)
    if s["op"] == "append":
        s["k"], s["v"] = (qkv[:, a * d:b * d].unflatten(1, (hkv, d)) for a, b in ((hq, hq + hkv), (hq + hkv, hq + 2 * hkv)))
        # tokens and heads of different sizes; a few channels of K much larger than the rest
        s["k"].mul_(torch.exp(torch.randn(s["T"], hkv, 1, generator=g, device=dev)).to(dt))
        s["v"].mul_(torch.exp(torch.randn(s["T"], hkv, 1, generator=g, device=dev)).to(dt))
        s["k"].mul_(torch.where(torch.rand(1, hkv, d, generator=g, device=dev) < 0.03, 8.0, 1.0).to(dt))
        pos = torch.cat([torch.arange(o, o + a, device=dev) for a, o in zip(new, old)])
        seq = torch.repeat_interleave(torch.arange(n, device=dev), s["new"].long())
        s["slot"] = s["table"].long()[seq, pos // page] * page + pos % page
    else:
        s["q"] = qkv[:, :hq * d].unflatten(1, (hq, d))
        s["pad"] = torch.arange(s["max_new"], device=dev)
        s["o"] = torch.empty(s["T"], hq, d, dtype=dt, device=dev)
        s["lse"] = torch.empty(s["T"], hq, dtype=torch.float32, device=dev)
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


def _own(s):
    import gated_deltanet_state_gb300 as gdn
    if "shape" not in s:
        from gated_deltanet_state_gb300 import inputs
        s["shape"] = inputs.AttnShape(s["hq"], s["hkv"], s["d"], s["page"], dtype=inputs.F32 if s["f32"] else inputs.BF16, kv_bits=4)
        s["pool"] = gdn.KVPool(s["shape"], s["num_pages"], buf=s["buf"])
        if s["op"] == "decode":
            s["ws"] = gdn.workspace_for(gdn.gdn_attn_decode_workspace_size(s["shape"], s["n"], s["T"], s["max_ctx"]))
    sh = s["shape"]
    if s["op"] == "append":
        gdn.gdn_kv_append(sh, s["pool"], k=s["k"], v=s["v"], slot_map=s["slot"], dev_error=s["err"])
        return _pool_outputs(s)
    if s["op"] == "gather":
        gdn.gdn_kv_gather(sh, s["pool"], cu_kv=s["cu_kv"], block_table=s["table"], k=s["k_out"], v=s["v_out"], dev_error=s["err"])
        return {"k": s["k_out"], "v": s["v_out"]}
    gdn.gdn_attn_decode(sh, s["pool"], q=s["q"], cu_seqlens=s["cu"], kv_len=s["ctx"], block_table=s["table"], o=s["o"],
                        lse=s["lse"], max_q_len=s["max_new"], max_kv_len=s["max_ctx"], workspace=s["ws"], dev_error=s["err"])
    return {"o": s["o"], "lse": s["lse"]}


def _pool_outputs(s):
    """The cache as it lies: whole numbers, two codes a byte, and the scales' bytes."""
    codes, nk, nv, _ = _sizes(s)
    return {"codes": s["buf"][:, :2 * codes], "scales": s["buf"][:, 2 * codes:2 * codes + nk + nv]}


def _scale_bytes(amax):
    """The least byte whose scale times 7 reaches amax (the greatest there is, if none does)."""
    top = _scale_table(amax.device)[:NAN] * 7        # exact: 3 and 4 bits
    return torch.searchsorted(top, amax.contiguous()).clamp(max=NAN - 1)


def _quantise(x):
    """x [..., m] in fp32 under one scale -> whole numbers -7 .. 7 and the scale's byte [...]."""
    nan = x.isnan().any(-1)
    b = _scale_bytes(torch.where(x.isfinite(), x.abs(), 0.0).amax(-1))
    # 64 bits: a quotient next to a half must not be rounded onto it
    s = _scale_table(x.device, torch.float64)[b][..., None]
    n = torch.floor(x.abs().double() / s + 0.5).clamp(max=7) * x.sign()
    return torch.where(nan[..., None], 0.0, n), torch.where(nan, NAN, b)


def _append(s):
    """K: every token writes its own bytes.  V: a block's tokens share bytes, so written blocks are read, merged and written back."""
    k, v, ks, vs = _parts(s)
    page, slot, d, hkv = s["page"], s["slot"], s["d"], s["hkv"]
    per = page // BLOCK
    blk, off = slot // BLOCK, slot % BLOCK
    pg, b = blk // per, blk % per
    n, sc = _quantise(s["k"].float().unflatten(-1, (-1, GROUP)))             # [T, hkv, d / 32, 32]
    k[pg, :, b, :, off] = _pack(n)
    ks[pg, :, b, :, off] = sc.to(torch.uint8)
    n, sc = _quantise(s["v"].float())                                        # [T, hkv, d]
    vs[pg, :, b, off] = sc.to(torch.uint8)
    ids, row = torch.unique_consecutive(blk, return_inverse=True)
    ip, ib = ids // per, ids % per
    held = _unpack(v[ip, :, ib])                                             # [U, hkv, d, 16]
    held[row, :, :, off] = n.float()
    v[ip, :, ib] = _pack(held)
    return _pool_outputs(s)


def _gather(s):
    t = torch.arange(s["T"], device=s["buf"].device)
    seq = torch.searchsorted(s["cu_kv"][1:].long(), t, right=True)
    pos = t - s["cu_kv"].long()[seq]
    for i in range(s["n"]):                                                  # a request's pages at a time
        m = seq == i
        kk, vv = _cached(s, s["table"][i:i + 1])
        s["k_out"][m] = kk[0, :, pos[m]].transpose(0, 1).to(s["k_out"].dtype)
        s["v_out"][m] = vv[0, :, pos[m]].transpose(0, 1).to(s["v_out"].dtype)
    return {"k": s["k_out"], "v": s["v_out"]}


def _decode(s):
    """softmax(q k^T / sqrt(d)) v over the keys that a row may see, some requests at a time; rows without keys give 0 and -inf."""
    n, h, R, d, T = s["n"], s["hkv"], s["max_new"], s["d"], s["T"]
    G, L = s["hq"] // h, s["table"].shape[1] * s["page"]
    keys = torch.arange(L, device=s["buf"].device)
    at = (s["cu"][:-1, None].long() + s["pad"]).clamp(max=T - 1)             # [n, R]
    step = max(1, (1 << 20) // L)
    for i in range(0, n, step):
        c = slice(i, min(n, i + step))
        m = c.stop - i
        kk, vv = _cached(s, s["table"][c])
        ctx, new = s["ctx"][c, None].long(), s["new"][c, None].long()
        q = s["q"][at[c]].float().reshape(m, R, h, G, d).permute(0, 2, 3, 1, 4)
        p = torch.matmul(q.reshape(m, h, G * R, d), kk.transpose(2, 3)).mul_(d ** -0.5).view(m, h, G, R, L)
        hide = keys >= (ctx - new + s["pad"] + 1)[:, :, None]                # [m, R, L]
        p.masked_fill_(hide[:, None, None], float("-inf"))
        top = p.amax(-1, keepdim=True)
        p.sub_(torch.where(top.isfinite(), top, 0.0)).exp_()
        l = p.sum(-1, keepdim=True)
        vv.masked_fill_((keys >= ctx)[:, None, :, None], 0.0)
        o = torch.matmul(p.view(m, h, G * R, L), vv).view(m, h, G, R, d) / torch.where(l > 0, l, 1.0)
        lse = torch.where(l > 0, top + torch.log(l), float("-inf"))[..., 0]
        own_row = s["pad"] < new
        s["o"][at[c][own_row]] = o.permute(0, 3, 1, 2, 4).reshape(m, R, h * G, d)[own_row].to(s["o"].dtype)
        s["lse"][at[c][own_row]] = lse.permute(0, 3, 1, 2).reshape(m, R, h * G)[own_row]
    return {"o": s["o"], "lse": s["lse"]}


_PLAIN = {"append": _append, "gather": _gather, "decode": _decode}


# ------------------------------------------------------------------ 64 bits, from the definitions

def _nibble(bytes_, i):
    """n - 8 in 64 bits of elements i (last dimension) of words in bytes_ [..., 4 m]."""
    word, e = i // 8, i % 8
    place = e // 2 + 4 * (e % 2)                     # which 4 bits of the word, from the lowest
    got = bytes_.index_select(-1, word * 4 + place // 2).double()
    return torch.where(place % 2 == 0, got - 16 * torch.floor(got / 16), torch.floor(got / 16)) - 8


def _scale64(b):
    b = b.double()
    s = (8 + b - 8 * torch.floor(b / 8)) * torch.exp2(torch.floor(b / 8) - 23)
    return torch.where(b == NAN, math.nan, s)


def _rows64(s, i, L):
    """K and V [L, hkv, d] in 64 bits of request i."""
    k, v, ks, vs = _parts(s)
    d, dev, pages = s["d"], s["buf"].device, _pages(L, s["page"])
    at = s["table"][i, :pages].long()
    e, t = torch.arange(GROUP, device=dev), torch.arange(BLOCK, device=dev)
    kk = _nibble(k[at], e) * _scale64(ks[at])[..., None]                     # [pages, hkv, blocks, groups, 16, 32]
    kk = kk.permute(0, 2, 4, 1, 3, 5).reshape(-1, s["hkv"], d)[:L]
    vv = _nibble(v[at], t) * _scale64(vs[at])[..., None, :]                  # [pages, hkv, blocks, d, 16]
    vv = vv.permute(0, 2, 4, 1, 3).reshape(-1, s["hkv"], d)[:L]
    return kk, vv


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "append":
        return _exact_append(s)
    new, old = _lens(case)
    dev, out = s["buf"].device, ([], [])
    q0, G = 0, s["hq"] // s["hkv"]
    for i in range(s["n"]):
        L = new[i] + old[i]
        k, v = _rows64(s, i, L)
        if s["op"] == "gather":
            out[0].append(k)
            out[1].append(v)
            continue
        o = torch.zeros(new[i], s["hq"], s["d"], dtype=torch.float64, device=dev)
        ls = torch.full((new[i], s["hq"]), -math.inf, dtype=torch.float64, device=dev)
        seen = torch.arange(L, device=dev)[None] <= torch.arange(L - new[i], L, device=dev)[:, None]
        for h in range(s["hkv"] if L and new[i] else 0):
            x = torch.einsum("rgd,ld->grl", s["q"][q0:q0 + new[i], h * G:(h + 1) * G].double(), k[:, h]) / math.sqrt(s["d"])
            x = torch.where(seen, x, -math.inf)
            ls[:, h * G:(h + 1) * G] = torch.logsumexp(x, 2).T
            o[:, h * G:(h + 1) * G] = torch.einsum("grl,ld->rgd", torch.softmax(x, 2), v[:, h])
        q0 += new[i]
        out[0].append(o)
        out[1].append(ls)
    a, b = torch.cat(out[0]), torch.cat(out[1])
    return {"k": a, "v": b} if s["op"] == "gather" else {"o": a, "lse": b}


def _exact_bytes(x):
    """Codes 1 .. 15 and scale byte of x [..., m] in 64 bits, by counting thresholds."""
    x = x.double()
    top = torch.where(x.isfinite(), x.abs(), 0.0).amax(-1)
    e = torch.floor(torch.log2((top / 56).clamp(min=2.0 ** -23)))            # 7 * 8 * 2^e <= top, about
    b = torch.zeros_like(top)
    for step in (-1, 0, 1):                                                  # count the scales that are too small
        for m in range(8):
            f = e + step
            b += ((f >= -23) & (7 * (8 + m) * torch.exp2(f) < top)).double()
    b = (b + 8 * (e - 1 + 23).clamp(min=0)).clamp(max=NAN - 1)
    s = _scale64(b)[..., None]
    n = 8 + sum((x >= (j - 0.5) * s).double() - (x <= -(j - 0.5) * s).double() for j in range(1, 8))
    bad = x.isnan().any(-1)
    return torch.where(bad[..., None], 8.0, n), torch.where(bad, float(NAN), b)


def _exact_append(s):
    """Every token by its own bytes, in 64 bits."""
    k, v, ks, vs = _parts(s)
    page, slot = s["page"], s["slot"]
    pg, b, t = slot // page, slot % page // BLOCK, slot % BLOCK
    n, sc = _exact_bytes(s["k"].unflatten(-1, (-1, GROUP)))
    # a word's four bytes hold elements 0 and 2, 4 and 6, 1 and 3, 5 and 7
    lo = torch.tensor([8 * (j // 4) + (0, 4, 1, 5)[j % 4] for j in range(16)], device=slot.device)
    k[pg, :, b, :, t] = (n.index_select(-1, lo) + 16 * n.index_select(-1, lo + 2)).to(torch.uint8)
    ks[pg, :, b, :, t] = sc.to(torch.uint8)
    n, sc = _exact_bytes(s["v"])
    vs[pg, :, b, t] = sc.to(torch.uint8)
    for j in range(BLOCK):                                                   # a block's tokens share bytes: one after another
        m = t == j
        e = j % 8
        byte, high = 4 * (j // 8) + (e // 2 + 4 * (e % 2)) // 2, e // 2 % 2
        held = v[pg[m], :, b[m], :, byte].double()
        upper = torch.floor(held / 16)
        put = held - 16 * upper + 16 * n[m] if high else 16 * upper + n[m]
        v[pg[m], :, b[m], :, byte] = put.to(torch.uint8)
    return _pool_outputs(s)
