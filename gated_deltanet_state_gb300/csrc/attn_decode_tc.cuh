// attn_decode_tc.cuh — what the two decode kernels on the tensor cores share:
// the work items, the loads of the cache's blocks, the products' forms.
//
// The cache's e4m3 codes are the products' operands as they lie in memory; no
// code is converted.  Q and P enter in 8-bit parts whose products are added:
//
// * A row of Q, scaled by a power of two so that its largest element is in (224,
//   448], as hi + lo: hi an e4m3 of 4 significant bits, lo what is left of the 8
//   of a bf16 (at most 3 bits and a sign), as an e4m3 of 16 times it or as an
//   e5m2.  All 8 bits are kept of elements down to 2^-13 of the largest; below,
//   an element is off by at most 2^-21 of the largest.
// * A weight p as three e5m2, of 3 significant bits each: 9 together, to at
//   most 2^-9 of the weight, half of what a rounding to bf16 may do.  e5m2
//   reaches down to 2^-16, and weights are scaled so that the reference is
//   2^11, so this holds down to 2^-19 of it; smaller weights are off by at most
//   2^-28 of the reference (and are not dropped: where one key takes most of
//   the softmax and its values are small, the outputs are theirs).
//
// A block's K scale multiplies its scores; its V scale goes into the weight's
// exponent, so a weight is 2^(s + log2(vs) - M) and the sum of the p is the sum
// of the weights over vs (in fp32, of the weights as they were before the split).
#pragma once

#include "attn.h"
#include "tc.cuh"

namespace gdn {
namespace dt {

constexpr int kDtTok = 128;           // tokens of a tile
constexpr int kDtBlocks = kDtTok / kKvBlock;
constexpr int kDtSeqs = 256;         // sequences a launch
constexpr int kDtMaxStages = 8;
constexpr long long kDtWait = 4000000000LL;
// Weights are scaled by 2^11 and may grow by 2^4.75 (55,109 < 57,344, the largest
// e5m2) before a row's reference moves (which costs a pass over its outputs).
constexpr float kDtBase = 11.f, kDtGrow = 4.75f;

struct DtParams {
  AttnDecodeParams a;
  int32_t s0, ns;       // this launch's sequences ...
  int32_t row_lo, row_hi;   // ... those with (row, head of the group) pairs in [row_lo, row_hi]
  int32_t k_stages, v_stages;
  long long wait;       // SM clocks that a wait may take; < 0: every one has run out
  uint32_t k_off, v_off, q_off, p_off, misc_off;   // dynamic shared memory
};

// Shared memory of either kernel.
struct DtBase {
  uint64_t k_full[kDtMaxStages], k_empty[kDtMaxStages], v_full[kDtMaxStages], v_empty[kDtMaxStages];
  uint64_t sc_full[kDtMaxStages + 2], s_full[2], p_full[2], o_done[2], q_full, drain;
  float ks[kDtMaxStages + 2][kDtBlocks], vs[kDtMaxStages + 2][kDtBlocks];
  int bad[2][256];          // (items alternate) first token with a NaN value that not every row sees, by element
  int items[kDtSeqs + 1];   // running sums of the sequences' work items ...
  long long work[kDtSeqs + 1];   // ... and of their weights (tiles of every head: past 32 bits for long shared contexts)
  uint32_t tmem;
  int fail;
};

__device__ __forceinline__ bool dt_wait(uint64_t* m, uint32_t parity, volatile int* fail, long long limit) {
  if (tc::mbar_test_wait(m, parity)) return true;
  const long long t0 = clock64();
  while (!tc::mbar_try_wait(m, parity)) {
    if (*fail) return false;
    if (clock64() - t0 > limit) {
      *fail = 1;
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ void dt_arrive(uint64_t* m) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(smem_u32(m)) : "memory");
}
__device__ __forceinline__ float dt_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// e4m3 x e4m3 -> fp32: D[tmem] (+)= A[smem] B[smem]^T, 32 deep; a whole warp
// runs it, the lane with `lead` issues (tc::elect_one).
__device__ __forceinline__ void mma_e4m3(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}
// Instruction descriptor: e4m3 A and B (both K-contiguous), fp32 sums, M = 128;
// and what makes A or B e5m2.
constexpr uint32_t kE5m2A = 1u << 7, kE5m2B = 1u << 10;
__host__ __device__ constexpr uint32_t idesc_e4m3(int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kDtTok >> 4) << 24);
}
constexpr uint32_t kTransposedB = 1u << 16;   // B's rows contiguous instead of the contraction
// Operand of unswizzled 8-row x 16-byte tiles: `lead` bytes to the next 16
// elements of the contraction, `stride` to the next 8 rows.
__device__ __forceinline__ uint64_t desc_tiles(uint32_t saddr, uint32_t lead, uint32_t stride) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)(lead >> 4) << 16 | (uint64_t)(stride >> 4) << 32 | (uint64_t)1 << 46;
}

// Work item -> sequence, kv head, row tile, piece.
struct DtItem {
  int s, h, r0, rows, piece, pieces, pt, rt;   // rows: (row, head) pairs of this item, from r0
  int q0, n, L, k0, k1, tiles;
};

// Whether item t has other rows than the one before it.
__device__ __forceinline__ bool dt_new_rows(const DtItem& t, bool first) { return first || t.rt > 1 || t.piece == 0; }
// Whether its rows then enter a product.  (Those of an item without keys do not,
// and no role waits for them: two such loads in a row would pass the product
// warp's wait by, since only an item's scores tell that it has seen them.)
__device__ __forceinline__ bool dt_load_rows(const DtItem& t, bool first) { return t.tiles > 0 && dt_new_rows(t, first); }

// Groups (kv head, row tile) of a sequence; 0: no rows, -1: out of bounds.
template <int NT>
__device__ __forceinline__ int dt_groups(const DtParams& w, int s) {
  const AttnDecodeParams& p = w.a;
  const int n = p.cu[s + 1] - p.cu[s], L = p.kv_len[s];
  if (n <= 0) return 0;
  if (n > p.max_q || L > p.max_kv || L < 0 || p.cu[s] < 0 || (int64_t)p.cu[s] + n > p.T) return -1;
  if (n * p.G < w.row_lo || n * p.G > w.row_hi) return 0;
  return p.c.Hkv * ((n * p.G + NT - 1) / NT);
}
// A tile of keys counts 1, an item's fixed cost as much again.
__device__ __forceinline__ int dt_piece_work(const AttnDecodeParams& p, int s) {
  return decode_piece_tokens(p.kv_len[s], (p.cu[s + 1] - p.cu[s]) * p.G) / kDtTok + 1;
}

// The last s with sums[s] <= i.
template <typename I>
__device__ __forceinline__ int dt_find(const I* sums, int n, I i) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

// First item of CTA b: the work before it is b / CTAs of all.
template <int NT>
__device__ __forceinline__ int dt_first(const DtParams& w, const int* items, const long long* work, int b, int ctas) {
  const long long at = work[w.ns] * b / ctas;
  if (at >= work[w.ns]) return items[w.ns];
  const int s = dt_find(work, w.ns, at);
  const int per = dt_piece_work(w.a, w.s0 + s);   // of each of its items
  return min(items[s + 1], items[s] + (int)((at - work[s] + per - 1) / per));
}

template <int NT>
__device__ __forceinline__ DtItem dt_item(const DtParams& w, const int* items, int i) {
  const AttnDecodeParams& p = w.a;
  const int lo = dt_find(items, w.ns, i);
  DtItem t;
  t.s = w.s0 + lo;
  const int k = i - items[lo];
  t.q0 = p.cu[t.s];
  t.n = p.cu[t.s + 1] - t.q0;
  t.L = p.kv_len[t.s];
  // of one head: piece after piece, of a piece its row tiles (with one tile a
  // CTA's run of items loads its rows once a head)
  t.pieces = decode_pieces(t.L, t.n * p.G);
  t.rt = (t.n * p.G + NT - 1) / NT;
  t.h = k / (t.pieces * t.rt);
  const int in = k - t.h * t.pieces * t.rt;
  t.piece = in / t.rt;
  t.r0 = (in - t.piece * t.rt) * NT;
  t.rows = min(NT, t.n * p.G - t.r0);
  t.pt = decode_piece_tokens(t.L, t.n * p.G);
  t.k0 = t.piece * t.pt;
  t.k1 = min(t.L, t.k0 + t.pt);
  t.tiles = (t.k1 - t.k0 + kDtTok - 1) / kDtTok;
  return t;
}
// The item after it.
template <int NT>
__device__ __forceinline__ void dt_next(const DtParams& w, const int* items, int i, DtItem& t) {
  if (t.rt == 1 && t.piece + 1 < t.pieces) {
    ++t.piece;
    t.k0 += t.pt;
    t.k1 = min(t.L, t.k0 + t.pt);
    t.tiles = (t.k1 - t.k0 + kDtTok - 1) / kDtTok;
  } else {
    t = dt_item<NT>(w, items, i);
  }
}

// One product's steps: KS of 32 elements, the operands' starts moving by a
// step's tiles (constants: with run-time steps the issue takes 130 cycles a
// product, which takes 41 at 16 columns and 67 at 128).
template <int KS>
__device__ __forceinline__ void mma_steps(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint64_t astep, uint64_t bstep, bool acc) {
#pragma unroll
  for (int c = 0; c < KS; ++c) mma_e4m3(lead, d, a + c * astep, b + c * bstep, id, acc || c != 0);
}
// Largest value of a warp (NaN falls out).
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;\n" : "=f"(r) : "f"(x));
  return r;
}

// ---- the parts of Q and P --------------------------------------------------------
// Two f16 to e5m2, nearest even (x in the low byte).
__device__ __forceinline__ uint32_t e5m2x2(__half2 x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t*>(&x)));
  return r;
}
// Four weights in three parts, four codes a word.  An e5m2 is the upper byte of
// an f16, so the first two parts are cut off without a conversion; the last is
// rounded.  (The differences are exact: f16 holds 11 bits.)
__device__ __forceinline__ void split_weights(float e0, float e1, float e2, float e3, uint32_t (&part)[3]) {
  __half2 a = __floats2half2_rn(e0, e1), b = __floats2half2_rn(e2, e3);
  auto bits = [](__half2& x) -> uint32_t& { return *reinterpret_cast<uint32_t*>(&x); };
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    part[i] = __byte_perm(bits(a), bits(b), 0x7531);
    __half2 u, v;
    bits(u) = bits(a) & 0xff00ff00u, bits(v) = bits(b) & 0xff00ff00u;
    a = __hsub2(a, u), b = __hsub2(b, v);
  }
  part[2] = e5m2x2(a) | e5m2x2(b) << 16;
}
// Eight elements of a row of Q (x; a warp holds the row) in two parts: LO_E5M2
// or, for sums of its own, 16 times the rest as e4m3 (kDtLo undoes it).  Returns
// the power of two that the codes are to be multiplied by; NaN where an element
// is infinite, which makes the row's scores NaN, as its codes would not.
constexpr float kDtLo = 1.f / 16.f;
template <bool LO_E5M2>
__device__ __forceinline__ float split_row(const uint4& x, uint2& hi, uint2& lo) {
  float f[8], amax = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t u = (&x.x)[k >> 1];
    f[k] = __uint_as_float(k & 1 ? u & 0xffff0000u : u << 16);
    amax = fmaxf(amax, fabsf(f[k]));
  }
  amax = warp_max(amax);
  // largest element to (224, 448]; exponents kept where both factors are normal
  int e = (int)(__float_as_uint(amax) >> 23) - 127 - 8 + ((__float_as_uint(amax) & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = max(-100, min(100, e));
  const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float g[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) g[u] = f[4 * k + u] * inv;
    const uint32_t h = e4m3x4(g[0], g[1], g[2], g[3]);
    const float2 a = e4m3_f32x2(h), b = e4m3_f32x2(h >> 16);
    (&hi.x)[k] = h;
    if constexpr (LO_E5M2)
      (&lo.x)[k] = e5m2x2(__floats2half2_rn(g[0] - a.x, g[1] - a.y)) | e5m2x2(__floats2half2_rn(g[2] - b.x, g[3] - b.y)) << 16;
    else
      (&lo.x)[k] = e4m3x4((g[0] - a.x) * 16.f, (g[1] - a.y) * 16.f, (g[2] - b.x) * 16.f, (g[3] - b.y) * 16.f);
  }
  return amax < INFINITY ? __uint_as_float((uint32_t)(127 + e) << 23) : __int_as_float(0x7fffffff);
}

// Running sums of the items (one warp); lengths out of bounds are reported and
// have none.
template <int NT>
__device__ __forceinline__ void dt_sums(const DtParams& w, DtBase& sh, int lane) {
  const AttnDecodeParams& p = w.a;
  int sum = 0;
  long long sumw = 0;
  if (lane == 0) sh.items[0] = sh.work[0] = 0;
  for (int c = 0; c < w.ns; c += 32) {
    int v = 0;
    long long x = 0;
    if (c + lane < w.ns) {
      const int s = w.s0 + c + lane;
      int g = dt_groups<NT>(w, s);
      if (g < 0) {
        if (blockIdx.x == 0) set_error(p.err, GDN_ERR_INVALID_ARG);
        g = 0;
      }
      if (g > 0) {
        const int pieces = decode_pieces(p.kv_len[s], (p.cu[s + 1] - p.cu[s]) * p.G);
        v = g * pieces;
        x = (long long)v * dt_piece_work(p, s);
      }
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, v, o);
      const long long b = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) v += a, x += b;
    }
    if (c + lane < w.ns) sh.items[c + lane + 1] = sum + v, sh.work[c + lane + 1] = sumw + x;
    sum += __shfl_sync(0xffffffffu, v, 31);
    sumw += __shfl_sync(0xffffffffu, x, 31);
  }
}

// A warp's loads of the CTA's items [i0, i1), K's codes and scales or V's:
// lane b < 8 the tile's block b.  Returns the tiles loaded.
template <int NT>
__device__ __forceinline__ int dt_load(const DtParams& w, DtBase& sh, uint8_t* base, int i0, int i1, bool is_v, int lane) {
  const AttnDecodeParams& p = w.a;
  volatile int* fail = &sh.fail;
  uint64_t *full = is_v ? sh.v_full : sh.k_full, *empty = is_v ? sh.v_empty : sh.k_empty;
  uint8_t* ring = base + (is_v ? w.v_off : w.k_off);
  const int ST = is_v ? w.v_stages : w.k_stages, NS = max(w.k_stages, w.v_stages) + 2, d = p.c.d;
  const uint32_t unit = (uint32_t)kDtTok * d;
  int loaded = 0;
  int st = 0, ph = 0, sc = 0;
  bool ok = true;
  DtItem t{};
  for (int i = i0; ok && i < i1; ++i) {
    if (i == i0) t = dt_item<NT>(w, sh.items, i);
    else dt_next<NT>(w, sh.items, i, t);
    const int32_t* bt = p.block_table + (int64_t)t.s * p.max_pages;
    auto page_of = [&](int j) {
      const int pos = t.k0 + j * kDtTok + lane * kKvBlock, at = pos / p.c.page_tokens;
      return lane < kDtBlocks && pos < t.k1 && at < p.max_pages ? bt[at] : -1;
    };
    int next = t.tiles > 0 ? page_of(0) : -1;
    for (int j = 0; j < t.tiles; ++j) {
      const int page = next, pos = t.k0 + j * kDtTok + lane * kKvBlock;
      if (j + 1 < t.tiles) next = page_of(j + 1);
      const bool in = lane < kDtBlocks && pos < t.k1, good = in && page >= 0 && page < p.c.num_pages;
      if (in && !good) set_error(p.err, GDN_ERR_PAGE_RANGE);
      if (loaded >= ST) ok = dt_wait(&empty[st], ph ^ 1, fail, w.wait);
      if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
      uint8_t* dst = ring + (uint32_t)st * unit;
      const unsigned have = __ballot_sync(0xffffffffu, good);
      if (have != (1u << kDtBlocks) - 1u) {
        // blocks that are not loaded: their weights are 0, and so must V be
        if (is_v)
          for (unsigned miss = ~have & ((1u << kDtBlocks) - 1u); miss; miss &= miss - 1) {
            uint4* z = reinterpret_cast<uint4*>(dst + (__ffs(miss) - 1) * kKvBlock * d);
            for (int x = lane; x < d; x += 32) z[x] = make_uint4(0, 0, 0, 0);
          }
        tc::fence_async_smem();
        if (lane < kDtBlocks && !good) {
          if (is_v) sh.vs[sc][lane] = 1.f;
          else sh.ks[sc][lane] = -1.f;   // a block to leave out
        }
        __syncwarp();
      }
      if (lane == 0) tc::mbar_expect_tx(&full[st], __popc(have) * kKvBlock * d);
      __syncwarp();
      if (lane < kDtBlocks) {
        if (good) {
          const int b = (pos - pos / p.c.page_tokens * p.c.page_tokens) / kKvBlock;
          tc::bulk_load(dst + lane * kKvBlock * d, is_v ? kv_v_block(p.c, page, t.h, b) : kv_k_block(p.c, page, t.h, b),
                        kKvBlock * d, &full[st]);
          if (is_v) cp_async4(&sh.vs[sc][lane], kv_v_scale(p.c, page, t.h, b), 4);
          else cp_async4(&sh.ks[sc][lane], kv_k_scale(p.c, page, t.h, b), 4);
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(smem_u32(&sh.sc_full[sc])) : "memory");
        } else {
          dt_arrive(&sh.sc_full[sc]);
        }
      }
      ++loaded;
      if (++st == ST) st = 0, ph ^= 1;
      if (++sc == NS) sc = 0;
    }
  }
  cp_async_commit();
  cp_async_wait<0>();
  return loaded;
}

// After a run-out: one more bounded wait for each copy in flight.
__device__ __forceinline__ void dt_drain(const DtParams& w, DtBase& sh, int loaded, bool is_v) {
  const int ST = is_v ? w.v_stages : w.k_stages;
  for (int n = max(0, loaded - ST); n < loaded; ++n)
    tc::mbar_wait_bounded(is_v ? &sh.v_full[n % ST] : &sh.k_full[n % ST], (uint32_t)(n / ST) & 1, kDtWait);
}

// Reports a run-out and marks the rows of the pieces that this CTA had, items
// [i0, i1): what it has not written of them must not be joined.
template <int NT>
__device__ __forceinline__ void dt_report(const DtParams& w, const DtBase& sh, int i0, int i1) {
  const AttnDecodeParams& p = w.a;
  if (threadIdx.x == 0) atomicExch(p.err, GDN_ERR_TIMEOUT);   // over an earlier code
  if (!p.part_o) return;
  for (int i = i0; i < i1; ++i) {
    const DtItem t = dt_item<NT>(w, sh.items, i);
    for (int n = threadIdx.x; n < t.rows; n += blockDim.x) {
      const int row = (t.r0 + n) / p.G, g = t.r0 + n - row * p.G;
      p.part_ml[t.piece * (p.T * p.Hq) + (int64_t)(t.q0 + row) * p.Hq + t.h * p.G + g] = make_float2(0.f, kLostPiece);
    }
  }
}

// Values of a tile (of its stage v) that some row may not see: past the
// sequence they become zero, and so do NaN codes (a weight of 0 would not keep
// them out of the product), noted by element for the rows that do see them.
// 128 threads, elements tid and tid + 128.
__device__ __forceinline__ void dt_clean(uint8_t* v, int* bad, const DtItem& t, int kb, int least, int d, int tid) {
  for (int e = tid; e < d; e += 128)
    for (int b = max(0, (least - kb) / kKvBlock); b < kDtBlocks && kb + b * kKvBlock < t.k1; ++b) {
      uint8_t* at = v + (b * d + e) * kKvBlock;
      for (int k = 0; k < kKvBlock; ++k) {
        const int pos = kb + b * kKvBlock + k;
        if (pos >= t.L) {
          at[k] = 0;
        } else if (pos >= least && (at[k] & 0x7f) == 0x7f) {
          at[k] = 0;
          atomicMin(&bad[e], pos);
        }
      }
    }
}

inline long long dt_limit(const AttnDecodeParams& p) {
  return p.wait_cycles > 0 ? p.wait_cycles : p.wait_cycles < 0 ? -1 : kDtWait;
}

// The cache's share of dynamic shared memory: K and V stages in what `fixed`
// leaves of `all` bytes; where d is no multiple of 128 a product's 128 rows of
// V read up to 2 KB past a stage (their sums are not used).  The offset behind.
inline uint32_t dt_rings(DtParams& w, uint32_t all, uint32_t fixed) {
  const uint32_t d = (uint32_t)w.a.c.d, unit = kDtTok * d, past = d % 128 ? 2048 : 0;
  const int units = all > fixed + past ? (int)((all - fixed - past) / unit) : 0;
  w.k_stages = units / 2 + units % 2 > kDtMaxStages ? kDtMaxStages : units / 2 + units % 2;
  w.v_stages = units / 2 > kDtMaxStages ? kDtMaxStages : units / 2;
  w.k_off = 0;
  w.v_off = w.k_stages * unit;
  return ((w.k_stages + w.v_stages) * unit + past + 127) / 128 * 128;
}

}  // namespace dt
}  // namespace gdn
