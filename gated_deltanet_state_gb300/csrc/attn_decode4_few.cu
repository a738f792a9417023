// attn_decode4_few.cu — attention over the 4-bit cache of up to 8 (row, head of
// the group) pairs a kv head, bf16 rows: a decode step.
//
// With so few rows the products are small and what decides is the way of the
// codes into them: 65,536 of a 128-token tile at d = 256, for which the memory
// takes 1,500 cycles an SM.  They go from shared memory into registers and, as
// operands of warp-wide products, nowhere else.  (By way of tensor memory, where
// the larger products take their operands from, the same step costs stores,
// hand-overs and waits on top: 256 sequences of 1,024 to 8,192 tokens, 24 heads, 4
// kv heads, d = 256, 425 us.)
//
//   S^T [16 tokens x 8 rows] = K Q^T,    O^T [16 channels x 8 rows] += V^T P^T
//
// K's and V's codes are whole numbers in f16, less 8 (pairs 1 and 3 of a word's four
// sixteenfold, whose partners in Q and whose weights carry 2^-4).  A group of 32
// channels of K is a product of its own, added under its tokens' scales in fp32.  (K's
// codes as they stand, as subnormals, with the offset of 8 taken out by the products'
// start value, took 2 % longer with half the instructions for it.  And what is then
// summed and taken away again is 8 times a group's largest q, also where its code is
// 0, so elements of 2^-10 of that lost bits.)  Which channel or token
// stands in which step of a product is chosen so that a lane's word is its operand:
// a lane holds eight channels of K, or eight tokens of V.
//
// Q is scaled by a power of two for each row, its largest element to [2^15, 2^16):
// all 8 bits of elements down to 2^-29 of the largest, off by 2^-36 of it at most
// below.  A weight times its V scale is an f16 against a reference of its row that is
// the first chunk's maximum and moves only when a weight would pass f16's range: 11
// bits down to 2^-20 of it, off by 2^-31 at most below.
//
// A warp takes 32 tokens of every tile of 128, with statistics and sums of its own,
// which the four bring together in a fixed order at the end of a piece; it waits for
// nothing but the tile.
//
// 256 sequences of 1,024 to 8,192 tokens, 24 heads, 4 kv heads, d = 256 (1.24 GB):
// 367 us, 3.4 TB/s; one of 229,376 tokens 72 us.  What bounds it is the warps' own
// chains: 6,000 instructions a tile at 2.0 a cycle (issue slots 51 % used, 27 % of a
// warp's time waiting for an instruction's fixed latency), which take 3,000 cycles
// where the memory takes 1,500.  Registers hold the warps at 12 an SM and one for
// loads a CTA: with four CTAs 96 registers a thread spill (495 us), with two 410 us.
#include "attn_decode_tc.cuh"
#include "kv4.cuh"

namespace gdn {

using namespace dt;

namespace {

constexpr int kFewRows = 8, kFewWarps = 4, kFewThreads = 32 * (kFewWarps + 1);   // and the loads' warp
constexpr int kFewTok = kDtTok / kFewWarps, kFewBlocks = kFewTok / kKvBlock;     // of a warp, in a tile
constexpr int kFewStages = 8;
constexpr float kFewBase = 10.f, kFewTop = 15.75f;   // a weight at its reference is 2^10, none passes 2^15.75
constexpr float kFewUnset = 3e38f;                   // the offset of a row that has seen no key

// A stage holds the tokens of kFewPer warps: K's codes, K's scales, V's codes, V's scales,
// as they lie in pages.  All four warps' up to d = 128, where a copy is short and its
// issue what counts; one's above, so that three CTAs an SM hold some ahead.
template <int GR>
constexpr int kFewPer = GR <= 4 ? kFewWarps : 1;
template <int GR>
constexpr bool kFewBulk = kFewPer<GR> < kFewWarps;   // scales in bulk copies
// CTAs on an SM: as many as registers allow without spills in the loop (at d = 128
// three 115 us for 64 sequences of 512 to 8,192 tokens, 32 heads, four 126).
template <int GR>
constexpr int kFewCtas = GR <= 2 ? 4 : 3;
struct FewStage {
  uint32_t ks, v, vs, bytes;
};
template <int GR>
__host__ __device__ inline FewStage few_stage(int d) {
  constexpr int kBlocks = kFewPer<GR> * kFewBlocks;
  FewStage s;
  s.ks = kBlocks * kv4_codes(d), s.v = s.ks + kBlocks * kv4_k_scales(d), s.vs = s.v + kBlocks * kv4_codes(d);
  s.bytes = (s.vs + kBlocks * kKvBlock + 127) / 128 * 128;
  return s;
}

struct FewShared : DtItems {
  uint64_t full[kFewStages], empty[kFewStages];
  uint32_t have[kFewStages];            // blocks of a stage that were loaded
  uint32_t issued;                      // stages whose loads have begun (one warp's stages)
  float2 stat[kFewWarps][kFewRows];     // a warp's offset and sum of each row
  uint4 q[8][32];                       // Q of row g, eight channels of a group, by lane
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(x));
  return r;
}
// D += A B: 16 x 16 by 16 x 8 in f16, fp32 sums.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float few_log2(float x) {   // (normal numbers)
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Largest and sum over the lanes of a column (every fourth lane).
__device__ __forceinline__ float column_max(float x) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float column_sum(float x) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
// Waits until the loads' warp has begun more than n stages.  A stage of one warp's
// tokens serves warp after warp, and copies end in any order: only when its n-th
// round has begun, which needs the round before to be consumed, does the parity of
// its barrier tell the n-th from the one before.
__device__ __forceinline__ bool few_issued(const uint32_t* issued, uint32_t n, volatile int* fail, long long limit) {
  auto begun = [&]() {
    uint32_t x;
    asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];\n" : "=r"(x) : "r"(smem_u32(issued)) : "memory");
    return x > n;
  };
  if (begun()) return true;
  const long long t0 = clock64();
  while (!begun()) {
    if (*fail) return false;
    if (clock64() - t0 > limit) {
      *fail = 1;
      return false;
    }
  }
  return true;
}
// The loads of the CTA's items [i0, i1).  Bulk copies, which the lanes with one issue in
// turn: lane 8 x + b has part x (K's codes, V's, K's scales, V's) of a tile's block b and
// of the blocks of the stage that follow it in its page (all, in pages of whole tiles).
// In stages of a whole tile the scales come 16 bytes a lane instead, all at once: bulk
// copies of them keep the issue busy where pages are small (64 sequences, 8 kv heads, d =
// 64, pages of 16: 104 us with, 92 without; at d = 256, where a stage is a warp's, 373
// with, 385 without).  Returns the stages loaded.
template <int GR>
__device__ __forceinline__ int few_load(const DtParams& w, FewShared& sh, uint8_t* base, int i0, int i1, int lane) {
  const AttnDecodeParams& p = w.a;
  volatile int* fail = &sh.fail;
  constexpr int kBlocks = kFewPer<GR> * kFewBlocks;   // of a stage
  const int ST = w.k_stages, d = p.c.d, part = lane >> 3, blk = lane & 7, groups = d / kKv4Group;
  const FewStage sg = few_stage<GR>(d);
  const uint32_t codes = kv4_codes(d), scales = kv4_k_scales(d);
  const uint32_t size = part < 2 ? codes : part == 2 ? scales : kKvBlock;
  const uint32_t to = (part == 0 ? 0u : part == 1 ? sg.v : part == 2 ? sg.ks : sg.vs) + blk % kBlocks * size;
  // this lane's 16 bytes of scales: the i-th group of K's of a block, or V's after those
  constexpr int kScales = (kBlocks * (GR + 1) + 31) / 32;
  int sblk[kScales], sgrp[kScales];
#pragma unroll
  for (int k = 0; k < kScales; ++k) sblk[k] = (lane + 32 * k) / (groups + 1), sgrp[k] = (lane + 32 * k) % (groups + 1);
  int loaded = 0, st = 0, ph = 0;
  bool ok = true;
  DtItem t{};
  for (int i = i0; ok && i < i1; ++i) {
    if (i == i0) t = dt_item<kFewRows, kMaxPieces4>(w, sh.items, i);
    else dt_next<kFewRows, kMaxPieces4>(w, sh.items, i, t);
    const int32_t* bt = p.block_table + (int64_t)t.s * p.max_pages;
    int next_at = 0, next = -1;
    auto look = [&](int j) {
      const int pos = t.k0 + j * kDtTok + blk * kKvBlock;
      next_at = pos / p.c.page_tokens;
      next = pos < t.k1 && next_at < p.max_pages ? bt[next_at] : -1;
    };
    if (t.tiles > 0) look(0);
    for (int j = 0; ok && j < t.tiles; ++j) {
      const int page = next, at = next_at, pos = t.k0 + j * kDtTok + blk * kKvBlock;
      if (j + 1 < t.tiles) look(j + 1);
      const bool in = pos < t.k1, good = in && page >= 0 && page < p.c.num_pages;
      if (in && !good && part == 0) set_error(p.err, GDN_ERR_PAGE_RANGE);
      const unsigned have = __ballot_sync(0xffffffffu, good) & 0xffu;
      const int b = (pos - at * p.c.page_tokens) / kKvBlock, before = __shfl_up_sync(0xffffffffu, page, 1);
      // (the same in every part)
      const unsigned first = __ballot_sync(0xffffffffu, good && !(blk % kBlocks > 0 && b > 0 && (have >> (blk - 1) & 1) && before == page)) & 0xffu;
      // up to the next copy's first block, or the first one that is not there
      const unsigned stop = (first | ~have) >> (blk + 1);
      const int n = min((int)kDtBlocks - blk, __ffs(stop));
      const uint8_t* from = nullptr;
      if ((first >> blk & 1) && (kFewBulk<GR> || part < 2))
        from = part == 0   ? kv4_k_block(p.c, page, t.h, b)
               : part == 1 ? kv4_v_block(p.c, page, t.h, b)
               : part == 2 ? kv4_k_scale(p.c, page, t.h, b)
                           : kv4_v_scale(p.c, page, t.h, b);
#pragma unroll 1
      for (int c = 0; c < kDtBlocks / kBlocks; ++c) {
        if (loaded >= ST) ok = dt_wait(&sh.empty[st], ph ^ 1, fail, w.wait);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        if (lane == 0) {
          const unsigned mine = have >> (c * kBlocks) & ((1u << kBlocks) - 1u);
          sh.have[st] = mine;
          tc::mbar_expect_tx(&sh.full[st], __popc(mine) * (2 * codes + (kFewBulk<GR> ? scales + kKvBlock : 0)));
          if (kFewBulk<GR>) asm volatile("st.release.cta.shared::cta.u32 [%0], %1;\n" ::"r"(smem_u32(&sh.issued)), "r"(loaded + 1) : "memory");
        }
        __syncwarp();
        uint8_t* stage = base + (uint32_t)st * sg.bytes;
        if (from && blk / kBlocks == c) tc::bulk_load(stage + to, from, n * size, &sh.full[st]);
        if constexpr (!kFewBulk<GR>) {
#pragma unroll
          for (int k = 0; k < kScales; ++k) {
            const int of = c * kBlocks + sblk[k], pg = __shfl_sync(0xffffffffu, page, of & 7), pb = __shfl_sync(0xffffffffu, b, of & 7);
            if (sblk[k] < kBlocks && (have >> of & 1)) {
              if (sgrp[k] < groups) cp_async16(stage + sg.ks + sblk[k] * scales + sgrp[k] * 16, kv4_k_scale(p.c, pg, t.h, pb) + sgrp[k] * 16, 16);
              else cp_async16(stage + sg.vs + sblk[k] * kKvBlock, kv4_v_scale(p.c, pg, t.h, pb), 16);
            }
          }
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(smem_u32(&sh.full[st])) : "memory");
        }
        ++loaded;
        if (++st == ST) st = 0, ph ^= 1;
      }
    }
  }
  cp_async_commit();
  cp_async_wait<0>();
  return loaded;
}

}  // namespace

// GR: groups of 32 channels (d up to 32 GR).
template <int GR>
__global__ void __launch_bounds__(kFewThreads, kFewCtas<GR>) attn_decode4_few_kernel(const DtParams w) {
  extern __shared__ uint8_t dyn[];
  const AttnDecodeParams& p = w.a;
  uint8_t* base = dyn + ((128u - (smem_u32(dyn) & 127u)) & 127u);
  FewShared& sh = *reinterpret_cast<FewShared*>(base + w.misc_off);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, d = p.c.d;
  const int ST = w.k_stages;
  volatile int* fail = &sh.fail;
  const long long limit = w.wait;

  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) tc::mbar_init(&sh.full[i], kFewBulk<GR> ? 1 : 33), tc::mbar_init(&sh.empty[i], kFewPer<GR>);   // (33: a lane's own copies each)
    sh.fail = limit < 0;
    sh.issued = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == 0) dt_sums<kFewRows, kMaxPieces4>(w, sh, lane);
  __syncthreads();
  // this CTA's run of items
  const int i0 = dt_first<kFewRows, kMaxPieces4>(w, sh.items, sh.work, blockIdx.x, gridDim.x);
  const int last_item = dt_first<kFewRows, kMaxPieces4>(w, sh.items, sh.work, blockIdx.x + 1, gridDim.x);
  const int i1 = limit < 0 ? i0 : last_item;
  int loaded = 0;   // stages (the loading warp's)

  if (warp == kFewWarps) {
    loaded = few_load<GR>(w, sh, base, i0, i1, lane);
  } else {
    const FewStage sg = few_stage<GR>(d);
    const int g = lane >> 2, t = lane & 3, groups = d / kKv4Group;
    const uint32_t ring = smem_u32(base);
    // a lane's places in a stage: the row of K's matrices that it points at (token
    // lane % 16 of the warp's first or second block), its tokens' scales (g and g + 8 of
    // either block), its words of V (the warp's t-th)
    constexpr int PER = kFewPer<GR>, kAhead = kFewWarps / PER;   // warps of a stage, stages of a tile
    const uint32_t block = kFewBlocks * (warp % PER), next_ks = kv4_k_scales(d);
    const uint32_t at_k = (block + (lane >> 4)) * kv4_codes(d) + (lane & 15) * 16;
    const uint32_t at_ks = sg.ks + block * next_ks + g;
    const uint32_t at_v = sg.v + (block + (t >> 1)) * kv4_codes(d) + g * 8 + (t & 1) * 4;
    const uint32_t at_vs = sg.vs + block * kKvBlock + g;
    // 16 of the warp's scales, of K's or behind those of V's
    const uint32_t k_parts = kFewBlocks * groups;
    const uint32_t at_nan = lane < k_parts ? sg.ks + block * next_ks + lane * 16 : sg.vs + (block + lane - k_parts) * kKvBlock;
    float4* red = reinterpret_cast<float4*>(base + w.p_off);   // [4 warps][4 tiles][32]
    float cs[2] = {};      // factors of the scores of rows 2 t, 2 t + 1 ...
    int lim[2] = {};       // ... and the keys that they see
    bool ok = true;
    int st = warp / PER, ph = 0;   // (fewer than the stages there are)
    uint32_t nth = warp;           // stages before this one
    DtItem u{};
    for (int i = i0; i < i1; ++i) {
      if (i == i0) u = dt_item<kFewRows, kMaxPieces4>(w, sh.items, i);
      else dt_next<kFewRows, kMaxPieces4>(w, sh.items, i, u);
      if (dt_new_rows(u, i == i0)) {
        uint4 x[GR];
        float amax = 0.f;
        const int row = g / p.G, head = g - row * p.G;
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.q) + (int64_t)(u.q0 + row) * p.q_stride +
                                   (int64_t)(u.h * p.G + head) * d + t * 8;
#pragma unroll
        for (int c = 0; c < GR; ++c)
          x[c] = g < u.rows && c < groups ? *reinterpret_cast<const uint4*>(src + c * kKv4Group) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int c = 0; c < GR; ++c)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t v = (&x[c].x)[k];
            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(v << 16)), fabsf(__uint_as_float(v & 0xffff0000u))));
          }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // the largest element to [2^15, 2^16), whatever finite size it has (from below 2^-111
        // as near as 2^e and its inverse are normal)
        const int e = max(-126, min(112, (int)(__float_as_uint(amax) >> 23) - 127 - 15));
        const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
        for (int c = 0; c < GR; ++c) {
          if (c % kFewWarps != warp) continue;   // (every warp has them all)
          uint4 q;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t v = (&x[c].x)[k];
            const float s = k & 1 ? inv * 0.0625f : inv;   // codes of pairs 1 and 3 stand four bits up
            (&q.x)[k] = half2_bits(__uint_as_float(v << 16) * s, __uint_as_float(v & 0xffff0000u) * s);
          }
          sh.q[c][lane] = q;
        }
        // (an infinite element makes its row's scores NaN)
        const float f = amax < INFINITY ? p.scale_log2 * __uint_as_float((uint32_t)(127 + e) << 23) : __int_as_float(0x7fffffff);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          cs[k] = __shfl_sync(0xffffffffu, f, 8 * t + 4 * k);
          lim[k] = u.L - u.n + (2 * t + k) / p.G + 1;
        }
        dt_any<32 * kFewWarps>(false);
      }
      float o[2 * GR][4], l[2] = {0.f, 0.f}, off[2] = {kFewUnset, kFewUnset};
#pragma unroll
      for (int c = 0; c < 2 * GR; ++c)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[c][k] = 0.f;
      const int least = u.L - u.n + 1;   // keys that every row sees
#pragma unroll 1
      for (int j = 0; j < u.tiles; ++j) {
        if constexpr (PER < kFewWarps) ok = few_issued(&sh.issued, nth, fail, limit), nth += kFewWarps;
        ok = __all_sync(0xffffffffu, ok && dt_wait(&sh.full[st], ph, fail, limit));
        if (!ok) break;
        const uint8_t* stage = base + st * sg.bytes;
        const uint32_t stage_k = ring + st * sg.bytes + at_k;
        const uint8_t *k_scale = stage + at_ks, *v_scale = stage + at_vs, *v_word = stage + at_v;
        const int kb = u.k0 + j * kDtTok + kFewTok * warp;
        const unsigned have = sh.have[st] >> block & 3u;
        if (kb < u.k1 && have) {
        // ---- scores: 16 tokens at a time ----
        float x[2][4] = {};   // of block s: token g of rows 2 t, 2 t + 1, token g + 8
#pragma unroll 2
        for (int c = 0; c < groups; ++c) {
          const uint4 q = sh.q[c][lane];
          uint32_t m[4];
          ldsm4(stage_k + c * 256, m);
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const uint32_t sa = k_scale[s * next_ks + c * 16], sb = k_scale[s * next_ks + c * 16 + 8];
            uint32_t ya[4], yb[4];
            kv4_halves(m[2 * s], ya);
            kv4_halves(m[2 * s + 1], yb);
            float y[4] = {};
            mma_f16(y, ya[0], yb[0], ya[1], yb[1], q.x, q.y);
            mma_f16(y, ya[2], yb[2], ya[3], yb[3], q.z, q.w);
            const float fa = kv4_number(sa), fb = kv4_number(sb);
            x[s][0] = fmaf(y[0], fa, x[s][0]), x[s][1] = fmaf(y[1], fa, x[s][1]);
            x[s][2] = fmaf(y[2], fb, x[s][2]), x[s][3] = fmaf(y[3], fb, x[s][3]);
          }
        }
        // a NaN scale (255, taken for a number) of K makes its token's scores NaN, one of V
        // its token's weights, but not their sum
        uint4 some = make_uint4(0, 0, 0, 0);
        if (lane < k_parts + kFewBlocks) some = *reinterpret_cast<const uint4*>(stage + at_nan);
        auto full_byte = [](uint32_t v) { return (~v - 0x01010101u) & v & 0x80808080u; };
        const bool nan = __any_sync(0xffffffffu, (full_byte(some.x) | full_byte(some.y) | full_byte(some.z) | full_byte(some.w)) != 0);
        if (nan) {
          for (int c = 0; c < groups; ++c)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              if (k_scale[s * next_ks + c * 16] == kKv4Nan) x[s][0] = x[s][1] = __int_as_float(0x7fffffff);
              if (k_scale[s * next_ks + c * 16 + 8] == kKv4Nan) x[s][2] = x[s][3] = __int_as_float(0x7fffffff);
            }
        }
        // ---- weights ----
        const bool edge = have != 3u || kb + kFewTok > u.k1 || kb + kFewTok > least;
        float rv[2][2];
        float top[2];
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            // of a token: the exponent of its V scale (less 4 where its codes stand four bits
            // up), and what undoes it in the sums
            const float lv = few_log2(kv4_number(v_scale[s * kKvBlock + 8 * k])) - (g & 2 ? 4.f : 0.f);
            rv[s][k] = dt_ex2(-lv);
#pragma unroll
            for (int h = 0; h < 2; ++h) x[s][2 * k + h] = fmaf(x[s][2 * k + h], cs[h], lv);
          }
        if (edge) {
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const int end = have >> s & 1 ? u.k1 : 0, pos = kb + s * kKvBlock + g;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (pos + 4 * (k & 2) >= min(end, lim[k & 1])) x[s][k] = -INFINITY;
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) top[h] = fmaxf(fmaxf(x[0][h], x[0][2 + h]), fmaxf(x[1][h], x[1][2 + h]));
        if (__any_sync(0xffffffffu, top[0] + off[0] > kFewTop || top[1] + off[1] > kFewTop)) {
          // a row's first keys, or one far above its reference
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float mx = column_max(top[h]);
            float alpha = 1.f;
            if (off[h] == kFewUnset) {
              if (mx > -INFINITY) off[h] = kFewBase - mx;
            } else if (mx + off[h] > kFewTop) {
              alpha = dt_ex2(kFewBase - mx - off[h]);
              off[h] = kFewBase - mx;
            }
            l[h] *= alpha;
#pragma unroll
            for (int c = 0; c < 2 * GR; ++c) o[c][h] *= alpha, o[c][2 + h] *= alpha;
          }
        }
        uint32_t pb[4];   // P of row g, first by word (its tokens 2 t, 2 t + 1), then by pair (of word t)
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float a = dt_ex2(x[s][2 * k] + off[0]), b = dt_ex2(x[s][2 * k + 1] + off[1]);
            l[0] = fmaf(a, rv[s][k], l[0]), l[1] = fmaf(b, rv[s][k], l[1]);
            pb[2 * s + k] = transposed(half2_bits(a, b));
          }
        if (nan) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {   // token 2 t + j of word i, where row g sees it
              const int at = i % 2 * 8 + 2 * t + j, end = min(have >> (i / 2) & 1 ? u.k1 : 0, least + g / p.G);
              if (stage[sg.vs + (block + i / 2) * kKvBlock + at] == kKv4Nan && kb + i / 2 * kKvBlock + at < end) pb[i] |= 0x7fffu << (16 * j);
            }
        }
        kv4_transpose(pb, t);
        // ---- outputs: 16 channels at a time ----
#pragma unroll
        for (int c = 0; c < 2 * GR; ++c) {
          if (c < 2 * groups) {
            uint32_t ya[4], yb[4];
            kv4_halves(*reinterpret_cast<const uint32_t*>(v_word + c * 128), ya);
            kv4_halves(*reinterpret_cast<const uint32_t*>(v_word + c * 128 + 64), yb);
#pragma unroll
            for (int s = 0; s < 2; ++s)
              mma_f16(o[c], ya[2 * s], yb[2 * s], ya[2 * s + 1], yb[2 * s + 1], pb[2 * s], pb[2 * s + 1]);
          }
        }
        }
        __syncwarp();
        if (lane == 0) dt_arrive(&sh.empty[st]);
        st += kAhead;
        if (st >= ST) st -= ST, ph ^= 1;
      }
      // ---- the four warps' sums, brought to the largest reference and added in order ----
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        l[h] = column_sum(l[h]);
        if (lane < 4) sh.stat[warp][2 * t + h] = make_float2(off[h], l[h]);
      }
      if (dt_any<32 * kFewWarps>(!ok)) { ok = false; break; }
      const int64_t R = p.T * p.Hq;
      float sum[2], mine[2];
      int64_t rh[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int col = 2 * t + h;
        float2 s[kFewWarps];
        float least_off = kFewUnset;
#pragma unroll
        for (int v = 0; v < kFewWarps; ++v) s[v] = sh.stat[v][col], least_off = fminf(least_off, s[v].x);
        sum[h] = 0.f;
#pragma unroll
        for (int v = 0; v < kFewWarps; ++v) {
          const float f = dt_ex2(least_off - s[v].x);
          sum[h] = fmaf(s[v].y, f, sum[h]);
          if (v == warp) mine[h] = f;
        }
        const int row = col / p.G;
        rh[h] = (int64_t)(u.q0 + row) * p.Hq + u.h * p.G + col - row * p.G;
        if (warp == 0 && g == 0 && col < u.rows) {
          const float m = sum[h] == 0.f ? -INFINITY : -least_off;
          if (p.part_o) p.part_ml[u.piece * R + rh[h]] = make_float2(m, sum[h]);
          else if (p.lse) p.lse[rh[h]] = sum[h] == 0.f ? -INFINITY : m * 0.693147180559945309f + logf(sum[h]);
        }
      }
#pragma unroll
      for (int c0 = 0; c0 < 2 * GR; c0 += kFewWarps) {   // a tile of 16 channels a warp
#pragma unroll
        for (int c = 0; c < kFewWarps; ++c) {
          const float(&v)[4] = o[c0 + c];
          red[(warp * kFewWarps + c) * 32 + lane] = make_float4(v[0] * mine[0], v[1] * mine[1], v[2] * mine[0], v[3] * mine[1]);
        }
        dt_any<32 * kFewWarps>(false);
        const int ch = (c0 + warp) * 16 + g;
        if (ch < d) {
          float4 v = red[warp * 32 + lane];
#pragma unroll
          for (int k = 1; k < kFewWarps; ++k) {
            const float4 x = red[(k * kFewWarps + warp) * 32 + lane];
            v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (2 * t + h < u.rows) {
              const float a = h ? v.y : v.x, b = h ? v.w : v.z;
              if (p.part_o) {
                float* to = p.part_o + (u.piece * R + rh[h]) * d + ch;
                to[0] = a, to[8] = b;
              } else {
                __nv_bfloat16* to = static_cast<__nv_bfloat16*>(p.o) + rh[h] * d + ch;
                to[0] = __float2bfloat16_rn(sum[h] == 0.f ? 0.f : a / sum[h]);
                to[8] = __float2bfloat16_rn(sum[h] == 0.f ? 0.f : b / sum[h]);
              }
            }
          }
        }
        dt_any<32 * kFewWarps>(false);
      }
    }
  }
  __syncwarp();
  __syncthreads();
  if (sh.fail) {
    // a wait ran out: report, then give the copies in flight one more bounded
    // wait each before their memory goes
    dt_report<kFewRows, kMaxPieces4>(w, sh, i0, last_item);
    if (warp == kFewWarps && lane == 0)
      for (int n = max(0, loaded - ST); n < loaded; ++n) tc::mbar_wait_bounded(&sh.full[n % ST], (uint32_t)(n / ST) & 1, kDtWait);
    __syncwarp();
    __syncthreads();
  }
  dt_end_after_first();
}

namespace {

template <int GR>
cudaError_t few(const AttnDecodeParams& p, int sms, bool follows, cudaStream_t st) {
  DtParams w{};
  w.a = p;
  w.wait = dt_limit(p);
  w.row_lo = 1, w.row_hi = kFewRows;
  // a CTA's share of 228 KB, of which 1 KB is the system's
  const uint32_t all = 233472 / kFewCtas<GR> - 1024, red = kFewWarps * kFewWarps * 32 * sizeof(float4), misc = (uint32_t)sizeof(FewShared) + 256;
  const FewStage sg = few_stage<GR>(p.c.d);
  const int stages = (int)((all - red - misc) / sg.bytes);
  w.k_stages = stages > kFewStages ? kFewStages : stages;
  if (w.k_stages < kFewWarps / kFewPer<GR>) return cudaErrorInvalidValue;
  w.p_off = w.k_stages * sg.bytes;
  w.misc_off = w.p_off + red;
  const uint32_t smem = w.misc_off + misc;
  cudaError_t e = allow_shared(attn_decode4_few_kernel<GR>);
  if (e != cudaSuccess) return e;
  for (int s0 = 0; s0 < p.N; s0 += kDtSeqs) {
    w.s0 = s0;
    w.ns = p.N - s0 < kDtSeqs ? p.N - s0 : kDtSeqs;
    const int64_t most = (int64_t)w.ns * p.max_pieces * p.c.Hkv;
    e = dt_launch(attn_decode4_few_kernel<GR>, w, most < kFewCtas<GR> * sms ? most : kFewCtas<GR> * sms, kFewThreads, smem, follows, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_attn_decode4_few(const AttnDecodeParams& p, int sms, bool follows, cudaStream_t st) {
  return p.c.d > 128 ? few<8>(p, sms, follows, st) : p.c.d > 64 ? few<4>(p, sms, follows, st) : few<2>(p, sms, follows, st);
}

}  // namespace gdn
