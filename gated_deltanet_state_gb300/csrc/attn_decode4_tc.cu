// attn_decode4_tc.cu — attention of 1 to 32 new rows a sequence over the 4-bit
// cache, on the tensor cores (bf16 and fp32 rows, every head size of the cache).
//
// The products have the cache as their 128 rows,
//   S^T [tokens x rows] = K Q^T,    O^T [elements x rows] += V^T P^T,
// and K and V^T come from tensor memory: two kinds of warps stand between the
// codes and the products, one that unpacks codes of shared memory into operands
// there, one that makes the weights.  A code under its scale is exact in bf16, so
// K enters as it is cached, in bf16, and Q as it is given (fp32 rows in three bf16
// parts, which hold their 24 bits).  V's codes enter as whole numbers in
// f16; V's scale, one for a token and head, goes into the token's weight, an
// f16 (two parts for fp32 rows).
//
// A weight times its V scale is 2^(s + log2(vs) - M) for a reference M of its row:
// the first tile's maximum, which moves only when a weight would pass f16's range,
// so a tile costs the softmax one vote.  Weights keep 11 bits down to 2^-20 of the
// reference and are off by at most 2^-31 of it below (fp32 rows: 23 bits down to
// 2^-10, 2^-33 of it below).
//
// 16 drafts of 16 rows over 2,048 to 32,768 tokens, 24 heads, 4 kv heads, d = 256 (117
// GF, 321 MB): 220 us, 200 of them here.  A tile takes 5,000 cycles with its share of
// the items' ends, 11,000 instructions of all kinds of warps at once (issue slots 55 %
// used, the ALU pipe 47 %, most of it unpacking; the tensor pipe 32 %); what waits is
// the softmax's chain of scores, vote and weights.  Pieces of other sizes, two
// softmax warpgroups on their own, and half the registers for twice the unpacking
// warps took as long or longer.
#include "attn_decode_tc.cuh"
#include "kv4.cuh"

namespace gdn {

using namespace dt;

namespace {

// A weight at its row's reference is 2^BASE, and none passes 2^kTop (f16 ends at
// 2^16); a token whose codes stand four bits up (kv4_halves) has 2^-4 of that.
constexpr float kTop = 15.75f;
constexpr float kUnset = 3e38f;        // the offset of a row that has seen no key
// Channels of K, or tokens of V, of an operand: 64 columns of tensor memory.  (64 of
// them, so twice the operands in twice the places: 16 drafts of 16 rows 236 us, 214.)
constexpr int kChunk = 128;

// Registers of a thread by kind of warp, with one CTA on an SM: together what the
// block is launched with (16 drafts of 16 rows 210 us; 136, 80, 48: 215; 128, 80, 64:
// 217; 144, 64, 64: 225).
constexpr int kLaunchRegs = 96, kSoftRegs = 136, kUnpackRegs = 72, kRestRegs = 64;

constexpr int round16(int x) { return (x + 15) / 16 * 16; }

// NT rows a tile, QP parts of Q and PP of P side by side as columns, SWG softmax
// and UWG unpacking warpgroups, CTAS on an SM.
template <typename T_, int NT_, int QP_, int PP_, int SWG_, int UWG_, int CTAS_>
struct D4Cfg {
  using T = T_;
  static constexpr int NT = NT_, QP = QP_, PP = PP_, SWG = SWG_, UWG = UWG_, CTAS = CTAS_;
  static constexpr float BASE = sizeof(T) == 2 ? 10.f : 12.f;
  static constexpr int CW = NT / SWG;                      // columns (rows) of a softmax warpgroup
  static constexpr int NQ = round16(NT * QP), NP = round16(NT * PP);
  static constexpr int SOFT = 128 * SWG, UNPACK = 128 * UWG;
  static constexpr int THREADS = SOFT + UNPACK + (CTAS == 1 ? 128 : 96);   // and K loads, V loads, products
  static constexpr uint32_t COLS = CTAS == 1 ? 512 : 256;
  static constexpr uint32_t O0 = 2 * NQ, R0 = O0 + 2 * NP; // tensor memory: scores of two tiles, O of 128 elements each, operands
  static constexpr int SLOT = kChunk / 2, FIT = (COLS - R0) / SLOT, RING = FIT < 8 ? FIT : 8;   // columns of an operand, operands
  static_assert(CTAS > 1 || kSoftRegs * SOFT + kUnpackRegs * UNPACK + kRestRegs * (THREADS - SOFT - UNPACK) <= kLaunchRegs * THREADS, "registers");
  static_assert(RING >= 2 && RING % UWG == 0 && NT % SWG == 0 && CW % 8 == 0, "tensor memory");
};

template <typename C>
struct D4Shared : DtItems {
  uint64_t k_full[kDtMaxStages], k_empty[kDtMaxStages], v_full[kDtMaxStages], v_empty[kDtMaxStages];
  uint64_t a_full[8], a_empty[8], s_full[2], p_full[2], o_done[2], q_full, drain;
  uint32_t have[kDtMaxStages];    // blocks of a tile that were loaded, by V stage
  uint32_t nan[4 * C::SWG];       // of a softmax warp's tokens, those with a NaN scale of V
  float4 lsum[C::NT];
  float cmax[4][C::NT];           // largest score of each column, by warp
  float off[C::NT], alpha[C::NT];   // what a row's exponents are moved by: BASE less its reference
  // of a head's rows, heads alternate: keys seen, place among the outputs
  int lim[2][C::NT];
  uint32_t out[2][C::NT];         // (row, head) counted from the item's first row's head 0
};

// 32-bit words of pairs (f16, or bf16): a rounding, and what it leaves, PARTS times.
// (In bf16 towards zero: three parts hold the 24 bits so too, and no finite number
// becomes infinite.)
template <int PARTS, bool BF16>
__device__ __forceinline__ void split_pairs(float a, float b, uint32_t (&w)[PARTS]) {
#pragma unroll
  for (int i = 0; i < PARTS; ++i) {
    float2 back;
    if constexpr (BF16) {
      asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(b), "f"(a));
      back = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    } else {
      const __half2 h = __floats2half2_rn(a, b);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
      back = __half22float2(h);
    }
    a -= back.x, b -= back.y;
  }
}

// CW columns of parts NT apart, added.
template <int CW, int NT, int PARTS>
__device__ __forceinline__ void read_columns(uint32_t col, float (&x)[CW]) {
  if constexpr (PARTS == 1 && CW % 16 == 0) {
    uint32_t v[CW / 16][16];   // all loads, then one wait
#pragma unroll
    for (int k = 0; k < CW / 16; ++k) tc::tmem_ld16_nowait(col + 16 * k, v[k]);
    tc::tmem_ld_wait();
#pragma unroll
    for (int k = 0; k < CW / 16; ++k) {
      tc::tmem_ld_fence(v[k]);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[16 * k + i] = __uint_as_float(v[k][i]);
    }
  } else {
    static_assert(CW == 8 && NT == 8 && PARTS > 1, "");
    float v[16];
    tc::tmem_ld16(col, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = v[i] + v[8 + i];
    if constexpr (PARTS == 3) {
      tc::tmem_ld16(col + 16, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] += v[i];
    }
  }
}

// Sums of l[16] over a warp's lanes, into out[column] at its warp's place.
__device__ __forceinline__ void sums16(const float* l, float4* out, int n, int lane, int quad) {
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = i < n ? l[i] : 0.f;
  int bit = 16, at = 0;
#pragma unroll
  for (int half = 8; half >= 1; half >>= 1, bit >>= 1) {
    const bool up = lane & bit;
    at = 2 * at + (up ? 1 : 0);
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float send = up ? v[i] : v[i + half], keep = up ? v[i + half] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
    }
  }
  v[0] += __shfl_xor_sync(0xffffffffu, v[0], 1);
  if ((lane & 1) == 0 && at < n) (&out[at].x)[quad] = v[0];
}

// Instruction descriptor: f16 A and B, fp32 sums, M = 128.
__host__ __device__ constexpr uint32_t idesc_f16(int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kDtTok >> 4) << 24);
}

// A warp's loads of the CTA's items [i0, i1), K's codes and scales or V's: lane b
// < 8 finds the tile's block b; blocks that lie one after another in a page (all
// eight, in pages of whole tiles) come in one copy.  Returns the tiles loaded.
template <int NT, typename SH>
__device__ __forceinline__ int d4_load(const DtParams& w, SH& sh, uint8_t* base, int i0, int i1, bool is_v, int lane) {
  const AttnDecodeParams& p = w.a;
  volatile int* fail = &sh.fail;
  uint64_t *full = is_v ? sh.v_full : sh.k_full, *empty = is_v ? sh.v_empty : sh.k_empty;
  uint8_t* ring = base + (is_v ? w.v_off : w.k_off);
  const int ST = is_v ? w.v_stages : w.k_stages, d = p.c.d;
  const uint32_t codes = kv4_codes(d), scales = is_v ? kKvBlock : kv4_k_scales(d), unit = kDtBlocks * (codes + scales);
  int loaded = 0, st = 0, ph = 0;
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
      const int page = next, pos = t.k0 + j * kDtTok + lane * kKvBlock, at = pos / p.c.page_tokens;
      if (j + 1 < t.tiles) next = page_of(j + 1);
      const bool in = lane < kDtBlocks && pos < t.k1, good = in && page >= 0 && page < p.c.num_pages;
      if (in && !good) set_error(p.err, GDN_ERR_PAGE_RANGE);
      if (loaded >= ST) ok = dt_wait(&empty[st], ph ^ 1, fail, w.wait);
      if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
      const unsigned have = __ballot_sync(0xffffffffu, good);
      const int b = (pos - at * p.c.page_tokens) / kKvBlock, before = __shfl_up_sync(0xffffffffu, page, 1);
      const unsigned first = __ballot_sync(0xffffffffu, good && !(lane > 0 && b > 0 && (have >> (lane - 1) & 1) && before == page));
      if (lane == 0) {
        if (is_v) sh.have[st] = have;
        tc::mbar_expect_tx(&full[st], __popc(have) * (codes + scales));
      }
      __syncwarp();
      if (first >> lane & 1) {
        // up to the next copy's first block, or the first one that is not there
        const unsigned stop = (first | ~have) >> (lane + 1);
        const int n = min((int)kDtBlocks - lane, __ffs(stop));
        uint8_t* dst = ring + (uint32_t)st * unit;
        tc::bulk_load(dst + lane * codes, is_v ? kv4_v_block(p.c, page, t.h, b) : kv4_k_block(p.c, page, t.h, b), n * codes, &full[st]);
        tc::bulk_load(dst + kDtBlocks * codes + lane * scales,
                      is_v ? kv4_v_scale(p.c, page, t.h, b) : kv4_k_scale(p.c, page, t.h, b), n * scales, &full[st]);
      }
      ++loaded;
      if (++st == ST) st = 0, ph ^= 1;
    }
  }
  return loaded;
}

}  // namespace

template <typename C>
__global__ void __launch_bounds__(C::THREADS, C::CTAS) attn_decode4_tc_kernel(const DtParams w) {
  using E = typename C::T;
  constexpr int NT = C::NT, CW = C::CW, SW = 4 * C::SWG, UW = 4 * C::UWG;   // warps of softmax, unpacking
  extern __shared__ uint8_t dyn[];
  const AttnDecodeParams& p = w.a;
  uint8_t* base = dyn + ((128u - (smem_u32(dyn) & 127u)) & 127u);
  D4Shared<C>& sh = *reinterpret_cast<D4Shared<C>*>(base + w.misc_off);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, d = p.c.d, quad = warp & 3;
  const int KS = w.k_stages, VS = w.v_stages;
  const int halves = (d + kChunk - 1) / kChunk;   // operands of K, and of V, a tile
  volatile int* fail = &sh.fail;
  const long long limit = w.wait;

  dt_let_next(w);
  if (threadIdx.x == 0) {
    for (int i = 0; i < KS; ++i) tc::mbar_init(&sh.k_full[i], 1), tc::mbar_init(&sh.k_empty[i], UW);
    for (int i = 0; i < VS; ++i) tc::mbar_init(&sh.v_full[i], 1), tc::mbar_init(&sh.v_empty[i], UW + SW);
    for (int i = 0; i < C::RING; ++i) tc::mbar_init(&sh.a_full[i], 4), tc::mbar_init(&sh.a_empty[i], 1);
    for (int i = 0; i < 2; ++i)
      tc::mbar_init(&sh.s_full[i], 1), tc::mbar_init(&sh.p_full[i], C::SOFT), tc::mbar_init(&sh.o_done[i], 1);
    tc::mbar_init(&sh.q_full, C::SOFT);
    tc::mbar_init(&sh.drain, 1);
    sh.fail = limit < 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == SW + UW) {
    tc::tmem_alloc(&sh.tmem, C::COLS);
    tc::tmem_relinquish();
  }
  if (warp == 0) dt_sums<NT>(w, sh, lane);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tb = sh.tmem;
  // this CTA's run of items
  const int i0 = dt_first<NT>(w, sh.items, sh.work, blockIdx.x, gridDim.x);
  const int last_item = dt_first<NT>(w, sh.items, sh.work, blockIdx.x + 1, gridDim.x);
  const int i1 = limit < 0 ? i0 : last_item;
  const uint32_t codes = kv4_codes(d), k_unit = kDtBlocks * (codes + kv4_k_scales(d)), v_unit = kDtBlocks * (codes + kKvBlock);
  int loaded = 0;                               // tiles loaded (a loading warp's)

  if (warp >= SW + UW) {
    if constexpr (C::CTAS == 1) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kRestRegs));
    if (warp < SW + UW + 2) {
      // ---- loads, a warp for K and one for V ----
      loaded = d4_load<NT>(w, sh, base, i0, i1, warp == SW + UW + 1, lane);
    } else if (warp == SW + UW + 2) {
      // ---- products: the whole warp, one lane issues ----
      const uint32_t lead = tc::elect_one();
      auto all = [](bool x) { return __all_sync(0xffffffffu, x) != 0; };
      constexpr uint32_t id_qk = tc::idesc_bf16_f32(128, C::NQ), id_pv = idesc_f16(C::NP) | kTransposedB;
      const uint64_t qd = desc_tiles(smem_u32(base + w.q_off), 128, 16u * d);
      // P: tokens of 8 columns (16 B), the next 8 columns a block of 128 tokens further
      const uint64_t pd = desc_tiles(smem_u32(base + w.p_off), 128, 16 * kDtTok);
      int r = 0, rp = 0, rows = 0;   // operand and its phase
      unsigned T = 0;                // tiles multiplied
      bool ok = true;
      auto operand = [&](uint32_t dst, uint64_t b, uint32_t id, int steps, bool acc) {
        if (!all(dt_wait(&sh.a_full[r], rp, fail, limit))) return false;
        tc::fence_after_sync();
        const uint32_t a = tb + C::R0 + r * C::SLOT;
        if (steps == kChunk / 16) {
#pragma unroll
          for (int k = 0; k < kChunk / 16; ++k) tc::mma_bf16_ts_if(lead, dst, a + 8 * k, b + 16 * k, id, acc || k != 0);
        } else {
          for (int k = 0; k < steps; ++k) tc::mma_bf16_ts_if(lead, dst, a + 8 * k, b + 16 * k, id, acc || k != 0);
        }
        tc::mma_commit_if(lead, &sh.a_empty[r]);
        if (++r == C::RING) r = 0, rp ^= 1;
        return true;
      };
      auto qk = [&](unsigned tt) {
        for (int c = 0; c < halves; ++c)
          if (!operand(tb + (tt & 1) * C::NQ, qd + c * kChunk, id_qk, min(kChunk, d - c * kChunk) / 16, c != 0)) return false;
        tc::mma_commit_if(lead, &sh.s_full[tt & 1]);
        return true;
      };
      DtItem t{};
      for (int i = i0; ok && i < i1; ++i) {
        if (i == i0) t = dt_item<NT>(w, sh.items, i);
        else dt_next<NT>(w, sh.items, i, t);
        if (dt_load_rows(t, i == i0)) ok = all(dt_wait(&sh.q_full, rows++ & 1, fail, limit));
        tc::fence_after_sync();
        if (ok && t.tiles > 0) ok = qk(T);
        for (int j = 0; ok && j < t.tiles; ++j, ++T) {
          if (j + 1 < t.tiles) ok = qk(T + 1);
          ok = ok && all(dt_wait(&sh.p_full[T & 1], (T >> 1) & 1, fail, limit));
          if (!ok) break;
          tc::fence_after_sync();
          for (int hf = 0; ok && hf < halves; ++hf)
            ok = operand(tb + C::O0 + hf * C::NP, pd + (T & 1) * (C::NP * kDtTok * 2 / 16), id_pv, kDtTok / 16, j != 0);
          tc::mma_commit_if(lead, &sh.o_done[T & 1]);
        }
      }
      // every product issued, and every arrival on a barrier, before the end
      tc::mma_commit_if(lead, &sh.drain);
      if (!tc::mbar_wait_bounded(&sh.drain, 0, kDtWait)) *fail = 1;
    }
  } else if (warp >= SW) {
    // ---- codes to operands: a thread a row of them, K's tokens or V's channels ----
    if constexpr (C::CTAS == 1) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kUnpackRegs));
    const int wg = (warp - SW) >> 2, row = quad * 32 + lane;
    const uint32_t lanes = tb + C::R0 + ((uint32_t)quad << 21);
    const uint8_t *kr = base + w.k_off, *vr = base + w.v_off;
    int n = 0, r = 0, rp = 0, ks = 0, kp = 0, vs = 0, vp = 0;   // operands so far, ring and stages with their phases
    bool ok = true;
    auto mine = [&]() { return C::UWG == 1 || n % C::UWG == wg; };
    // an operand's place is free; afterwards it is there
    auto free_wait = [&]() {
      const bool x = n < C::RING || dt_wait(&sh.a_empty[r], rp ^ 1, fail, limit);
      const bool y = __all_sync(0xffffffffu, x) != 0;
      tc::fence_after_sync();
      return y;
    };
    auto done = [&]() {
      tc::tmem_st_wait();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) dt_arrive(&sh.a_full[r]);
    };
    auto next = [&]() {
      ++n;
      if (++r == C::RING) r = 0, rp ^= 1;
    };
    DtItem t{};
    for (int i = i0; ok && i < i1; ++i) {
      if (i == i0) t = dt_item<NT>(w, sh.items, i);
      else dt_next<NT>(w, sh.items, i, t);
      // in the order of the products: K of tile j, then V of the tile before
      for (int j = 0; ok && j <= t.tiles && t.tiles > 0; ++j) {
        if (j < t.tiles) {
          ok = __all_sync(0xffffffffu, dt_wait(&sh.k_full[ks], kp, fail, limit));
          const uint8_t* blk = kr + (uint32_t)ks * k_unit + (row >> 4) * codes + (row & 15) * 16;
          const uint8_t* sc = kr + (uint32_t)ks * k_unit + kDtBlocks * codes + (row >> 4) * kv4_k_scales(d) + (row & 15);
          for (int c = 0; ok && c < halves; ++c, next()) {
            if (!mine()) continue;
            const int groups = min(kChunk, d - c * kChunk) / kKv4Group;
            uint4 x[kChunk / 32];
            uint32_t s[kChunk / 32];
#pragma unroll
            for (int g = 0; g < kChunk / 32; ++g)
              if (g < groups) x[g] = *reinterpret_cast<const uint4*>(blk + (c * (kChunk / 32) + g) * 256), s[g] = sc[(c * (kChunk / 32) + g) * 16];
            ok = free_wait();
            if (!ok) break;
#pragma unroll
            for (int g = 0; g < kChunk / 32; ++g)
              if (g < groups) {
                const uint32_t s1 = kv4_scale_bf16(s[g]), s2 = s1 << 16 | s1, off = kv4_offset(s2);
                uint32_t y[16];
#pragma unroll
                for (int u = 0; u < 16; ++u) y[u] = kv4_fma(kv4_pair((&x[g].x)[u >> 2] >> (4 * (u & 3))), s2, off);
                tc::tmem_st16u(lanes + r * C::SLOT + g * 16, y);
              }
            done();
          }
          __syncwarp();
          if (lane == 0) dt_arrive(&sh.k_empty[ks]);
          if (++ks == KS) ks = 0, kp ^= 1;
        }
        if (ok && j > 0) {
          ok = __all_sync(0xffffffffu, dt_wait(&sh.v_full[vs], vp, fail, limit));
          const uint8_t* blk = vr + (uint32_t)vs * v_unit + row * 8;
          for (int hf = 0; ok && hf < halves; ++hf, next()) {
            if (!mine()) continue;
            const bool live = hf * 128 + quad * 32 < d;   // (channels past the head's: rows of O that no one reads)
            uint2 x[kDtBlocks];
#pragma unroll
            for (int b = 0; b < kDtBlocks; ++b)
              if (live) x[b] = *reinterpret_cast<const uint2*>(blk + b * codes + hf * 1024);
            ok = free_wait();
            if (!ok) break;
            if (live) {
#pragma unroll
              for (int g = 0; g < kChunk / 32; ++g) {
                uint32_t y[4][4], z[16];
#pragma unroll
                for (int u = 0; u < 4; ++u) kv4_halves(u & 1 ? x[2 * g + (u >> 1)].y : x[2 * g + (u >> 1)].x, y[u]);
#pragma unroll
                for (int u = 0; u < 16; ++u) z[u] = y[u >> 2][u & 3];
                tc::tmem_st16u(lanes + r * C::SLOT + g * 16, z);
              }
            }
            done();
          }
          __syncwarp();
          if (lane == 0) dt_arrive(&sh.v_empty[vs]);
          if (++vs == VS) vs = 0, vp ^= 1;
        }
      }
    }
  } else {
    // ---- softmax: a thread a token of the tile, CW rows ----
    if constexpr (C::CTAS == 1) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kSoftRegs));
    const int wg = warp >> 2, tid = threadIdx.x & 127, c0 = wg * CW;   // this warpgroup's first column
    const uint32_t lanes = tb + ((uint32_t)quad << 21);
    uint8_t *qs = base + w.q_off, *ps = base + w.p_off;
    const float cs = p.scale_log2;
    bool ok = true;
    // an item's rows as the products' columns, a warp a row at a time, loads
    // first; where they belong is noted for an item without keys too
    auto load_q = [&](const DtItem& t, int par) {
      const int e0 = lane * 8;
      constexpr int ROWS = NT / SW, NB = ROWS > 4 ? 4 : ROWS;   // of a warp; loaded at once
#pragma unroll 1
      for (int b0 = 0; b0 < ROWS; b0 += NB) {
        uint4 x[NB][sizeof(E) / 2];
#pragma unroll
        for (int u = 0; u < NB; ++u) {
          const int n = (b0 + u) * SW + warp;
#pragma unroll
          for (int v = 0; v < (int)sizeof(E) / 2; ++v) x[u][v] = make_uint4(0, 0, 0, 0);
          if (n < t.rows) {
            const int row = (t.r0 + n) / p.G, g = t.r0 + n - row * p.G;
            const E* src = static_cast<const E*>(p.q) + (int64_t)(t.q0 + row) * p.q_stride + (int64_t)(t.h * p.G + g) * d + e0;
            if (t.tiles > 0 && e0 < d)
#pragma unroll
              for (int v = 0; v < (int)sizeof(E) / 2; ++v) x[u][v] = reinterpret_cast<const uint4*>(src)[v];
            if (lane == 0) {
              sh.lim[par][n] = t.L - t.n + row + 1;
              sh.out[par][n] = (uint32_t)((row - t.r0 / p.G) * p.Hq + t.h * p.G + g);
            }
          }
        }
        if (t.tiles == 0 || e0 >= d) continue;
#pragma unroll
        for (int u = 0; u < NB; ++u) {
          const int n = (b0 + u) * SW + warp;
          auto at = [&](int col) { return reinterpret_cast<uint4*>(qs + (col >> 3) * 16 * d + lane * 128 + (col & 7) * 16); };
          if constexpr (sizeof(E) == 2) {
            *at(n) = x[u][0];
          } else {
            uint32_t part[4][C::QP];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint4& f = x[u][k >> 1];
              split_pairs<C::QP, true>(__uint_as_float(k & 1 ? f.z : f.x), __uint_as_float(k & 1 ? f.w : f.y), part[k]);
            }
#pragma unroll
            for (int v = 0; v < C::QP; ++v) *at(v * NT + n) = make_uint4(part[0][v], part[1][v], part[2][v], part[3][v]);
          }
        }
      }
      if (t.tiles == 0) return;
      tc::fence_async_smem();
      dt_arrive(&sh.q_full);
    };
    unsigned T = 0;
    int st = 0, vp = 0, par = 0;   // V stage and its phase; head
    DtItem t{};
    if (threadIdx.x < NT) sh.off[threadIdx.x] = kUnset;
    if (i0 < i1) {
      t = dt_item<NT>(w, sh.items, i0);
      load_q(t, 0);
    }
    dt_any<C::SOFT>(false);
    for (int i = i0; i < i1; ++i) {
      float l[CW];
#pragma unroll
      for (int n = 0; n < CW; ++n) l[n] = 0.f;
      const int least = t.L - t.n + t.r0 / p.G + 1;   // keys that every row of the tile sees
      for (int j = 0; j < t.tiles; ++j, ++T) {
        const int kb = t.k0 + j * kDtTok, pos = kb + tid;
        const uint32_t scol = lanes + (T & 1) * C::NQ + c0;
        // V's part first: it is there before the scores
        ok = dt_wait(&sh.v_full[st], vp, fail, limit);
        const uint32_t vbyte = (base + w.v_off + (uint32_t)st * v_unit + kDtBlocks * codes)[tid];
        const bool valid = pos < t.k1 && (sh.have[st] >> (tid >> 4) & 1);
        // (kept in shared memory until the weights: in a register, 16 drafts of 16 rows 202 us, 199)
        const unsigned nan = __ballot_sync(0xffffffffu, valid && vbyte == kKv4Nan);
        if (lane == 0) sh.nan[warp] = nan;
        __syncwarp();
        if (lane == 0) dt_arrive(&sh.v_empty[st]);
        // of this token: the exponent of its V scale, and what undoes it in the sums of
        // weights (a NaN scale counts as a number until the weights are made)
        const float vscale = kv4_number(vbyte), lv = __log2f(vscale) - (tid & 2 ? 4.f : 0.f);
        const float rv = __fdividef(tid & 2 ? 16.f : 1.f, vscale);
        const bool part = !__all_sync(0xffffffffu, valid), edge = kb + kDtTok > least;   // some row does not see some token
        ok = ok && dt_wait(&sh.s_full[T & 1], (T >> 1) & 1, fail, limit);
        __syncwarp();
        tc::fence_after_sync();
        float x[CW];
        // s + log2(vs) + off, where off is the rows' offsets or nothing; masked -inf
        auto scores = [&](bool against) {
          read_columns<CW, NT, C::QP>(scol, x);
          const float4* r4 = reinterpret_cast<const float4*>(&sh.off[c0]);
          const f32x2 cc = pack2(cs, cs), ll = pack2(lv, lv);
#pragma unroll
          for (int k = 0; k < CW; k += 4) {
            float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
            if (against) r = r4[k / 4];
            const float2 a = unpack2(fma2(pack2(x[k], x[k + 1]), cc, add2(pack2(r.x, r.y), ll)));
            const float2 b = unpack2(fma2(pack2(x[k + 2], x[k + 3]), cc, add2(pack2(r.z, r.w), ll)));
            x[k] = a.x, x[k + 1] = a.y, x[k + 2] = b.x, x[k + 3] = b.y;
          }
          if (part || edge) {
#pragma unroll
            for (int k = 0; k < CW; ++k)
              if (!valid || pos >= sh.lim[par][c0 + k]) x[k] = -INFINITY;
          }
        };
        scores(true);
        float top[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int k = 4; k < CW; ++k) top[k & 3] = fmaxf(top[k & 3], x[k]);
        if (dt_any<C::SOFT>(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) > kTop || !ok)) {
          // a row's first keys, or one far above its reference (or a wait that ran
          // out): a row's reference moves by that row's scores alone
          scores(false);
#pragma unroll
          for (int k = 0; k < CW; k += 4) {
            const float a = warp_max(x[k]), b = warp_max(x[k + 1]), c = warp_max(x[k + 2]), e = warp_max(x[k + 3]);
            if (lane == 0) *reinterpret_cast<float4*>(&sh.cmax[quad][c0 + k]) = make_float4(a, b, c, e);
          }
          // the products before this tile's are done with O
          if (j > 0) ok = ok && dt_wait(&sh.o_done[(T - 1) & 1], ((T - 1) >> 1) & 1, fail, limit);
          if (dt_any<C::SOFT>(!ok)) { ok = false; break; }
          if (tid < CW) {
            const int n = c0 + tid;
            const float mx = fmaxf(fmaxf(sh.cmax[0][n], sh.cmax[1][n]), fmaxf(sh.cmax[2][n], sh.cmax[3][n]));
            const float off = sh.off[n];
            float alpha = 1.f;
            if (off == kUnset) {
              if (mx > -INFINITY) sh.off[n] = C::BASE - mx;
            } else if (mx + off > kTop) {
              alpha = dt_ex2(C::BASE - mx - off);
              sh.off[n] = C::BASE - mx;
            }
            sh.alpha[n] = alpha;
          }
          dt_any<C::SOFT>(false);
          if (j > 0) {
            tc::fence_after_sync();
#pragma unroll
            for (int n = 0; n < CW; ++n) l[n] *= sh.alpha[c0 + n];
            for (int hf = 0; hf < halves; ++hf) {
#pragma unroll 1
              for (int v = 0; v < C::PP; ++v) {
#pragma unroll 1
                for (int c = 0; c < CW; c += 8) {
                  const uint32_t col = lanes + C::O0 + hf * C::NP + v * NT + c0 + c;
                  uint32_t o[8];
                  tc::tmem_ld8(col, o);
#pragma unroll
                  for (int k = 0; k < 8; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * sh.alpha[c0 + c + k]);
                  tc::tmem_st8(col, o);
                }
              }
            }
            tc::tmem_st_wait();
          }
          scores(true);
        }
        // the weights (the products of two tiles ago, which read this place, were done
        // before this tile's scores)
        uint8_t* pw = ps + (T & 1) * (C::NP * kDtTok * 2) + tid * 16;
        const f32x2 rr = pack2(rv, rv);
#pragma unroll
        for (int k = 0; k < CW; k += 8) {
          uint32_t word[4][C::PP];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int n = k + 2 * u;
            const float a = dt_ex2(x[n]), b = dt_ex2(x[n + 1]);
            const float2 sum = unpack2(fma2(pack2(a, b), rr, pack2(l[n], l[n + 1])));
            l[n] = sum.x, l[n + 1] = sum.y;
            split_pairs<C::PP, false>(a, b, word[u]);
          }
#pragma unroll
          for (int v = 0; v < C::PP; ++v)
            *reinterpret_cast<uint4*>(pw + ((v * NT + c0 + k) >> 3) * (16 * kDtTok)) =
                make_uint4(word[0][v], word[1][v], word[2][v], word[3][v]);
        }
        // a NaN scale of V makes the weights of the rows that see its token NaN, not their sums
        if (sh.nan[warp] >> lane & 1) {
#pragma unroll 1
          for (int n = c0; n < c0 + CW; ++n)
            if (pos < sh.lim[par][n]) reinterpret_cast<uint16_t*>(pw + (n >> 3) * (16 * kDtTok))[n & 7] = 0x7fff;
        }
        __syncwarp();
        tc::fence_async_smem();
        tc::fence_before_sync();
        dt_arrive(&sh.p_full[T & 1]);
        if (++st == VS) st = 0, vp ^= 1;
      }
      if (!ok) break;
      // the next head's rows: its scores may then start while this item ends
      const DtItem u = t;
      const int was = par;
      if (i + 1 < i1) {
        dt_next<NT>(w, sh.items, i + 1, t);
        if (dt_new_rows(t, false)) load_q(t, par ^= 1);
      }
#pragma unroll
      for (int k = 0; k < CW; k += 16) sums16(l + k, sh.lsum + c0 + k, CW - k < 16 ? CW - k : 16, lane, quad);
      if (u.tiles > 0) ok = dt_wait(&sh.o_done[(T - 1) & 1], ((T - 1) >> 1) & 1, fail, limit);
      if (dt_any<C::SOFT>(!ok)) { ok = false; break; }
      tc::fence_after_sync();
      const int64_t R = p.T * p.Hq, rh0 = (int64_t)(u.q0 + u.r0 / p.G) * p.Hq;
      const int rows = min(CW, u.rows - c0);   // columns of this warpgroup that are rows
      auto total = [&](int n) {
        const float4 c = sh.lsum[n];
        return (c.x + c.y) + (c.z + c.w);
      };
      if (tid < rows) {
        const int n = c0 + tid;
        const float sum = u.tiles > 0 ? total(n) : 0.f, m = sum == 0.f ? -INFINITY : -sh.off[n];
        const int64_t rh = rh0 + sh.out[was][n];
        if (p.part_o) p.part_ml[u.piece * R + rh] = make_float2(m, sum);
        else if (p.lse) p.lse[rh] = sum == 0.f ? -INFINITY : m * 0.693147180559945309f + logf(sum);
      }
      __syncwarp();
      for (int hf = 0; hf < halves; ++hf) {
        const int e = hf * 128 + tid;
        float* po = p.part_o + (u.piece * R + rh0) * d + e;
        E* oo = static_cast<E*>(p.o) + rh0 * d + e;
#pragma unroll
        for (int k0 = 0; k0 < CW; k0 += 16) {
          constexpr int W = CW < 16 ? CW : 16;
          float o[W];
          if (u.tiles > 0) {
            read_columns<W, NT, C::PP>(lanes + C::O0 + hf * C::NP + c0 + k0, o);
          } else {
#pragma unroll
            for (int k = 0; k < W; ++k) o[k] = 0.f;
          }
          if (e < d) {
#pragma unroll
            for (int k = 0; k < W; ++k) {
              if (k0 + k < rows) {
                const uint32_t at = sh.out[was][c0 + k0 + k] * (uint32_t)d;   // at most 32 rows of 1,024 heads of 256 elements
                if (p.part_o) {
                  po[at] = o[k];
                } else {
                  const float sum = u.tiles > 0 ? total(c0 + k0 + k) : 0.f;
                  oo[at] = from_f32<E>(sum == 0.f ? 0.f : o[k] / sum);
                }
              }
            }
          }
          __syncwarp();
        }
      }
      tc::fence_before_sync();
      dt_any<C::SOFT>(false);   // lsum, references and O are free
      if (threadIdx.x < NT) sh.off[threadIdx.x] = kUnset;
      dt_any<C::SOFT>(false);
    }
  }
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  if (sh.fail) {
    // a wait ran out: report, then give the copies in flight one more bounded
    // wait each before their memory goes
    dt_report<NT>(w, sh, i0, last_item);
    if ((warp == SW + UW || warp == SW + UW + 1) && lane == 0) dt_drain(w, sh, loaded, warp == SW + UW + 1);
    __syncwarp();
    __syncthreads();
  }
  tc::fence_after_sync();
  if (warp == SW + UW) tc::tmem_dealloc(tb, C::COLS);
}

namespace {

template <typename C>
cudaError_t decode4(const AttnDecodeParams& p, int sms, int lo, bool first, cudaStream_t st) {
  DtParams w{};
  w.a = p;
  w.wait = dt_limit(p);
  w.row_lo = lo, w.row_hi = 0x7fffffff;
  w.first = first;
  const uint32_t d = (uint32_t)p.c.d, q = C::NQ * d * 2, pp = 2 * C::NP * kDtTok * 2, misc = (uint32_t)sizeof(D4Shared<C>);
  // 227 KB, or half of them a CTA, of which 1 KB is the system's
  const uint32_t all = C::CTAS == 1 ? 232448 : 115712;
  const uint32_t ku = kDtBlocks * (kv4_codes(d) + kv4_k_scales(d)), vu = kDtBlocks * (kv4_codes(d) + kKvBlock);
  const int units = (int)((all - q - pp - misc - 512) / ku);
  w.k_stages = units - units / 2 > kDtMaxStages ? kDtMaxStages : units - units / 2;
  w.v_stages = units / 2 > kDtMaxStages ? kDtMaxStages : units / 2;
  if (w.v_stages < 1) return cudaErrorInvalidValue;
  w.k_off = 0;
  w.v_off = w.k_stages * ku;
  w.q_off = (w.v_off + w.v_stages * vu + 127) / 128 * 128;
  w.p_off = w.q_off + q;
  w.misc_off = w.p_off + pp;
  uint32_t smem = w.misc_off + misc + 128;
  // no more than CTAS on an SM, which share its tensor memory
  const uint32_t least = C::CTAS == 1 ? 120 * 1024 : 80 * 1024;
  if (smem < least) smem = least;
  cudaError_t e = allow_shared(attn_decode4_tc_kernel<C>);
  if (e != cudaSuccess) return e;
  const int tiles = (p.max_q * p.G + C::NT - 1) / C::NT;
  for (int s0 = 0; s0 < p.N; s0 += kDtSeqs) {
    w.s0 = s0;
    w.ns = p.N - s0 < kDtSeqs ? p.N - s0 : kDtSeqs;
    const int64_t most = (int64_t)w.ns * p.max_pieces * p.c.Hkv * tiles, run = (int64_t)C::CTAS * sms;
    attn_decode4_tc_kernel<C><<<(unsigned)(most < run ? most : run), C::THREADS, smem, st>>>(w);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

using Mid = D4Cfg<__nv_bfloat16, 16, 1, 1, 1, 1, 2>;
using Some = D4Cfg<__nv_bfloat16, 32, 1, 1, 2, 2, 1>;
using Many = D4Cfg<__nv_bfloat16, 96, 1, 1, 2, 2, 1>;
using Full8 = D4Cfg<float, 8, 3, 2, 1, 1, 2>;

}  // namespace

cudaError_t launch_attn_decode4_tc(const AttnDecodeParams& p, int dtype, cudaStream_t st) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  if (dtype == GDN_F32) return decode4<Full8>(p, sms, 1, false, st);
  // a sequence's kernel goes by its own rows (a row's bits with it): up to 8 (row,
  // head) pairs of a kv head, or more, of which either form gives the same bits; a
  // call that may have both launches both.  (What rows there are in all does not
  // tell: one sequence may have too many and be left out, or rows may stand behind
  // the last sequence.)
  const int most = p.max_q * p.G;
  const bool few = p.G <= kD4Few, many = most > kD4Few;
  const int lo = few ? kD4Few + 1 : 1;
  if (many) e = most <= 16   ? decode4<Mid>(p, sms, lo, few, st)
                : most <= 32 ? decode4<Some>(p, sms, lo, few, st)
                             : decode4<Many>(p, sms, lo, few, st);
  return e == cudaSuccess && few ? launch_attn_decode4_few(p, sms, many, st) : e;
}

}  // namespace gdn
