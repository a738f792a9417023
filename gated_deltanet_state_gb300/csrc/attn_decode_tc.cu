// attn_decode_tc.cu — attention of a few new rows a sequence over the 8-bit
// cache, on the tensor cores (bf16 rows, d a multiple of 32).
//
// The cache's e4m3 codes are the operands as they lie in memory: with 128
// tokens as the rows of the first product and the head's elements as the rows
// of the second,
//   S^T [tokens x rows] = K Q^T,    O^T [elements x rows] += V^T P^T,
// no code is converted, and the few query rows are the products' narrow side
// (NT columns).  Q and P enter as two e4m3 parts each, x = hi + lo, both
// accumulated into the same sums: hi keeps 4 significant bits, lo 4 more of
// what is left, which is all 8 of a bf16 q (scaled by a power of two so that
// its largest element is in (224, 448]; parts below 2^-9 vanish, 2^-18 of that
// element) and rounds p like bf16 would.  A block's K scale multiplies its
// scores; its V scale goes into the weight's exponent, so a weight is
// 2^(s + log2(vs) - M) and the sum of the p is the sum of the weights over vs.
#include "attn.h"
#include "tc.cuh"

namespace gdn {

namespace {

constexpr int kDtTok = 128;           // tokens of a tile
constexpr int kDtBlocks = kDtTok / kKvBlock;
constexpr int kDtSeqs = 512;         // sequences a launch
constexpr int kDtMaxStages = 8;
constexpr long long kDtWait = 4000000000LL;
constexpr float kDtBase = 7.f;        // weights are scaled by 2^7 ...
constexpr float kDtGrow = 1.75f;      // ... and may exceed that by 2^1.75: 430 < 448

// NT columns; CW of them a softmax warpgroup (128 threads, a token each).
template <int NT>
struct DtCfg {
  static constexpr int CW = NT < 32 ? NT : 32, WGS = NT / CW;
  static constexpr int THREADS = WGS * 128 + 96;       // and K loads, V loads, products
  // narrow tiles: two CTAs an SM, one's softmax under the other's products and loads
  static constexpr int CTAS = NT <= 32 ? 2 : 1;
  static constexpr int PB = NT <= 64 ? 2 : 1;          // weights of two tiles while shared memory allows it
  static constexpr uint32_t COLS = NT <= 16 ? 64 : NT <= 32 ? 128 : NT <= 64 ? 256 : 512;
  static constexpr uint32_t O0 = 2 * NT;               // scores of two tiles, then O of 128 elements each
};

struct DtParams {
  AttnDecodeParams a;
  int32_t s0, ns;       // this launch's sequences
  int32_t stages;
  uint32_t k_off, v_off, q_off, p_off, misc_off;   // dynamic shared memory
};

template <int NT>
struct DtShared {
  uint64_t k_full[kDtMaxStages], k_empty[kDtMaxStages], v_full[kDtMaxStages], v_empty[kDtMaxStages];
  uint64_t sc_full[kDtMaxStages + 2], s_full[2], p_full[2], o_done[2], q_full, drain;
  float ks[kDtMaxStages + 2][kDtBlocks], vs[kDtMaxStages + 2][kDtBlocks];
  float4 lsum[NT];
  float cmax[4][NT];        // largest score of each column, by warp
  float ref[NT], alpha[NT];
  // of an item's columns, items alternate: score factor, keys seen, place among the outputs
  float fq[2][NT];
  int lim[2][NT];
  int64_t out[2][NT];
  int bad[2][256];          // first token with a NaN value that not every row sees, by element
  int items[kDtSeqs + 1];   // running sum of the sequences' work items
  uint32_t tmem;
  int fail;
  unsigned grow[DtCfg<NT>::WGS];   // the last tile (from 1) that moved a column's reference
};

__device__ __forceinline__ bool dt_wait(uint64_t* m, uint32_t parity, volatile int* fail) {
  if (tc::mbar_test_wait(m, parity)) return true;
  const long long t0 = clock64();
  while (!tc::mbar_try_wait(m, parity)) {
    if (*fail) return false;
    if (clock64() - t0 > kDtWait) {
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

// e4m3 x e4m3 -> fp32: D[tmem] (+)= A[smem] B[smem]^T, 32 deep.
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// Instruction descriptor: e4m3 A and B (both K-contiguous), fp32 sums, M = 128.
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
  int s, h, r0, rows, piece;   // rows: (row, head) pairs of this item, from r0
  int q0, n, L, k0, k1, tiles;
};

template <int NT>
__device__ __forceinline__ int dt_items(const AttnDecodeParams& p, int s) {
  const int n = p.cu[s + 1] - p.cu[s], L = p.kv_len[s];
  if (n <= 0) return 0;
  if (n > p.max_q || L > p.max_kv || L < 0 || p.cu[s] < 0 || (int64_t)p.cu[s] + n > p.T) return -1;
  return decode_pieces(L, n * p.G) * p.c.Hkv * ((n * p.G + NT - 1) / NT);
}

template <int NT>
__device__ __forceinline__ DtItem dt_item(const DtParams& w, const int* items, int i) {
  const AttnDecodeParams& p = w.a;
  int lo = 0, hi = w.ns;   // the last s with items[s] <= i
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (items[mid] <= i) lo = mid;
    else hi = mid;
  }
  DtItem t;
  t.s = w.s0 + lo;
  int k = i - items[lo];
  t.q0 = p.cu[t.s];
  t.n = p.cu[t.s + 1] - t.q0;
  t.L = p.kv_len[t.s];
  const int rt = (t.n * p.G + NT - 1) / NT;
  t.r0 = k % rt * NT;
  k /= rt;
  t.h = k % p.c.Hkv;
  t.piece = k / p.c.Hkv;
  t.rows = min(NT, t.n * p.G - t.r0);
  const int pt = decode_piece_tokens(t.L, t.n * p.G);
  t.k0 = t.piece * pt;
  t.k1 = min(t.L, t.k0 + pt);
  t.tiles = (t.k1 - t.k0 + kDtTok - 1) / kDtTok;
  return t;
}

// Sums of v[16] over 32 lanes: lane l ends with column l >> 1, 16 shuffles.
__device__ __forceinline__ float sum16(float (&v)[16], int lane) {
#pragma unroll
  for (int half = 8, bit = 16; half >= 1; half >>= 1, bit >>= 1) {
    const bool up = lane & bit;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float send = up ? v[i] : v[i + half], keep = up ? v[i + half] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
    }
  }
  return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
}
// Largest value of a warp (NaN falls out).
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;\n" : "=f"(r) : "f"(x));
  return r;
}

// Barrier of a softmax warpgroup; true when all of it says so, which keeps it
// together when a wait has run out.
__device__ __forceinline__ bool bar_and(bool ok, int id) {
  int r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n barrier.cta.red.and.pred q, %2, 128, p;\n"
      " selp.s32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((int)ok), "r"(id)
      : "memory");
  __syncwarp();
  return r != 0;
}

}  // namespace

template <int NT>
__global__ void __launch_bounds__(DtCfg<NT>::THREADS, DtCfg<NT>::CTAS) attn_decode_tc_kernel(const DtParams w) {
  using C = DtCfg<NT>;
  constexpr int CW = C::CW, WARPS = C::WGS * 4;   // softmax warps; then K loads, V loads, products
  extern __shared__ uint8_t dyn[];
  const AttnDecodeParams& p = w.a;
  uint8_t* base = dyn + ((128u - (smem_u32(dyn) & 127u)) & 127u);
  DtShared<NT>& sh = *reinterpret_cast<DtShared<NT>*>(base + w.misc_off);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, d = p.c.d, ST = w.stages, NS = ST + 2;
  volatile int* fail = &sh.fail;

  if (threadIdx.x == 0) {
    sh.items[0] = 0;
    for (int i = 0; i < ST; ++i) {
      tc::mbar_init(&sh.k_full[i], 1), tc::mbar_init(&sh.k_empty[i], 1);
      tc::mbar_init(&sh.v_full[i], 1), tc::mbar_init(&sh.v_empty[i], 1);
    }
    for (int i = 0; i < NS; ++i) tc::mbar_init(&sh.sc_full[i], 2 * kDtBlocks);
    for (int i = 0; i < 2; ++i)
      tc::mbar_init(&sh.s_full[i], 1), tc::mbar_init(&sh.p_full[i], C::WGS * 128), tc::mbar_init(&sh.o_done[i], 1);
    tc::mbar_init(&sh.q_full, C::WGS * 128);
    tc::mbar_init(&sh.drain, 1);
    sh.fail = 0;
    for (int i = 0; i < C::WGS; ++i) sh.grow[i] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == WARPS) {
    tc::tmem_alloc(&sh.tmem, C::COLS);
    tc::tmem_relinquish();
  }
  // running sum of the items; lengths out of bounds are reported and have none
  if (warp == 0) {
    int sum = 0;
    for (int c = 0; c < w.ns; c += 32) {
      int v = c + lane < w.ns ? dt_items<NT>(p, w.s0 + c + lane) : 0;
      if (v < 0) {
        if (blockIdx.x == 0) set_error(p.err, GDN_ERR_INVALID_ARG);
        v = 0;
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
      }
      if (c + lane < w.ns) sh.items[c + lane + 1] = sum + v;
      sum += __shfl_sync(0xffffffffu, v, 31);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tb = sh.tmem;
  const int total = sh.items[w.ns];
  const uint32_t unit = (uint32_t)kDtTok * d;   // bytes of a tile's K (or V) codes
  int loaded = 0;                               // tiles loaded (a loading warp's)

  if (warp == WARPS || warp == WARPS + 1) {
    // ---- loads, a warp for K and one for V: lane b < 8 the tile's block b ----
    const bool is_v = warp == WARPS + 1;
    uint64_t *full = is_v ? sh.v_full : sh.k_full, *empty = is_v ? sh.v_empty : sh.k_empty;
    uint8_t* ring = base + (is_v ? w.v_off : w.k_off);
    int st = 0, ph = 0, sc = 0;
    bool ok = true;
    for (int i = blockIdx.x; ok && i < total; i += gridDim.x) {
      const DtItem t = dt_item<NT>(w, sh.items, i);
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
        if (loaded >= ST) ok = dt_wait(&empty[st], ph ^ 1, fail);
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
  } else if (warp == WARPS + 2) {
    // ---- products ----
    if (lane == 0) {
      constexpr uint32_t id = idesc_e4m3(NT);
      const uint32_t k0 = smem_u32(base + w.k_off), v0 = smem_u32(base + w.v_off), qa = smem_u32(base + w.q_off),
                     pa = smem_u32(base + w.p_off);
      const uint32_t rows8 = 8u * d;   // 8 tokens of K (or 8 rows of Q)
      const int halves = (d + 127) / 128;
      int ks = 0, kp = 0, vs = 0, vp = 0, item = 0;
      unsigned T = 0;   // tiles multiplied
      bool ok = true;
      auto qk = [&](unsigned tt) {
        if (!dt_wait(&sh.k_full[ks], kp, fail)) return false;
        tc::fence_after_sync();
        const uint64_t a = desc_tiles(k0 + ks * unit, 128, rows8);
        for (int part = 0; part < 2; ++part) {
          const uint64_t b = desc_tiles(qa + part * NT * d, 128, rows8);
          for (int c = 0; c < d / 32; ++c) mma_e4m3(tb + (tt & 1) * NT, a + c * 16, b + c * 16, id, part | c);
        }
        tc::mma_commit(&sh.k_empty[ks]);
        tc::mma_commit(&sh.s_full[tt & 1]);
        if (++ks == ST) ks = 0, kp ^= 1;
        return true;
      };
      for (int i = blockIdx.x; ok && i < total; i += gridDim.x, ++item) {
        const DtItem t = dt_item<NT>(w, sh.items, i);
        ok = dt_wait(&sh.q_full, item & 1, fail);
        if (ok && t.tiles > 0) ok = qk(T);
        for (int j = 0; ok && j < t.tiles; ++j, ++T) {
          if (j + 1 < t.tiles) ok = qk(T + 1);
          ok = ok && dt_wait(&sh.p_full[T & 1], (T >> 1) & 1, fail) && dt_wait(&sh.v_full[vs], vp, fail);
          if (!ok) break;
          tc::fence_after_sync();
          for (int hf = 0; hf < halves; ++hf)
            for (int part = 0; part < 2; ++part) {
              const uint64_t a = desc_tiles(v0 + vs * unit + hf * 2048u, 16u * d, 128);
              // P: tokens of 16 columns (16 B), the next 16 columns a block of 128 tokens further
              const uint64_t b = desc_tiles(pa + ((T & (C::PB - 1)) * 2 + part) * NT * kDtTok, 128, 16 * kDtTok);
#pragma unroll
              for (int c = 0; c < kDtTok / 32; ++c)
                mma_e4m3(tb + C::O0 + hf * NT, a + ((uint32_t)c * 32u * d >> 4), b + c * 32, id | kTransposedB, j | part | c);
            }
          tc::mma_commit(&sh.v_empty[vs]);
          tc::mma_commit(&sh.o_done[T & 1]);
          if (++vs == ST) vs = 0, vp ^= 1;
        }
      }
      // every product issued, and every arrival on a barrier, before the end
      tc::mma_commit(&sh.drain);
      if (!tc::mbar_wait_bounded(&sh.drain, 0, kDtWait)) *fail = 1;
    }
  } else {
    // ---- softmax: a thread a token of the tile, a warpgroup CW columns ----
    const int wg = warp >> 2, quad = warp & 3, tid = threadIdx.x & 127, c0 = wg * CW, bar = 1 + wg;
    const uint32_t lanes = tb + ((uint32_t)quad << 21);
    uint8_t* qd = base + w.q_off;
    uint8_t* pd = base + w.p_off;
    bool ok = true;
    // an item's rows as hi and lo codes, a warp a row at a time, all loads first
    auto load_q = [&](const DtItem& t, int par) {
      const int e0 = lane * 8;
      constexpr int NR = CW / 4;
      uint4 x[NR];
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const int n = c0 + r * 4 + quad;
        x[r] = make_uint4(0, 0, 0, 0);
        if (n < t.rows) {
          const int row = (t.r0 + n) / p.G, g = t.r0 + n - row * p.G;
          if (e0 < d)
            x[r] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + (int64_t)(t.q0 + row) * p.q_stride +
                                                   (int64_t)(t.h * p.G + g) * d + e0);
          if (lane == 0) {
            sh.lim[par][n] = t.L - t.n + row + 1;
            sh.out[par][n] = (int64_t)(t.q0 + row) * p.Hq + t.h * p.G + g;
          }
        }
      }
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const int n = c0 + r * 4 + quad;
        float f[8], amax = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t u = (&x[r].x)[k >> 1];
          f[k] = __uint_as_float(k & 1 ? u & 0xffff0000u : u << 16);
          amax = fmaxf(amax, fabsf(f[k]));
        }
        amax = warp_max(amax);
        // largest element to (224, 448]; exponents kept where both factors are normal
        int e = (int)(__float_as_uint(amax) >> 23) - 127 - 8 + ((__float_as_uint(amax) & 0x7fffffu) > 0x600000u ? 1 : 0);
        e = max(-100, min(100, e));
        const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
        uint32_t hi[2], lo[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float g4[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) g4[u] = f[4 * k + u] * inv;
          hi[k] = e4m3x4(g4[0], g4[1], g4[2], g4[3]);
          const float2 a = e4m3_f32x2(hi[k]), b = e4m3_f32x2(hi[k] >> 16);
          lo[k] = e4m3x4(g4[0] - a.x, g4[1] - a.y, g4[2] - b.x, g4[3] - b.y);
        }
        if (e0 < d) {
          uint8_t* at = qd + (n >> 3) * 8 * d + (e0 >> 4) * 128 + (n & 7) * 16 + (e0 & 8);
          *reinterpret_cast<uint2*>(at) = make_uint2(hi[0], hi[1]);
          *reinterpret_cast<uint2*>(at + NT * d) = make_uint2(lo[0], lo[1]);
        }
        // an infinite element makes the row NaN, as its codes would not
        if (lane == 0)
          sh.fq[par][n] = amax < INFINITY ? p.scale_log2 * __uint_as_float((uint32_t)(127 + e) << 23)
                                          : __int_as_float(0x7fffffff);
      }
      tc::fence_async_smem();
      dt_arrive(&sh.q_full);
    };
    unsigned T = 0;
    int st = 0, sc = 0, scp = 0, vp = 0, par = 0;   // V stage and its phase, scale slot and its phase, item
    DtItem t{};
    if ((int)blockIdx.x < total) {
      t = dt_item<NT>(w, sh.items, blockIdx.x);
      load_q(t, 0);
    }
    bar_and(true, bar);
    for (int i = blockIdx.x; i < total; i += gridDim.x, par ^= 1) {
      float l[CW];
#pragma unroll
      for (int n = 0; n < CW; ++n) l[n] = 0.f;
      float ref = -INFINITY;                          // of column c0 + tid
      if (wg == 0) sh.bad[par][tid] = sh.bad[par][tid + 128] = 0x7fffffff;
      const int least = t.L - t.n + 1;                // keys that every row sees
      for (int j = 0; j < t.tiles; ++j, ++T) {
        const int kb = t.k0 + j * kDtTok, pos = kb + tid;
        const uint32_t scol = lanes + (T & 1) * NT + c0;
        ok = dt_wait(&sh.sc_full[sc], scp, fail) && dt_wait(&sh.s_full[T & 1], (T >> 1) & 1, fail);
        __syncwarp();
        tc::fence_after_sync();
        const float kscale = sh.ks[sc][tid >> 4], vscale = sh.vs[sc][tid >> 4];
        const bool valid = pos < t.k1 && kscale >= 0.f;
        const bool part = !__all_sync(0xffffffffu, valid);
        // scales are powers of two from 2^-64 up: exponent and reciprocal are exact
        const int ve = (int)(__float_as_uint(vscale) >> 23);
        const float lv = (float)(ve - 127);
        const float rv = valid ? __uint_as_float((uint32_t)(254 - ve) << 23) : 0.f;
        const bool edge = kb + kDtTok > least;        // some row does not see some token
        // weight exponents s + log2(vs) of 16 columns, -inf where masked
        auto scores = [&](int ch, float (&x)[16]) {
          tc::tmem_ld16(scol + ch * 16, x);
          const float4* f4 = reinterpret_cast<const float4*>(&sh.fq[par][c0 + ch * 16]);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float4 f = f4[u];
#pragma unroll
            for (int k = 0; k < 4; ++k) x[4 * u + k] = fmaf(x[4 * u + k], kscale * (&f.x)[k], lv);
          }
          if (part || edge) {
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if (!valid || pos >= sh.lim[par][c0 + ch * 16 + k]) x[k] = -INFINITY;
          }
        };
        float x[CW / 16][16];
#pragma unroll
        for (int ch = 0; ch < CW / 16; ++ch) {
          scores(ch, x[ch]);
#pragma unroll
          for (int k = 0; k < 16; k += 4) {
            const float a = warp_max(x[ch][k]), b = warp_max(x[ch][k + 1]), c = warp_max(x[ch][k + 2]),
                        e = warp_max(x[ch][k + 3]);
            if (lane == 0) *reinterpret_cast<float4*>(&sh.cmax[quad][c0 + ch * 16 + k]) = make_float4(a, b, c, e);
          }
        }
        ok = bar_and(ok, bar);
        if (!ok) break;
        if (tid < CW) {
          const int n = c0 + tid;
          const float mx = fmaxf(fmaxf(sh.cmax[0][n], sh.cmax[1][n]), fmaxf(sh.cmax[2][n], sh.cmax[3][n]));
          float alpha = 1.f;
          if (j == 0) {
            ref = mx;
          } else if (mx - ref > kDtGrow) {
            // the reference moves only past the codes' headroom: a column's
            // choice depends on that column alone
            alpha = dt_ex2(ref - mx);
            ref = mx;
            *(volatile unsigned*)&sh.grow[wg] = T + 1;
          }
          sh.ref[n] = (ref == -INFINITY ? 0.f : ref) - kDtBase;
          sh.alpha[n] = alpha;
        }
        bar_and(true, bar);
        if (*(volatile unsigned*)&sh.grow[wg] == T + 1) {
          // the products before this tile's: done, then scaled column by column
          ok = bar_and(dt_wait(&sh.o_done[(T - 1) & 1], ((T - 1) >> 1) & 1, fail), bar);
          if (!ok) break;
          tc::fence_after_sync();
#pragma unroll
          for (int ch = 0; ch < CW / 16; ++ch) {
            float al[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) al[k] = sh.alpha[c0 + ch * 16 + k], l[ch * 16 + k] *= al[k];
            for (int hf = 0; hf < (d + 127) / 128; ++hf) {
              float o[16];
              tc::tmem_ld16(lanes + C::O0 + hf * NT + c0 + ch * 16, o);
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] *= al[k];
              tc::tmem_st16(lanes + C::O0 + hf * NT + c0 + ch * 16, o);
            }
          }
          tc::tmem_st_wait();
        }
        if (C::PB == 1 && j > 0) {   // one buffer of weights: the product before has read it
          ok = bar_and(dt_wait(&sh.o_done[(T - 1) & 1], ((T - 1) >> 1) & 1, fail), bar);
          if (!ok) break;
        }
        uint8_t* pw = pd + (T & (C::PB - 1)) * 2 * NT * kDtTok + c0 * kDtTok + tid * 16;
#pragma unroll
        for (int ch = 0; ch < CW / 16; ++ch) {
          uint4 hi, lo;
          const float4* r4 = reinterpret_cast<const float4*>(&sh.ref[c0 + ch * 16]);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float4 r = r4[u];
            float e[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              e[k] = dt_ex2(x[ch][4 * u + k] - (&r.x)[k]);
              l[ch * 16 + 4 * u + k] = fmaf(e[k], rv, l[ch * 16 + 4 * u + k]);
            }
            const uint32_t h = e4m3x4(e[0], e[1], e[2], e[3]);
            const float2 a = e4m3_f32x2(h), b = e4m3_f32x2(h >> 16);
            (&hi.x)[u] = h;
            (&lo.x)[u] = e4m3x4(e[0] - a.x, e[1] - a.y, e[2] - b.x, e[3] - b.y);
          }
          *reinterpret_cast<uint4*>(pw + ch * 16 * kDtTok) = hi;
          *reinterpret_cast<uint4*>(pw + ch * 16 * kDtTok + NT * kDtTok) = lo;
        }
        if (edge && wg == 0) {
          // values that some row may not see: past the sequence they become
          // zero, and so do NaN codes (a weight of 0 would not keep them out),
          // noted by element for the rows that do see them
          ok = bar_and(dt_wait(&sh.v_full[st], vp, fail), bar);
          if (!ok) break;
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const int e = hf * 128 + tid;
            if (e >= d) break;
            for (int b = max(0, (least - kb) / kKvBlock); b < kDtBlocks && kb + b * kKvBlock < t.k1; ++b) {
              uint8_t* v = base + w.v_off + (uint32_t)st * unit + (b * d + e) * kKvBlock;
              for (int k = 0; k < kKvBlock; ++k) {
                const int at = kb + b * kKvBlock + k;
                if (at >= t.L) {
                  v[k] = 0;
                } else if (at >= least && (v[k] & 0x7f) == 0x7f) {
                  v[k] = 0;
                  sh.bad[par][e] = min(sh.bad[par][e], at);
                }
              }
            }
          }
        }
        __syncwarp();
        tc::fence_async_smem();
        tc::fence_before_sync();
        dt_arrive(&sh.p_full[T & 1]);
        if (++st == ST) st = 0, vp ^= 1;
        if (++sc == NS) sc = 0, scp ^= 1;
      }
      if (!ok) break;
      // the next item's rows: its scores may then start while this one ends
      const DtItem u = t;
      if (i + (int)gridDim.x < total) {
        t = dt_item<NT>(w, sh.items, i + gridDim.x);
        load_q(t, par ^ 1);
      }
#pragma unroll
      for (int ch = 0; ch < CW / 16; ++ch) {
        float x[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) x[k] = l[ch * 16 + k];
        const float sum = sum16(x, lane);
        if (!(lane & 1)) (&sh.lsum[c0 + ch * 16 + (lane >> 1)].x)[quad] = sum;
      }
      if (u.tiles > 0) ok = dt_wait(&sh.o_done[(T - 1) & 1], ((T - 1) >> 1) & 1, fail);
      ok = bar_and(ok, bar);
      if (!ok) break;
      tc::fence_after_sync();
      const int64_t R = p.T * p.Hq;
      const int mine = min(CW, u.rows - c0);   // columns of this warpgroup that are rows
      if (tid < mine) {
        const float4 c = sh.lsum[c0 + tid];
        const float sum = (c.x + c.y) + (c.z + c.w), m = sum == 0.f ? -INFINITY : sh.ref[c0 + tid];
        const int64_t rh = sh.out[par][c0 + tid];
        if (p.part_o) p.part_ml[u.piece * R + rh] = make_float2(m, sum);
        else if (p.lse) p.lse[rh] = sum == 0.f ? -INFINITY : m * 0.693147180559945309f + logf(sum);
      }
      __syncwarp();
      const bool check = u.k0 + u.tiles * kDtTok > least;   // some tile had values that not every row sees
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int e = hf * 128 + tid;
        if (hf * 128 >= d) break;
        const int bad = check && e < d ? sh.bad[par][e] : 0x7fffffff;
        float* po = p.part_o + u.piece * R * d + e;
#pragma unroll
        for (int ch = 0; ch < CW / 16; ++ch) {
          if (ch * 16 >= mine) break;
          float o[16];
          if (u.tiles > 0) {
            tc::tmem_ld16(lanes + C::O0 + hf * NT + c0 + ch * 16, o);
          } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = 0.f;
          }
          if (e < d) {
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const int n = c0 + ch * 16 + k;
              if (ch * 16 + k >= mine) break;
              const float v = bad < sh.lim[par][n] ? __int_as_float(0x7fffffff) : o[k];
              if (p.part_o) {
                po[sh.out[par][n] * d] = v;
              } else {
                const float4 c = sh.lsum[n];
                const float sum = (c.x + c.y) + (c.z + c.w);
                static_cast<__nv_bfloat16*>(p.o)[sh.out[par][n] * d + e] = __float2bfloat16_rn(sum == 0.f ? 0.f : v / sum);
              }
            }
          }
          __syncwarp();
        }
      }
      tc::fence_before_sync();
      bar_and(true, bar);   // lsum, ref and O are free
    }
  }
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  if (sh.fail) {
    // a wait ran out: report, then give the copies in flight one more bounded
    // wait each before their memory goes
    if (threadIdx.x == 0) set_error(p.err, GDN_ERR_TIMEOUT);
    if ((warp == WARPS || warp == WARPS + 1) && lane == 0)
      for (int n = max(0, loaded - ST); n < loaded; ++n)
        tc::mbar_wait_bounded(warp == WARPS ? &sh.k_full[n % ST] : &sh.v_full[n % ST], (uint32_t)(n / ST) & 1, kDtWait);
    __syncwarp();
    __syncthreads();
  }
  tc::fence_after_sync();
  if (warp == WARPS) tc::tmem_dealloc(tb, C::COLS);
}

namespace {

template <int NT>
cudaError_t decode_tc(const AttnDecodeParams& p, int sms, cudaStream_t st) {
  using C = DtCfg<NT>;
  DtParams w{};
  w.a = p;
  const uint32_t d = (uint32_t)p.c.d, unit = kDtTok * d, q = 2 * NT * d, pp = 2 * C::PB * NT * kDtTok;
  // K and V stages in what is left of 227 KB (1 KB a CTA is the system's);
  // below 128 elements the second product's 128 rows read up to 2 KB past a
  // stage (their sums are not used)
  const uint32_t all = C::CTAS == 2 ? 115712 : 232448;
  const uint32_t fixed = q + pp + (uint32_t)sizeof(DtShared<NT>) + 2048 + 512;
  const uint32_t stages = (all - fixed) / (2 * unit);
  w.stages = stages > kDtMaxStages ? kDtMaxStages : (int)stages;
  if (w.stages < 1) return cudaErrorInvalidValue;
  w.k_off = 0;
  w.v_off = w.stages * unit;
  w.q_off = (2 * w.stages * unit + 2048 + 127) / 128 * 128;
  w.p_off = w.q_off + q;
  w.misc_off = (w.p_off + pp + 127) / 128 * 128;
  uint32_t smem = w.misc_off + (uint32_t)sizeof(DtShared<NT>) + 128;
  // no more CTAs an SM than share its tensor memory
  const uint32_t least = C::CTAS == 2 ? 80 * 1024 : 120 * 1024;
  if (smem < least) smem = least;
  cudaError_t e = cudaFuncSetAttribute(attn_decode_tc_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int rt = (p.max_q * p.G + NT - 1) / NT;
  for (int s0 = 0; s0 < p.N; s0 += kDtSeqs) {
    w.s0 = s0;
    w.ns = p.N - s0 < kDtSeqs ? p.N - s0 : kDtSeqs;
    const int64_t most = (int64_t)w.ns * p.max_pieces * p.c.Hkv * rt;
    attn_decode_tc_kernel<NT><<<(unsigned)(most < C::CTAS * sms ? most : C::CTAS * sms), C::THREADS, smem, st>>>(w);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

bool attn_decode_tc_supported(const AttnDecodeParams& p, int dtype) {
  return dtype == GDN_BF16 && p.c.d % 32 == 0;
}

cudaError_t launch_attn_decode_tc(const AttnDecodeParams& p, cudaStream_t st) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  // the narrowest tile that holds a sequence's (row, head) pairs of a kv head
  const int rows = p.max_q * p.G;
  if (rows <= 16) return decode_tc<16>(p, sms, st);
  if (rows <= 32) return decode_tc<32>(p, sms, st);
  if (rows <= 64) return decode_tc<64>(p, sms, st);
  return decode_tc<96>(p, sms, st);
}

}  // namespace gdn
