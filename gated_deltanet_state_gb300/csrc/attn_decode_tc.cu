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
constexpr int kDtSeqs = 256;         // sequences a launch
constexpr int kDtMaxStages = 8;
constexpr long long kDtWait = 4000000000LL;
// Weights are scaled by 2^6 and may grow by 2^2.75 (430 < 448) before a
// column's reference moves: a lower scale would lose small weights' bits (parts
// vanish below 2^-16 of the reference), a higher one moves more often.
constexpr float kDtBase = 6.f, kDtGrow = 2.75f;

// NT query rows; CW of them a softmax warpgroup (128 threads, a token each).
template <int NT>
struct DtCfg {
  static constexpr int CW = NT < 32 ? NT : 32, WGS = NT / CW, CH = CW < 16 ? CW : 16;
  static constexpr int N = NT < 16 ? 16 : NT;          // columns of a product; those past NT are not read
  static constexpr int THREADS = WGS * 128 + 96;       // and K loads, V loads, products
  // narrow tiles: two CTAs an SM, one's softmax under the other's products and loads
  static constexpr int CTAS = NT <= 32 ? 2 : 1;
  static constexpr uint32_t COLS = NT <= 16 ? 64 : NT <= 32 ? 128 : 512;
  static constexpr uint32_t O0 = 2 * N;                // scores of two tiles, then O of 128 elements each
};

struct DtParams {
  AttnDecodeParams a;
  int32_t s0, ns;       // this launch's sequences
  int32_t k_stages, v_stages;
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
  // of a head's rows, heads alternate: score factor, keys seen, place among the outputs
  float fq[2][NT];
  int lim[2][NT];
  uint32_t out[2][NT];      // (row, head) counted from the item's first row's head 0
  int bad[2][256];          // (items alternate) first token with a NaN value that not every row sees, by element
  int items[kDtSeqs + 1];   // running sums of the sequences' work items ...
  int work[kDtSeqs + 1];    // ... and of their weights
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
  int s, h, r0, rows, piece, pieces, pt;   // rows: (row, head) pairs of this item, from r0
  int q0, n, L, k0, k1, tiles;
};

// Groups (kv head, row tile) of a sequence; 0: no rows, -1: out of bounds.
template <int NT>
__device__ __forceinline__ int dt_groups(const AttnDecodeParams& p, int s) {
  const int n = p.cu[s + 1] - p.cu[s], L = p.kv_len[s];
  if (n <= 0) return 0;
  if (n > p.max_q || L > p.max_kv || L < 0 || p.cu[s] < 0 || (int64_t)p.cu[s] + n > p.T) return -1;
  return p.c.Hkv * ((n * p.G + NT - 1) / NT);
}
// A tile of keys counts 1, an item's fixed cost as much again.
__device__ __forceinline__ int dt_piece_work(const AttnDecodeParams& p, int s) {
  return decode_piece_tokens(p.kv_len[s], (p.cu[s + 1] - p.cu[s]) * p.G) / kDtTok + 1;
}

// The last s with sums[s] <= i.
__device__ __forceinline__ int dt_find(const int* sums, int n, int i) {
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
__device__ __forceinline__ int dt_first(const DtParams& w, const int* items, const int* work, int b, int ctas) {
  const int at = (int)((int64_t)work[w.ns] * b / ctas);
  if (at >= work[w.ns]) return items[w.ns];
  const int s = dt_find(work, w.ns, at);
  const int groups = dt_groups<NT>(w.a, w.s0 + s), per = (work[s + 1] - work[s]) / groups, pieces = (items[s + 1] - items[s]) / groups;
  const int g = (at - work[s]) / per;
  return items[s] + g * pieces + min(pieces, (at - work[s] - g * per + dt_piece_work(w.a, w.s0 + s) - 1) / dt_piece_work(w.a, w.s0 + s));
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
  // pieces of one head's rows one after another: a CTA's run of items loads
  // its rows once a head
  t.pieces = decode_pieces(t.L, t.n * p.G);
  const int group = k / t.pieces;
  t.piece = k - group * t.pieces;
  const int rt = (t.n * p.G + NT - 1) / NT;
  t.h = group / rt;
  t.r0 = (group - t.h * rt) * NT;
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
  if (t.piece + 1 < t.pieces) {
    ++t.piece;
    t.k0 += t.pt;
    t.k1 = min(t.L, t.k0 + t.pt);
    t.tiles = (t.k1 - t.k0 + kDtTok - 1) / kDtTok;
  } else {
    t = dt_item<NT>(w, items, i);
  }
}

// CW or 16 columns of a product's sums.
template <int CH>
__device__ __forceinline__ void read_columns(uint32_t col, float (&x)[CH]) {
  if constexpr (CH == 8) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(col));
    tc::tmem_ld_wait();
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = __uint_as_float(r[k]);
  } else {
    tc::tmem_ld16(col, x);
  }
}
// One product's steps: KS of 32 elements, the operands' starts moving by a
// step's tiles (constants, so that the issuing thread spends an add or two a
// step: with run-time steps it takes 130 cycles a product, which takes 51 to 60).
template <int KS>
__device__ __forceinline__ void mma_steps(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint64_t astep, uint64_t bstep, bool acc) {
#pragma unroll
  for (int c = 0; c < KS; ++c) mma_e4m3(d, a + c * astep, b + c * bstep, id, acc || c != 0);
}
// Sums of l[CW] over a warp's lanes, into out[column] at its warp's place.  By
// halves: after log2(CW) exchanges a lane holds one column of its part.
template <int CW>
__device__ __forceinline__ void column_sums(const float (&l)[CW], float4* out, int lane, int quad) {
  float v[CW];
#pragma unroll
  for (int i = 0; i < CW; ++i) v[i] = l[i];
  int bit = 16, at = 0;
#pragma unroll
  for (int half = CW / 2; half >= 1; half >>= 1, bit >>= 1) {
    const bool up = lane & bit;
    at = 2 * at + (up ? 1 : 0);
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float send = up ? v[i] : v[i + half], keep = up ? v[i + half] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
    }
  }
  for (; bit >= 1; bit >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], bit);
  if ((lane & (32 / CW - 1)) == 0) (&out[at].x)[quad] = v[0];
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
  constexpr int CW = C::CW, CH = C::CH, WARPS = C::WGS * 4;   // softmax warps; then K loads, V loads, products
  extern __shared__ uint8_t dyn[];
  const AttnDecodeParams& p = w.a;
  uint8_t* base = dyn + ((128u - (smem_u32(dyn) & 127u)) & 127u);
  DtShared<NT>& sh = *reinterpret_cast<DtShared<NT>*>(base + w.misc_off);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, d = p.c.d;
  const int KS = w.k_stages, VS = w.v_stages, NS = max(KS, VS) + 2;
  volatile int* fail = &sh.fail;

  if (threadIdx.x == 0) {
    for (int i = 0; i < KS; ++i) tc::mbar_init(&sh.k_full[i], 1), tc::mbar_init(&sh.k_empty[i], 1);
    for (int i = 0; i < VS; ++i) tc::mbar_init(&sh.v_full[i], 1), tc::mbar_init(&sh.v_empty[i], 1);
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
  // running sums of the items; lengths out of bounds are reported and have none
  if (warp == 0) {
    int sum = 0, sumw = 0;
    if (lane == 0) sh.items[0] = sh.work[0] = 0;
    for (int c = 0; c < w.ns; c += 32) {
      int v = 0, x = 0;
      if (c + lane < w.ns) {
        const int s = w.s0 + c + lane;
        int g = dt_groups<NT>(p, s);
        if (g < 0) {
          if (blockIdx.x == 0) set_error(p.err, GDN_ERR_INVALID_ARG);
          g = 0;
        }
        if (g > 0) {
          const int pieces = decode_pieces(p.kv_len[s], (p.cu[s + 1] - p.cu[s]) * p.G);
          v = g * pieces;
          x = g * pieces * dt_piece_work(p, s);
        }
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, v, o), b = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) v += a, x += b;
      }
      if (c + lane < w.ns) sh.items[c + lane + 1] = sum + v, sh.work[c + lane + 1] = sumw + x;
      sum += __shfl_sync(0xffffffffu, v, 31);
      sumw += __shfl_sync(0xffffffffu, x, 31);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tb = sh.tmem;
  // this CTA's run of items
  const int i0 = dt_first<NT>(w, sh.items, sh.work, blockIdx.x, gridDim.x);
  const int i1 = dt_first<NT>(w, sh.items, sh.work, blockIdx.x + 1, gridDim.x);
  const uint32_t unit = (uint32_t)kDtTok * d;   // bytes of a tile's K (or V) codes
  int loaded = 0;                               // tiles loaded (a loading warp's)

  if (warp == WARPS || warp == WARPS + 1) {
    // ---- loads, a warp for K and one for V: lane b < 8 the tile's block b ----
    const bool is_v = warp == WARPS + 1;
    uint64_t *full = is_v ? sh.v_full : sh.k_full, *empty = is_v ? sh.v_empty : sh.k_empty;
    uint8_t* ring = base + (is_v ? w.v_off : w.k_off);
    const int ST = is_v ? VS : KS;
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
      constexpr uint32_t id = idesc_e4m3(C::N);
      const uint32_t k0 = smem_u32(base + w.k_off), v0 = smem_u32(base + w.v_off), qa = smem_u32(base + w.q_off),
                     pa = smem_u32(base + w.p_off);
      const uint32_t rows8 = 8u * d;   // 8 tokens of K (or 8 rows of Q)
      const int halves = (d + 127) / 128;
      const uint64_t vstep = (uint64_t)(32u * d >> 4);
      int ks = 0, kp = 0, vs = 0, vp = 0, heads = 0;
      unsigned T = 0;   // tiles multiplied
      bool ok = true;
      auto qk = [&](unsigned tt) {
        if (!dt_wait(&sh.k_full[ks], kp, fail)) return false;
        tc::fence_after_sync();
        const uint64_t a = desc_tiles(k0 + ks * unit, 128, rows8);
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          const uint64_t b = desc_tiles(qa + part * NT * d, 128, rows8);
          const uint32_t dst = tb + (tt & 1) * C::N;
          if (d == 256) {
            mma_steps<8>(dst, a, b, id, 16, 16, part);
          } else if (d == 128) {
            mma_steps<4>(dst, a, b, id, 16, 16, part);
          } else {
            for (int c = 0; c < d / 32; ++c) mma_e4m3(dst, a + c * 16, b + c * 16, id, part | c);
          }
        }
        tc::mma_commit(&sh.k_empty[ks]);
        tc::mma_commit(&sh.s_full[tt & 1]);
        if (++ks == KS) ks = 0, kp ^= 1;
        return true;
      };
      DtItem t{};
      for (int i = i0; ok && i < i1; ++i) {
        if (i == i0) t = dt_item<NT>(w, sh.items, i);
        else dt_next<NT>(w, sh.items, i, t);
        if (i == i0 || t.piece == 0) ok = dt_wait(&sh.q_full, heads++ & 1, fail);
        if (ok && t.tiles > 0) ok = qk(T);
        for (int j = 0; ok && j < t.tiles; ++j, ++T) {
          if (j + 1 < t.tiles) ok = qk(T + 1);
          ok = ok && dt_wait(&sh.p_full[T & 1], (T >> 1) & 1, fail) && dt_wait(&sh.v_full[vs], vp, fail);
          if (!ok) break;
          tc::fence_after_sync();
          for (int hf = 0; hf < halves; ++hf) {
            const uint64_t a = desc_tiles(v0 + vs * unit + hf * 2048u, 16u * d, 128);
            // P: tokens of 16 columns (16 B), the next 16 columns a block of 128 tokens further
#pragma unroll
            for (int part = 0; part < 2; ++part)
              mma_steps<kDtTok / 32>(tb + C::O0 + hf * C::N, a, desc_tiles(pa + part * C::N * kDtTok, 128, 16 * kDtTok),
                                     id | kTransposedB, vstep, 32, j | part);
          }
          tc::mma_commit(&sh.v_empty[vs]);
          tc::mma_commit(&sh.o_done[T & 1]);
          if (++vs == VS) vs = 0, vp ^= 1;
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
    bool ok = true, okp = true;
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
            sh.out[par][n] = (uint32_t)((row - t.r0 / p.G) * p.Hq + t.h * p.G + g);
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
    int st = 0, sc = 0, scp = 0, vp = 0, par = 0, ip = 0;   // V stage, scale slot and their phases; head, item
    DtItem t{};
    if (i0 < i1) {
      t = dt_item<NT>(w, sh.items, i0);
      load_q(t, 0);
    }
    bar_and(true, bar);
    for (int i = i0; i < i1; ++i) {
      float l[CW];
#pragma unroll
      for (int n = 0; n < CW; ++n) l[n] = 0.f;
      float ref = -INFINITY;                          // of column c0 + tid
      if (wg == 0 && t.tiles > 0) sh.bad[ip][tid] = sh.bad[ip][tid + 128] = 0x7fffffff;
      const int least = t.L - t.n + 1;                // keys that every row sees
      for (int j = 0; j < t.tiles; ++j, ++T) {
        const int kb = t.k0 + j * kDtTok, pos = kb + tid;
        const uint32_t scol = lanes + (T & 1) * C::N + c0;
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
        // weight exponents s + log2(vs), -inf where masked
        float x[CW / CH][CH];
#pragma unroll
        for (int ch = 0; ch < CW / CH; ++ch) {
          read_columns(scol + ch * CH, x[ch]);
          const float4* f4 = reinterpret_cast<const float4*>(&sh.fq[par][c0 + ch * CH]);
#pragma unroll
          for (int k = 0; k < CH; k += 4) {
            const float4 f = f4[k / 4];
#pragma unroll
            for (int u = 0; u < 4; ++u) x[ch][k + u] = fmaf(x[ch][k + u], kscale * (&f.x)[u], lv);
          }
          if (part || edge) {
#pragma unroll
            for (int k = 0; k < CH; ++k)
              if (!valid || pos >= sh.lim[par][c0 + ch * CH + k]) x[ch][k] = -INFINITY;
          }
#pragma unroll
          for (int k = 0; k < CH; k += 4) {
            const float a = warp_max(x[ch][k]), b = warp_max(x[ch][k + 1]), c = warp_max(x[ch][k + 2]),
                        e = warp_max(x[ch][k + 3]);
            if (lane == 0) *reinterpret_cast<float4*>(&sh.cmax[quad][c0 + ch * CH + k]) = make_float4(a, b, c, e);
          }
        }
        ok = bar_and(ok && okp, bar);
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
          // (one that runs out shows at the next barrier)
          okp = dt_wait(&sh.o_done[(T - 1) & 1], ((T - 1) >> 1) & 1, fail);
          __syncwarp();
          tc::fence_after_sync();
#pragma unroll
          for (int n = 0; n < CW; ++n) l[n] *= sh.alpha[c0 + n];
          for (int hf = 0; hf < (d + 127) / 128; ++hf)
#pragma unroll
            for (int ch = 0; ch < (CW + 15) / 16; ++ch) {
              const uint32_t col = lanes + C::O0 + hf * C::N + c0 + ch * 16;
              float o[16];
              tc::tmem_ld16(col, o);
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] *= sh.alpha[c0 + (ch * 16 + k) % CW];   // (of 8 rows the other 8 are not read)
              tc::tmem_st16(col, o);
            }
          tc::tmem_st_wait();
        }
        // the weights' place: read by the product before
        if (j > 0) okp = dt_wait(&sh.o_done[(T - 1) & 1], ((T - 1) >> 1) & 1, fail) && okp;
        uint8_t* pw = pd + c0 * kDtTok + tid * 16;
#pragma unroll
        for (int ch = 0; ch < CW / CH; ++ch) {
          uint32_t hi[CH / 4], lo[CH / 4];
          const float4* r4 = reinterpret_cast<const float4*>(&sh.ref[c0 + ch * CH]);
#pragma unroll
          for (int u = 0; u < CH / 4; ++u) {
            const float4 r = r4[u];
            float e[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              e[k] = dt_ex2(x[ch][4 * u + k] - (&r.x)[k]);
              l[ch * CH + 4 * u + k] = fmaf(e[k], rv, l[ch * CH + 4 * u + k]);
            }
            hi[u] = e4m3x4(e[0], e[1], e[2], e[3]);
            const float2 a = e4m3_f32x2(hi[u]), b = e4m3_f32x2(hi[u] >> 16);
            lo[u] = e4m3x4(e[0] - a.x, e[1] - a.y, e[2] - b.x, e[3] - b.y);
          }
          if constexpr (CH == 8) {
            *reinterpret_cast<uint2*>(pw) = make_uint2(hi[0], hi[1]);
            *reinterpret_cast<uint2*>(pw + C::N * kDtTok) = make_uint2(lo[0], lo[1]);
          } else {
            *reinterpret_cast<uint4*>(pw + ch * 16 * kDtTok) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(pw + ch * 16 * kDtTok + C::N * kDtTok) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
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
                  sh.bad[ip][e] = min(sh.bad[ip][e], at);
                }
              }
            }
          }
        }
        __syncwarp();
        tc::fence_async_smem();
        tc::fence_before_sync();
        dt_arrive(&sh.p_full[T & 1]);
        if (++st == VS) st = 0, vp ^= 1;
        if (++sc == NS) sc = 0, scp ^= 1;
      }
      if (!ok) break;
      // the next head's rows: its scores may then start while this item ends
      const DtItem u = t;
      const int was = par;
      if (i + 1 < i1) {
        dt_next<NT>(w, sh.items, i + 1, t);
        if (t.piece == 0) load_q(t, par ^= 1);
      }
      column_sums<CW>(l, sh.lsum + c0, lane, quad);
      if (u.tiles > 0) ok = dt_wait(&sh.o_done[(T - 1) & 1], ((T - 1) >> 1) & 1, fail);
      ok = bar_and(ok && okp, bar);
      if (!ok) break;
      tc::fence_after_sync();
      const int64_t R = p.T * p.Hq, rh0 = (int64_t)(u.q0 + u.r0 / p.G) * p.Hq;
      const int mine = min(CW, u.rows - c0);   // columns of this warpgroup that are rows
      if (tid < mine) {
        const float4 c = sh.lsum[c0 + tid];
        const float sum = (c.x + c.y) + (c.z + c.w), m = sum == 0.f ? -INFINITY : sh.ref[c0 + tid];
        const int64_t rh = rh0 + sh.out[was][c0 + tid];
        if (p.part_o) p.part_ml[u.piece * R + rh] = make_float2(m, sum);
        else if (p.lse) p.lse[rh] = sum == 0.f ? -INFINITY : m * 0.693147180559945309f + logf(sum);
      }
      __syncwarp();
      const bool check = u.tiles > 0 && u.k0 + u.tiles * kDtTok > least;   // some tile had values that not every row sees
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        if (hf * 128 >= d) break;
        const int e = hf * 128 + tid;
        float* po = p.part_o + (u.piece * R + rh0) * d + e;
        __nv_bfloat16* oo = static_cast<__nv_bfloat16*>(p.o) + rh0 * d + e;
#pragma unroll
        for (int ch = 0; ch < CW / CH; ++ch) {
          if (ch * CH >= mine) break;
          float o[CH];
          if (u.tiles > 0) {
            read_columns(lanes + C::O0 + hf * C::N + c0 + ch * CH, o);
          } else {
#pragma unroll
            for (int k = 0; k < CH; ++k) o[k] = 0.f;
          }
          if (e < d) {
            if (check) {
              const int bad = sh.bad[ip][e];
#pragma unroll
              for (int k = 0; k < CH; ++k)
                if (bad < sh.lim[was][c0 + ch * CH + k]) o[k] = __int_as_float(0x7fffffff);
            }
#pragma unroll
            for (int k = 0; k < CH; ++k) {
              const int n = c0 + ch * CH + k;
              const uint32_t at = sh.out[was][n] * (uint32_t)d;   // at most 32 rows of 1,024 heads of 256 elements
              if (ch * CH + k < mine) {
                if (p.part_o) {
                  po[at] = o[k];
                } else {
                  const float4 c = sh.lsum[n];
                  const float sum = (c.x + c.y) + (c.z + c.w);
                  oo[at] = __float2bfloat16_rn(sum == 0.f ? 0.f : o[k] / sum);
                }
              }
            }
          }
          __syncwarp();
        }
      }
      tc::fence_before_sync();
      bar_and(true, bar);   // lsum, ref and O are free
      // (a buffer comes back after an item whose tiles every warpgroup has passed)
      if (u.tiles > 0) ip ^= 1;
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
    {
      const int ST = warp == WARPS ? KS : VS;
      for (int n = max(0, loaded - ST); n < loaded; ++n)
        tc::mbar_wait_bounded(warp == WARPS ? &sh.k_full[n % ST] : &sh.v_full[n % ST], (uint32_t)(n / ST) & 1, kDtWait);
    }
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
  const uint32_t d = (uint32_t)p.c.d, unit = kDtTok * d, q = 2 * NT * d, pp = 2 * C::N * kDtTok;
  // K and V stages in what is left of 227 KB (1 KB a CTA is the system's);
  // where d is no multiple of 128 the second product's 128 rows read up to
  // 2 KB past a stage (their sums are not used)
  const uint32_t past = d % 128 ? 2048 : 0;
  const uint32_t all = C::CTAS == 2 ? 115712 : 232448;
  const uint32_t fixed = q + pp + (uint32_t)sizeof(DtShared<NT>) + past + 512;
  const uint32_t units = (all - fixed) / unit;
  if (units < 2) return cudaErrorInvalidValue;
  w.k_stages = units / 2 + units % 2 > kDtMaxStages ? kDtMaxStages : (int)(units / 2 + units % 2);
  w.v_stages = units / 2 > kDtMaxStages ? kDtMaxStages : (int)(units / 2);
  w.k_off = 0;
  w.v_off = w.k_stages * unit;
  w.q_off = ((w.k_stages + w.v_stages) * unit + past + 127) / 128 * 128;
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
  if (rows <= 8) return decode_tc<8>(p, sms, st);
  if (rows <= 16) return decode_tc<16>(p, sms, st);
  if (rows <= 32) return decode_tc<32>(p, sms, st);
  return decode_tc<96>(p, sms, st);
}

}  // namespace gdn
