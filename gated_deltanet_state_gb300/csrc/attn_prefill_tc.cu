// attn_prefill_tc.cu — causal attention over packed prompts on the tensor
// cores (bf16, d = 64, 128, 256).
//
// S = Q K^T and O += P V are tcgen05 products of 128 query rows (row i of a
// tile: token i / G, head i % G of the group, so that the group shares the
// keys) with 128 keys, accumulated in tensor memory.  The softmax runs between
// them, the running maximum and sum of a row in the threads that hold it.  How
// long that takes decides how idle the tensor cores are, so each of two row
// tiles (up to d = 128) has two warpgroups, a row's 128 scores in two threads
// which exchange their maxima; at d = 256, where the outputs of one row tile
// take half of tensor memory and its keys and values more of L2 than there is,
// two CTAs share every key tile (cta_group::2: half of its keys and half of its
// values' elements in each) and two warpgroups take its key tiles in turn, the
// running maximum passing from one to the other before the exponentials, so
// that those of two key tiles overlap.
#include <cuda.h>

#include "attn.h"
#include "launch.h"
#include "tc.cuh"

namespace gdn {

namespace {

constexpr int kTile = 128;          // rows and keys of a tile
constexpr long long kPreWait = 4000000000LL;

template <int D, bool PAIR>
struct PreCfg {
  static constexpr int NQ = D == 256 ? 1 : 2;            // row tiles a CTA
  static constexpr int SLOTS = D == 256 ? 2 : 1;         // score buffers a row tile
  static constexpr int UD = D < 128 ? D : 128;           // head elements of a staged unit
  static constexpr int U = D / UD;                       // units of a key tile
  static constexpr int CTAS = PAIR ? 2 : 1;              // that share a key tile
  static constexpr uint32_t UNIT = kTile * UD * 2 / CTAS;
  static constexpr int STAGES = D == 64 ? 8 : 5 * CTAS;
  static constexpr int KROWS = kTile / CTAS, VCOLS = UD / CTAS;   // of a unit of K, of V, in this CTA
  static constexpr uint32_t Q_BYTES = kTile * D * 2;
  static constexpr uint32_t DATA = NQ * Q_BYTES + STAGES * UNIT;
  static constexpr bool ALT = D == 256;                  // key tiles in turn instead of rows in two halves
  static constexpr int SW = ALT ? 8 : 16;                // softmax warps
  static constexpr int THREADS = SW * 32 + 128;          // and loads, products, guards
  // registers a thread: what the guards' group gives up goes to the softmax,
  // together at most what the block starts with (168 x 384, 96 x 640)
  static constexpr int REGS = ALT ? 216 : 104, REGS_REST = ALT ? 72 : 64;
  // tensor memory columns: scores (the weights overwrite them), then outputs
  static constexpr uint32_t S0 = 0, O0 = 256;
};

template <class C, int D>
struct PreShared {
  uint64_t full[C::STAGES], empty[C::STAGES], s_full[2], p_full[2], o_done[2], q_full[2], v_raw[8], v_ok[8], m_ready[4], fin[2], drain;
  float m[C::SW / 4][kTile];   // by warpgroup: d = 256: its reference of each row; else its scores' maxima; at the end its sums
  uint32_t tmem;
  int fail, bad_any, issued[2];   // (issued: units loaded by each CTA of a pair)
  // by element of V the first key with +inf, -inf, NaN, counted from the first
  // guarded tile's (a pair's rows guard at most 768): 10 bits each, ones: none
  uint32_t bad[D];
};
template <int D, bool PAIR>
constexpr uint32_t kPreSmem = PreCfg<D, PAIR>::DATA + sizeof(PreShared<PreCfg<D, PAIR>, D>);
static_assert(kPreSmem<256, true> <= 232448 && kPreSmem<256, false> <= 232448 && kPreSmem<128, false> <= 232448 &&
                  kPreSmem<64, false> <= 232448,
              "227 KB a CTA");

// ---- the two CTAs of a pair -----------------------------------------------------
// The same place of shared memory in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t peer_smem(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
template <typename T>
__device__ __forceinline__ T* peer_ptr(T* p, uint32_t rank) {   // for ordinary loads, stores and atomics
  uint64_t r;
  asm volatile("mapa.u64 %0, %1, %2;\n" : "=l"(r) : "l"(reinterpret_cast<uint64_t>(p)), "r"(rank));
  return reinterpret_cast<T*>(r);
}
__device__ __forceinline__ void arrive_at(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(cluster_addr) : "memory");
}
// What orders tensor memory is the fence before it, not this.
__device__ __forceinline__ void arrive_at_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
// A tile load that reports to a barrier of either CTA.
__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3, %4}], "
      "[%5];\n" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
// Products of a pair: 256 rows, 128 in each CTA, against an operand of which
// each CTA holds half; issued by one CTA for both.
template <bool PAIR>
__device__ __forceinline__ void pre_mma(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  if constexpr (!PAIR) {
    tc::mma_bf16_if(lead, d, a, b, id, acc);
  } else {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
        " @q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(acc), "r"(lead)
        : "memory");
  }
}
template <bool PAIR>
__device__ __forceinline__ void pre_mma_ts(uint32_t lead, uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) {
  if constexpr (!PAIR) {
    tc::mma_bf16_ts_if(lead, d, a, b, id, acc);
  } else {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
        " @q tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(id), "r"(acc), "r"(lead)
        : "memory");
  }
}
// Arrival, on this barrier in every CTA of the pair, once the products so far are done.
template <bool PAIR>
__device__ __forceinline__ void pre_commit(uint32_t lead, uint64_t* m) {
  if constexpr (!PAIR) {
    tc::mma_commit_if(lead, m);
  } else {
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
        " @q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %2;\n}\n" ::"r"(
            smem_u32(m)),
        "r"(lead), "h"((uint16_t)3)
        : "memory");
  }
}
// As if bytes of a copy had arrived.
__device__ __forceinline__ void mbar_complete_tx(uint64_t* m, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cta.b64 [%0], %1;\n" ::"r"(smem_u32(m)), "r"(bytes) : "memory");
}
// The wait of one who then reads what the other CTA has written.
__device__ __forceinline__ bool mbar_test_cluster(uint64_t* m, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(m)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Minimum of the 10-bit field of a word in shared memory that starts at bit `at`.
__device__ __forceinline__ void min10(uint32_t* w, int at, uint32_t v) {
  uint32_t old = *w;
  while (((old >> at) & 0x3ffu) > v) {
    const uint32_t seen = atomicCAS(w, old, (old & ~(0x3ffu << at)) | (v << at));
    if (seen == old) break;
    old = seen;
  }
}

// Waits for a phase: bounded, and given up at once when another role has.
template <bool CLUSTER = false>
__device__ __forceinline__ bool pre_wait(uint64_t* m, uint32_t parity, long long limit, volatile int* fail) {
  if (CLUSTER ? mbar_test_cluster(m, parity) : tc::mbar_test_wait(m, parity)) return true;
  const long long t0 = clock64();
  while (!(CLUSTER ? mbar_test_cluster(m, parity) : tc::mbar_try_wait(m, parity))) {
    if (*fail) return false;
    if (clock64() - t0 > limit) {
      *fail = 1;
      return false;
    }
  }
  return true;
}

__device__ __forceinline__ void mbar_arrive(uint64_t* m) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(smem_u32(m)) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Largest of three (NaN falls out).
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Shared-memory descriptor of V as the N x K operand with N contiguous: rows of
// 64 elements (128 B, swizzled) for one key, 8-key groups 1,024 B apart, the
// next 64 elements (which a CTA of a pair does not hold) a whole block of keys
// (128 x 128 B) further.
__device__ __forceinline__ uint64_t desc_v(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)((kTile * 128) >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
constexpr uint32_t kTransposedB = 1u << 16;   // instruction descriptor: B is N-contiguous

// Geometry of one CTA's row tiles.
struct PreTile {
  int s, h, q0, n, k0, L;
  int64_t r0;            // first row (token * G + head) of the CTA's first tile
  int nk[2], nkmax;      // key tiles of each row tile
  int least;             // keys that every row sees (of the pair)
};

template <class C>
__device__ __forceinline__ bool pre_tile(const AttnPrefillParams& p, PreTile& t, bool report) {
  constexpr int NQ = C::NQ, ROWS = C::CTAS * NQ * kTile;   // rows of the CTA, or of the pair's
  const int groups = p.N * p.Hkv, block = blockIdx.x / C::CTAS, rank = blockIdx.x % C::CTAS;
  const int back = block / groups, pr = block - back * groups;
  t.s = pr / p.Hkv;
  t.h = pr - t.s * p.Hkv;
  t.q0 = p.cu_q[t.s];
  t.n = p.cu_q[t.s + 1] - t.q0;
  t.k0 = p.cu_kv[t.s];
  t.L = p.cu_kv[t.s + 1] - t.k0;
  if (t.n <= 0) return false;
  if (t.n > p.max_q || t.L > p.max_kv || t.L < 0 || t.q0 < 0 || t.k0 < 0 || (int64_t)t.q0 + t.n > p.Tq ||
      (int64_t)t.k0 + t.L > p.Tk) {
    if (report) set_error(p.err, GDN_ERR_INVALID_ARG);
    return false;
  }
  const int64_t rows = (int64_t)t.n * p.G;
  const int tiles = (int)((rows + ROWS - 1) / ROWS);
  if (back >= tiles) return false;
  const int64_t first = (int64_t)(tiles - 1 - back) * ROWS;   // the last rows, which see the most keys, first
  t.r0 = first + rank * NQ * kTile;
  t.nkmax = 0;
  for (int q = 0; q < 2; ++q) {
    // key tiles of row tile q: of a pair's two the more (its products are one)
    t.nk[q] = 0;
    for (int c = 0; c < C::CTAS; ++c) {
      const int64_t r = first + (c * NQ + q) * kTile;
      if (q >= NQ || r >= rows) continue;
      const int last = (int)min((int64_t)t.n - 1, (r + kTile - 1) / p.G);
      t.nk[q] = max(t.nk[q], (max(0, t.L - t.n + last + 1) + kTile - 1) / kTile);
    }
    t.nkmax = max(t.nkmax, t.nk[q]);
  }
  t.least = max(0, t.L - t.n + (int)(first / p.G) + 1);
  return true;
}

// Whether unit n in the ring's order (K 0, with one row tile K 1; then V j and
// the next K in turn) is one of V for the guards.
template <class C>
__device__ __forceinline__ bool pre_guarded(const PreTile& t, int n) {
  constexpr int ahead = C::NQ == 1 ? 2 : 1;
  int tile = n / C::U;
  const int lead = min(ahead, t.nkmax), both = 2 * (t.nkmax - lead);
  if (tile < lead) return false;
  tile -= lead;
  if (tile < both && (tile & 1)) return false;
  const int j = tile < both ? tile >> 1 : (both >> 1) + tile - both;
  return (j + 1) * kTile > t.least;
}

}  // namespace

template <int D, bool PAIR>
__global__ void __launch_bounds__(PreCfg<D, PAIR>::THREADS, 1)
    attn_prefill_tc_kernel(const AttnPrefillParams p, const __grid_constant__ CUtensorMap kmap,
                           const __grid_constant__ CUtensorMap vmap) {
  using C = PreCfg<D, PAIR>;
  extern __shared__ __align__(1024) uint8_t base[];
  PreTile t;
  if (!pre_tile<C>(p, t, threadIdx.x == 0)) return;   // (both CTAs of a pair)
  // the swizzled tiles need the 1,024-byte alignment that shared memory without
  // static variables starts with: there is no room to make it up
  if (smem_u32(base) & 1023u) {
    if (threadIdx.x == 0) set_error(p.err, GDN_ERR_CUDA);
    return;
  }
  uint8_t* sq = base;
  uint8_t* ring = base + C::NQ * C::Q_BYTES;
  PreShared<C, D>& sh = *reinterpret_cast<PreShared<C, D>*>(base + C::DATA);
  const uint32_t rank = PAIR ? blockIdx.x & 1 : 0;   // 0: the CTA that issues the products
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long limit = p.wait_cycles > 0 ? p.wait_cycles : p.wait_cycles < 0 ? -1 : kPreWait;
  volatile int* fail = &sh.fail;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::STAGES; ++i) tc::mbar_init(&sh.full[i], 1), tc::mbar_init(&sh.empty[i], 1);
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sh.s_full[i], 1);
      tc::mbar_init(&sh.p_full[i], (C::ALT ? 4 : 8) * C::CTAS);   // a warp arrives once
      tc::mbar_init(&sh.o_done[i], 1);
      tc::mbar_init(&sh.q_full[i], 8 * C::CTAS);
    }
    for (int i = 0; i < 8; ++i) tc::mbar_init(&sh.v_raw[i], 1), tc::mbar_init(&sh.v_ok[i], (C::U == 2 ? 1 : 2) * C::CTAS);
    for (int i = 0; i < 4; ++i) tc::mbar_init(&sh.m_ready[i], 128);
    for (int i = 0; i < 2; ++i) tc::mbar_init(&sh.fin[i], C::ALT ? 128 : 256);
    tc::mbar_init(&sh.drain, 1);
    sh.fail = limit < 0, sh.bad_any = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  for (int i = threadIdx.x; i < D; i += C::THREADS) sh.bad[i] = 0x3fffffffu;
  if (warp == 0) {
    if constexpr (PAIR) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(smem_u32(&sh.tmem)) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n" ::: "memory");
    } else {
      tc::tmem_alloc(&sh.tmem, 512);
      tc::tmem_relinquish();
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (PAIR) cluster_sync();   // the other's barriers are there too
  tc::fence_after_sync();
  // one arrival of a warp on a barrier of the CTA that issues the products
  auto arrive_lead = [&](uint64_t* m) {
    __syncwarp();
    if (lane != 0) return;
    if (PAIR) arrive_at(peer_smem(m, 0));
    else mbar_arrive(m);
  };
  const uint32_t tb = sh.tmem;
  const int wg = warp >> 2;
  int issued = 0, raw = 0;   // units loaded, those of them for the guards first (the loading thread's)

  if (warp < C::SW) {
    // ---- softmax: row i of tile q; its keys' half, or (d = 256) every second key tile ----
    constexpr bool ALT = C::ALT;
    constexpr int SC = ALT ? kTile : kTile / 2, NU = SC / 32;   // scores of a thread
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(C::REGS));
    const int q = ALT ? 0 : wg >> 1, half = wg & 1, i = threadIdx.x & 127;
    const int nk = t.nk[q];
    const int64_t rbase = t.r0 + q * kTile, r = rbase + i;
    const int tok = (int)(r / p.G), g = (int)(r - (int64_t)tok * p.G);
    const bool valid = tok < t.n;
    const int lim = valid ? max(0, t.L - t.n + tok + 1) : 0;
    const int64_t row_off = ((int64_t)(t.q0 + tok) * p.Hq + t.h * p.G + g);
    const uint32_t lanes = tb + ((uint32_t)(warp & 3) << 21);   // this warp's 32 lanes
    const __nv_bfloat16* qg = static_cast<const __nv_bfloat16*>(p.q);
    if (nk > 0 && limit >= 0) {
      // 16 rows a warp, all their loads before the first store (one after
      // another they take 19,000 cycles of a tile's 80,000)
      constexpr int CH = D / 8, RP = 32 / CH, NP = 16 / RP;   // 16-byte chunks of a row, rows a pass, passes
      const int w0 = (half * 4 + (warp & 3)) * 16 + lane / CH, c8 = lane % CH * 8;
      const int tok0 = (int)(rbase / p.G), rem0 = (int)(rbase - (int64_t)tok0 * p.G);   // of the tile's first row
      uint4 w[NP];
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        const int x = rem0 + w0 + k * RP, tk = tok0 + x / p.G, gg = x % p.G;
        w[k] = make_uint4(0, 0, 0, 0);
        if (tk < t.n)
          w[k] = *reinterpret_cast<const uint4*>(qg + (int64_t)(t.q0 + tk) * p.q_stride + (int64_t)(t.h * p.G + gg) * D + c8);
      }
#pragma unroll
      for (int k = 0; k < NP; ++k)
        *reinterpret_cast<uint4*>(sq + q * C::Q_BYTES + tc::sw128_offset(w0 + k * RP, c8, kTile)) = w[k];
      tc::fence_async_smem();
      arrive_lead(&sh.q_full[q]);
    }
    float m = -INFINITY, l = 0.f;
    const float c = p.scale_log2;
    // O of tiles 0 .. j: with two score buffers two barriers in turn, since
    // scores j only say that O of tile j - 2 is done
    auto o_wait = [&](int j) {
      return ALT ? pre_wait(&sh.o_done[j & 1], (uint32_t)(j >> 1) & 1, limit, fail)
                 : pre_wait(&sh.o_done[q], (uint32_t)j & 1, limit, fail);
    };
    // keys that all of this warp's rows see: below it no mask
    int wlim = valid ? lim : 0x7fffffff;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) wlim = min(wlim, __shfl_xor_sync(0xffffffffu, wlim, o));
    bool ok = nk == 0 || limit >= 0;
    for (int j = ALT ? half : 0; ok && j < nk; j += ALT ? 2 : 1) {
      const int b = ALT ? half : q;   // score buffer
      ok = pre_wait(&sh.s_full[b], (uint32_t)(ALT ? j >> 1 : j) & 1, limit, fail);
      if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
      tc::fence_after_sync();
      const uint32_t scol = lanes + C::S0 + (uint32_t)b * 128;
      uint32_t s[NU][32];
#pragma unroll
      for (int u = 0; u < NU; ++u) tc::tmem_ld32_nowait(scol + (ALT ? 0 : half * SC) + u * 32, s[u]);
      tc::tmem_ld_wait();
#pragma unroll
      for (int u = 0; u < NU; ++u) tc::tmem_ld_fence(s[u]);
      if ((j + 1) * kTile > wlim) {
        const int seen = lim - j * kTile - (ALT ? 0 : half * SC);   // of these scores, those that the row sees
#pragma unroll
        for (int u = 0; u < NU; ++u)
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (u * 32 + k >= seen) s[u][k] = 0xff800000u;
      }
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int u = 0; u < NU; ++u)
#pragma unroll
        for (int k = 0; k < 32; k += 2)
          mx[k >> 1 & 3] = max3(mx[k >> 1 & 3], __uint_as_float(s[u][k]), __uint_as_float(s[u][k + 1]));
      float mt = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
      const float before = m;
      if (!ALT) {
        // the row's other half: its maximum, and that its scores have been read
        // (the weights below overwrite them)
        sh.m[wg][i] = mt;
        mbar_arrive(&sh.m_ready[wg]);
        ok = pre_wait(&sh.m_ready[wg ^ 1], (uint32_t)j & 1, limit, fail);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        mt = fmaxf(mt, sh.m[wg ^ 1][i]);
      } else if (j > 0) {   // the reference after the tile before, the other warpgroup's
        ok = pre_wait(&sh.m_ready[wg ^ 1], (uint32_t)((j - 1) >> 1) & 1, limit, fail);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        m = sh.m[wg ^ 1][i];
      }
      // the reference of the weights moves only when the maximum has grown by
      // 2^8: weights stay below 2^8, and a row's choice depends on that row alone
      float alpha = 1.f;
      if (j == 0) {
        m = mt;
      } else if ((mt - m) * c > 8.f) {
        alpha = ex2((m - mt) * c);
        m = mt;
      }
      if (ALT) {
        sh.m[wg][i] = m;
        mbar_arrive(&sh.m_ready[wg]);
        if (j > 1 && m != before) l *= ex2((before - m) * c);
      } else {
        l *= alpha;
      }
      if (__any_sync(0xffffffffu, alpha != 1.f)) {
        // O of the tiles before: wait for their products, scale this warp's rows
        // (of two halves each half of the row)
        ok = o_wait(j - 1);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        tc::fence_after_sync();
#pragma unroll 1
        for (int e = ALT ? 0 : half * (D / 2); e < (ALT ? D : (half + 1) * (D / 2)); e += 16) {
          float o[16];
          const uint32_t col = lanes + C::O0 + (uint32_t)q * D + e;
          tc::tmem_ld16(col, o);
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] *= alpha;
          tc::tmem_st16(col, o);
        }
        tc::tmem_st_wait();
      }
      const float ref = m == -INFINITY ? 0.f : -m * c;
      const f32x2 cc = pack2(c, c), rr = pack2(ref, ref);
      f32x2 sum[2] = {pack2(0.f, 0.f), pack2(0.f, 0.f)};
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        uint32_t w[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const float2 x = unpack2(fma2(pack2(__uint_as_float(s[u][2 * k]), __uint_as_float(s[u][2 * k + 1])), cc, rr));
          const float a = ex2(x.x), b2 = ex2(x.y);
          sum[k & 1] = add2(sum[k & 1], pack2(a, b2));
          const __nv_bfloat162 h2 = __floats2bfloat162_rn(a, b2);
          w[k] = *reinterpret_cast<const uint32_t*>(&h2);
        }
        tc::tmem_st16u(scol + (ALT ? 0 : half * (SC / 2)) + u * 16, w);
      }
      l += sum2(add2(sum[0], sum[1]));
      tc::tmem_st_wait();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if (PAIR) arrive_at_relaxed(peer_smem(&sh.p_full[b], 0));
        else mbar_arrive(&sh.p_full[b]);
      }
    }
    // ---- outputs ----
    if (nk > 0 && limit >= 0) {
      if (!ok) *fail = 1;
      if (!ALT) {
        // the row's sum: the two halves', where the maxima were once the last
        // products say that both halves have had those
        ok = ok && o_wait(nk - 1);
        sh.m[wg][i] = l;
        mbar_arrive(&sh.fin[q]);
        ok = pre_wait(&sh.fin[q], 0, limit, fail) && ok;
        l = sh.m[wg & ~1][i] + sh.m[wg | 1][i];
      } else {
        // the warpgroup that had the last tile takes the other's sum, brought to
        // its reference, and hands the total back
        const int last = (nk - 1) & 1;
        if (wg != last) {
          ok = pre_wait(&sh.m_ready[last], (uint32_t)((nk - 1) >> 1) & 1, limit, fail) && ok;
          const float mine = m;
          m = sh.m[last][i];
          sh.m[wg][i] = l == 0.f ? 0.f : l * ex2((mine - m) * c);
          mbar_arrive(&sh.fin[0]);
          ok = pre_wait(&sh.fin[1], 0, limit, fail) && ok;
          l = sh.m[last][i];
        } else {
          ok = pre_wait(&sh.fin[0], 0, limit, fail) && ok;
          l += sh.m[wg ^ 1][i];
          sh.m[wg][i] = l;
          mbar_arrive(&sh.fin[1]);
        }
      }
    }
    if (ok && nk > 0) ok = o_wait(nk - 1);
    if (PAIR) asm volatile("fence.acq_rel.cluster;\n" ::: "memory");   // and what the other CTA noted of V
    if (__all_sync(0xffffffffu, ok)) {
      tc::fence_after_sync();
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const bool bad = nk > 0 && *(volatile int*)&sh.bad_any;
      // Rows leave through shared memory (this tile's Q, which every product has
      // read), each warp its half of 32 rows, so that whole stretches of a row are
      // written: 16-byte chunk ch of row i at place ch ^ (i % CH) of the row.
      constexpr int W = D / 2, CH = W / 8, RP = 32 / CH;   // elements of a row here, its chunks, rows a pass
      const int e0 = half * W;
      uint8_t* so = sq + q * C::Q_BYTES + half * (kTile * W * 2) + (warp & 3) * 32 * (W * 2);
#pragma unroll 1
      for (int e = 0; e < W; e += 32) {
        float o[32];
        if (nk > 0) {
          tc::tmem_ld32(lanes + C::O0 + (uint32_t)q * D + e0 + e, o);
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0.f;
        }
        if (bad) {
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const int mine = lim - t.least / kTile * kTile;
            const uint32_t w = sh.bad[e0 + e + k];
            const bool hi = (int)(w & 0x3ffu) < mine, lo = (int)(w >> 10 & 0x3ffu) < mine;
            if (hi) o[k] = INFINITY;
            if (lo) o[k] = -INFINITY;
            if ((int)(w >> 20) < mine || (hi && lo)) o[k] = __int_as_float(0x7fffffff);
          }
        }
#pragma unroll
        for (int k = 0; k < 32; k += 8) {
          uint32_t w[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            // a row that sees no key is 0, whatever its lanes of O hold
            const __nv_bfloat162 h2 = l == 0.f ? __floats2bfloat162_rn(0.f, 0.f)
                                               : __floats2bfloat162_rn(o[k + 2 * u] * inv, o[k + 2 * u + 1] * inv);
            w[u] = *reinterpret_cast<const uint32_t*>(&h2);
          }
          *reinterpret_cast<uint4*>(so + lane * (W * 2) + ((((e + k) >> 3) ^ (lane & (CH - 1))) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      __syncwarp();
      const int64_t mine = valid ? row_off : -1;
      __nv_bfloat16* og = static_cast<__nv_bfloat16*>(p.o) + e0 + (lane % CH) * 8;
#pragma unroll 4
      for (int r0 = 0; r0 < 32; r0 += RP) {
        const int rr = r0 + lane / CH;
        const int64_t at = __shfl_sync(0xffffffffu, mine, rr);
        if (at >= 0)
          *reinterpret_cast<uint4*>(og + at * D) =
              *reinterpret_cast<const uint4*>(so + rr * (W * 2) + (((lane % CH) ^ (rr & (CH - 1))) << 4));
      }
      if (valid && p.lse && half == 0) p.lse[row_off] = l == 0.f ? -INFINITY : (m * c + log2f(l)) * 0.693147180559945309f;
    }
  } else {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(C::REGS_REST));
  if (warp == C::SW && lane == 0) {
    // ---- loads ----
    // a V tile that some row sees in part arrives on the guards' barriers, who
    // hand it on; they follow within the ring, so 8 barriers never alias
    auto tile = [&](const CUtensorMap* map, int j, bool guarded) {
      for (int u = 0; u < C::U; ++u) {
        const int st = issued % C::STAGES;
        if (issued >= C::STAGES && !pre_wait(&sh.empty[st], (uint32_t)(issued / C::STAGES - 1) & 1, limit, fail)) return false;
        if constexpr (PAIR) {
          // each CTA its half: keys of K, elements of V; the bytes of both count
          // on the issuing CTA's barrier, what the guards take on their own CTA's
          const bool is_v = map == &vmap;
          uint64_t* bar = guarded ? &sh.v_raw[raw++ & 7] : &sh.full[st];
          if (guarded) tc::mbar_expect_tx(bar, C::UNIT);
          else if (rank == 0) tc::mbar_expect_tx(bar, 2 * C::UNIT);
          const uint32_t at = guarded ? peer_smem(bar, rank) : peer_smem(bar, 0);
          if (is_v) {
            tma_load_3d_pair(ring + st * C::UNIT, map, u * C::UD + rank * C::VCOLS, t.h, t.k0 + j * kTile, at);
          } else {
            for (int b = 0; b < C::UD / 64; ++b)
              tma_load_3d_pair(ring + st * C::UNIT + b * (C::KROWS * 128), map, u * C::UD + b * 64, t.h,
                               t.k0 + j * kTile + rank * C::KROWS, at);
          }
        } else {
          uint64_t* bar = guarded ? &sh.v_raw[raw++ & 7] : &sh.full[st];
          tc::mbar_expect_tx(bar, C::UNIT);
          for (int b = 0; b < C::UD / 64; ++b)
            tc::tma_load_3d(ring + st * C::UNIT + b * (kTile * 128), map, u * C::UD + b * 64, t.h, t.k0 + j * kTile, bar);
        }
        ++issued;
      }
      return true;
    };
    // in the order the products take them
    bool ok = limit >= 0 && (t.nkmax == 0 || tile(&kmap, 0, false));
    if (ok && C::NQ == 1 && t.nkmax > 1) ok = tile(&kmap, 1, false);
    constexpr int ahead = C::NQ == 1 ? 2 : 1;
    for (int j = 0; ok && j < t.nkmax; ++j) 
      ok = tile(&vmap, j, (j + 1) * kTile > t.least) && (j + ahead >= t.nkmax || tile(&kmap, j + ahead, false));
  } else if (warp == C::SW + 1 && limit >= 0 && rank == 0) {
    // ---- products: the whole warp, one lane issues ----
    const uint32_t lead = tc::elect_one();
    constexpr uint32_t id_qk = tc::idesc_bf16_f32(C::CTAS * kTile, kTile);
    constexpr uint32_t id_pv = tc::idesc_bf16_f32(C::CTAS * kTile, C::UD) | kTransposedB;
    const uint64_t qdesc = tc::desc_sw128(smem_u32(sq)), kdesc = tc::desc_sw128(smem_u32(ring)), vdesc = desc_v(smem_u32(ring));
    int st = 0, guarded = 0;   // the ring's place that is taken next
    uint32_t ph = 0;
    bool ok = true;
    auto step = [&](int& s, uint32_t& p) {
      if (++s == C::STAGES) s = 0, p ^= 1;
    };
    auto qk_unit = [&](int q, uint32_t scol, int s, int u) {
      const uint64_t a = qdesc + ((q * C::Q_BYTES + u * (C::UD / 64) * (kTile * 128)) >> 4), b = kdesc + (s * C::UNIT >> 4);
#pragma unroll
      for (int ks = 0; ks < C::UD / 16; ++ks) {
        const uint64_t oa = ((uint32_t)(ks >> 2) * (kTile * 128) + (uint32_t)(ks & 3) * 32u) >> 4;
        const uint64_t ob = ((uint32_t)(ks >> 2) * (C::KROWS * 128) + (uint32_t)(ks & 3) * 32u) >> 4;
        pre_mma<PAIR>(lead, tb + scol, a + oa, b + ob, id_qk, u != 0 || ks != 0);
      }
    };
    auto pv_unit = [&](int q, uint32_t pcol, int s, int u, bool acc) {
      const uint64_t b = vdesc + (s * C::UNIT >> 4);
#pragma unroll
      for (int ks = 0; ks < kTile / 16; ++ks)
        pre_mma_ts<PAIR>(lead, tb + C::O0 + q * D + u * C::UD, tb + pcol + 8 * ks, b + ((uint32_t)ks * 2048u >> 4), id_pv,
                           acc || ks != 0);
    };
    // a look at a barrier ahead of its use, so that the answer is there when
    // the products in between are issued
    auto peek = [&](uint64_t* m, uint32_t p) { return __all_sync(0xffffffffu, tc::mbar_test_wait(m, p)) != 0; };
    auto full = [&](int s, uint32_t p) { return pre_wait(&sh.full[s], p, limit, fail); };
    // a guarded V unit: from the guards, and its place's phase moves on here
    auto v_ready = [&](int s, uint32_t p, int j) {
      if ((j + 1) * kTile <= t.least) return full(s, p);
      const int k = guarded++;
      if (!pre_wait<PAIR>(&sh.v_ok[k & 7], (uint32_t)(k >> 3) & 1, limit, fail)) return false;
      if (lead) mbar_arrive(&sh.full[s]);
      __syncwarp();
      return true;
    };
    // ok is the same in every lane: after each wait the warp agrees
    auto all = [&](bool x) { return __all_sync(0xffffffffu, x) != 0; };
    if constexpr (C::NQ == 1) {
      static_assert(C::U == 2, "two units a key tile");
      ok = t.nkmax == 0 || all(pre_wait<PAIR>(&sh.q_full[0], 0, limit, fail));
      // a wait for each unit of 32 KB: the ring holds five, so the next one is
      // often still on its way
      bool seen = false;   // whether the next unit has been seen to be there
      auto unit = [&](bool last_unit) {   // the next unit's place is st; look at the one behind it
        int s1 = st;
        uint32_t p1 = ph;
        step(s1, p1);
        seen = !last_unit && peek(&sh.full[s1], p1);
      };
      auto qk = [&](int j) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (!seen && !all(full(st, ph))) return false;
          unit(false);
          qk_unit(0, C::S0 + (j & 1) * 128, st, u);
          pre_commit<PAIR>(lead, &sh.empty[st]);
          step(st, ph);
        }
        pre_commit<PAIR>(lead, &sh.s_full[j & 1]);
        return true;
      };
      auto pv = [&](int j) {
        const bool guards = (j + 1) * kTile > t.least;
        if (!all(pre_wait(&sh.p_full[j & 1], (uint32_t)(j >> 1) & 1, limit, fail))) return false;
        tc::fence_after_sync();
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if ((guards || !seen) && !all(v_ready(st, ph, j))) return false;
          unit(guards);
          pv_unit(0, C::S0 + (j & 1) * 128, st, u, j != 0);
          pre_commit<PAIR>(lead, &sh.empty[st]);
          step(st, ph);
        }
        pre_commit<PAIR>(lead, &sh.o_done[j & 1]);
        return true;
      };
      if (ok && t.nkmax > 0) ok = qk(0);
      if (ok && t.nkmax > 1) ok = qk(1);
      for (int j = 0; ok && j < t.nkmax; ++j) ok = pv(j) && (j + 2 >= t.nkmax || qk(j + 2));
    } else {
      for (int q = 0; ok && q < 2; ++q) ok = t.nk[q] == 0 || all(pre_wait<PAIR>(&sh.q_full[q], 0, limit, fail));
      if (ok && t.nkmax > 0) {
        ok = all(full(0, 0));
        if (ok) {
          tc::fence_after_sync();
          for (int q = 0; q < 2; ++q)
            if (t.nk[q] > 0) {
              qk_unit(q, C::S0 + q * 128, 0, 0);
              pre_commit<PAIR>(lead, &sh.s_full[q]);
            }
          pre_commit<PAIR>(lead, &sh.empty[0]);
        }
        step(st, ph);
      }
      for (int j = 0; ok && j < t.nkmax; ++j) {
        int s1 = st;
        uint32_t p1 = ph;
        step(s1, p1);
        const bool more = j + 1 < t.nkmax;
        ok = all(v_ready(st, ph, j) && (!more || full(s1, p1)));
        for (int q = 0; ok && q < 2; ++q) {
          if (j >= t.nk[q]) continue;
          ok = all(pre_wait(&sh.p_full[q], (uint32_t)j & 1, limit, fail));
          if (!ok) break;
          tc::fence_after_sync();
          pv_unit(q, C::S0 + q * 128, st, 0, j != 0);
          pre_commit<PAIR>(lead, &sh.o_done[q]);
          if (j + 1 < t.nk[q]) {
            qk_unit(q, C::S0 + q * 128, s1, 0);
            pre_commit<PAIR>(lead, &sh.s_full[q]);
          }
        }
        if (!ok) break;
        pre_commit<PAIR>(lead, &sh.empty[st]);
        if (more) {
          pre_commit<PAIR>(lead, &sh.empty[s1]);
          step(st, ph);
        }
        step(st, ph);
      }
    }
    // every product issued, and every arrival on a barrier, before the end
    pre_commit<PAIR>(lead, &sh.drain);
    if (!tc::mbar_wait_bounded(&sh.drain, 0, kPreWait)) *fail = 1;
  } else if (warp >= C::SW + 2 && limit >= 0) {
    // ---- guards: in V tiles that some row sees in part, keys past the
    // sequence become zero and so do NaN and infinities, which a weight of 0
    // would not keep out of the product; where those were is noted by element
    // for the rows that do see them ----
    // (two units of a tile: a warp each; one: both warps)
    constexpr int GT = C::U == 2 ? 32 : 64;
    const int me = (threadIdx.x - (C::SW + 2) * 32) % GT;
    bool ok = true;
    int done = 0;
    for (int j = t.least / kTile; ok && j < t.nkmax; ++j) {
      for (int u = C::U == 2 ? warp - (C::SW + 2) : 0, one = 1; ok && one; one = 0) {
        // position of unit u of V tile j in the ring's order
        int n;
        if constexpr (C::NQ == 1) n = min(t.nkmax, j + 2) * C::U + j * C::U + u;
        else n = 1 + 2 * j;
        const int k = done * C::U + u;   // of the guarded units
        ok = pre_wait(&sh.v_raw[k & 7], (uint32_t)(k >> 3) & 1, limit, fail);
        if (!ok) break;
        ++done;
        uint8_t* v = ring + (n % C::STAGES) * C::UNIT;
        // 16-byte chunks x = me + GT k: block x / 1024, key x / 8 % 128
        const int left = t.L - j * kTile;   // keys of the tile in the sequence
        if (left < kTile)
          for (int x = me; x < (int)C::UNIT / 16; x += GT)
            if ((x >> 3 & (kTile - 1)) >= left) *reinterpret_cast<uint4*>(v + x * 16) = make_uint4(0, 0, 0, 0);
        // eight chunks at a time: 0 times an infinity or NaN is NaN, and so is a sum with it
        for (int x0 = me; x0 < (int)C::UNIT / 16; x0 += 8 * GT) {
          __nv_bfloat162 sum[4] = {};
          const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint4 w = *reinterpret_cast<const uint4*>(v + (x0 + GT * k) * 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[i] = __hfma2(reinterpret_cast<const __nv_bfloat162*>(&w)[i], zero, sum[i]);
          }
          const __nv_bfloat162 a = __hadd2(__hadd2(sum[0], sum[1]), __hadd2(sum[2], sum[3]));
          if (!__hisnan(a.x) && !__hisnan(a.y)) continue;
          for (int x = x0; x < x0 + 8 * GT; x += GT) {
            const int row = x >> 3 & (kTile - 1), col = u * C::UD + rank * C::VCOLS + (x >> 10) * 64 + (((x & 7) ^ (row & 7)) << 3);
            for (int i = 0; i < 8; ++i) {
              uint16_t* el = reinterpret_cast<uint16_t*>(v + x * 16) + i;
              const uint16_t b = *el;
              if ((b & 0x7f80u) != 0x7f80u) continue;
              const int bit = (b & 0x7f) ? 20 : (b & 0x8000u) ? 10 : 0, key = j * kTile + row - t.least / kTile * kTile;
              min10(&sh.bad[col + i], bit, key);
              if (PAIR) min10(peer_ptr(&sh.bad[col + i], rank ^ 1), bit, key);
              *el = 0;
            }
          }
          *(volatile int*)&sh.bad_any = 1;
          if (PAIR) *(volatile int*)peer_ptr(&sh.bad_any, rank ^ 1) = 1;
        }
        tc::fence_async_smem();
        if (PAIR) asm volatile("fence.acq_rel.cluster;\n" ::: "memory");
        arrive_lead(&sh.v_ok[k & 7]);
      }
    }
  }
  }
  if constexpr (PAIR) {   // each CTA learns how far the other came
    if (warp == C::SW && lane == 0) sh.issued[rank] = issued, *(volatile int*)peer_ptr(&sh.issued[rank], rank ^ 1) = issued;
  }
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  if constexpr (PAIR) {
    if (threadIdx.x == 0 && *fail) *(volatile int*)peer_ptr(&sh.fail, rank ^ 1) = 1;
    __syncwarp();
    cluster_sync();
    // the last arrival from the issuing CTA
    if (rank == 1 && threadIdx.x == 0 && limit >= 0) tc::mbar_wait_bounded(&sh.drain, 0, kPreWait);
    __syncwarp();
  }
  if (*fail) {
    // a wait ran out: report, then give the copies in flight one more bounded
    // wait each before their memory goes
    if (threadIdx.x == 0) set_error(p.err, GDN_ERR_TIMEOUT);
    if (warp == C::SW && lane == 0) {
      // a pair's bytes of K and of whole V tiles count on the issuing CTA's
      // barriers, which waits for both: with the same units on both sides
      int first = issued, last = issued, k = raw - 1;
      if (PAIR && rank == 0) {
        const int other = *(volatile int*)&sh.issued[1];
        first = min(first, other), last = max(last, other);
      }
      for (int n = last - 1; n >= 0 && n >= last - C::STAGES; --n) {
        const bool mine = n < issued, guarded = pre_guarded<C>(t, n);
        if (guarded) {
          if (mine) tc::mbar_wait_bounded(&sh.v_raw[k & 7], (uint32_t)(k >> 3) & 1, kPreWait), --k;
        } else if (rank == 0) {
          uint64_t* bar = &sh.full[n % C::STAGES];
          if (PAIR && n >= first) {
            if (mine) mbar_complete_tx(bar, C::UNIT);   // the other's half does not come
            else tc::mbar_expect_tx(bar, C::UNIT);      // only the other's half comes
          }
          tc::mbar_wait_bounded(bar, (uint32_t)(n / C::STAGES) & 1, kPreWait);
        }
      }
    }
    __syncwarp();
    __syncthreads();
  }
  __syncwarp();
  if (PAIR) cluster_sync();   // nobody leaves while the other may still reach it
  tc::fence_after_sync();
  if (warp == 0) {
    if constexpr (PAIR) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;\n" ::"r"(tb) : "memory");
    else tc::tmem_dealloc(tb, 512);
  }
  if (PAIR) cluster_sync();
}

namespace {

cudaError_t rows_map(CUtensorMap* map, const void* base, int d, int heads, int64_t rows, int64_t stride, int box_rows) {
  auto encode = tensor_map_encoder();
  if (!encode) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, 1, (cuuint32_t)box_rows}, estr[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

template <int D, bool PAIR>
cudaError_t prefill_tc(const AttnPrefillParams& p, cudaStream_t st) {
  using C = PreCfg<D, PAIR>;
  CUtensorMap kmap, vmap;
  cudaError_t e = rows_map(&kmap, p.k, D, p.Hkv, p.Tk, p.k_stride, C::KROWS);
  if (e == cudaSuccess) e = rows_map(&vmap, p.v, D, p.Hkv, p.Tk, p.v_stride, kTile);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(attn_prefill_tc_kernel<D, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPreSmem<D, PAIR>);
  if (e != cudaSuccess) return e;
  constexpr int ROWS = C::CTAS * C::NQ * kTile;
  const int64_t grid = ((int64_t)p.max_q * p.G + ROWS - 1) / ROWS * p.N * p.Hkv * C::CTAS;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = kPreSmem<D, PAIR>;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = C::CTAS;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_prefill_tc_kernel<D, PAIR>, p, kmap, vmap);
}

}  // namespace

bool attn_prefill_tc_supported(const AttnPrefillParams& p, int dtype) {
  return dtype == GDN_BF16 && (p.d == 64 || p.d == 128 || p.d == 256) && p.Tk > 0 && p.k_stride < (1LL << 38) &&
         p.v_stride < (1LL << 38);
}

cudaError_t launch_attn_prefill_tc(const AttnPrefillParams& p, cudaStream_t st) {
  // d = 256: a CTA's 128 rows take 128 KB of keys and values for 2,144 cycles of
  // products, more than L2 gives (2 x 8,192 tokens: 1,235 us), so two share
  // them (1,072 us) unless a sequence's rows fit one.  Two row tiles of d <= 128
  // need half of that and only lose by moving together (d = 128, chunks of 101
  // to 2,003 tokens: 525 us alone, 563 us in pairs).
  if (p.d == 64) return prefill_tc<64, false>(p, st);
  if (p.d == 128) return prefill_tc<128, false>(p, st);
  return (int64_t)p.max_q * p.G > kTile ? prefill_tc<256, true>(p, st) : prefill_tc<256, false>(p, st);
}

}  // namespace gdn
