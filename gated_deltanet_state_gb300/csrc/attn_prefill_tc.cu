// attn_prefill_tc.cu — causal attention over packed prompts on the tensor
// cores (bf16, d = 64, 128, 256).
//
// S = Q K^T and O += P V are tcgen05 products of 128 query rows (row i of a
// tile: token i / G, head i % G of the group, so that the group shares the
// keys) with 128 keys, accumulated in tensor memory; P = 2^(c S - m), rounded
// to bf16 (as O is in the end), goes back over the scores it comes from; the
// running maximum m and sum of a row stay in fp32 registers.  A key tile takes
// D / 8 products of 67 cycles, and everything else has to hide under them:
//
// * Two warpgroups take the key tiles in turn (a row in a thread, 1,900 cycles a
//   tile), the reference m passing from one to the other before the
//   exponentials, so that those of two key tiles overlap; two score buffers
//   cover that at d = 256 (2,144 cycles of products), three at d = 128 (1,069,
//   of about 1,400 that a key tile takes in the six chunks below: latency, since
//   neither the tensor pipe nor the issue slots are full) and 64 (680, which the
//   exponentials' 950 exceed).
// * At d = 256 and 128 a CTA would load a key tile's 128 or 64 KB in that time,
//   more than L2 gives, so two CTAs share it (cta_group::2: half of its keys and
//   half of its values' elements in each, 256 query rows a product).
// * Blocks take further row tiles while they run: what surrounds the key tiles
//   (set-up, queries, outputs: 21,000 cycles of a block with one row tile, 33
//   key tiles of 2,100 on average at 8,192 tokens) comes under the products of
//   the tile before or after, about 9,000 of it still in the way.
//
// Measured (24 heads, 4 kv heads, d = 256; 32, 8, d = 128): two prompts of
// 8,192 tokens 1,002 to 1,017 us, 1.62 to 1.65 PFLOP/s or 83 to 84 % of a library
// product's burst, 94 to 95 % of its sustained rate, under the power limit (900 us
// at 1.85 GHz); six chunks of 101 to 2,003 tokens after up to 6,007 keys 457 to
// 465 us, 1.37 to 1.39 PFLOP/s; two prompts of 8,192 at d = 64 (32 heads, 8)
// 666 us, 0.83 PFLOP/s.
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
  static constexpr int NB = D == 256 ? 2 : 3;            // score buffers
  static constexpr int UD = D < 128 ? D : 128;           // head elements of a staged unit
  static constexpr int U = D / UD;                       // units of a key tile
  static constexpr int CTAS = PAIR ? 2 : 1;              // that share a key tile
  static constexpr uint32_t UNIT = kTile * UD * 2 / CTAS;
  static constexpr int STAGES = D == 64 ? 10 : (D == 128 ? 5 : 4) * CTAS;
  static constexpr int NV = 8;                           // barriers of guarded units: no more are in the ring at once
  static constexpr int KROWS = kTile / CTAS, VCOLS = UD / CTAS;   // of a unit of K, of V, in this CTA
  static constexpr uint32_t Q_BYTES = kTile * D * 2;
  static constexpr int SW = 8;                           // softmax warps
  static constexpr int THREADS = SW * 32 + 128;          // and loads, products, guards
  static constexpr int OW = D == 64 ? 32 : 64;               // elements of a row that leave a warp at a time
  static constexpr uint32_t O_BYTES = SW * 32 * OW * 2;
  static constexpr uint32_t DATA = Q_BYTES + STAGES * UNIT + O_BYTES;
  // registers a thread: what the others give up goes to the softmax, together at
  // most what the block starts with (168 x 384)
  static constexpr int REGS = 216, REGS_REST = 72;
  // tensor memory columns: scores (the weights overwrite them), then outputs
  static constexpr uint32_t S0 = 0, O0 = NB * 128;
};

// Geometry of a CTA's row tile.
struct PreTile {
  int s, h, q0, n, k0, L;   // n < 0: there are no more
  int64_t r0;            // first row (token * G + head)
  int nk;                // key tiles
  int least;             // keys that every row sees (of the pair)
};

template <class C, int D>
struct PreShared {
  uint4 next;            // what the request for another block's tile brought
  uint64_t full[C::STAGES], empty[C::STAGES], s_full[3], p_full[3], o_done[3], q_full, q_free, v_raw[C::NV], v_ok[C::NV], m_ready[2],
      fin[2], drain, o_free, tile_full[2], tile_empty[2], next_full, next_empty;
  float m[2][kTile];     // a warpgroup's reference of each row; at the end its sum
  PreTile tile[2];       // tiles k and k + 1 in slots k % 2
  uint32_t tmem;
  int fail, bad_any;
  int out_read, out_done;   // warps that have read what bad holds for a tile; that are done with it, the pair's, counted over all tiles
  int issued[2], bits[2], asked[2];   // by CTA of a pair at the end: units loaded, which of the last 32 for the guards, requests
  // by element of V the first key with +inf, -inf, NaN, counted from the first
  // guarded tile's (the rows guard at most 768 keys): 10 bits each, ones: none
  uint32_t bad[D];
};
template <int D, bool PAIR>
constexpr uint32_t kPreSmem = PreCfg<D, PAIR>::DATA + sizeof(PreShared<PreCfg<D, PAIR>, D>);
static_assert(kPreSmem<256, true> <= 232448 && kPreSmem<128, true> <= 232448 && kPreSmem<256, false> <= 232448 && kPreSmem<128, false> <= 232448 &&
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

// A block takes its own row tiles and then, one after another, those of blocks
// that have not started (cluster launch control), so that barriers and tensor
// memory are set up once and a tile's first loads and products go on under the
// outputs of the tile before.
__device__ __forceinline__ void ask_next(uint4* answer, uint64_t* bar, bool cluster) {
  if (cluster)
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.multicast::cluster::all.b128 [%0], [%1];\n" ::"r"(
            smem_u32(answer)),
        "r"(smem_u32(bar))
        : "memory");
  else
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];\n" ::"r"(
                     smem_u32(answer)),
                 "r"(smem_u32(bar))
                 : "memory");
}
// First block of the cluster that will not start on its own, -1: all have.
__device__ __forceinline__ int next_block(const uint4* answer) {
  uint32_t got, x;
  asm volatile(
      "{\n .reg .b128 a;\n .reg .pred p;\n .reg .b32 y, z, w;\n ld.shared.b128 a, [%2];\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n selp.u32 %0, 1, 0, p;\n mov.u32 %1, 0;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, y, z, w}, a;\n}\n"
      : "=r"(got), "=r"(x)
      : "r"(smem_u32(answer))
      : "memory");
  return got ? (int)x : -1;
}

template <class C>
__device__ __forceinline__ bool pre_tile(const AttnPrefillParams& p, PreTile& t, int block, int rank, bool report) {
  constexpr int ROWS = C::CTAS * kTile;
  int back;
  prefill_place(p, ROWS, block / C::CTAS, t.s, t.h, back);
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
  if (back < 0 || back >= tiles) return false;
  const int64_t first = (int64_t)(tiles - 1 - back) * ROWS;   // the last rows, which see the most keys, first
  t.r0 = first + rank * kTile;
  // the key tiles of the last row (a pair's two have the same: its products are one)
  const int last = (int)min((int64_t)t.n - 1, (first + ROWS - 1) / p.G);
  t.nk = (max(0, t.L - t.n + last + 1) + kTile - 1) / kTile;
  t.least = max(0, t.L - t.n + (int)(first / p.G) + 1);
  return true;
}

}  // namespace

template <int D, bool PAIR>
__global__ void __launch_bounds__(PreCfg<D, PAIR>::THREADS, 1)
    attn_prefill_tc_kernel(const AttnPrefillParams p, const __grid_constant__ CUtensorMap kmap,
                           const __grid_constant__ CUtensorMap vmap) {
  using C = PreCfg<D, PAIR>;
  extern __shared__ __align__(1024) uint8_t base[];
  const uint32_t rank = PAIR ? blockIdx.x & 1 : 0;   // 0: the CTA that issues the products
  PreTile first;
  if (!pre_tile<C>(p, first, blockIdx.x, rank, threadIdx.x == 0)) return;   // (both CTAs of a pair)
  // the swizzled tiles need the 1,024-byte alignment that shared memory without
  // static variables starts with: there is no room to make it up
  if (smem_u32(base) & 1023u) {
    if (threadIdx.x == 0) set_error(p.err, GDN_ERR_CUDA);
    return;
  }
  uint8_t* sq = base;
  uint8_t* ring = base + C::Q_BYTES;
  uint8_t* out = ring + C::STAGES * C::UNIT;
  PreShared<C, D>& sh = *reinterpret_cast<PreShared<C, D>*>(base + C::DATA);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long limit = p.wait_cycles > 0 ? p.wait_cycles : p.wait_cycles < 0 ? -1 : kPreWait;
  volatile int* fail = &sh.fail;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::STAGES; ++i) tc::mbar_init(&sh.full[i], 1), tc::mbar_init(&sh.empty[i], 1);
    for (int i = 0; i < 3; ++i) {
      tc::mbar_init(&sh.s_full[i], 1);
      tc::mbar_init(&sh.p_full[i], 4 * C::CTAS);   // a warp arrives once
      tc::mbar_init(&sh.o_done[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sh.fin[i], 128);
      tc::mbar_init(&sh.m_ready[i], 128);
      tc::mbar_init(&sh.tile_full[i], 1);
      tc::mbar_init(&sh.tile_empty[i], C::SW + 2 + (rank == 0 ? 1 : 0));
    }
    for (int i = 0; i < C::NV; ++i) tc::mbar_init(&sh.v_raw[i], 1), tc::mbar_init(&sh.v_ok[i], (C::U == 2 ? 1 : 2) * C::CTAS);
    tc::mbar_init(&sh.q_full, 2 * C::CTAS);
    tc::mbar_init(&sh.q_free, 1);
    tc::mbar_init(&sh.drain, 1);
    tc::mbar_init(&sh.o_free, 8 * C::CTAS);
    tc::mbar_init(&sh.next_full, 1);
    tc::mbar_init(&sh.next_empty, 1);
    sh.fail = limit < 0, sh.bad_any = sh.out_read = sh.out_done = 0;
    sh.tile[0] = first;
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
  // one arrival of a warp on a barrier of the CTA that issues the products; with
  // `relaxed` what it orders is tensor memory, by the fence before it (a release
  // to the cluster costs about 1,300 cycles)
  auto arrive_lead = [&](uint64_t* m, bool relaxed = false) {
    __syncwarp();
    if (lane != 0) return;
    if (!PAIR) mbar_arrive(m);
    else if (relaxed) arrive_at_relaxed(peer_smem(m, 0));
    else arrive_at(peer_smem(m, 0));
  };
  // tile k's slot is filled, and is done with
  auto tile_wait = [&](int k) { return k == 0 || pre_wait(&sh.tile_full[k & 1], (uint32_t)((k - 1) >> 1) & 1, limit, fail); };
  auto tile_release = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.tile_empty[k & 1]);
  };
  // ok of a warp: the same in every lane
  auto all = [&](bool x) { return __all_sync(0xffffffffu, x) != 0; };
  const uint32_t tb = sh.tmem;
  const int wg = warp >> 2;
  int issued = 0, raw = 0, asked = 0, answered = 0;   // units loaded, those of them for the guards first, requests (the loading thread's)
  uint32_t raw_bits = 0;     // which of the last 32 went to the guards

  if (warp < C::SW) {
    // ---- softmax: row i, every second key tile ----
    constexpr int NU = kTile / 32;
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(C::REGS));
    const int i = threadIdx.x & 127;
    const uint32_t lanes = tb + ((uint32_t)(warp & 3) << 21);   // this warp's 32 lanes
    const float c = p.scale_log2;
    // O of the J-th key tile and those before: a barrier for each score buffer
    // in turn, since scores J only say that O of J - NB is done
    auto o_wait = [&](int J) { return pre_wait(&sh.o_done[J % C::NB], (uint32_t)(J / C::NB) & 1, limit, fail); };
    int nk = 0, before_nk = 0, turns = 0;   // key tiles of this row tile, of all before; row tiles before that had any
    int lim = 0;
    bool valid = false;
    int64_t row_off = 0;
    float m = -INFINITY, l = 0.f;
    bool ok = limit >= 0;
    for (int k = 0; ok; ++k) {
      ok = all(tile_wait(k));
      if (!ok) break;
      const PreTile& t = sh.tile[k & 1];
      const bool more = t.n >= 0;
      // ---- outputs of the tile before ----
      if (k > 0) {
        const PreTile& b = sh.tile[(k - 1) & 1];
        if (nk > 0) {
          const int J = before_nk + nk - 1;
          // the warpgroup that had the last tile takes the other's sum, brought to
          // its reference, and hands the total back
          const int last = J & 1;
          if (wg != last) {
            ok = pre_wait(&sh.m_ready[last], (uint32_t)(J >> 1) & 1, limit, fail);
            const float mine = m;
            m = sh.m[last][i];
            sh.m[wg][i] = l == 0.f ? 0.f : l * ex2((mine - m) * c);
            mbar_arrive(&sh.fin[0]);
            ok = pre_wait(&sh.fin[1], (uint32_t)turns & 1, limit, fail) && ok;
            l = sh.m[last][i];
          } else {
            ok = pre_wait(&sh.fin[0], (uint32_t)turns & 1, limit, fail);
            l += sh.m[wg ^ 1][i];
            sh.m[wg][i] = l;
            mbar_arrive(&sh.fin[1]);
          }
          ok = o_wait(J) && ok;
          ok = all(ok);
          if (!ok) break;
          if (PAIR) asm volatile("fence.acq_rel.cluster;\n" ::: "memory");   // and what the other CTA noted of V
          tc::fence_after_sync();
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const bool bad = nk > 0 && *(volatile int*)&sh.bad_any;
        // Rows leave through shared memory, each warp its half of 32 rows, so that
        // stretches of 64 or 128 bytes are written: 16-byte chunk ch of row i at
        // place ch ^ f(i) of the row.
        constexpr int W = D / 2, OW = C::OW, CH = OW / 8, RP = 32 / CH;   // elements of a row here, at a time, chunks, rows a pass
        auto f = [](int row) { return CH == 8 ? row & 7 : row >> 1 & (CH - 1); };
        const int e0 = wg * W;
        uint8_t* so = out + warp * (32 * OW * 2);
        const int64_t mine = valid ? row_off : -1;
#pragma unroll 1
        for (int e = 0; e < W; e += OW) {
#pragma unroll
          for (int e1 = 0; e1 < OW; e1 += 32) {
            float o[32];
            if (nk > 0) {
              tc::tmem_ld32(lanes + C::O0 + e0 + e + e1, o);
            } else {
#pragma unroll
              for (int x = 0; x < 32; ++x) o[x] = 0.f;
            }
            if (bad) {
#pragma unroll
              for (int x = 0; x < 32; ++x) {
                const int mine_ = lim - b.least / kTile * kTile;
                const uint32_t w = sh.bad[e0 + e + e1 + x];
                const bool hi = (int)(w & 0x3ffu) < mine_, lo = (int)(w >> 10 & 0x3ffu) < mine_;
                if (hi) o[x] = INFINITY;
                if (lo) o[x] = -INFINITY;
                if ((int)(w >> 20) < mine_ || (hi && lo)) o[x] = __int_as_float(0x7fffffff);
              }
            }
#pragma unroll
            for (int x = 0; x < 32; x += 8) {
              uint32_t w[4];
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                // a row that sees no key is 0, whatever its lanes of O hold
                const __nv_bfloat162 h2 = l == 0.f ? __floats2bfloat162_rn(0.f, 0.f)
                                                   : __floats2bfloat162_rn(o[x + 2 * u] * inv, o[x + 2 * u + 1] * inv);
                w[u] = *reinterpret_cast<const uint32_t*>(&h2);
              }
              *reinterpret_cast<uint4*>(so + lane * (OW * 2) + ((((e1 + x) >> 3) ^ f(lane)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          if (nk > 0 && e + OW >= W) {   // the next tile's products may overwrite O
            tc::fence_before_sync();
            arrive_lead(&sh.o_free, true);
          }
          __syncwarp();
          __nv_bfloat16* og = static_cast<__nv_bfloat16*>(p.o) + e0 + e + (lane % CH) * 8;
#pragma unroll 4
          for (int r0 = 0; r0 < 32; r0 += RP) {
            const int rr = r0 + lane / CH;
            const int64_t at = __shfl_sync(0xffffffffu, mine, rr);
            if (at >= 0)
              *reinterpret_cast<uint4*>(og + at * D) = *reinterpret_cast<const uint4*>(so + rr * (OW * 2) + (((lane % CH) ^ f(rr)) << 4));
          }
          __syncwarp();
        }
        if (valid && p.lse && wg == 0) p.lse[row_off] = l == 0.f ? -INFINITY : (m * c + log2f(l)) * 0.693147180559945309f;
        // the last warp done clears what was noted of V; then the guards may note for the next tile
        __syncwarp();
        if (lane == 0) {
          if (bad) __threadfence_block();
          const int n = atomicAdd(&sh.out_read, 1) + 1;
          if (n == k * C::SW && *(volatile int*)&sh.bad_any) {
            for (int x = 0; x < D; ++x) sh.bad[x] = 0x3fffffffu;
            *(volatile int*)&sh.bad_any = 0;
            if (PAIR) asm volatile("fence.acq_rel.cluster;\n" ::: "memory");
            else __threadfence_block();
          }
          atomicAdd(&sh.out_done, 1);
          if (PAIR) atomicAdd(peer_ptr(&sh.out_done, rank ^ 1), 1);
        }
        tile_release(k - 1);
        before_nk += nk;
        if (nk > 0) ++turns;
      }
      if (!more) break;
      // ---- this tile's key tiles ----
      {
        const int64_t r = t.r0 + i;
        const int tok = (int)(r / p.G), g = (int)(r - (int64_t)tok * p.G);
        valid = tok < t.n;
        lim = valid ? max(0, t.L - t.n + tok + 1) : 0;
        row_off = (int64_t)(t.q0 + tok) * p.Hq + t.h * p.G + g;
      }
      nk = t.nk;
      m = -INFINITY, l = 0.f;
      // keys that all of this warp's rows see: below it no mask
      int wlim = valid ? lim : 0x7fffffff;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) wlim = min(wlim, __shfl_xor_sync(0xffffffffu, wlim, o));
      for (int j = (wg ^ before_nk) & 1; ok && j < nk; j += 2) {
        const int J = before_nk + j;
        const int b = J % C::NB;   // score buffer
        ok = all(pre_wait(&sh.s_full[b], (uint32_t)(J / C::NB) & 1, limit, fail));
        if (!ok) break;
        tc::fence_after_sync();
        const uint32_t scol = lanes + C::S0 + (uint32_t)b * 128;
        uint32_t s[NU][32];
#pragma unroll
        for (int u = 0; u < NU; ++u) tc::tmem_ld32_nowait(scol + u * 32, s[u]);
        tc::tmem_ld_wait();
#pragma unroll
        for (int u = 0; u < NU; ++u) tc::tmem_ld_fence(s[u]);
        if ((j + 1) * kTile > wlim) {
          const int seen = lim - j * kTile;   // of these scores, those that the row sees
#pragma unroll
          for (int u = 0; u < NU; ++u)
#pragma unroll
            for (int x = 0; x < 32; ++x)
              if (u * 32 + x >= seen) s[u][x] = 0xff800000u;
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int u = 0; u < NU; ++u)
#pragma unroll
          for (int x = 0; x < 32; x += 2)
            mx[x >> 1 & 3] = max3(mx[x >> 1 & 3], __uint_as_float(s[u][x]), __uint_as_float(s[u][x + 1]));
        const float mt = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
        const float before = m;
        if (j > 0) {   // the reference after the tile before, the other warpgroup's
          ok = all(pre_wait(&sh.m_ready[wg ^ 1], (uint32_t)((J - 1) >> 1) & 1, limit, fail));
          if (!ok) break;
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
        sh.m[wg][i] = m;
        mbar_arrive(&sh.m_ready[wg]);
        if (j > 1 && m != before) l *= ex2((before - m) * c);
        if (__any_sync(0xffffffffu, alpha != 1.f)) {
          // O of the tiles before: wait for their products, scale this warp's rows
          ok = all(o_wait(J - 1));
          if (!ok) break;
          tc::fence_after_sync();
#pragma unroll 1
          for (int e = 0; e < D; e += 16) {
            float o[16];
            const uint32_t col = lanes + C::O0 + e;
            tc::tmem_ld16(col, o);
#pragma unroll
            for (int x = 0; x < 16; ++x) o[x] *= alpha;
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
          for (int x = 0; x < 16; ++x) {
            const float2 y = unpack2(fma2(pack2(__uint_as_float(s[u][2 * x]), __uint_as_float(s[u][2 * x + 1])), cc, rr));
            const float a = ex2(y.x), b2 = ex2(y.y);
            sum[x & 1] = add2(sum[x & 1], pack2(a, b2));
            const __nv_bfloat162 h2 = __floats2bfloat162_rn(a, b2);
            w[x] = *reinterpret_cast<const uint32_t*>(&h2);
          }
          tc::tmem_st16u(scol + u * 16, w);
        }
        l += sum2(add2(sum[0], sum[1]));
        tc::tmem_st_wait();
        tc::fence_before_sync();
        arrive_lead(&sh.p_full[b], true);
      }
    }
    if (!ok) *fail = 1;
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(C::REGS_REST));
    if (warp == C::SW && lane == 0) {
      // ---- loads, and the requests for more tiles ----
      bool ok = limit >= 0;
      auto ask = [&] {
        // (the other CTA has read the answer before)
        if (PAIR && rank == 0 && asked > 0 && !pre_wait(&sh.next_empty, (uint32_t)(asked - 1) & 1, limit, fail)) return false;
        tc::mbar_expect_tx(&sh.next_full, 16);
        if (rank == 0) ask_next(&sh.next, &sh.next_full, PAIR);
        ++asked;
        return true;
      };
      for (int k = 0; ok; ++k) {
        PreTile t = sh.tile[k & 1];
        ok = ask();
        // a V tile that some row sees in part arrives on the guards' barriers,
        // who hand it on; they follow within the ring
        auto tile = [&](const CUtensorMap* map, int j, bool guarded) {
          for (int u = 0; u < C::U; ++u) {
            const int st = issued % C::STAGES;
            if (issued >= C::STAGES && !pre_wait(&sh.empty[st], (uint32_t)(issued / C::STAGES - 1) & 1, limit, fail)) return false;
            uint64_t* bar = guarded ? &sh.v_raw[raw++ % C::NV] : &sh.full[st];
            if constexpr (PAIR) {
              // each CTA its half: keys of K, elements of V; the bytes of both count
              // on the issuing CTA's barrier, what the guards take on their own CTA's
              if (guarded) tc::mbar_expect_tx(bar, C::UNIT);
              else if (rank == 0) tc::mbar_expect_tx(bar, 2 * C::UNIT);
              const uint32_t at = peer_smem(bar, guarded ? rank : 0);
              if (map == &vmap) {
                tma_load_3d_pair(ring + st * C::UNIT, map, u * C::UD + rank * C::VCOLS, t.h, t.k0 + j * kTile, at);
              } else {
                for (int b = 0; b < C::UD / 64; ++b)
                  tma_load_3d_pair(ring + st * C::UNIT + b * (C::KROWS * 128), map, u * C::UD + b * 64, t.h,
                                   t.k0 + j * kTile + rank * C::KROWS, at);
              }
            } else {
              tc::mbar_expect_tx(bar, C::UNIT);
              for (int b = 0; b < C::UD / 64; ++b)
                tc::tma_load_3d(ring + st * C::UNIT + b * (kTile * 128), map, u * C::UD + b * 64, t.h, t.k0 + j * kTile, bar);
            }
            ++issued;
            raw_bits = raw_bits << 1 | (guarded ? 1u : 0u);
          }
          return true;
        };
        // in the order the products take them
        for (int j = 0; ok && j < C::NB && j < t.nk; ++j) ok = tile(&kmap, j, false);
        for (int j = 0; ok && j < t.nk; ++j)
          ok = tile(&vmap, j, (j + 1) * kTile > t.least) && (j + C::NB >= t.nk || tile(&kmap, j + C::NB, false));
        // the next tile with rows
        while (ok) {
          ok = pre_wait(&sh.next_full, (uint32_t)answered & 1, limit, fail);
          if (!ok) break;
          ++answered;
          const int block = next_block(&sh.next);
          tc::fence_async_smem();   // read before the next answer comes
          if (PAIR && rank == 1) arrive_at(peer_smem(&sh.next_empty, 0));
          t.n = -1;
          if (block < 0 || pre_tile<C>(p, t, block, rank, rank == 0)) break;
          ok = ask();
        }
        const int s1 = (k + 1) & 1;
        if (ok && k > 0) ok = pre_wait(&sh.tile_empty[s1], (uint32_t)((k - 1) >> 1) & 1, limit, fail);
        if (!ok) break;
        sh.tile[s1] = t;
        mbar_arrive(&sh.tile_full[s1]);
        if (t.n < 0) break;
      }
      if (!ok) *fail = 1;
    } else if (warp == C::SW + 1 && limit >= 0 && rank == 0) {
      // ---- products: the whole warp, one lane issues ----
      const uint32_t lead = tc::elect_one();
      constexpr uint32_t id_qk = tc::idesc_bf16_f32(C::CTAS * kTile, kTile);
      constexpr uint32_t id_pv = tc::idesc_bf16_f32(C::CTAS * kTile, C::UD) | kTransposedB;
      const uint64_t qdesc = tc::desc_sw128(smem_u32(sq)), kdesc = tc::desc_sw128(smem_u32(ring)), vdesc = desc_v(smem_u32(ring));
      int st = 0, guarded = 0;   // the ring's place that is taken next; guarded units so far
      uint32_t ph = 0;
      int before_nk = 0, turns = 0;   // key tiles before, row tiles that had any
      bool ok = true;
      auto step = [&](int& s, uint32_t& p) {
        if (++s == C::STAGES) s = 0, p ^= 1;
      };
      auto qk_unit = [&](uint32_t scol, int s, int u) {
        const uint64_t a = qdesc + ((u * (C::UD / 64) * (kTile * 128)) >> 4), b = kdesc + (s * C::UNIT >> 4);
#pragma unroll
        for (int ks = 0; ks < C::UD / 16; ++ks) {
          const uint64_t oa = ((uint32_t)(ks >> 2) * (kTile * 128) + (uint32_t)(ks & 3) * 32u) >> 4;
          const uint64_t ob = ((uint32_t)(ks >> 2) * (C::KROWS * 128) + (uint32_t)(ks & 3) * 32u) >> 4;
          pre_mma<PAIR>(lead, tb + scol, a + oa, b + ob, id_qk, u != 0 || ks != 0);
        }
      };
      auto pv_unit = [&](uint32_t pcol, int s, int u, bool acc) {
        const uint64_t b = vdesc + (s * C::UNIT >> 4);
#pragma unroll
        for (int ks = 0; ks < kTile / 16; ++ks)
          pre_mma_ts<PAIR>(lead, tb + C::O0 + u * C::UD, tb + pcol + 8 * ks, b + ((uint32_t)ks * 2048u >> 4), id_pv,
                           acc || ks != 0);
      };
      // a look at a barrier ahead of its use, so that the answer is there when
      // the products in between are issued
      auto peek = [&](uint64_t* m, uint32_t p) { return all(tc::mbar_test_wait(m, p)); };
      auto full = [&](int s, uint32_t p) { return pre_wait(&sh.full[s], p, limit, fail); };
      // a guarded V unit: from the guards, and its place's phase moves on here
      auto v_ready = [&](int s, uint32_t p, bool guards) {
        if (!guards) return full(s, p);
        const int k = guarded++;
        if (!pre_wait<PAIR>(&sh.v_ok[k % C::NV], (uint32_t)(k / C::NV) & 1, limit, fail)) return false;
        if (lead) mbar_arrive(&sh.full[s]);
        __syncwarp();
        return true;
      };
      bool seen = false;   // whether the next unit has been seen to be there
      for (int k = 0; ok; ++k) {
        ok = all(tile_wait(k));
        if (!ok) break;
        const PreTile t = sh.tile[k & 1];
        tile_release(k);
        if (t.n < 0) break;
        if (t.nk > 0) ok = all(pre_wait<PAIR>(&sh.q_full, (uint32_t)turns++ & 1, limit, fail));
        auto unit = [&](bool guards) {   // the next unit's place is st; look at the one behind it
          int s1 = st;
          uint32_t p1 = ph;
          step(s1, p1);
          seen = !guards && peek(&sh.full[s1], p1);
        };
        auto qk = [&](int j) {
          const int J = before_nk + j;
#pragma unroll
          for (int u = 0; u < C::U; ++u) {
            if (!seen && !all(full(st, ph))) return false;
            unit(false);
            qk_unit(C::S0 + (J % C::NB) * 128, st, u);
            pre_commit<PAIR>(lead, &sh.empty[st]);
            step(st, ph);
          }
          pre_commit<PAIR>(lead, &sh.s_full[J % C::NB]);
          if (j + 1 == t.nk) pre_commit<PAIR>(lead, &sh.q_free);
          return true;
        };
        auto pv = [&](int j) {
          const int J = before_nk + j;
          const bool guards = (j + 1) * kTile > t.least;
          if (!all(pre_wait(&sh.p_full[J % C::NB], (uint32_t)(J / C::NB) & 1, limit, fail))) return false;
          // O of the row tile before has been read
          if (j == 0 && turns > 1 && !all(pre_wait(&sh.o_free, (uint32_t)turns & 1, limit, fail))) return false;
          tc::fence_after_sync();
#pragma unroll
          for (int u = 0; u < C::U; ++u) {
            if ((guards || !seen) && !all(v_ready(st, ph, guards))) return false;
            unit(guards);
            pv_unit(C::S0 + (J % C::NB) * 128, st, u, j != 0);
            pre_commit<PAIR>(lead, &sh.empty[st]);
            step(st, ph);
          }
          pre_commit<PAIR>(lead, &sh.o_done[J % C::NB]);
          return true;
        };
        tc::fence_after_sync();
        for (int j = 0; ok && j < C::NB && j < t.nk; ++j) ok = qk(j);
        for (int j = 0; ok && j < t.nk; ++j) ok = pv(j) && (j + C::NB >= t.nk || qk(j + C::NB));
        before_nk += t.nk;
      }
      if (!ok) *fail = 1;
      // every product issued, and every arrival on a barrier, before the end
      pre_commit<PAIR>(lead, &sh.drain);
      if (!tc::mbar_wait_bounded(&sh.drain, 0, kPreWait)) *fail = 1;
    } else if (warp >= C::SW + 2 && limit >= 0) {
      // ---- Q, and guards: in V tiles that some row sees in part, keys past the
      // sequence become zero and so do NaN and infinities, which a weight of 0
      // would not keep out of the product; where those were is noted by element
      // for the rows that do see them ----
      // (two units of a tile: a warp each; one: both warps)
      constexpr int GT = C::U == 2 ? 32 : 64;
      const int me = (threadIdx.x - (C::SW + 2) * 32) % GT;
      const int u = C::U == 2 ? warp - (C::SW + 2) : 0;
      bool ok = true;
      int done = 0, units = 0;   // guarded tiles, units of the ring before this tile's
      int turns = 0;             // row tiles that had key tiles
      for (int k = 0; ok; ++k) {
        ok = all(tile_wait(k));
        if (!ok) break;
        const PreTile t = sh.tile[k & 1];
        if (t.n < 0) break;
        // Q, once the products of the row tile before have read theirs; zeros past
        // the last row.  A warp every second group of rows.
        if (t.nk > 0) {
          constexpr int CH = D / 8, RP = 32 / CH;   // 16-byte chunks of a row, rows a pass
          const int64_t rbase = t.r0;
          const int w0 = (warp - (C::SW + 2)) * RP + lane / CH, c8 = lane % CH * 8;
          const int tok0 = (int)(rbase / p.G), y = (int)(rbase - (int64_t)tok0 * p.G) + w0;
          const int dt = 2 * RP / p.G, dg = 2 * RP - dt * p.G;   // from pass to pass
          int tk = tok0 + y / p.G, g = y % p.G;
          const __nv_bfloat16* qg = static_cast<const __nv_bfloat16*>(p.q) + (int64_t)t.q0 * p.q_stride + (int64_t)t.h * p.G * D + c8;
          if (turns > 0) ok = all(pre_wait(&sh.q_free, (uint32_t)(turns - 1) & 1, limit, fail));
          ++turns;
          if (!ok) break;
          for (int x = w0; x < kTile; x += 2 * RP) {
            const bool in = tk < t.n;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(
                             smem_u32(sq + tc::sw128_offset(x, c8, kTile))),
                         "l"(in ? qg + (int64_t)tk * p.q_stride + (int64_t)g * D : qg), "r"(in ? 16 : 0)
                         : "memory");
            tk += dt, g += dg;
            if (g >= p.G) g -= p.G, ++tk;
          }
          asm volatile("cp.async.wait_all;\n" ::: "memory");
          tc::fence_async_smem();
          arrive_lead(&sh.q_full);
        }
        for (int j = t.least / kTile; ok && j < t.nk; ++j) {
          // position of unit u of V tile j in the ring's order
          const int n = units + (min(t.nk, j + C::NB) + j) * C::U + u;
          const int g = done * C::U + u;   // of the guarded units
          ok = all(pre_wait(&sh.v_raw[g % C::NV], (uint32_t)(g / C::NV) & 1, limit, fail));
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
            for (int y = 0; y < 8; ++y) {
              const uint4 w = *reinterpret_cast<const uint4*>(v + (x0 + GT * y) * 16);
#pragma unroll
              for (int i = 0; i < 4; ++i) sum[i] = __hfma2(reinterpret_cast<const __nv_bfloat162*>(&w)[i], zero, sum[i]);
            }
            const __nv_bfloat162 a = __hadd2(__hadd2(sum[0], sum[1]), __hadd2(sum[2], sum[3]));
            if (!__hisnan(a.x) && !__hisnan(a.y)) continue;
            // the notes of the tile before have been read and cleared, in both CTAs
            const long long t0 = clock64();
            while (*(volatile int*)&sh.out_done < k * C::SW * C::CTAS && !*fail)
              if (clock64() - t0 > limit) *fail = 1;
            // (the other CTA's clearing, before notes go there)
            if (PAIR) asm volatile("fence.acq_rel.cluster;\n" ::: "memory");
            else __threadfence_block();
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
          arrive_lead(&sh.v_ok[g % C::NV]);
        }
        if (!ok) break;
        tile_release(k);
        units += 2 * t.nk * C::U;
      }
      if (!ok) *fail = 1;
    }
  }
  if constexpr (PAIR) {   // each CTA learns how far the other came
    if (warp == C::SW && lane == 0) {
      const int o = rank ^ 1;
      *(volatile int*)peer_ptr(&sh.issued[rank], o) = issued;
      *(volatile int*)peer_ptr(&sh.bits[rank], o) = (int)raw_bits;
      *(volatile int*)peer_ptr(&sh.asked[rank], o) = asked;
    }
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
    if (threadIdx.x == 0) atomicExch(p.err, GDN_ERR_TIMEOUT);   // over an earlier code
    if (warp == C::SW && lane == 0) {
      // a pair's bytes of K and of whole V tiles count on the issuing CTA's
      // barriers, which waits for both: with the same units on both sides
      int both = issued, last = issued, k = raw - 1, requests = asked;
      uint32_t bits = raw_bits;
      if constexpr (PAIR) {
        const int other = *(volatile int*)&sh.issued[rank ^ 1];
        both = min(issued, other), last = max(issued, other);
        if (other > issued) bits = (uint32_t)*(volatile int*)&sh.bits[rank ^ 1];
        if (rank == 1) requests = *(volatile int*)&sh.asked[0];
      }
      for (int n = last - 1; n >= 0 && n >= last - C::STAGES; --n, bits >>= 1) {
        const bool mine = n < issued;
        if (bits & 1) {
          if (mine) tc::mbar_wait_bounded(&sh.v_raw[k % C::NV], (uint32_t)(k / C::NV) & 1, kPreWait), --k;
        } else if (rank == 0) {
          uint64_t* bar = &sh.full[n % C::STAGES];
          if (PAIR && n >= both) {
            if (mine) mbar_complete_tx(bar, C::UNIT);   // the other's half does not come
            else tc::mbar_expect_tx(bar, C::UNIT);      // only the other's half comes
          }
          tc::mbar_wait_bounded(bar, (uint32_t)(n / C::STAGES) & 1, kPreWait);
        }
      }
      if (requests > answered) {   // an answer on its way
        if (asked < requests) tc::mbar_expect_tx(&sh.next_full, 16);
        tc::mbar_wait_bounded(&sh.next_full, (uint32_t)answered & 1, kPreWait);
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
cudaError_t prefill_tc(AttnPrefillParams p, cudaStream_t st) {
  using C = PreCfg<D, PAIR>;
  CUtensorMap kmap, vmap;
  cudaError_t e = rows_map(&kmap, p.k, D, p.Hkv, p.Tk, p.k_stride, C::KROWS);
  if (e == cudaSuccess) e = rows_map(&vmap, p.v, D, p.Hkv, p.Tk, p.v_stride, kTile);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(attn_prefill_tc_kernel<D, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPreSmem<D, PAIR>);
  if (e != cudaSuccess) return e;
  constexpr int ROWS = C::CTAS * kTile;
  const int64_t grid = prefill_grid(p, ROWS, 1) * C::CTAS;
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
  // d >= 128: a CTA's 128 rows take a key tile's 64 or 128 KB for 1,069 or 2,144
  // cycles of products, more than L2 gives, so two share them unless a
  // sequence's rows fit one.
  const bool pair = (int64_t)p.max_q * p.G > kTile;
  if (p.d == 64) return prefill_tc<64, false>(p, st);
  if (p.d == 128) return pair ? prefill_tc<128, true>(p, st) : prefill_tc<128, false>(p, st);
  return pair ? prefill_tc<256, true>(p, st) : prefill_tc<256, false>(p, st);
}

}  // namespace gdn
