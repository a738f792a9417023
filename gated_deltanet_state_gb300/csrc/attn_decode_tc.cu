// attn_decode_tc.cu — attention of a few new rows a sequence over the 8-bit
// cache, on the tensor cores (bf16 rows, d a multiple of 32, up to 16 (row,
// head of the group) pairs a kv head).
//
// With 128 tokens as the rows of the first product and the head's elements as
// the rows of the second,
//   S^T [tokens x rows] = K Q^T,    O^T [elements x rows] += V^T P^T,
// the few query rows are the products' narrow side; the two parts of Q and the
// three of P stand side by side as columns whose sums are added when read (a
// product of up to 64 columns takes the time that reading the 128 rows of
// codes takes, 52 cycles).
//
// Bound by HBM: 256 sequences over 1,024 to 8,192 tokens (24 heads, 4 kv heads,
// d = 256: 2.45 GB) take 403 to 407 us with the join, 6.0 TB/s or 89 % of a
// copy's rate; one over 777 tokens 13.5 to 14 us, two launches and the chain of a
// piece's loads, two products and softmax.  The third part of P doubles the
// columns of 8 rows' output products (16 to 32): nothing at d = 256, 7 to 10 % at
// narrow heads (64 sequences of 1,024 to 8,192 tokens, 32 heads, 8, d = 64: 113 us).
#include "attn_decode_tc.cuh"

namespace gdn {

using namespace dt;

namespace {

// NT query rows (8 or 16), a softmax warpgroup of 128 threads, a token each.
// Two CTAs an SM: one's softmax runs under the other's products and loads.
template <int NT>
struct DtCfg {
  static constexpr int CW = NT;
  static constexpr int NQ = 2 * NT;                    // columns of the scores' products
  static constexpr int NP = NT <= 8 ? 32 : 48;         // of the outputs': 3 NT, in blocks of 16
  static constexpr int THREADS = 128 + 96;             // and K loads, V loads, products
  static constexpr uint32_t COLS = NT <= 8 ? 128 : 256;   // two CTAs an SM
  static constexpr uint32_t O0 = 2 * NQ;               // scores of two tiles, then O of 128 elements each
  static_assert(O0 + 2 * NP <= COLS, "tensor memory");
};

template <int NT>
struct DtShared : DtBase {
  float4 lsum[NT];
  float cmax[4][NT];        // largest score of each column, by warp
  float ref[NT], alpha[NT];
  // of a head's rows, heads alternate: score factor, keys seen, place among the outputs
  float fq[2][NT];
  int lim[2][NT];
  uint32_t out[2][NT];      // (row, head) counted from the item's first row's head 0
  unsigned grow;            // the last tile (from 1) that moved a column's reference
};

// The rows' scores: hi and lo parts added.
template <int CW>
__device__ __forceinline__ void read_scores(uint32_t col, float (&x)[CW]) {
  if constexpr (CW == 8) {
    float v[16];
    tc::tmem_ld16(col, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = fmaf(v[8 + k], kDtLo, v[k]);
  } else {
    float v[16];
    tc::tmem_ld16x2(col, col + 16, x, v);
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] = fmaf(v[k], kDtLo, x[k]);
  }
}
// The rows' outputs: three parts added.
template <int CW>
__device__ __forceinline__ void read_outputs(uint32_t col, float (&x)[CW]) {
  float v[16];
  if constexpr (CW == 8) {
    float u[16];
    tc::tmem_ld16x2(col, col + 16, u, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = u[k] + (u[8 + k] + v[k]);
  } else {
    tc::tmem_ld16x2(col + 16, col + 32, x, v);
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] += v[k];
    tc::tmem_ld16(col, v);
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] += v[k];
  }
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
// Barrier of the softmax warps; true when all of them say so, which keeps them
// together when a wait has run out.
__device__ __forceinline__ bool bar_and(bool ok) {
  int r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n barrier.cta.red.and.pred q, 1, 128, p;\n"
      " selp.s32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((int)ok)
      : "memory");
  __syncwarp();
  return r != 0;
}

}  // namespace

template <int NT>
__global__ void __launch_bounds__(DtCfg<NT>::THREADS, 2) attn_decode_tc_kernel(const DtParams w) {
  using C = DtCfg<NT>;
  constexpr int CW = C::CW, WARPS = 4;   // softmax warps; then K loads, V loads, products
  extern __shared__ uint8_t dyn[];
  const AttnDecodeParams& p = w.a;
  uint8_t* base = dyn + ((128u - (smem_u32(dyn) & 127u)) & 127u);
  DtShared<NT>& sh = *reinterpret_cast<DtShared<NT>*>(base + w.misc_off);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, d = p.c.d;
  const int KS = w.k_stages, VS = w.v_stages, NS = max(KS, VS) + 2;
  volatile int* fail = &sh.fail;
  const long long limit = w.wait;

  if (threadIdx.x == 0) {
    for (int i = 0; i < KS; ++i) tc::mbar_init(&sh.k_full[i], 1), tc::mbar_init(&sh.k_empty[i], 1);
    for (int i = 0; i < VS; ++i) tc::mbar_init(&sh.v_full[i], 1), tc::mbar_init(&sh.v_empty[i], 1);
    for (int i = 0; i < NS; ++i) tc::mbar_init(&sh.sc_full[i], 2 * kDtBlocks);
    for (int i = 0; i < 2; ++i)
      tc::mbar_init(&sh.s_full[i], 1), tc::mbar_init(&sh.p_full[i], 128), tc::mbar_init(&sh.o_done[i], 1);
    tc::mbar_init(&sh.q_full, 128);
    tc::mbar_init(&sh.drain, 1);
    sh.fail = limit < 0;
    sh.grow = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == WARPS) {
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
  const uint32_t unit = (uint32_t)kDtTok * d;   // bytes of a tile's K (or V) codes
  int loaded = 0;                               // tiles loaded (a loading warp's)

  if (warp == WARPS || warp == WARPS + 1) {
    // ---- loads, a warp for K and one for V ----
    loaded = dt_load<NT>(w, sh, base, i0, i1, warp == WARPS + 1, lane);
  } else if (warp == WARPS + 2) {
    // ---- products: the whole warp, one lane issues ----
    const uint32_t lead = tc::elect_one();
    auto all = [](bool x) { return __all_sync(0xffffffffu, x) != 0; };
    constexpr uint32_t id_qk = idesc_e4m3(C::NQ), id_pv = idesc_e4m3(C::NP) | kE5m2B | kTransposedB;
    const uint32_t k0 = smem_u32(base + w.k_off), v0 = smem_u32(base + w.v_off), qa = smem_u32(base + w.q_off),
                   pa = smem_u32(base + w.p_off);
    const uint32_t rows8 = 8u * d;   // 8 tokens of K (or 8 rows of Q)
    const int halves = (d + 127) / 128;
    const uint64_t vstep = (uint64_t)(32u * d >> 4);
    int ks = 0, kp = 0, vs = 0, vp = 0, rows = 0;
    unsigned T = 0;   // tiles multiplied
    bool ok = true;
    auto qk = [&](unsigned tt) {
      if (!all(dt_wait(&sh.k_full[ks], kp, fail, limit))) return false;
      tc::fence_after_sync();
      const uint64_t a = desc_tiles(k0 + ks * unit, 128, rows8);
      const uint64_t b = desc_tiles(qa, 128, rows8);
      const uint32_t dst = tb + (tt & 1) * C::NQ;
      if (d == 256) {
        mma_steps<8>(lead, dst, a, b, id_qk, 16, 16, false);
      } else if (d == 128) {
        mma_steps<4>(lead, dst, a, b, id_qk, 16, 16, false);
      } else {
        for (int c = 0; c < d / 32; ++c) mma_e4m3(lead, dst, a + c * 16, b + c * 16, id_qk, c);
      }
      tc::mma_commit_if(lead, &sh.k_empty[ks]);
      tc::mma_commit_if(lead, &sh.s_full[tt & 1]);
      if (++ks == KS) ks = 0, kp ^= 1;
      return true;
    };
    DtItem t{};
    for (int i = i0; ok && i < i1; ++i) {
      if (i == i0) t = dt_item<NT>(w, sh.items, i);
      else dt_next<NT>(w, sh.items, i, t);
      if (dt_load_rows(t, i == i0)) ok = all(dt_wait(&sh.q_full, rows++ & 1, fail, limit));
      if (ok && t.tiles > 0) ok = qk(T);
      for (int j = 0; ok && j < t.tiles; ++j, ++T) {
        if (j + 1 < t.tiles) ok = qk(T + 1);
        ok = ok && all(dt_wait(&sh.p_full[T & 1], (T >> 1) & 1, fail, limit) && dt_wait(&sh.v_full[vs], vp, fail, limit));
        if (!ok) break;
        tc::fence_after_sync();
        for (int hf = 0; hf < halves; ++hf) {
          const uint64_t a = desc_tiles(v0 + vs * unit + hf * 2048u, 16u * d, 128);
          // P: tokens of 16 columns (16 B), the next 16 columns a block of 128 tokens further
          mma_steps<kDtTok / 32>(lead, tb + C::O0 + hf * C::NP, a, desc_tiles(pa, 128, 16 * kDtTok), id_pv, vstep, 32, j != 0);
        }
        tc::mma_commit_if(lead, &sh.v_empty[vs]);
        tc::mma_commit_if(lead, &sh.o_done[T & 1]);
        if (++vs == VS) vs = 0, vp ^= 1;
      }
    }
    // every product issued, and every arrival on a barrier, before the end
    tc::mma_commit_if(lead, &sh.drain);
    if (!tc::mbar_wait_bounded(&sh.drain, 0, kDtWait)) *fail = 1;
  } else {
    // ---- softmax: a thread a token of the tile ----
    const int quad = warp, tid = threadIdx.x;
    const uint32_t lanes = tb + ((uint32_t)quad << 21);
    uint8_t* qd = base + w.q_off;
    uint8_t* pd = base + w.p_off;
    bool ok = true, okp = true;
    // an item's rows as hi and lo codes, a warp a row at a time, all loads first;
    // where they belong is noted for an item without keys too
    auto load_q = [&](const DtItem& t, int par) {
      const int e0 = lane * 8;
      constexpr int NR = CW / 4;
      uint4 x[NR];
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const int n = r * 4 + quad;
        x[r] = make_uint4(0, 0, 0, 0);
        if (n < t.rows) {
          const int row = (t.r0 + n) / p.G, g = t.r0 + n - row * p.G;
          if (t.tiles > 0 && e0 < d)
            x[r] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + (int64_t)(t.q0 + row) * p.q_stride +
                                                   (int64_t)(t.h * p.G + g) * d + e0);
          if (lane == 0) {
            sh.lim[par][n] = t.L - t.n + row + 1;
            sh.out[par][n] = (uint32_t)((row - t.r0 / p.G) * p.Hq + t.h * p.G + g);
          }
        }
      }
      if (t.tiles == 0) return;
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const int n = r * 4 + quad;
        uint2 hi, lo;
        const float factor = split_row<false>(x[r], hi, lo);
        if (e0 < d) {
          uint8_t* at = qd + (n >> 3) * 8 * d + (e0 >> 4) * 128 + (n & 7) * 16 + (e0 & 8);
          *reinterpret_cast<uint2*>(at) = hi;
          *reinterpret_cast<uint2*>(at + NT * d) = lo;
        }
        if (lane == 0) sh.fq[par][n] = p.scale_log2 * factor;
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
    bar_and(true);
    for (int i = i0; i < i1; ++i) {
      float l[CW];
#pragma unroll
      for (int n = 0; n < CW; ++n) l[n] = 0.f;
      float ref = -INFINITY;                          // of column tid
      if (t.tiles > 0) sh.bad[ip][tid] = sh.bad[ip][tid + 128] = 0x7fffffff;
      const int least = t.L - t.n + 1;                // keys that every row sees
      for (int j = 0; j < t.tiles; ++j, ++T) {
        const int kb = t.k0 + j * kDtTok, pos = kb + tid;
        const uint32_t scol = lanes + (T & 1) * C::NQ;
        ok = dt_wait(&sh.sc_full[sc], scp, fail, limit) && dt_wait(&sh.s_full[T & 1], (T >> 1) & 1, fail, limit);
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
        float x[CW];
        read_scores(scol, x);
        const float4* f4 = reinterpret_cast<const float4*>(&sh.fq[par][0]);
#pragma unroll
        for (int k = 0; k < CW; k += 4) {
          const float4 f = f4[k / 4];
#pragma unroll
          for (int u = 0; u < 4; ++u) x[k + u] = fmaf(x[k + u], kscale * (&f.x)[u], lv);
        }
        if (part || edge) {
#pragma unroll
          for (int k = 0; k < CW; ++k)
            if (!valid || pos >= sh.lim[par][k]) x[k] = -INFINITY;
        }
#pragma unroll
        for (int k = 0; k < CW; k += 4) {
          const float a = warp_max(x[k]), b = warp_max(x[k + 1]), c = warp_max(x[k + 2]), e = warp_max(x[k + 3]);
          if (lane == 0) *reinterpret_cast<float4*>(&sh.cmax[quad][k]) = make_float4(a, b, c, e);
        }
        ok = bar_and(ok && okp);
        if (!ok) break;
        if (tid < CW) {
          const int n = tid;
          const float mx = fmaxf(fmaxf(sh.cmax[0][n], sh.cmax[1][n]), fmaxf(sh.cmax[2][n], sh.cmax[3][n]));
          float alpha = 1.f;
          if (j == 0) {
            ref = mx;
          } else if (mx - ref > kDtGrow) {
            // the reference moves only past the codes' headroom: a column's
            // choice depends on that column alone
            alpha = dt_ex2(ref - mx);
            ref = mx;
            *(volatile unsigned*)&sh.grow = T + 1;
          }
          sh.ref[n] = (ref == -INFINITY ? 0.f : ref) - kDtBase;
          sh.alpha[n] = alpha;
        }
        bar_and(true);
        if (*(volatile unsigned*)&sh.grow == T + 1) {
          // the products before this tile's: done, then scaled column by column
          // (one that runs out shows at the next barrier)
          okp = dt_wait(&sh.o_done[(T - 1) & 1], ((T - 1) >> 1) & 1, fail, limit);
          __syncwarp();
          tc::fence_after_sync();
          float al[CW];
#pragma unroll
          for (int n = 0; n < CW; ++n) al[n] = sh.alpha[n], l[n] *= al[n];
          for (int hf = 0; hf < (d + 127) / 128; ++hf) {
#pragma unroll
            for (int c = 0; c < C::NP; c += 16) {
              const uint32_t col = lanes + C::O0 + hf * C::NP + c;
              float o[16];
              tc::tmem_ld16(col, o);
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] *= al[k % CW];
              tc::tmem_st16(col, o);
            }
          }
          tc::tmem_st_wait();
        }
        // the weights' place: read by the product before
        if (j > 0) okp = dt_wait(&sh.o_done[(T - 1) & 1], ((T - 1) >> 1) & 1, fail, limit) && okp;
        uint8_t* pw = pd + tid * 16;
        uint32_t w4[3][CW / 4];
        const float4* r4 = reinterpret_cast<const float4*>(&sh.ref[0]);
#pragma unroll
        for (int u = 0; u < CW / 4; ++u) {
          const float4 r = r4[u];
          float e[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            e[k] = dt_ex2(x[4 * u + k] - (&r.x)[k]);
            l[4 * u + k] = fmaf(e[k], rv, l[4 * u + k]);
          }
          uint32_t part[3];
          split_weights(e[0], e[1], e[2], e[3], part);
#pragma unroll
          for (int k = 0; k < 3; ++k) w4[k][u] = part[k];
        }
        if constexpr (CW == 8) {
          *reinterpret_cast<uint4*>(pw) = make_uint4(w4[0][0], w4[0][1], w4[1][0], w4[1][1]);
          *reinterpret_cast<uint4*>(pw + 16 * kDtTok) = make_uint4(w4[2][0], w4[2][1], 0, 0);
        } else {
#pragma unroll
          for (int k = 0; k < 3; ++k)
            *reinterpret_cast<uint4*>(pw + k * 16 * kDtTok) = make_uint4(w4[k][0], w4[k][1], w4[k][2], w4[k][3]);
        }
        if (edge) {
          ok = bar_and(dt_wait(&sh.v_full[st], vp, fail, limit));
          if (!ok) break;
          dt_clean(base + w.v_off + (uint32_t)st * unit, sh.bad[ip], t, kb, least, d, tid);
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
        if (dt_new_rows(t, false)) load_q(t, par ^= 1);
      }
      column_sums<CW>(l, sh.lsum, lane, quad);
      if (u.tiles > 0) ok = dt_wait(&sh.o_done[(T - 1) & 1], ((T - 1) >> 1) & 1, fail, limit);
      ok = bar_and(ok && okp);
      if (!ok) break;
      tc::fence_after_sync();
      const int64_t R = p.T * p.Hq, rh0 = (int64_t)(u.q0 + u.r0 / p.G) * p.Hq;
      const int mine = u.rows;   // columns of this warpgroup that are rows
      if (tid < mine) {
        const float4 c = sh.lsum[tid];
        const float sum = (c.x + c.y) + (c.z + c.w), m = sum == 0.f ? -INFINITY : sh.ref[tid];
        const int64_t rh = rh0 + sh.out[was][tid];
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
        float o[CW];
        if (u.tiles > 0) {
          read_outputs(lanes + C::O0 + hf * C::NP, o);
        } else {
#pragma unroll
          for (int k = 0; k < CW; ++k) o[k] = 0.f;
        }
        if (e < d) {
          if (check) {
            const int bad = sh.bad[ip][e];
#pragma unroll
            for (int k = 0; k < CW; ++k)
              if (bad < sh.lim[was][k]) o[k] = __int_as_float(0x7fffffff);
          }
#pragma unroll
          for (int k = 0; k < CW; ++k) {
            const uint32_t at = sh.out[was][k] * (uint32_t)d;   // at most 32 rows of 1,024 heads of 256 elements
            if (k < mine) {
              if (p.part_o) {
                po[at] = o[k];
              } else {
                const float4 c = sh.lsum[k];
                const float sum = (c.x + c.y) + (c.z + c.w);
                oo[at] = __float2bfloat16_rn(sum == 0.f ? 0.f : o[k] / sum);
              }
            }
          }
        }
        __syncwarp();
      }
      tc::fence_before_sync();
      bar_and(true);   // lsum, ref and O are free
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
    dt_report<NT>(w, sh, i0, last_item);
    if ((warp == WARPS || warp == WARPS + 1) && lane == 0) dt_drain(w, sh, loaded, warp == WARPS + 1);
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
  w.wait = dt_limit(p);
  w.row_lo = 1, w.row_hi = kDtNarrow;
  const uint32_t q = C::NQ * (uint32_t)p.c.d, pp = C::NP * kDtTok;
  // half of 227 KB a CTA, of which 1 KB is the system's
  w.q_off = dt_rings(w, 115712, q + pp + (uint32_t)sizeof(DtShared<NT>) + 512);
  if (w.v_stages < 1) return cudaErrorInvalidValue;
  w.p_off = w.q_off + q;
  w.misc_off = (w.p_off + pp + 127) / 128 * 128;
  uint32_t smem = w.misc_off + (uint32_t)sizeof(DtShared<NT>) + 128;
  if (smem < 80 * 1024) smem = 80 * 1024;   // no more than two CTAs an SM share its tensor memory
  cudaError_t e = cudaFuncSetAttribute(attn_decode_tc_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  for (int s0 = 0; s0 < p.N; s0 += kDtSeqs) {
    w.s0 = s0;
    w.ns = p.N - s0 < kDtSeqs ? p.N - s0 : kDtSeqs;
    const int64_t most = (int64_t)w.ns * p.max_pieces * p.c.Hkv;
    attn_decode_tc_kernel<NT><<<(unsigned)(most < 2 * sms ? most : 2 * sms), C::THREADS, smem, st>>>(w);
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
  // a sequence's kernel goes by its own rows (a row's bits with it): up to 16
  // (row, head) pairs of a kv head here, more with the rows as the products'
  // 128 (attn_draft_tc.cu); a call that may have both launches both
  if (p.max_q * p.G > kDtNarrow) {
    // (none has few where all rows together say that each has max_q: a launch, 6 us, less)
    const bool few = p.G <= kDtNarrow && (int64_t)p.N * p.max_q != p.T;
    if (few) e = decode_tc<16>(p, sms, st);
    return e != cudaSuccess ? e : launch_attn_draft_tc(p, sms, few, st);
  }
  return p.max_q * p.G <= 8 ? decode_tc<8>(p, sms, st) : decode_tc<16>(p, sms, st);
}

}  // namespace gdn
