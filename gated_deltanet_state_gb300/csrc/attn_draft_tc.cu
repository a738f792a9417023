// attn_draft_tc.cu — attention of a draft's rows over the 8-bit cache, on the
// tensor cores (bf16 rows, d a multiple of 32, more than 16 (row, head of the
// group) pairs a kv head).
//
// The pairs are the 128 rows of both products,
//   S [rows x tokens] = Q K^T,    O [rows x elements] += P V,
// with the cache's blocks as the second operands.  A softmax thread holds one
// row, so no maximum or sum crosses lanes; the parts of Q (two) and of P (three)
// are products of their own into the same sums, and P goes back to tensor
// memory over the scores it comes from.  A tile of 128 tokens takes 16 products
// of 67 cycles (scores) and 12 of 134 (outputs), 2,680 in all, as many as its
// 64 KB at d = 256 take at the memory's rate (2,700); the softmax of a tile
// takes 2,600, so two warpgroups take the tiles in turn, the reference passing
// from one to the other before the exponentials.
//
// Measured: 16 drafts of 16 rows over 2,048 to 32,768 tokens (606 MB of codes)
// 225 to 235 us with the join, 2.6 TB/s (with P in two e4m3 parts on one scale 216 us,
// but then what lies below 2^-14 of the reference was lost).  A score buffer's
// own chain (scores, softmax, outputs one after another, and what passes between
// them) is the longest part of a tile; an item's end (128 rows x 1 KB on their
// way out, the next rows' way in) takes about as long as seven tiles, since one
// set of sums and two score tiles fill tensor memory; the join takes 22 us.
#include "attn_decode_tc.cuh"

namespace gdn {

using namespace dt;

namespace {

constexpr int kDrRows = 128;
constexpr int kDrThreads = 256 + 128;      // softmax; K loads, V loads, products (and a warp that idles)
constexpr uint32_t kDrO = 256;             // tensor memory: scores of two tiles, then O

struct DrShared : DtBase {
  uint64_t m_ready[2], fin[2], o_free;
  float m[2][kDrRows];      // a warpgroup's reference of each row, its sum at the end
  float fq[2][kDrRows];     // score factors (heads alternate)
  float4 turn[8][32][5];    // a warp's 32 rows x 16 elements on their way out
};

// D[tmem] (+)= A[tmem] B[smem]^T, e4m3, 32 deep: eight columns of A hold four codes each.
__device__ __forceinline__ void mma_e4m3_ts(uint32_t lead, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}

}  // namespace

__global__ void __launch_bounds__(kDrThreads, 1) attn_draft_tc_kernel(const DtParams w) {
  constexpr int NT = kDrRows;
  extern __shared__ uint8_t dyn[];
  const AttnDecodeParams& p = w.a;
  uint8_t* base = dyn + ((128u - (smem_u32(dyn) & 127u)) & 127u);
  DrShared& sh = *reinterpret_cast<DrShared*>(base + w.misc_off);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, d = p.c.d;
  const int KS = w.k_stages, VS = w.v_stages, NS = max(KS, VS) + 2;
  volatile int* fail = &sh.fail;
  const long long limit = w.wait;

  if (threadIdx.x == 0) {
    for (int i = 0; i < KS; ++i) tc::mbar_init(&sh.k_full[i], 1), tc::mbar_init(&sh.k_empty[i], 1);
    for (int i = 0; i < VS; ++i) tc::mbar_init(&sh.v_full[i], 1), tc::mbar_init(&sh.v_empty[i], 1);
    for (int i = 0; i < NS; ++i) tc::mbar_init(&sh.sc_full[i], 2 * kDtBlocks);
    for (int i = 0; i < 2; ++i) tc::mbar_init(&sh.s_full[i], 1), tc::mbar_init(&sh.p_full[i], 128), tc::mbar_init(&sh.o_done[i], 1);
    tc::mbar_init(&sh.q_full, 256);
    for (int i = 0; i < 2; ++i) tc::mbar_init(&sh.m_ready[i], 128), tc::mbar_init(&sh.fin[i], 128);
    tc::mbar_init(&sh.o_free, 256);
    tc::mbar_init(&sh.drain, 1);
    sh.fail = limit < 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == 8) {
    tc::tmem_alloc(&sh.tmem, 512);
    tc::tmem_relinquish();
  }
  if (warp == 0) dt_sums<NT>(w, sh, lane);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tb = sh.tmem;
  const int i0 = dt_first<NT>(w, sh.items, sh.work, blockIdx.x, gridDim.x);
  const int last_item = dt_first<NT>(w, sh.items, sh.work, blockIdx.x + 1, gridDim.x);
  const int i1 = limit < 0 ? i0 : last_item;
  const uint32_t unit = (uint32_t)kDtTok * d;
  int loaded = 0;

  if (warp < 8) {
    // registers: what the last warpgroup gives up goes to the softmax, together
    // no more than the 168 x 384 that the block starts with
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;\n");
    // ---- softmax: a thread a row, a warpgroup every second tile ----
    const int tid = threadIdx.x & 127, wg = warp >> 2;
    const uint32_t lanes = tb + ((uint32_t)(warp & 3) << 21);
    uint8_t* qd = base + w.q_off;
    bool ok = true;
    // the rows of this warp as hi and lo codes, a row at a time, eight loads ahead
    auto load_q = [&](const DtItem& t, int par) {
      const int e0 = lane * 8;
#pragma unroll 1
      for (int r0 = warp * 16; r0 < warp * 16 + 16; r0 += 8) {
        uint4 x[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int n = r0 + u;
          x[u] = make_uint4(0, 0, 0, 0);
          if (n < t.rows && e0 < d) {
            const int row = (t.r0 + n) / p.G, g = t.r0 + n - row * p.G;
            x[u] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + (int64_t)(t.q0 + row) * p.q_stride +
                                                   (int64_t)(t.h * p.G + g) * d + e0);
          }
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int n = r0 + u;
          uint2 hi, lo;
          const float factor = split_row<true>(x[u], hi, lo);
          if (e0 < d) {
            uint8_t* at = qd + (n >> 3) * 8 * d + (e0 >> 4) * 128 + (n & 7) * 16 + (e0 & 8);
            *reinterpret_cast<uint2*>(at) = hi;
            *reinterpret_cast<uint2*>(at + kDrRows * d) = lo;
          }
          if (lane == 0) sh.fq[par][n] = p.scale_log2 * factor;
        }
      }
      tc::fence_async_smem();
      dt_arrive(&sh.q_full);
    };
    unsigned T = 0;
    int ip = 0, par = 0, items = 0;   // item and head parity, items with tiles
    DtItem t{};
    if (i0 < i1) {
      t = dt_item<NT>(w, sh.items, i0);
      if (dt_load_rows(t, true)) load_q(t, 0);
    }
    for (int i = i0; i < i1; ++i) {
      float l = 0.f, ref = -INFINITY;
      const int row = (t.r0 + tid) / p.G, g = t.r0 + tid - row * p.G;
      const int lim = t.L - t.n + row + 1;            // keys that the row sees (rows past the last: masked as the last)
      const int least = t.L - t.n + t.r0 / p.G + 1;   // keys that every row of the tile sees
      for (int j = 0; j < t.tiles; ++j, ++T) {
        if ((int)(T & 1) != wg) continue;
        const int kb = t.k0 + j * kDtTok, sc = T % NS, st = T % VS;   // scale slot, V stage
        const uint32_t scol = lanes + (T & 1) * kDtTok;
        ok = dt_wait(&sh.sc_full[sc], T / NS & 1, fail, limit) && dt_wait(&sh.s_full[T & 1], (T >> 1) & 1, fail, limit);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        tc::fence_after_sync();
        const float fq = sh.fq[par][tid];
        if (j == 0) sh.bad[ip][tid] = sh.bad[ip][tid + 128] = 0x7fffffff;   // before the other warpgroup's next tile
        uint32_t s[4][32];
#pragma unroll
        for (int u = 0; u < 4; ++u) tc::tmem_ld32_nowait(scol + u * 32, s[u]);
        // factors of the tile's blocks
        float kf[kDtBlocks], lv[kDtBlocks];
        bool part = kb + kDtTok > t.k1;
#pragma unroll
        for (int b = 0; b < kDtBlocks; ++b) {
          const float ks = sh.ks[sc][b], vs = sh.vs[sc][b];
          part = part || !(ks >= 0.f);
          // scales are powers of two from 2^-64 up: the exponent is exact
          lv[b] = (float)((int)(__float_as_uint(vs) >> 23) - 127);
          kf[b] = ks * fq;
          if (kf[b] < 1.2e-38f) kf[b] = 1.2e-38f;   // stays positive: times -inf is a mask (NaN stays)
        }
        tc::tmem_ld_wait();
#pragma unroll
        for (int u = 0; u < 4; ++u) tc::tmem_ld_fence(s[u]);
        const bool edge = kb + kDtTok > least;        // some row does not see some token
        if (part || edge) {
          const int seen = min(lim, t.k1) - kb;
#pragma unroll
          for (int b = 0; b < kDtBlocks; ++b) {
            const bool out = !(sh.ks[sc][b] >= 0.f);
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if (out || b * 16 + k >= seen) s[b / 2][b % 2 * 16 + k] = 0xff800000u;
          }
        }
        // the weight's exponent x = s kf + lv grows with s: the block's largest s gives its largest x
        float mx = -INFINITY;
#pragma unroll
        for (int b = 0; b < kDtBlocks; ++b) {
          float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
          for (int k = 0; k < 16; k += 2) {
            m0 = fmaxf(m0, __uint_as_float(s[b / 2][b % 2 * 16 + k]));
            m1 = fmaxf(m1, __uint_as_float(s[b / 2][b % 2 * 16 + k + 1]));
          }
          mx = fmaxf(mx, fmaf(fmaxf(m0, m1), kf[b], lv[b]));
        }
        float alpha = 1.f;
        const float before = ref;
        if (j > 0) {   // the reference after the tile before, the other warpgroup's
          ok = dt_wait(&sh.m_ready[wg ^ 1], ((T - 1) >> 1) & 1, fail, limit);
          if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
          ref = sh.m[wg ^ 1][tid];
        }
        if (j == 0) {
          ref = mx;
        } else if (mx - ref > kDtGrow) {
          // the reference moves only past the codes' headroom: a row's choice
          // depends on that row alone
          alpha = dt_ex2(ref - mx);
          ref = mx;
        }
        sh.m[wg][tid] = ref;
        dt_arrive(&sh.m_ready[wg]);
        if (j > 1 && ref != before) l *= dt_ex2(before - ref);
        if (__any_sync(0xffffffffu, alpha != 1.f)) {
          ok = dt_wait(&sh.o_done[(T - 1) & 1], ((T - 1) >> 1) & 1, fail, limit);
          if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
          tc::fence_after_sync();
#pragma unroll 1
          for (int e = 0; e < d; e += 32) {
            uint32_t a[16], b[16];
            float o[16], o2[16];
            tc::tmem_ld16x2(lanes + kDrO + e, lanes + kDrO + e + 16, o, o2);
#pragma unroll
            for (int k = 0; k < 16; ++k) a[k] = __float_as_uint(o[k] * alpha), b[k] = __float_as_uint(o2[k] * alpha);
            tc::tmem_st16u(lanes + kDrO + e, a);
            tc::tmem_st16u(lanes + kDrO + e + 16, b);
          }
          tc::tmem_st_wait();
        }
        const float r = (ref == -INFINITY ? 0.f : ref) - kDtBase;
#pragma unroll
        for (int u = 0; u < 4; ++u) {   // 32 tokens: 8 columns of codes of each part
          uint32_t code[3][8];
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const int blk = u * 2 + b;
            const f32x2 kk = pack2(kf[blk], kf[blk]), rr = pack2(lv[blk] - r, lv[blk] - r);
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t* q4 = &s[blk / 2][blk % 2 * 16 + 4 * k];
              const float2 x = unpack2(fma2(pack2(__uint_as_float(q4[0]), __uint_as_float(q4[1])), kk, rr));
              const float2 y = unpack2(fma2(pack2(__uint_as_float(q4[2]), __uint_as_float(q4[3])), kk, rr));
              const float e0 = dt_ex2(x.x), e1 = dt_ex2(x.y), e2 = dt_ex2(y.x), e3 = dt_ex2(y.y);
              sum += (e0 + e1) + (e2 + e3);
              uint32_t part[3];
              split_weights(e0, e1, e2, e3, part);
#pragma unroll
              for (int i2 = 0; i2 < 3; ++i2) code[i2][b * 4 + k] = part[i2];
            }
            l = fmaf(sum, __uint_as_float((uint32_t)(127 - (int)lv[blk]) << 23), l);   // over the V scale
          }
#pragma unroll
          for (int k = 0; k < 3; ++k) tc::tmem_st8(scol + 32 * k + u * 8, code[k]);
        }
        tc::tmem_st_wait();
        if (edge) {
          ok = dt_wait(&sh.v_full[st], T / VS & 1, fail, limit);
          if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
          dt_clean(base + w.v_off + (uint32_t)st * unit, sh.bad[ip], t, kb, least, d, tid);
          tc::fence_async_smem();
        }
        __syncwarp();
        tc::fence_before_sync();
        dt_arrive(&sh.p_full[T & 1]);
      }
      if (!ok) break;
      // the next head's rows: its scores may then start while this item ends
      const DtItem u = t;
      const unsigned last = T - 1;   // the item's last tile
      if (i + 1 < i1) {
        dt_next<NT>(w, sh.items, i + 1, t);
        if (dt_load_rows(t, false)) {
          // (the last scores, if the other warpgroup's, have to be done with the rows)
          if (u.tiles > 0) ok = dt_wait(&sh.s_full[last & 1], (last >> 1) & 1, fail, limit);
          if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
          load_q(t, par ^= 1);
        }
      }
      if (u.tiles > 0) {
        // the row's sum: the warpgroup that had the last tile takes the other's,
        // brought to its reference, and hands the total back; each then writes
        // every second 32 elements
        const int w1 = (int)(last & 1);
        if (wg != w1) {
          ok = dt_wait(&sh.m_ready[w1], (last >> 1) & 1, fail, limit);
          const float mine = ref;
          ref = sh.m[w1][tid];
          sh.m[wg][tid] = l == 0.f ? 0.f : l * dt_ex2(mine - ref);
          dt_arrive(&sh.fin[0]);
          ok = dt_wait(&sh.fin[1], items & 1, fail, limit) && ok;
          l = sh.m[w1][tid];
        } else {
          ok = dt_wait(&sh.fin[0], items & 1, fail, limit);
          l += sh.m[wg ^ 1][tid];
          sh.m[wg][tid] = l;
          dt_arrive(&sh.fin[1]);
        }
        ++items;
        ok = ok && dt_wait(&sh.o_done[last & 1], (last >> 1) & 1, fail, limit);
      }
      if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
      tc::fence_after_sync();
      const bool mine = tid < u.rows;
      const int64_t R = p.T * p.Hq, rh = (int64_t)(u.q0 + row) * p.Hq + u.h * p.G + g;
      const float m = l == 0.f ? -INFINITY : (ref == -INFINITY ? 0.f : ref) - kDtBase;
      if (mine && wg == 0) {
        if (p.part_o) p.part_ml[u.piece * R + rh] = make_float2(m, l);
        else if (p.lse) p.lse[rh] = l == 0.f ? -INFINITY : m * 0.693147180559945309f + logf(l);
      }
      __syncwarp();
      const bool check = u.tiles > 0 && u.k0 + u.tiles * kDtTok > least;   // some tile had values that not every row sees
      float* po = p.part_o + (u.piece * R + rh) * d;
      __nv_bfloat16* oo = static_cast<__nv_bfloat16*>(p.o) + rh * d;
#pragma unroll 1
      for (int e = 32 * wg; e < d; e += 64) {
        float o[32];
        if (u.tiles > 0) {
          tc::tmem_ld32(lanes + kDrO + e, o);
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0.f;
        }
        if (check) {
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (sh.bad[ip][e + k] < lim) o[k] = __int_as_float(0x7fffffff);
        }
        if (p.part_o) {
          // through shared memory, so that a warp writes 64 bytes of eight rows at a time
          const int rows = min(32, u.rows - (warp & 3) * 32), c4 = lane & 3;
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float* x = o + hf * 16 + 4 * k;
              sh.turn[warp][lane][k] = make_float4(x[0], x[1], x[2], x[3]);
            }
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 32; k += 8) {
              const int r = k + (lane >> 2);
              const uintptr_t at = __shfl_sync(0xffffffffu, reinterpret_cast<uintptr_t>(po + e + hf * 16), r);
              if (r < rows) reinterpret_cast<float4*>(at)[c4] = sh.turn[warp][r][c4];
            }
            __syncwarp();
          }
        } else if (mine) {
#pragma unroll
          for (int k = 0; k < 32; k += 8) {
            uint32_t b[4];
#pragma unroll
            for (int i2 = 0; i2 < 4; ++i2) {
              const float x = l == 0.f ? 0.f : o[k + 2 * i2] / l, y = l == 0.f ? 0.f : o[k + 2 * i2 + 1] / l;
              const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
              b[i2] = *reinterpret_cast<const uint32_t*>(&h);
            }
            *reinterpret_cast<uint4*>(oo + e + k) = make_uint4(b[0], b[1], b[2], b[3]);
          }
        }
        __syncwarp();
      }
      tc::fence_before_sync();
      if (u.tiles > 0) dt_arrive(&sh.o_free);
      // (a buffer comes back after an item whose tiles every warp has passed)
      if (u.tiles > 0) ip ^= 1;
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;\n");
    if (warp == 8 || warp == 9) {
      // ---- loads, a warp for K and one for V ----
      loaded = dt_load<NT>(w, sh, base, i0, i1, warp == 9, lane);
    } else if (warp == 10) {
      // ---- products: the whole warp, one lane issues ----
      const uint32_t lead = tc::elect_one();
      auto all = [](bool x) { return __all_sync(0xffffffffu, x) != 0; };
      constexpr uint32_t id_qk = idesc_e4m3(kDtTok);
      const uint32_t id_pv = idesc_e4m3(d) | kE5m2A;
      const uint32_t k0 = smem_u32(base + w.k_off), v0 = smem_u32(base + w.v_off), qa = smem_u32(base + w.q_off);
      const uint32_t rows8 = 8u * d;
      const uint64_t vstep = (uint64_t)(32u * d >> 4);
      int ks = 0, kp = 0, vs = 0, vp = 0, rows = 0;
      unsigned T = 0;   // tiles multiplied
      bool ok = true;
      auto qk = [&](unsigned tt) {
        if (!all(dt_wait(&sh.k_full[ks], kp, fail, limit))) return false;
        tc::fence_after_sync();
        const uint64_t b = desc_tiles(k0 + ks * unit, 128, rows8);
        const uint32_t dst = tb + (tt & 1) * kDtTok;
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          const uint32_t id = id_qk | (part ? kE5m2A : 0u);
          const uint64_t a = desc_tiles(qa + part * kDrRows * d, 128, rows8);
          if (d == 256) {
            mma_steps<8>(lead, dst, a, b, id, 16, 16, part);
          } else if (d == 128) {
            mma_steps<4>(lead, dst, a, b, id, 16, 16, part);
          } else {
            for (int c = 0; c < d / 32; ++c) mma_e4m3(lead, dst, a + c * 16, b + c * 16, id, part | c);
          }
        }
        tc::mma_commit_if(lead, &sh.k_empty[ks]);
        tc::mma_commit_if(lead, &sh.s_full[tt & 1]);
        if (++ks == KS) ks = 0, kp ^= 1;
        return true;
      };
      DtItem t{};
      int items = 0;   // with tiles
      for (int i = i0; ok && i < i1; ++i) {
        if (i == i0) t = dt_item<NT>(w, sh.items, i);
        else dt_next<NT>(w, sh.items, i, t);
        if (dt_load_rows(t, i == i0)) ok = all(dt_wait(&sh.q_full, rows++ & 1, fail, limit));
        if (ok && t.tiles > 0) ok = qk(T);
        for (int j = 0; ok && j < t.tiles; ++j, ++T) {
          if (j + 1 < t.tiles) ok = qk(T + 1);
          ok = ok && all(dt_wait(&sh.p_full[T & 1], (T >> 1) & 1, fail, limit) && dt_wait(&sh.v_full[vs], vp, fail, limit));
          // O of the item before has been read, by both warpgroups
          if (ok && j == 0 && items++ > 0) ok = all(dt_wait(&sh.o_free, items & 1, fail, limit));
          if (!ok) break;
          tc::fence_after_sync();
          const uint64_t b = desc_tiles(v0 + vs * unit, 16u * d, 128);
#pragma unroll
          for (int part = 0; part < 3; ++part)
#pragma unroll
            for (int c = 0; c < kDtTok / 32; ++c)
              mma_e4m3_ts(lead, tb + kDrO, tb + (T & 1) * kDtTok + part * 32 + c * 8, b + c * vstep, id_pv, j | part | c);
          tc::mma_commit_if(lead, &sh.v_empty[vs]);
          tc::mma_commit_if(lead, &sh.o_done[T & 1]);
          if (++vs == VS) vs = 0, vp ^= 1;
        }
      }
      // every product issued, and every arrival on a barrier, before the end
      tc::mma_commit_if(lead, &sh.drain);
      if (!tc::mbar_wait_bounded(&sh.drain, 0, kDtWait)) *fail = 1;
    }
  }
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  if (sh.fail) {
    // a wait ran out: report, then give the copies in flight one more bounded
    // wait each before their memory goes
    dt_report<NT>(w, sh, i0, last_item);
    if ((warp == 8 || warp == 9) && lane == 0) dt_drain(w, sh, loaded, warp == 9);
    __syncwarp();
    __syncthreads();
  }
  tc::fence_after_sync();
  if (warp == 8) tc::tmem_dealloc(tb, 512);
  // done when the kernel before this one (the call's other sequences) is
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
}

cudaError_t launch_attn_draft_tc(const AttnDecodeParams& p, int sms, bool overlap, cudaStream_t st) {
  DtParams w{};
  w.a = p;
  w.wait = dt_limit(p);
  w.row_lo = overlap ? kDtNarrow + 1 : 1, w.row_hi = 0x7fffffff;
  const uint32_t q = 2 * kDrRows * (uint32_t)p.c.d;
  w.q_off = dt_rings(w, 232448, q + (uint32_t)sizeof(DrShared) + 512);
  if (w.v_stages < 1) return cudaErrorInvalidValue;
  w.misc_off = (w.q_off + q + 127) / 128 * 128;
  uint32_t smem = w.misc_off + (uint32_t)sizeof(DrShared) + 128;
  if (smem < 120 * 1024) smem = 120 * 1024;   // one CTA an SM: it takes the tensor memory whole
  cudaError_t e = allow_shared(attn_draft_tc_kernel);
  if (e != cudaSuccess) return e;
  const int rt = (p.max_q * p.G + kDrRows - 1) / kDrRows;
  for (int s0 = 0; s0 < p.N; s0 += kDtSeqs) {
    w.s0 = s0;
    w.ns = p.N - s0 < kDtSeqs ? p.N - s0 : kDtSeqs;
    const int64_t most = (int64_t)w.ns * p.max_pieces * p.c.Hkv * rt;
    // behind the kernel of the sequences with few rows, which share nothing with these
    e = dt_launch(attn_draft_tc_kernel, w, most < sms ? most : sms, kDrThreads, smem, overlap, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace gdn
