// kv_cache.cu — the paged 8-bit K / V cache of the attention layers: a step's
// tables, the append of new rows and the read-back of a cached prefix
// (layout and rules: include/gdn.h).
#include "attn.h"

namespace gdn {

namespace {

// Exclusive prefix sums of two ints over a CTA of 256 threads; the totals come
// back in ta, tb.
__device__ __forceinline__ void scan2_256(int& a, int& b, int& ta, int& tb, int* sh /* [16] */) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int ia = a, ib = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int xa = __shfl_up_sync(0xffffffffu, ia, o), xb = __shfl_up_sync(0xffffffffu, ib, o);
    if (lane >= o) ia += xa, ib += xb;
  }
  if (lane == 31) sh[w] = ia, sh[8 + w] = ib;
  __syncthreads();
  int ba = 0, bb = 0;
  ta = tb = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (i == w) ba = ta, bb = tb;
    ta += sh[i], tb += sh[8 + i];
  }
  __syncthreads();
  a = ba + ia - a;
  b = bb + ib - b;
}

}  // namespace

// Tables of a step.  CTA (x, y): requests [x * seqs_per_cta, ...), slice y of
// their tokens.  Every CTA forms the running sums up to its own requests from
// the lengths themselves (N loads of 8 bytes from L2), so one launch does all
// and no CTA waits on another.  Bound by the launch and a few dependent loads:
// 256 requests of one token 8.8 us for the whole call, 67 prompts 9.6 us.
__global__ void __launch_bounds__(256) kv_tables_kernel(const KvTablesParams p) {
  __shared__ int sh[16];
  __shared__ int s_first[64], s_row[64], s_ok[64];   // of this CTA's requests
  const int s0 = blockIdx.x * p.seqs_per_cta, s1 = min(p.N, s0 + p.seqs_per_cta);
  int need0 = 0, row0 = 0, kv0 = 0, taken = 0;   // running sums before the scanned chunk
  for (int c0 = 0; c0 < s1; ) {
    // chunks of 256 requests up to s0, then the CTA's own (at most 64)
    const int c1 = c0 < s0 ? min(s0, c0 + 256) : s1;
    const int s = c0 + threadIdx.x;
    int kv = 0, add = 0, need = 0, have = 0;
    bool ok = true;
    if (s < c1) {
      kv = p.kv_len[s], add = p.new_len[s];
      const int64_t total = (int64_t)kv + add;
      ok = kv >= 0 && add >= 0 && total <= 0x7fffffff && (total + p.page_tokens - 1) / p.page_tokens <= p.max_pages;
      if (kv < 0) kv = 0;
      if (add < 0) add = 0;
      have = (int)(((int64_t)kv + p.page_tokens - 1) / p.page_tokens);
      need = ok ? (int)((total + p.page_tokens - 1) / p.page_tokens) - have : 0;
    }
    int first = need, row = add, tn, ta;
    scan2_256(first, row, tn, ta, sh);
    first += need0, row += row0;
    ok = ok && (need == 0 || first + need <= p.num_free);
    int out = s < c1 ? kv + (ok ? add : 0) : 0, got = s < c1 && ok ? need : 0, to, tg;
    const int kv_out = out;
    scan2_256(out, got, to, tg, sh);
    if (c0 >= s0 && s < c1) {
      s_first[s - s0] = first, s_row[s - s0] = row, s_ok[s - s0] = ok;
      if (blockIdx.y == 0) {
        if (!ok) set_error(p.err, GDN_ERR_PAGE_RANGE);
        p.cu_seqlens[s] = row;
        p.cu_kv[s] = kv0 + out;
        p.kv_len_out[s] = kv_out;
        if (s == p.N - 1) {
          p.cu_seqlens[p.N] = row0 + ta;
          p.cu_kv[p.N] = kv0 + to;
          p.pages_taken[0] = taken + tg;
        }
      }
    }
    need0 += tn, row0 += ta, kv0 += to, taken += tg;
    c0 = c1;
  }
  __syncthreads();
  const int me = blockIdx.y * blockDim.x + threadIdx.x, step = gridDim.y * blockDim.x;
  for (int s = s0; s < s1; ++s) {
    const int first = s_first[s - s0], kv = max(0, p.kv_len[s]), add = max(0, p.new_len[s]);
    const bool ok = s_ok[s - s0];
    const int have = (int)(((int64_t)kv + p.page_tokens - 1) / p.page_tokens);
    int32_t* bt = p.block_table + (int64_t)s * p.max_pages;
    if (ok) {
      const int want = (int)(((int64_t)kv + add + p.page_tokens - 1) / p.page_tokens);
      for (int j = have + me; j < want; j += step) bt[j] = p.free_pages[first + j - have];
    }
    const int64_t r0 = s_row[s - s0];
    for (int i = me; i < add; i += step) {
      if (r0 + i >= p.T) break;
      const int64_t pos = (int64_t)kv + i;
      int64_t slot = -1;
      if (ok) {
        const int j = (int)(pos / p.page_tokens);
        // a fresh page's id comes from the list: the table's entry may not be written yet
        const int page = j < have ? bt[j] : p.free_pages[first + j - have];
        if (page >= 0 && page < p.num_pages)
          slot = (int64_t)page * p.page_tokens + (int)(pos - (int64_t)j * p.page_tokens);
        else
          set_error(p.err, GDN_ERR_PAGE_RANGE);
      }
      p.positions[r0 + i] = pos;
      p.slot_map[r0 + i] = slot;
    }
  }
  // rows past the last request's
  if (s1 == p.N)
    for (int64_t t = (int64_t)row0 + me; t < p.T; t += step) p.positions[t] = 0, p.slot_map[t] = -1;
}

cudaError_t launch_kv_tables(const KvTablesParams& q, cudaStream_t st) {
  KvTablesParams p = q;
  // at most 1,024 groups of requests re-form the sums before them; tokens
  // beyond about 1,024 a CTA spread over y
  p.seqs_per_cta = (p.N + 1023) / 1024;
  const int gx = (p.N + p.seqs_per_cta - 1) / p.seqs_per_cta;
  int64_t gy = p.T / ((int64_t)gx * 1024);
  gy = gy < 1 ? 1 : gy > 64 ? 64 : gy;
  kv_tables_kernel<<<dim3(gx, (unsigned)gy), 256, 0, st>>>(p);
  return cudaGetLastError();
}

// ---- append -------------------------------------------------------------------------
namespace {

// The smallest power of two, at least 2^-64, with amax / scale <= 448 (finite amax >= 0).
__device__ __forceinline__ float pow2_scale(float amax) {
  const uint32_t b = __float_as_uint(amax);
  // 448 = 1.75 * 2^8: amax = 1.m * 2^e needs 2^(e - 8), one more when 1.m > 1.75
  int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  if (b < 0x00800000u || e < -64) e = -64;   // subnormal amax: far below 448 * 2^-64
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Largest magnitude of eight elements; NaN falls out, an infinity stays.
__device__ __forceinline__ float max8(const Row8<__nv_bfloat16>& r) {
  __nv_bfloat162 m = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = (&r.w.x)[i] & 0x7fff7fffu;
    m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162*>(&w));
  }
  return fmaxf(__bfloat162float(m.x), __bfloat162float(m.y));
}
__device__ __forceinline__ float max8(const Row8<float>& r) {
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(r.get(e)));
  return m;
}
template <typename T>
__device__ __forceinline__ float max8_finite(const Row8<T>& r) {
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float x = fabsf(r.get(e));
    if (x < __int_as_float(0x7f800000)) m = fmaxf(m, x);
  }
  return m;
}
template <int LPT>
__device__ __forceinline__ float lanes_max(float m, unsigned mask) {
#pragma unroll
  for (int o = LPT / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(mask, m, o));
  return m;
}
template <typename T>
__device__ __forceinline__ uint2 codes8(const Row8<T>& r, float inv) {
  return make_uint2(e4m3x4(r.get(0) * inv, r.get(1) * inv, r.get(2) * inv, r.get(3) * inv),
                    e4m3x4(r.get(4) * inv, r.get(5) * inv, r.get(6) * inv, r.get(7) * inv));
}
// Four codes times a power of two.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
  const float2 a = e4m3_f32x2(w), b = e4m3_f32x2(w >> 16);
  return e4m3x4(a.x * ratio, a.y * ratio, b.x * ratio, b.y * ratio);
}

// Where a task's lane writes: blk is its block of K or V, elements 8 lane .. 8 lane + 7.
struct AppendAt {
  uint8_t* blk;
  float* scale;
  int d, lane;
  __device__ uint2* k(int t) const {   // token t of K
    return reinterpret_cast<uint2*>(blk + (t >> 3) * (d / 16 * 128) + (t & 7) * 16 + (lane / 2) * 128 + (lane & 1) * 8);
  }
  __device__ uint8_t* v(int e) const { return blk + (lane * 8 + e) * kKvBlock; }   // element e's 16 tokens of V
};

// A whole block: its 16 rows into registers once, then the scale, then the codes.
template <typename T, int LPT>
__device__ __forceinline__ void append_block(const T* src, int64_t stride, const AppendAt& at, bool is_v, unsigned mask) {
  const bool on = at.lane * 8 < at.d;
  Row8<T> r[kKvBlock];
#pragma unroll
  for (int t = 0; t < kKvBlock; ++t) {
    if (on) r[t].load(src + t * stride);
    else r[t].zero();
  }
  float m = 0.f;
#pragma unroll
  for (int t = 0; t < kKvBlock; ++t) m = fmaxf(m, max8(r[t]));
  if (__any_sync(mask, !(m < __int_as_float(0x7f800000)))) {
    m = 0.f;
#pragma unroll
    for (int t = 0; t < kKvBlock; ++t) m = fmaxf(m, max8_finite(r[t]));
  }
  const float now = pow2_scale(lanes_max<LPT>(m, mask)), inv = 1.0f / now;   // a power of two: exact
  if (at.lane == 0) *at.scale = now;
  const unsigned live = __ballot_sync(mask, on);   // (whole pairs of lanes)
  if (!on) return;
  // Two lanes exchange halves, so that together they write 32 bytes at once.
  const bool odd = at.lane & 1;
  if (!is_v) {
#pragma unroll
    for (int t = 0; t < kKvBlock; t += 2) {   // the even lane token t, the odd one t + 1
      const uint2 a = codes8(r[t], inv), b = codes8(r[t + 1], inv);
      const uint2 other = make_uint2(__shfl_xor_sync(live, odd ? a.x : b.x, 1), __shfl_xor_sync(live, odd ? a.y : b.y, 1));
      uint8_t* to = reinterpret_cast<uint8_t*>(at.k(t + odd)) - (odd ? 8 : 0);
      *reinterpret_cast<uint4*>(to) = odd ? make_uint4(other.x, other.y, b.x, b.y) : make_uint4(a.x, a.y, other.x, other.y);
    }
  } else {
    auto tokens = [&](int e) {   // of element e
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = e4m3x4(r[4 * i].get(e) * inv, r[4 * i + 1].get(e) * inv, r[4 * i + 2].get(e) * inv, r[4 * i + 3].get(e) * inv);
      return make_uint4(w[0], w[1], w[2], w[3]);
    };
#pragma unroll
    for (int e = 0; e < 8; e += 2) {   // the even lane element e of both, the odd one e + 1
      const uint4 a = tokens(e), b = tokens(e + 1), give = odd ? a : b;
      const uint4 other = make_uint4(__shfl_xor_sync(live, give.x, 1), __shfl_xor_sync(live, give.y, 1),
                                     __shfl_xor_sync(live, give.z, 1), __shfl_xor_sync(live, give.w, 1));
      const int from = odd ? 8 : 0;   // the even lane's elements, from this lane's
      *reinterpret_cast<uint4*>(at.v(e + odd - from)) = odd ? other : a;
      *reinterpret_cast<uint4*>(at.v(e + odd - from + 8)) = odd ? b : other;
    }
  }
}

// Tokens [off, off + run) of a block that is not written whole.  More than two
// (a prompt's ends, a draft; HOLD): the rows into registers at once, as a whole
// block's, for one wait instead of one a row.  A decode step's single tokens: row
// by row, in little code (a step's kernel is as long as its instructions take to
// arrive: 256 of them 5.5 us, 6.1 through the other).  The codes before the run
// are read only when the scale rises.
template <typename T, int LPT, bool HOLD>
__device__ __forceinline__ void append_part(const T* src, int64_t stride, const AppendAt& at, bool is_v, int off, int run,
                                            unsigned mask) {
  const bool on = at.lane * 8 < at.d;
  const float before = off ? *at.scale : 0.f;
  float m = 0.f;
  Row8<T> held[HOLD ? kKvBlock - 1 : 1];
  auto most = [&](const Row8<T>& r) {
    const float x = max8(r);
    m = fmaxf(m, x < __int_as_float(0x7f800000) ? x : max8_finite(r));
  };
  if constexpr (HOLD) {
#pragma unroll
    for (int t = 0; t < kKvBlock - 1; ++t) {
      held[t].zero();
      if (on && t < run) held[t].load(src + t * stride);
    }
#pragma unroll
    for (int t = 0; t < kKvBlock - 1; ++t) most(held[t]);
  } else {
#pragma unroll 1
    for (int t = 0; t < run; ++t) {
      Row8<T> r;
      r.zero();
      if (on) r.load(src + t * stride);
      most(r);
    }
  }
  const float now = fmaxf(pow2_scale(lanes_max<LPT>(m, mask)), before), inv = 1.0f / now;
  __syncwarp(mask);   // the scale before has been read by every lane
  if (at.lane == 0) *at.scale = now;
  if (!on) return;
  if (off && now > before) {
    const float ratio = before * inv;
    if (!is_v) {
#pragma unroll 1
      for (int t = 0; t < off; ++t) {
        const uint2 o = *at.k(t);
        *at.k(t) = make_uint2(rescale4(o.x, ratio), rescale4(o.y, ratio));
      }
    } else {
      // bytes of tokens before the run
      const uint32_t full = off >> 2, rest = (1u << (8 * (off & 3))) - 1u;
      uint4 o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = *reinterpret_cast<const uint4*>(at.v(e));
#pragma unroll
      for (int e = 0; e < 8; ++e) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t& w = (&o[e].x)[i];
          const uint32_t keep = i < (int)full ? 0xffffffffu : i == (int)full ? rest : 0u;
          w = (rescale4(w, ratio) & keep) | (w & ~keep);
        }
        *reinterpret_cast<uint4*>(at.v(e)) = o[e];
      }
    }
  }
  auto put = [&](int t, const Row8<T>& r) {
    const uint2 c = codes8(r, inv);
    if (!is_v) {
      *at.k(off + t) = c;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) at.v(e)[off + t] = (uint8_t)((e < 4 ? c.x : c.y) >> (8 * (e & 3)));
    }
  };
  if constexpr (HOLD) {
#pragma unroll
    for (int t = 0; t < kKvBlock - 1; ++t)
      if (t < run) put(t, held[t]);
  } else {
#pragma unroll 1
    for (int t = 0; t < run; ++t) {
      Row8<T> r;
      r.load(src + t * stride);
      put(t, r);
    }
  }
}

}  // namespace

// New rows into the cache.  A CTA takes W rows; a run of rows of one block of
// 16 tokens is handled, for one kv head and K or V, by LPT lanes with 8
// elements of the head each.  The block's largest value decides its scale, so
// the rows are held in registers from the load to the store.  Prompts are bound
// by what a CTA does before its first row arrives (slots, list, two barriers) and
// by whole waves of CTAs more than by HBM.  Measured (4 kv heads, d = 256, bf16):
// five prompts, 29,500 rows (6.05 waves of 608 CTAs), 181 MB read and written
// 39 us, 4.6 TB/s (fp32: 301 MB 65 us); 256 single rows 5.5 us.
template <typename T, int LPT, int W, int THREADS>
__global__ void __launch_bounds__(THREADS, sizeof(T) == 2 ? 512 / THREADS : 256 / THREADS) kv_append_kernel(const KvAppendParams p) {
  constexpr int kSlots = THREADS / LPT;   // runs in work at once
  __shared__ int64_t s_slot[W + kKvBlock];
  __shared__ int s_lead[W], s_len[W], s_n;
  const int64_t t0 = (int64_t)blockIdx.x * W;
  for (int i = threadIdx.x; i < W + kKvBlock; i += THREADS) s_slot[i] = t0 + i < p.T ? p.slot_map[t0 + i] : -1;
  int64_t before0 = -1;
  if (threadIdx.x == 0) {
    s_n = 0;
    if (t0 > 0) before0 = p.slot_map[t0 - 1];
  }
  __syncthreads();
  if (threadIdx.x < W) {
    const int i = threadIdx.x;
    const int64_t slot = s_slot[i];
    const int64_t before = i > 0 ? s_slot[i - 1] : before0;
    if (slot >= 0 && !(before >= 0 && slot == before + 1 && slot % kKvBlock != 0)) {
      int n = 1;
      while (n < kKvBlock && (slot + n) % kKvBlock != 0 && s_slot[i + n] == slot + n) ++n;
      // the order of the list does not matter: runs are independent
      const int at = atomicAdd(&s_n, 1);
      s_lead[at] = i, s_len[at] = n;
    }
  }
  __syncthreads();
  const int sub = threadIdx.x / LPT, lane = threadIdx.x % LPT;
  const unsigned mask = (LPT == 32 ? 0xffffffffu : ((1u << (LPT & 31)) - 1u) << (threadIdx.x % 32 / LPT * LPT));
  const int d = p.c.d, h = blockIdx.y, runs = s_n;
  for (int task = sub; task < 2 * runs; task += kSlots) {
    const bool is_v = task >= runs;
    const int i = s_lead[is_v ? task - runs : task], run = s_len[is_v ? task - runs : task];
    const int64_t slot = s_slot[i];
    const int64_t page = slot / p.c.page_tokens;
    if (page >= p.c.num_pages) {
      if (lane == 0) set_error(p.err, GDN_ERR_PAGE_RANGE);
      continue;
    }
    const int in_page = (int)(slot - page * p.c.page_tokens), b = in_page / kKvBlock, off = in_page % kKvBlock;
    const int64_t stride = is_v ? p.v_stride : p.k_stride;
    const T* src = static_cast<const T*>(is_v ? p.v : p.k) + (t0 + i) * stride + (int64_t)h * d + lane * 8;
    const AppendAt at{const_cast<uint8_t*>(is_v ? kv_v_block(p.c, (int)page, h, b) : kv_k_block(p.c, (int)page, h, b)),
                      const_cast<float*>(is_v ? kv_v_scale(p.c, (int)page, h, b) : kv_k_scale(p.c, (int)page, h, b)), d, lane};
    if (run == kKvBlock) append_block<T, LPT>(src, stride, at, is_v, mask);
    else if (run > 2) append_part<T, LPT, true>(src, stride, at, is_v, off, run, mask);
    else append_part<T, LPT, false>(src, stride, at, is_v, off, run, mask);
  }
}

namespace {

template <typename T, int LPT>
cudaError_t append_rows(const KvAppendParams& p, cudaStream_t st) {
  // few rows (a decode step: every row a run of its own): 4 a CTA of 8 warps,
  // so that the runs of a step spread over the SMs (256 single rows 5.5 us, 31
  // with 32 rows a CTA); many (prompts): 32 a CTA of 4 warps, about two runs of K
  // and of V (one prompt of 4,000 rows 9.5 us, 19 with 4 rows; 2,000 rows 9.9
  // and 11.4)
  if (p.T <= 2048) {
    kv_append_kernel<T, LPT, 4, 256><<<dim3((unsigned)((p.T + 3) / 4), p.c.Hkv), 256, 0, st>>>(p);
  } else {
    kv_append_kernel<T, LPT, 32, 128><<<dim3((unsigned)((p.T + 31) / 32), p.c.Hkv), 128, 0, st>>>(p);
  }
  return cudaGetLastError();
}
template <typename T>
cudaError_t append_dtype(const KvAppendParams& p, cudaStream_t st) {
  if (p.c.d > 128) return append_rows<T, 32>(p, st);
  if (p.c.d > 64) return append_rows<T, 16>(p, st);
  return append_rows<T, 8>(p, st);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendParams& p, int dtype, cudaStream_t st) {
  return dtype == GDN_BF16 ? append_dtype<__nv_bfloat16>(p, st) : append_dtype<float>(p, st);
}

// ---- gather ---------------------------------------------------------------------------
namespace {

__device__ __forceinline__ void put8(__nv_bfloat16* p, const float (&f)[8]) {
  uint4 w;
  __nv_bfloat162* b = reinterpret_cast<__nv_bfloat162*>(&w);
#pragma unroll
  for (int i = 0; i < 4; ++i) b[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  *reinterpret_cast<uint4*>(p) = w;
}
__device__ __forceinline__ void put8(float* p, const float (&f)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

}  // namespace

// The cached rows of a prefix back as plain rows.  A CTA takes 16 output rows;
// each block of 16 tokens that starts among them is read, for one head and K or
// V, by LPT lanes with 8 elements each (V's operand tiles are transposed in
// registers) and written as row pieces of 8 elements.  Bound by HBM: two
// prefixes, 1.06 GB (4 kv heads, d = 256), 159 us, 6.6 TB/s or 97 % of a copy's
// rate; 19 ragged ones, 242 MB (8 kv heads, d = 128), 44 us (171 and 54 us with
// 64 rows a CTA, whose last ones leave SMs idle).
template <typename T, int LPT>
__global__ void __launch_bounds__(256) kv_gather_kernel(const KvGatherParams p) {
  constexpr int kSlots = 256 / LPT, W = 16;
  __shared__ int s_row[W], s_len[W], s_page[W], s_blk[W], s_n;
  const int64_t t0 = (int64_t)blockIdx.x * W;
  if (threadIdx.x == 0) s_n = 0;
  __syncthreads();
  if (threadIdx.x < W && t0 + threadIdx.x < p.T) {
    const int64_t t = t0 + threadIdx.x;
    int lo = 0, hi = p.N;   // the sequence s with cu[s] <= t < cu[s + 1]
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (p.cu_kv[mid + 1] > t) hi = mid;
      else lo = mid + 1;
    }
    if (lo < p.N && t >= p.cu_kv[lo]) {
      const int64_t pos = t - p.cu_kv[lo];
      if (pos % kKvBlock == 0) {
        const int64_t j = pos / p.c.page_tokens;
        int page = j < p.max_pages ? p.block_table[(int64_t)lo * p.max_pages + j] : -1;
        if (page < 0 || page >= p.c.num_pages) {
          set_error(p.err, GDN_ERR_PAGE_RANGE);
          page = -1;
        }
        const int64_t left = min((int64_t)p.cu_kv[lo + 1], p.T) - t;
        const int at = atomicAdd(&s_n, 1);
        s_row[at] = threadIdx.x;
        s_len[at] = left < kKvBlock ? (int)left : kKvBlock;
        s_page[at] = page;
        s_blk[at] = (int)(pos - j * p.c.page_tokens) / kKvBlock;
      }
    }
  }
  __syncthreads();
  const int sub = threadIdx.x / LPT, lane = threadIdx.x % LPT;
  const int e0 = lane * 8, d = p.c.d, Hkv = p.c.Hkv;
  if (e0 >= d) return;
  for (int task = sub; task < 2 * s_n * Hkv; task += kSlots) {
    const bool is_v = task & 1;
    const int i = (task >> 1) / Hkv, h = (task >> 1) % Hkv;
    const int page = s_page[i], b = s_blk[i], len = s_len[i];
    T* dst = static_cast<T*>(is_v ? p.v : p.k) + ((t0 + s_row[i]) * Hkv + h) * d + e0;
    const int64_t stride = (int64_t)Hkv * d;
    if (page < 0) {
      const float z[8] = {};
      for (int t = 0; t < len; ++t) put8(dst + t * stride, z);
      continue;
    }
    const float scale = *(is_v ? kv_v_scale(p.c, page, h, b) : kv_k_scale(p.c, page, h, b));
    if (!is_v) {
      const uint8_t* src = kv_k_block(p.c, page, h, b) + (e0 / 16) * 128 + (e0 & 8);
      const int half = d / 16 * 128;
      uint2 w[kKvBlock];
#pragma unroll
      for (int t = 0; t < kKvBlock; ++t) w[t] = *reinterpret_cast<const uint2*>(src + (t >> 3) * half + (t & 7) * 16);
#pragma unroll
      for (int t = 0; t < kKvBlock; ++t) {
        if (t >= len) break;
        const float2 a = e4m3_f32x2(w[t].x), b2 = e4m3_f32x2(w[t].x >> 16), c = e4m3_f32x2(w[t].y), f = e4m3_f32x2(w[t].y >> 16);
        const float x[8] = {a.x * scale, a.y * scale, b2.x * scale, b2.y * scale,
                            c.x * scale, c.y * scale, f.x * scale, f.y * scale};
        put8(dst + t * stride, x);
      }
    } else {
      const uint4* src = reinterpret_cast<const uint4*>(kv_v_block(p.c, page, h, b) + e0 * kKvBlock);
      uint4 w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = src[e];
#pragma unroll
      for (int t = 0; t < kKvBlock; t += 2) {
        float x[8], y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 f = e4m3_f32x2((&w[e].x)[t >> 2] >> (8 * (t & 2)));
          x[e] = f.x * scale, y[e] = f.y * scale;
        }
        if (t < len) put8(dst + t * stride, x);
        if (t + 1 < len) put8(dst + (t + 1) * stride, y);
      }
    }
  }
}

namespace {

template <typename T>
cudaError_t gather_dtype(const KvGatherParams& p, cudaStream_t st) {
  const unsigned g = (unsigned)((p.T + 15) / 16);
  if (p.c.d > 128) kv_gather_kernel<T, 32><<<g, 256, 0, st>>>(p);
  else if (p.c.d > 64) kv_gather_kernel<T, 16><<<g, 256, 0, st>>>(p);
  else kv_gather_kernel<T, 8><<<g, 256, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_gather(const KvGatherParams& p, int dtype, cudaStream_t st) {
  return dtype == GDN_BF16 ? gather_dtype<__nv_bfloat16>(p, st) : gather_dtype<float>(p, st);
}

}  // namespace gdn
