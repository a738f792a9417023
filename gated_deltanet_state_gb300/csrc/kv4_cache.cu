// kv4_cache.cu — the 4-bit cache of the attention layers: the append of new
// rows and the read-back of a cached prefix.
//
// Both walk the rows in windows: a warp takes 16 rows (or one, where a call has
// few) of as many kv heads as its lanes hold at 8 elements each, finds the blocks
// of 16 tokens that start there from the slots (or lengths) by itself, and moves
// K or V of each.  No warp waits on another, so the chain before the first row is
// the slots' loads alone.
#include "kv4.cuh"

namespace gdn {

namespace {

constexpr int kKv4Warps = 4;   // of a CTA

// Largest of each of N values over the LPT lanes of a head, by halves: lane l ends
// up with value l N / LPT's (LPT >= N).
template <int LPT, int N>
__device__ __forceinline__ uint32_t lanes_umax(const uint32_t (&in)[N], int l) {
  uint32_t v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = in[i];
  int bit = LPT / 2;
#pragma unroll
  for (int half = N / 2; half >= 1; half >>= 1, bit >>= 1) {
    const bool up = l & bit;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const uint32_t send = up ? v[i] : v[i + half], keep = up ? v[i + half] : v[i];
      v[i] = max(keep, __shfl_xor_sync(0xffffffffu, send, bit));
    }
  }
  for (; bit >= 1; bit >>= 1) v[0] = max(v[0], __shfl_xor_sync(0xffffffffu, v[0], bit));
  return v[0];
}

// Largest magnitude of eight elements as fp32 bits: an infinity or a NaN gives
// bits above every finite value's.
__device__ __forceinline__ uint32_t max8_bits(const Row8<__nv_bfloat16>& r) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = __vmaxu2(m, (&r.w.x)[i] & 0x7fff7fffu);
  return max(m << 16, m & 0xffff0000u);
}
__device__ __forceinline__ uint32_t max8_bits(const Row8<float>& r) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(r.get(i)) & 0x7fffffffu);
  return m;
}
// The same of the finite elements; ~0 if one is a NaN.
template <typename T>
__device__ __forceinline__ uint32_t max8_finite(const Row8<T>& r) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t x = __float_as_uint(r.get(i)) & 0x7fffffffu;
    m = max(m, x < 0x7f800000u ? x : x > 0x7f800000u ? ~0u : 0u);
  }
  return m;
}

// A scale, as quantising takes it.
struct Scale {
  float inv, s;   // 0, 0: of NaN
  // lane i's, of each `width` lanes
  __device__ __forceinline__ Scale of(int i, int width) const {
    return {__shfl_sync(0xffffffffu, inv, i, width), __shfl_sync(0xffffffffu, s, i, width)};
  }
};
__device__ __forceinline__ Scale make_scale(uint32_t byte) {
  if (byte == kKv4Nan) return {0.f, 0.f};
  const float s = kv4_scale(byte);
  return {__uint_as_float(__float_as_uint(__frcp_rn(s)) + 1u), s};
}

// An element's code as the last bits of an fp32 of 3 2^22 + n: the nearest, halves
// away from zero.  x inv is past a half where x / s is one (inv is above 1 / s by
// 2^-25 to 2^-22 of it), and a bf16 x that is not stays on its side, since x / s
// differs from a half by 2^-9 of it at least.  fp32 has values in between: what is
// left of x decides (exact: k s has 7 bits, and |x - k s| <= s).  SAFE: also where
// elements pass 7 s, or are no numbers.
constexpr uint32_t kCodeBits = 0x4b400000u;
template <bool SAFE>
__device__ __forceinline__ uint32_t code_bits(float x, const Scale& s, __nv_bfloat16) {
  if (SAFE) x = fminf(fmaxf(x, -7.f * s.s), 7.f * s.s);
  return __float_as_uint(fmaf(x, s.inv, 12582920.f));
}
template <bool SAFE>
__device__ __forceinline__ uint32_t code_bits(float x, const Scale& s, float) {
  if (SAFE) x = fminf(fmaxf(x, -7.f * s.s), 7.f * s.s);
  const float a = fabsf(x);
  float k = rintf(a * s.inv);
  const float t = fmaf(-k, s.s, a);
  if (s.s > 0.f) k += t >= 0.5f * s.s ? 1.f : t < -0.5f * s.s ? -1.f : 0.f;
  return __float_as_uint(copysignf(k, x) + 12582920.f);
}

// Bits of element i of a word.
__host__ __device__ constexpr int word_shift(int i) { return 4 * (i / 2) + 16 * (i % 2); }
// What the fp32s' own bits add up to in a word whose elements were added shifted.
constexpr uint32_t word_bias() {
  uint32_t c = 0;
  for (int i = 0; i < 8; ++i) c += kCodeBits << word_shift(i);
  return c;
}

// New rows of one block: row i of the run, 0 <= i < run, is token off + i.
template <typename T, int LPT>
struct AppendRun {
  const T* src;      // this lane's elements of the run's first row
  int64_t stride;
  int off, run, lane;   // lane within its head
  bool on, head;        // whether the lane has elements, and whether its head is one

  __device__ __forceinline__ bool has(int t) const { return t >= off && t < off + run; }
  __device__ __forceinline__ void load(Row8<T>& r, int t) const {
    r.zero();
    if (on && has(t)) r.load(src + (int64_t)(t - off) * stride);
  }

  // K: codes [d/32][16][16 B], scales [d/32][16].  Four tokens at a time, eight loaded.
  template <bool SAFE>
  __device__ __forceinline__ bool k_tokens(uint8_t* codes, uint8_t* scales, int t0, const Row8<T>* r) const {
    uint32_t m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = SAFE ? max8_finite(r[i]) : max8_bits(r[i]);
    const int q = lane & 3;
    const uint32_t top = lanes_umax<4>(m, q);   // of token t0 + q
    if (!SAFE && __any_sync(0xffffffffu, top > __float_as_uint(kKv4Most))) return false;
    const uint32_t mine = top == ~0u ? kKv4Nan : kv4_byte(top);
    const Scale own = make_scale(mine);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const Scale s = own.of(i, 4);
      uint32_t x = 0u - word_bias();
#pragma unroll
      for (int e = 0; e < 8; ++e) x += code_bits<SAFE>(r[i].get(e), s, T()) << word_shift(e);
      w[i] = x;
    }
    kv4_transpose(w, q);
    if (on && has(t0 + q)) {
      const int at = lane / 4 * kKvBlock + t0 + q;
      *reinterpret_cast<uint4*>(codes + at * 16) = make_uint4(w[0], w[1], w[2], w[3]);
      scales[at] = (uint8_t)mine;
    }
    return true;
  }
  __device__ __forceinline__ void k(uint8_t* codes, uint8_t* scales) const {
#pragma unroll 1
    for (int t0 = 0; t0 < kKvBlock; t0 += 8) {
      if (off >= t0 + 8 || off + run <= t0) continue;
      Row8<T> r[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) load(r[i], t0 + i);
#pragma unroll
      for (int i = 0; i < 8; i += 4)
        if (off < t0 + i + 4 && off + run > t0 + i)
          if (!k_tokens<false>(codes, scales, t0 + i, r + i)) k_tokens<true>(codes, scales, t0 + i, r + i);
    }
  }

  // V: codes [d][8 B], scales [16].  Eight tokens at a time, a word of each channel.
  template <bool SAFE>
  __device__ __forceinline__ bool v_tokens(uint8_t* scales, int t0, uint32_t (&w)[8]) const {
    Row8<T> r[8];
    uint32_t m[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) load(r[i], t0 + i);
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = SAFE ? max8_finite(r[i]) : max8_bits(r[i]);
    // lane l of a head: token t0 + l / STEP (of four lanes each has two)
    constexpr int N = LPT < 8 ? LPT : 8, STEP = LPT / N;
    Scale own[8 / N];
    uint32_t mine[8 / N];
#pragma unroll
    for (int k = 0; k < 8 / N; ++k) {
      uint32_t part[N];
#pragma unroll
      for (int i = 0; i < N; ++i) part[i] = m[k * N + i];
      const uint32_t top = lanes_umax<LPT>(part, lane);
      if (!SAFE && __any_sync(0xffffffffu, top > __float_as_uint(kKv4Most))) return false;
      mine[k] = top == ~0u ? kKv4Nan : kv4_byte(top);
      own[k] = make_scale(mine[k]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = 0u - word_bias();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const Scale s = own[i / N].of(i % N * STEP, LPT);
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] += code_bits<SAFE>(r[i].get(e), s, T()) << word_shift(i);
    }
#pragma unroll
    for (int k = 0; k < 8 / N; ++k) {
      const int at = t0 + k * N + lane / STEP;
      if (head && lane % STEP == 0 && has(at)) scales[at] = (uint8_t)mine[k];
    }
    return true;
  }
  __device__ __forceinline__ void v(uint8_t* codes, uint8_t* scales) const {
    if (run == kKvBlock) {
      uint32_t w[2][8];
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (!v_tokens<false>(scales, 8 * k, w[k])) v_tokens<true>(scales, 8 * k, w[k]);
      // a lane's 64 bytes, 16 at a time to four lanes, so that four write 64 in a row
      const int q = lane & 3;
      uint32_t to[4][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {   // word k of each 16 bytes: channels 2 i, 2 i + 1, tokens 0 .. 7, 8 .. 15
#pragma unroll
        for (int i = 0; i < 4; ++i) to[k][i] = w[k & 1][2 * i + (k >> 1)];
        kv4_transpose(to[k], q);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (on) *reinterpret_cast<uint4*>(codes + ((lane & ~3) + i) * 64 + q * 16) = make_uint4(to[0][i], to[1][i], to[2][i], to[3][i]);
      return;
    }
    // a word with other tokens in it is merged with what it holds
#pragma unroll 1
    for (int t0 = 0; t0 < kKvBlock; t0 += 8) {
      if (off >= t0 + 8 || off + run <= t0) continue;
      uint32_t w[8], keep = 0;
      if (!v_tokens<false>(scales, t0, w)) v_tokens<true>(scales, t0, w);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (!has(t0 + i)) keep |= 15u << word_shift(i);
      if (!on) continue;
      uint32_t* to = reinterpret_cast<uint32_t*>(codes + lane * 64 + t0 / 2);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (keep) w[e] = (w[e] & ~keep) | (to[2 * e] & keep);
        to[2 * e] = w[e];
      }
    }
  }
};

}  // namespace

// New rows into the cache.  Window w of W rows; grid y: K or V of 32 / LPT heads.
// A head's rows are read once; a group's or row's largest value is a maximum over
// lanes, and codes leave as whole words: K's word of eight channels is a lane's own,
// V's of eight tokens are formed in the lane that has their channel.  27,057 rows of
// 4 heads, d = 256, bf16 (139.5 MB, 20.5 us of memory): 34.8 us, five CTAs an SM; a
// warp's time goes to waits for its loads (36 %), and the 3,384 CTAs
// take 4.5 rounds of what is resident.  CTAs of 1 or 2 warps: the same.
template <typename T, int LPT, int W>
__global__ void __launch_bounds__(32 * kKv4Warps, sizeof(T) == 2 ? 5 : 4) kv4_append_kernel(const KvAppendParams p) {
  constexpr int HPW = 32 / LPT;
  const int lane = threadIdx.x & 31, sub = lane / LPT;
  const int64_t t0 = ((int64_t)blockIdx.x * kKv4Warps + (threadIdx.x >> 5)) * W;
  if (t0 >= p.T) return;
  const bool is_v = blockIdx.y & 1;
  const int h = (blockIdx.y >> 1) * HPW + sub, d = p.c.d;
  // lane i: the slot of row t0 + i; whether it goes on in the block of the row before
  const int64_t slot = t0 + lane < p.T ? p.slot_map[t0 + lane] : -1;
  int64_t before = __shfl_up_sync(0xffffffffu, slot, 1);
  if (lane == 0) before = t0 > 0 ? p.slot_map[t0 - 1] : -1;
  const unsigned cont = __ballot_sync(0xffffffffu, slot >= 0 && before >= 0 && slot == before + 1 && slot % kKvBlock != 0);
  unsigned starts = __ballot_sync(0xffffffffu, lane < W && slot >= 0) & ~cont;
  AppendRun<T, LPT> a;
  a.lane = lane % LPT;
  a.head = h < p.c.Hkv;
  a.on = a.lane * 8 < d && a.head;
  a.stride = is_v ? p.v_stride : p.k_stride;
  const T* rows = static_cast<const T*>(is_v ? p.v : p.k) + t0 * a.stride + (int64_t)h * d + a.lane * 8;
  for (; starts; starts &= starts - 1) {
    const int i = __ffs(starts) - 1;
    const int64_t first = __shfl_sync(0xffffffffu, slot, i), page = first / p.c.page_tokens;
    if (page >= p.c.num_pages) {
      if (lane == 0) set_error(p.err, GDN_ERR_PAGE_RANGE);
      continue;
    }
    const int in_page = (int)(first - page * p.c.page_tokens), b = in_page / kKvBlock;
    a.off = in_page % kKvBlock;
    a.run = __ffs(~(cont >> (i + 1)));   // (i < W <= 16: rows up to t0 + 31 reach a run's end)
    a.src = rows + i * a.stride;
    const int hh = h < p.c.Hkv ? h : 0;
    if (is_v) a.v(kv4_v_block(p.c, (int)page, hh, b), kv4_v_scale(p.c, (int)page, hh, b));
    else a.k(kv4_k_block(p.c, (int)page, hh, b), kv4_k_scale(p.c, (int)page, hh, b));
  }
}

namespace {

template <typename T, int LPT>
cudaError_t append4_rows(const KvAppendParams& p, cudaStream_t st) {
  const unsigned gy = 2u * ((p.c.Hkv + 32 / LPT - 1) / (32 / LPT));
  // Few rows are often each of a sequence of their own, and a window's runs go one
  // after another: 256 such rows 6.2 us in windows of 1, 35.9 of 16 (2 and 4: 8.3, 11.8).
  // A run's rows are better off in windows of 16 from few rows on, but the host does
  // not know the runs: up to 2,048 rows it takes them for single ones, where one run
  // loses least (2,048 rows 8.1 and 4.5 us, 8,192 rows 22.7 and 8.7; 4 heads, d = 256, bf16).
  if (p.T <= 2048) kv4_append_kernel<T, LPT, 1><<<dim3((unsigned)((p.T + kKv4Warps - 1) / kKv4Warps), gy), 32 * kKv4Warps, 0, st>>>(p);
  else kv4_append_kernel<T, LPT, 16><<<dim3((unsigned)((p.T + 16 * kKv4Warps - 1) / (16 * kKv4Warps)), gy), 32 * kKv4Warps, 0, st>>>(p);
  return cudaGetLastError();
}
template <typename T>
cudaError_t append4_dtype(const KvAppendParams& p, cudaStream_t st) {
  if (p.c.d > 128) return append4_rows<T, 32>(p, st);
  if (p.c.d > 64) return append4_rows<T, 16>(p, st);
  if (p.c.d > 32) return append4_rows<T, 8>(p, st);
  return append4_rows<T, 4>(p, st);
}

}  // namespace

cudaError_t launch_kv4_append(const KvAppendParams& p, int dtype, cudaStream_t st) {
  return dtype == GDN_BF16 ? append4_dtype<__nv_bfloat16>(p, st) : append4_dtype<float>(p, st);
}

// ---- gather ---------------------------------------------------------------------------
namespace {

// Eight bf16 (four words) to eight elements of a row.
__device__ __forceinline__ void put8(__nv_bfloat16* p, const uint32_t (&w)[4]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void put8(float* p, const uint32_t (&w)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    reinterpret_cast<float4*>(p)[i] =
        make_float4(__uint_as_float(w[2 * i] << 16), __uint_as_float(w[2 * i] & 0xffff0000u), __uint_as_float(w[2 * i + 1] << 16),
                    __uint_as_float(w[2 * i + 1] & 0xffff0000u));
}

}  // namespace

// The cached rows of a prefix back as plain rows: a warp takes 16 output rows,
// K or V of 32 / LPT heads.  (n - 8) scale is exact in bf16, one operation for a
// pair.  The rows that go out are four fifths of the bytes: 961 MB in 148 to 150 us
// (6.4 to 6.5 TB/s, 95 % of a copy's rate), 202 MB of 19 ragged prefixes in 36 us.
template <typename T, int LPT>
__global__ void __launch_bounds__(32 * kKv4Warps) kv4_gather_kernel(const KvGatherParams p) {
  constexpr int HPW = 32 / LPT;
  const int lane = threadIdx.x & 31, sub = lane / LPT, l = lane % LPT;
  const int64_t t0 = ((int64_t)blockIdx.x * kKv4Warps + (threadIdx.x >> 5)) * kKvBlock;
  if (t0 >= p.T) return;
  const bool is_v = blockIdx.y & 1;
  const int h = (blockIdx.y >> 1) * HPW + sub, d = p.c.d, hh = h < p.c.Hkv ? h : 0;
  const bool on = l * 8 < d && h < p.c.Hkv;
  // lane i < 16: the block that starts at row t0 + i, if one does
  int page = -1, blk = 0, len = 0;
  if (lane < kKvBlock && t0 + lane < p.T) {
    const int64_t t = t0 + lane;
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
        page = j < p.max_pages ? p.block_table[(int64_t)lo * p.max_pages + j] : -1;
        if (page < 0 || page >= p.c.num_pages) {
          set_error(p.err, GDN_ERR_PAGE_RANGE);
          page = -1;
        }
        blk = (int)(pos - j * p.c.page_tokens) / kKvBlock;
        len = (int)min((int64_t)kKvBlock, min((int64_t)p.cu_kv[lo + 1], p.T) - t);
      }
    }
  }
  const int64_t stride = (int64_t)p.c.Hkv * d;
  T* rows = static_cast<T*>(is_v ? p.v : p.k) + (t0 * p.c.Hkv + h) * d + l * 8;
  for (unsigned starts = __ballot_sync(0xffffffffu, len > 0); starts; starts &= starts - 1) {
    const int i = __ffs(starts) - 1;
    const int pg = __shfl_sync(0xffffffffu, page, i), b = __shfl_sync(0xffffffffu, blk, i), n = __shfl_sync(0xffffffffu, len, i);
    T* dst = rows + i * stride;
    if (pg < 0) {
      const uint32_t z[4] = {};
      for (int t = 0; t < n; ++t)
        if (on) put8(dst + t * stride, z);
      continue;
    }
    if (!is_v) {
      const uint8_t *codes = kv4_k_block(p.c, pg, hh, b), *scales = kv4_k_scale(p.c, pg, hh, b);
      const int q = l & 3, at = l / 4 * kKvBlock;
      uint4 c[4] = {}, s4 = {};
      if (on) {
#pragma unroll
        for (int k = 0; k < 4; ++k) c[k] = *reinterpret_cast<const uint4*>(codes + (at + 4 * k + q) * 16);
        s4 = *reinterpret_cast<const uint4*>(scales + at);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t w[4] = {c[k].x, c[k].y, c[k].z, c[k].w};
        kv4_transpose(w, q);   // this lane's 8 channels of tokens 4 k .. 4 k + 3
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint32_t s1 = kv4_scale_bf16((&s4.x)[k] >> (8 * u) & 255u), s = s1 << 16 | s1, off = kv4_offset(s);
          uint32_t x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = kv4_fma(kv4_pair(w[u] >> (4 * e)), s, off);
          if (on && 4 * k + u < n) put8(dst + (4 * k + u) * stride, x);
        }
      }
    } else if (on) {
      const uint4* codes = reinterpret_cast<const uint4*>(kv4_v_block(p.c, pg, hh, b) + l * 64);
      const uint4 s4 = *reinterpret_cast<const uint4*>(kv4_v_scale(p.c, pg, hh, b));
      uint4 c[4];   // channels 2 k, 2 k + 1: tokens 0 .. 7, 8 .. 15 of each
#pragma unroll
      for (int k = 0; k < 4; ++k) c[k] = codes[k];
#pragma unroll
      for (int t = 0; t < kKvBlock; t += 2) {
        const uint32_t sb = (&s4.x)[t / 4] >> (8 * (t % 4)), s = kv4_scale_bf16(sb & 255u) | kv4_scale_bf16(sb >> 8 & 255u) << 16,
                       off = kv4_offset(s);
        uint32_t x[4], y[4];   // tokens t and t + 1
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int sh = t % 8 * 2;
          const uint32_t a = kv4_fma(kv4_pair((t < 8 ? c[k].x : c[k].y) >> sh), s, off);
          const uint32_t e = kv4_fma(kv4_pair((t < 8 ? c[k].z : c[k].w) >> sh), s, off);
          x[k] = __byte_perm(a, e, 0x5410), y[k] = __byte_perm(a, e, 0x7632);
        }
        if (t < n) put8(dst + t * stride, x);
        if (t + 1 < n) put8(dst + (t + 1) * stride, y);
      }
    }
  }
}

namespace {

template <typename T, int LPT>
cudaError_t gather4_rows(const KvGatherParams& p, cudaStream_t st) {
  const unsigned gy = 2u * ((p.c.Hkv + 32 / LPT - 1) / (32 / LPT));
  kv4_gather_kernel<T, LPT><<<dim3((unsigned)((p.T + 16 * kKv4Warps - 1) / (16 * kKv4Warps)), gy), 32 * kKv4Warps, 0, st>>>(p);
  return cudaGetLastError();
}
template <typename T>
cudaError_t gather4_dtype(const KvGatherParams& p, cudaStream_t st) {
  if (p.c.d > 128) return gather4_rows<T, 32>(p, st);
  if (p.c.d > 64) return gather4_rows<T, 16>(p, st);
  if (p.c.d > 32) return gather4_rows<T, 8>(p, st);
  return gather4_rows<T, 4>(p, st);
}

}  // namespace

cudaError_t launch_kv4_gather(const KvGatherParams& p, int dtype, cudaStream_t st) {
  return dtype == GDN_BF16 ? gather4_dtype<__nv_bfloat16>(p, st) : gather4_dtype<float>(p, st);
}

}  // namespace gdn
