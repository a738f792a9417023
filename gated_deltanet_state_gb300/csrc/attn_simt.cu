// attn_simt.cu — attention over the 8-bit cache and over packed prompts with
// fp32 arithmetic on the CUDA cores: every dtype, head size and group size;
// and the kernel that joins the pieces of a decode row.
#include "attn.h"

namespace gdn {

namespace {

constexpr int kDecRows = 8;        // (row, head of the group) pairs a CTA
constexpr int kDecWarps = 4;

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <typename T> __device__ __forceinline__ void put1(void* o, int64_t i, float v) {
  static_cast<T*>(o)[i] = from_f32<T>(v);
}

}  // namespace

// One piece of one sequence's keys, for one kv head and up to 8 of its query
// rows.  A warp takes every fourth block of 16 tokens: the lanes hold one
// token each (two lanes share one, half of d each) for the scores, one element
// of the head each (d / 32 of them) for the values; each warp keeps its own
// softmax statistics, joined at the end.  Serves what the tensor-core kernels do
// not (fp32 rows, d not a multiple of 32), bound by the conversions and fp32
// arithmetic: 256 sequences over 1,024 to 8,192 tokens (24 heads, 4 kv heads) take
// 5,045 us at d = 256 in fp32, against 404 there in bf16, and 1,823 at d = 80.
template <typename T>
__global__ void __launch_bounds__(32 * kDecWarps) attn_decode_simt_kernel(const AttnDecodeParams p) {
  extern __shared__ float smem[];
  const int d = p.c.d, piece = blockIdx.x, s = blockIdx.z;
  const int groups = (p.max_q * p.G + kDecRows - 1) / kDecRows;
  const int h = blockIdx.y / groups, r0 = blockIdx.y % groups * kDecRows;
  const int q0 = p.cu[s], n = p.cu[s + 1] - q0, L = p.kv_len[s];
  if (n <= 0) return;
  if (n > p.max_q || L > p.max_kv || L < 0 || q0 < 0 || (int64_t)q0 + n > p.T) {
    if (threadIdx.x == 0) set_error(p.err, GDN_ERR_INVALID_ARG);
    return;
  }
  const int pt = decode_piece_tokens(L, n * p.G, p.c.bits);
  const int k0 = piece * pt, k1 = min(L, k0 + pt);
  if (r0 >= n * p.G || (piece > 0 && k0 >= L)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows = min(kDecRows, n * p.G - r0);
  float* sq = smem;                                  // [8][d]
  float* sp = smem + kDecRows * d + warp * kDecRows * 16;   // [8][16] of this warp
  for (int i = threadIdx.x; i < kDecRows * d; i += blockDim.x) {
    const int r = i / d, e = i - r * d;
    float x = 0.f;
    if (r < rows) {
      const int row = (r0 + r) / p.G, g = (r0 + r) % p.G;
      x = to_f32(static_cast<const T*>(p.q)[(int64_t)(q0 + row) * p.q_stride + (int64_t)(h * p.G + g) * d + e]);
    }
    sq[i] = x * p.scale_log2;
  }
  __syncthreads();
  float O[kDecRows][8], m[kDecRows], l[kDecRows];
#pragma unroll
  for (int r = 0; r < kDecRows; ++r) {
    m[r] = -INFINITY, l[r] = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) O[r][i] = 0.f;
  }
  const int t = lane & 15, hf = lane >> 4;
  for (int kb = k0 + warp * kKvBlock; kb < k1; kb += kDecWarps * kKvBlock) {
    const int j = kb / p.c.page_tokens, b = (kb - j * p.c.page_tokens) / kKvBlock;
    const int page = j < p.max_pages ? p.block_table[(int64_t)s * p.max_pages + j] : -1;
    if (page < 0 || page >= p.c.num_pages) {
      if (lane == 0) set_error(p.err, GDN_ERR_PAGE_RANGE);
      continue;
    }
    const uint8_t* kp = kv_k_block(p.c, page, h, b) + (t >> 3) * (d / 16) * 128 + (t & 7) * 16;
    float acc[kDecRows] = {};
    for (int c = hf; c < d / 16; c += 2) {
      float f[16];
      e4m3_f32x16(*reinterpret_cast<const uint4*>(kp + c * 128), f);
#pragma unroll
      for (int r = 0; r < kDecRows; ++r) {
        const float4* q4 = reinterpret_cast<const float4*>(sq + r * d + c * 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 q = q4[i];
          acc[r] = fmaf(q.x, f[4 * i], acc[r]);
          acc[r] = fmaf(q.y, f[4 * i + 1], acc[r]);
          acc[r] = fmaf(q.z, f[4 * i + 2], acc[r]);
          acc[r] = fmaf(q.w, f[4 * i + 3], acc[r]);
        }
      }
    }
    const float ks = *kv_k_scale(p.c, page, h, b), vs = *kv_v_scale(p.c, page, h, b);
    const int pos = kb + t;
#pragma unroll
    for (int r = 0; r < kDecRows; ++r) {
      float x = acc[r] + __shfl_xor_sync(0xffffffffu, acc[r], 16);
      // keys that this row sees: L - n + row + 1
      x = pos < L - n + (r0 + r) / p.G + 1 ? x * ks : -INFINITY;
      // the largest over the block's finite and infinite scores; NaN reaches l
      float mx = x;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float mn = fmaxf(m[r], mx);
      const float ref = mn == -INFINITY ? 0.f : mn;
      const float a = fast_exp2(m[r] - ref), e = fast_exp2(x - ref);
      float sum = e;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      m[r] = mn;
      l[r] = l[r] * a + sum;
#pragma unroll
      for (int i = 0; i < 8; ++i) O[r][i] *= a;
      if (hf == 0) sp[r * 16 + t] = e * vs;
    }
    __syncwarp();
    const uint8_t* vp = kv_v_block(p.c, page, h, b);
    const bool edge = kb + kKvBlock > L - n + 1;   // some row does not see some token
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = lane + 32 * i;
      if (e < d) {
        float f[16];
        e4m3_f32x16(*reinterpret_cast<const uint4*>(vp + e * kKvBlock), f);
#pragma unroll
        for (int r = 0; r < kDecRows; ++r) {
          const int seen = L - n + (r0 + r) / p.G + 1 - kb;
          const float4* p4 = reinterpret_cast<const float4*>(sp + r * 16);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float4 w = p4[u];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              // a masked token's value may be NaN: it is left out, not times 0
              const float v = edge && 4 * u + k >= seen ? 0.f : f[4 * u + k];
              O[r][i] = fmaf((&w.x)[k], v, O[r][i]);
            }
          }
        }
      }
    }
    __syncwarp();
  }
  // join the warps: through shared memory, in the order of the warps
  __syncthreads();
  float* so = smem;                         // [4][8][d]
  float* sm = smem + kDecWarps * kDecRows * d;   // [4][8]
  float* sl = sm + kDecWarps * kDecRows;
#pragma unroll
  for (int r = 0; r < kDecRows; ++r) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (lane + 32 * i < d) so[(warp * kDecRows + r) * d + lane + 32 * i] = O[r][i];
    if (lane == 0) sm[warp * kDecRows + r] = m[r], sl[warp * kDecRows + r] = l[r];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < rows * d; i += blockDim.x) {
    const int r = i / d, e = i - r * d;
    float mx = -INFINITY;
    for (int w = 0; w < kDecWarps; ++w) mx = fmaxf(mx, sm[w * kDecRows + r]);
    const float ref = mx == -INFINITY ? 0.f : mx;
    float acc = 0.f, sum = 0.f;
    for (int w = 0; w < kDecWarps; ++w) {
      const float a = fast_exp2(sm[w * kDecRows + r] - ref);
      acc += a * so[(w * kDecRows + r) * d + e];
      sum += a * sl[w * kDecRows + r];
    }
    const int64_t rh = (int64_t)(q0 + (r0 + r) / p.G) * p.Hq + h * p.G + (r0 + r) % p.G;
    if (p.part_o) {
      p.part_o[((int64_t)piece * p.T * p.Hq + rh) * d + e] = acc;
      if (e == 0) p.part_ml[(int64_t)piece * p.T * p.Hq + rh] = make_float2(mx, sum);
    } else {
      put1<T>(p.o, rh * d + e, sum == 0.f ? 0.f : acc / sum);
      if (p.lse && e == 0) p.lse[rh] = sum == 0.f ? -INFINITY : mx * 0.693147180559945309f + logf(sum);
    }
  }
}

// The pieces of a sequence of n rows, as the kernel that served it cut them.
template <typename T, int K>
__device__ __forceinline__ int join_pieces(const AttnDecodeParams& p, int L, int n) {
  if (sizeof(T) == 2 && 32 * K >= kMaxPieces4 && n * p.G <= kD4Few) return decode_pieces<kMaxPieces4>(L, n * p.G, p.c.bits);
  return decode_pieces(L, n * p.G, p.c.bits);
}

// Joins the pieces of every row in their order: o = sum_i w_i O_i / sum_i w_i l_i,
// w_i = 2^(m_i - max m).  A warp a (row, head): the lanes hold the pieces'
// weights (32 K at most), then an element of the head each.  Bound by the pieces'
// bytes: 15.6 us after 256 single rows (24 heads, d = 256), 22 us after 16 drafts of 16.
// (Four CTAs an SM leave 128 registers, which hold eight pieces' loads; with the
// bound open the compiler loads one by one: 417 us for the 256 rows' call, 405.)
template <typename T, int K>
__global__ void __launch_bounds__(128, 4) attn_decode_join_kernel(const AttnDecodeParams p) {
  const int s = blockIdx.y, lane = threadIdx.x & 31, d = p.c.d;
  const int q0 = p.cu[s], n = p.cu[s + 1] - q0, L = p.kv_len[s];
  asm volatile("griddepcontrol.wait;\n" ::: "memory");   // the pieces' kernel before this one
  if (n <= 0 || n > p.max_q || L > p.max_kv || L < 0 || q0 < 0 || (int64_t)q0 + n > p.T) return;
  const int pieces = join_pieces<T, K>(p, L, n);
  const int64_t R = p.T * p.Hq;
  for (int i = blockIdx.x * 4 + (threadIdx.x >> 5); i < n * p.Hq; i += gridDim.x * 4) {
    const int64_t rh = (int64_t)q0 * p.Hq + i;
    float2 ml[K];
    float mx = -INFINITY;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      ml[k] = lane + 32 * k < pieces ? p.part_ml[(lane + 32 * k) * R + rh] : make_float2(-INFINITY, 0.f);
      mx = fmaxf(mx, ml[k].x);
    }
    // a wait ran out in a piece of this row: the row is not written
    bool lost = false;
#pragma unroll
    for (int k = 0; k < K; ++k) lost = lost || ml[k].y == kLostPiece;
    lost = __any_sync(0xffffffffu, lost);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float ref = mx == -INFINITY ? 0.f : mx;
    float w[K];
#pragma unroll
    for (int k = 0; k < K; ++k) w[k] = fast_exp2(ml[k].x - ref);
    float sum = 0.f;
    float4 acc[2] = {};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int most = min(32, pieces - 32 * k);
      const float4* o = reinterpret_cast<const float4*>(p.part_o + (32 * k * R + rh) * d) + lane;
      // eight pieces' loads at once; those past the last have weight 0
#pragma unroll 1
      for (int j0 = 0; j0 < most; j0 += 8) {
        float4 v[8][2];
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            v[j][h] = j0 + j < most && lane * 4 + 128 * h < d ? o[(j0 + j) * (R * d / 4) + 32 * h] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float wj = __shfl_sync(0xffffffffu, w[k], j0 + j);
          sum = fmaf(wj, __shfl_sync(0xffffffffu, ml[k].y, j0 + j), sum);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            acc[h].x = fmaf(wj, v[j][h].x, acc[h].x), acc[h].y = fmaf(wj, v[j][h].y, acc[h].y);
            acc[h].z = fmaf(wj, v[j][h].z, acc[h].z), acc[h].w = fmaf(wj, v[j][h].w, acc[h].w);
          }
        }
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (lane * 4 + 128 * h < d && !lost)
#pragma unroll
        for (int e = 0; e < 4; ++e) put1<T>(p.o, rh * d + lane * 4 + 128 * h + e, sum == 0.f ? 0.f : (&acc[h].x)[e] / sum);
    if (p.lse && lane == 0 && !lost) p.lse[rh] = sum == 0.f ? -INFINITY : mx * 0.693147180559945309f + logf(sum);
  }
}

// The same for a few rows, where rounds of loads are what the time goes to: a warp
// takes 32 elements of a (row, head), 32 pieces at once.  (One row of 24 heads over 112
// pieces, d = 256: the call takes 72 us, with the kernel above 75; over 4 pieces 17.3
// and 16.9.)
template <typename T, int K>
__global__ void __launch_bounds__(128, 4) attn_decode_join_few_kernel(const AttnDecodeParams p) {
  const int s = blockIdx.y, lane = threadIdx.x & 31, d = p.c.d, parts = (d + 31) / 32;
  const int q0 = p.cu[s], n = p.cu[s + 1] - q0, L = p.kv_len[s];
  asm volatile("griddepcontrol.wait;\n" ::: "memory");   // the pieces' kernel before this one
  if (n <= 0 || n > p.max_q || L > p.max_kv || L < 0 || q0 < 0 || (int64_t)q0 + n > p.T) return;
  const int pieces = join_pieces<T, K>(p, L, n);
  const int64_t R = p.T * p.Hq;
  for (int i = blockIdx.x * 4 + (threadIdx.x >> 5); i < n * p.Hq * parts; i += gridDim.x * 4) {
    const int64_t rh = (int64_t)q0 * p.Hq + i / parts;
    const int e = i % parts * 32 + lane;
    float2 ml[K];
    float mx = -INFINITY;
    bool lost = false;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      ml[k] = lane + 32 * k < pieces ? p.part_ml[(lane + 32 * k) * R + rh] : make_float2(-INFINITY, 0.f);
      mx = fmaxf(mx, ml[k].x);
      lost = lost || ml[k].y == kLostPiece;
    }
    lost = __any_sync(0xffffffffu, lost);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float ref = mx == -INFINITY ? 0.f : mx;
    float sum = 0.f, acc = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (32 * k >= pieces) break;
      const float w = fast_exp2(ml[k].x - ref);
      const float* o = p.part_o + (32 * k * R + rh) * d + e;
      float v[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = 32 * k + j < pieces && e < d ? o[j * (R * d)] : 0.f;
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const float wj = __shfl_sync(0xffffffffu, w, j);
        sum = fmaf(wj, __shfl_sync(0xffffffffu, ml[k].y, j), sum);
        acc = fmaf(wj, v[j], acc);
      }
    }
    if (lost) continue;
    if (e < d) put1<T>(p.o, rh * d + e, sum == 0.f ? 0.f : acc / sum);
    if (p.lse && e == 0) p.lse[rh] = sum == 0.f ? -INFINITY : mx * 0.693147180559945309f + logf(sum);
  }
}

namespace {

template <typename T>
cudaError_t decode_simt(const AttnDecodeParams& p, cudaStream_t st) {
  const int groups = (p.max_q * p.G + kDecRows - 1) / kDecRows;
  const size_t sm_run = (size_t)(kDecRows * p.c.d + kDecWarps * kDecRows * 16) * 4;
  const size_t sm_join = (size_t)(kDecWarps * kDecRows * (p.c.d + 2)) * 4;
  const size_t sm = sm_run > sm_join ? sm_run : sm_join;   // at most 33 KB
  attn_decode_simt_kernel<T><<<dim3(p.max_pieces, p.c.Hkv * groups, p.N), 32 * kDecWarps, sm, st>>>(p);
  return cudaGetLastError();
}

// The join of a few rows is taken up to about the warps that 152 SMs hold at once (16
// each: 2,432), over more pieces than its lanes load in one round.
constexpr int64_t kJoinFew = 2400;

// A join with so many warps a (row, head), launched as the last CTAs of the pieces'
// kernel leave, waiting on the device for its end.
cudaError_t join(const AttnDecodeParams& p, void (*kernel)(AttnDecodeParams), int parts, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((p.max_q * p.Hq * parts + 3) / 4), p.N);
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <typename T>
cudaError_t decode_dtype(const AttnDecodeParams& p, int dtype, cudaStream_t st) {
  const cudaError_t e = p.c.bits == 4                      ? launch_attn_decode4_tc(p, dtype, st)
                        : attn_decode_tc_supported(p, dtype) ? launch_attn_decode_tc(p, st)
                                                             : decode_simt<T>(p, st);
  if (e != cudaSuccess || !p.part_o) return e;
  constexpr int K8 = (kMaxPieces + 31) / 32, K4 = (kMaxPieces4 + 31) / 32;
  if (p.c.bits == 8) return join(p, attn_decode_join_kernel<T, K8>, 1, st);
  const int parts = (p.c.d + 31) / 32;
  return p.max_pieces > 32 && (int64_t)p.N * p.max_q * p.Hq * parts <= kJoinFew ? join(p, attn_decode_join_few_kernel<T, K4>, parts, st)
                                                           : join(p, attn_decode_join_kernel<T, K4>, 1, st);
}

}  // namespace

cudaError_t launch_attn_decode(const AttnDecodeParams& p, int dtype, cudaStream_t st) {
  return dtype == GDN_BF16 ? decode_dtype<__nv_bfloat16>(p, dtype, st) : decode_dtype<float>(p, dtype, st);
}

// ---- prefill ----------------------------------------------------------------------------
namespace {

constexpr int kPreKeys = 64, kPreLdP = kPreKeys + 4;
// Rows of a tile, four threads' worth each: 32 up to D = 64, so that a small
// model's prompts make more CTAs and their longest one is shorter (nine prompts
// of up to 1,000 tokens: 75 us with 64, 53 with 32, one group each), 64 above,
// where the keys' tiles take the shared memory.
template <int D> constexpr int kPreRows = D <= 64 ? 32 : 64;
// Groups of threads that take a tile's keys in turn, each with sums of its own:
// at D = 32 the longest prompt's last tile, which decides, has twice the threads
// (54 us with one group, 46 with two, 50 with four); at D = 64 two do not fit
// their registers (four prompts of 2,000: 758 us with one, 809 with two).
template <int D> constexpr int kPreGroups = D <= 32 ? 2 : 1;

// Four consecutive elements of a row as fp32.
__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xffff0000u));
}

}  // namespace

// A tile of query rows of one kv head's group (row i of the tile: token i / G, head
// i % G, so that the group shares the keys) against its keys, 64 at a time.
// 16 threads a row group: each 4 rows by 4 keys of the scores and 4 rows by
// D / 16 elements of the outputs (D: the head size rounded up to 32, 64, 128
// or 256).  Bound by fp32 arithmetic out of shared memory; a small model's
// prompts by the longest tile's way through its keys, which the next keys' loads
// (up to D = 64 held in registers while the present ones are used) leave.  Nine
// fp32 prompts of up to 1,000 tokens (4 heads, 2 kv heads, d = 32; 0.47 GFLOP of
// visible pairs): 43 us.
template <typename T, int D>
__global__ void __launch_bounds__(4 * kPreRows<D> * kPreGroups<D>, D <= 32 ? 2 : 1) attn_prefill_simt_kernel(const AttnPrefillParams p) {
  extern __shared__ float smem[];
  constexpr int VW = D == 32 ? 2 : 4, VN = D / 16 / VW;   // a thread's elements: VN groups of VW
  constexpr int ROWS = kPreRows<D>, THREADS = 4 * ROWS, GROUPS = kPreGroups<D>;   // threads of a group
  constexpr int NL = kPreKeys * D / 4 / THREADS;              // 4-element loads a thread for a tile of K (or V)
  constexpr bool AHEAD = D <= 64;
  const int d = p.d, ld = d + 4;
  int s, h, back;
  prefill_place(p, ROWS, (int)blockIdx.x, s, h, back);
  const int q0 = p.cu_q[s], n = p.cu_q[s + 1] - q0, k0 = p.cu_kv[s], L = p.cu_kv[s + 1] - k0;
  if (n <= 0) return;
  if (n > p.max_q || L > p.max_kv || L < 0 || q0 < 0 || k0 < 0 || (int64_t)q0 + n > p.Tq || (int64_t)k0 + L > p.Tk) {
    if (threadIdx.x == 0) set_error(p.err, GDN_ERR_INVALID_ARG);
    return;
  }
  const int tiles = (int)(((int64_t)n * p.G + ROWS - 1) / ROWS);
  const int tile = tiles - 1 - back;
  if (tile < 0 || back < 0) return;
  const int64_t r0 = (int64_t)tile * ROWS;
  float* sq = smem;                       // [ROWS][ld]
  const int group = threadIdx.x / THREADS, tid = threadIdx.x % THREADS;
  float* sk = sq + ROWS * ld + group * (2 * kPreKeys * ld + ROWS * kPreLdP);   // [64][ld]
  float* sv = sk + kPreKeys * ld;         // [64][ld]
  float* sp = sv + kPreKeys * ld;         // [ROWS][68]
  const int tx = tid & 15, ty = tid >> 4;
  auto sync = [&] {   // of this group
    if (GROUPS == 1) __syncthreads();
    else if (group == 0) asm volatile("bar.sync 1, %0;\n" ::"n"(THREADS) : "memory");
    else asm volatile("bar.sync 2, %0;\n" ::"n"(THREADS) : "memory");
  };
  static_assert(GROUPS <= 2, "a barrier each");
  // element group and row of this thread's loads: D / 4 groups a row
  constexpr int LG = D / 4;
  const int le = tid % LG * 4, lr = tid / LG, lstep = THREADS / LG;
  for (int r = lr + group * lstep; r < ROWS; r += GROUPS * lstep) {
    const int64_t row = (r0 + r) / p.G;
    const int g = (int)((r0 + r) - row * p.G);
    if (le < d) {
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row < n) x = load4(static_cast<const T*>(p.q) + (q0 + row) * p.q_stride + (int64_t)(h * p.G + g) * d + le);
      *reinterpret_cast<float4*>(sq + r * ld + le) =
          make_float4(x.x * p.scale_log2, x.y * p.scale_log2, x.z * p.scale_log2, x.w * p.scale_log2);
    }
  }
  float O[4][VN * VW], m[4], l[4];
  int lim[4];   // keys that each of this thread's rows sees
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY, l[i] = 0.f;
    const int64_t row = (r0 + 4 * ty + i) / p.G;
    lim[i] = row < n ? max(0, (int)(L - n + row + 1)) : 0;
#pragma unroll
    for (int j = 0; j < VN * VW; ++j) O[i][j] = 0.f;
  }
  const int last = (int)min((int64_t)n - 1, (r0 + ROWS - 1) / p.G), most = max(0, L - n + last + 1);
  const int least = max(0, (int)(L - n + r0 / p.G + 1));
  const T* kg = static_cast<const T*>(p.k) + (int64_t)k0 * p.k_stride + (int64_t)h * d + le;
  const T* vg = static_cast<const T*>(p.v) + (int64_t)k0 * p.v_stride + (int64_t)h * d + le;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  float4 ak[AHEAD ? NL : 1], av[AHEAD ? NL : 1];
  auto fetch = [&](int kb) {
#pragma unroll
    for (int i = 0; i < (AHEAD ? NL : 1); ++i) {
      const int key = kb + lr + i * lstep;
      const bool in = key < most && le < d;   // keys that no row sees may hold anything
      ak[i] = in ? load4(kg + key * p.k_stride) : zero;
      av[i] = in ? load4(vg + key * p.v_stride) : zero;
    }
  };
  if (AHEAD) fetch(group * kPreKeys);
  __syncthreads();   // the rows are there
  for (int kb = group * kPreKeys; kb < most; kb += GROUPS * kPreKeys) {
    sync();
    if (le < d) {
      if (AHEAD) {
#pragma unroll
        for (int i = 0; i < NL; ++i) {
          *reinterpret_cast<float4*>(sk + (lr + i * lstep) * ld + le) = ak[i];
          *reinterpret_cast<float4*>(sv + (lr + i * lstep) * ld + le) = av[i];
        }
      } else {
#pragma unroll 4
        for (int i = 0; i < NL; ++i) {
          const int key = kb + lr + i * lstep;
          *reinterpret_cast<float4*>(sk + (lr + i * lstep) * ld + le) = key < most ? load4(kg + key * p.k_stride) : zero;
          *reinterpret_cast<float4*>(sv + (lr + i * lstep) * ld + le) = key < most ? load4(vg + key * p.v_stride) : zero;
        }
      }
    }
    sync();
    if (AHEAD && kb + GROUPS * kPreKeys < most) fetch(kb + GROUPS * kPreKeys);
    float x[4][4] = {};
#pragma unroll 4
    for (int e = 0; e < d; e += 4) {
      float4 a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(sq + (4 * ty + i) * ld + e);
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(sk + (tx + 16 * j) * ld + e);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[i][j] = fmaf(a[i].x, b[j].x, x[i][j]);
          x[i][j] = fmaf(a[i].y, b[j].y, x[i][j]);
          x[i][j] = fmaf(a[i].z, b[j].z, x[i][j]);
          x[i][j] = fmaf(a[i].w, b[j].w, x[i][j]);
        }
    }
    const bool edge = kb + kPreKeys > least;   // some row does not see some key
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (edge) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (kb + tx + 16 * j >= lim[i]) x[i][j] = -INFINITY;
      }
      float mx = fmaxf(fmaxf(x[i][0], x[i][1]), fmaxf(x[i][2], x[i][3]));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float mn = fmaxf(m[i], mx), ref = mn == -INFINITY ? 0.f : mn;
      const float a = fast_exp2(m[i] - ref);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float e = fast_exp2(x[i][j] - ref);
        sum += e;
        sp[(4 * ty + i) * kPreLdP + tx + 16 * j] = e;
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      m[i] = mn, l[i] = l[i] * a + sum;
#pragma unroll
      for (int j = 0; j < VN * VW; ++j) O[i][j] *= a;
    }
    __syncwarp();   // a row's 16 threads are in one warp
#pragma unroll 2
    for (int k = 0; k < kPreKeys; k += 4) {
      float4 w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4*>(sp + (4 * ty + i) * kPreLdP + k);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
#pragma unroll
        for (int j = 0; j < VN; ++j) {
          const int e = VW * (tx + 16 * j);
          if (e >= d) continue;
          float v[VW];
#pragma unroll
          for (int c = 0; c < VW; c += 2)
            *reinterpret_cast<float2*>(v + c) = *reinterpret_cast<const float2*>(sv + (k + u) * ld + e + c);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // a masked key's value may be NaN: it is left out, not times 0
            const bool see = !edge || kb + k + u < lim[i];
#pragma unroll
            for (int c = 0; c < VW; ++c) O[i][j * VW + c] = fmaf((&w[i].x)[u], see ? v[c] : 0.f, O[i][j * VW + c]);
          }
        }
      }
    }
  }
  if constexpr (GROUPS > 1) {
    // the groups' sums joined in their order, through where their keys were
    constexpr int NO = VN * VW;
    auto part = [&](int g) { return sq + ROWS * ld + g * (2 * kPreKeys * ld + ROWS * kPreLdP) + tid; };
    sync();
    if (group > 0) {
      float* to = part(group);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        to[(2 * i) * THREADS] = m[i], to[(2 * i + 1) * THREADS] = l[i];
#pragma unroll
        for (int j = 0; j < NO; ++j) to[(8 + i * NO + j) * THREADS] = O[i][j];
      }
    }
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float mn = m[i];
#pragma unroll
      for (int g = 1; g < GROUPS; ++g) mn = fmaxf(mn, part(g)[(2 * i) * THREADS]);
      const float ref = mn == -INFINITY ? 0.f : mn, a = fast_exp2(m[i] - ref);
      m[i] = mn, l[i] *= a;
#pragma unroll
      for (int j = 0; j < NO; ++j) O[i][j] *= a;
#pragma unroll
      for (int g = 1; g < GROUPS; ++g) {
        const float* of = part(g);
        const float b = fast_exp2(of[(2 * i) * THREADS] - ref);
        l[i] = fmaf(of[(2 * i + 1) * THREADS], b, l[i]);
#pragma unroll
        for (int j = 0; j < NO; ++j) O[i][j] = fmaf(of[(8 + i * NO + j) * THREADS], b, O[i][j]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + 4 * ty + i, row = r / p.G;
    if (row >= n) continue;
    const int64_t rh = (q0 + row) * p.Hq + h * p.G + (r - row * p.G);
#pragma unroll
    for (int j = 0; j < VN; ++j)
#pragma unroll
      for (int c = 0; c < VW; ++c) {
        const int e = VW * (tx + 16 * j) + c;
        if (e < d) put1<T>(p.o, rh * d + e, l[i] == 0.f ? 0.f : O[i][j * VW + c] / l[i]);
      }
    if (p.lse && tx == 0) p.lse[rh] = l[i] == 0.f ? -INFINITY : m[i] * 0.693147180559945309f + logf(l[i]);
  }
}

namespace {

template <typename T, int D>
cudaError_t prefill_simt(AttnPrefillParams p, cudaStream_t st) {
  const int64_t grid = prefill_grid(p, kPreRows<D>, 8);
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  const size_t sm =   // 217,088 B at d = 256
      (size_t)(kPreRows<D> * (p.d + 4) + kPreGroups<D> * (2 * kPreKeys * (p.d + 4) + kPreRows<D> * kPreLdP)) * 4;
  cudaError_t e = allow_shared(attn_prefill_simt_kernel<T, D>);
  if (e != cudaSuccess) return e;
  attn_prefill_simt_kernel<T, D><<<(unsigned)grid, 4 * kPreRows<D> * kPreGroups<D>, sm, st>>>(p);
  return cudaGetLastError();
}
template <typename T>
cudaError_t prefill_dtype(const AttnPrefillParams& p, cudaStream_t st) {
  if (p.d <= 32) return prefill_simt<T, 32>(p, st);
  if (p.d <= 64) return prefill_simt<T, 64>(p, st);
  if (p.d <= 128) return prefill_simt<T, 128>(p, st);
  return prefill_simt<T, 256>(p, st);
}

}  // namespace

cudaError_t launch_attn_prefill(const AttnPrefillParams& p, int dtype, cudaStream_t st) {
  if (attn_prefill_tc_supported(p, dtype)) return launch_attn_prefill_tc(p, st);
  return dtype == GDN_BF16 ? prefill_dtype<__nv_bfloat16>(p, st) : prefill_dtype<float>(p, st);
}

}  // namespace gdn
