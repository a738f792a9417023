// attn.h — parameters and launchers of the attention layers' kernels (the
// 8-bit and 4-bit K / V caches and the attention that reads them; not exported).
#pragma once

#include "common.cuh"

namespace gdn {

constexpr int kKvBlock = GDN_KV_BLOCK;

// The cache of one layer: page layout of include/gdn.h.
struct KvCache {
  char* base;
  int64_t page_bytes;
  int32_t num_pages;
  int32_t page_tokens;
  int32_t Hkv, d;
  int32_t bits;   // 8 or 4
};

// Offsets within a page: block b of head h.
__host__ __device__ inline int64_t kv_block_index(const KvCache& c, int h, int b) {
  return (int64_t)h * (c.page_tokens / kKvBlock) + b;
}
__host__ __device__ inline int64_t kv_codes_bytes(const KvCache& c) { return (int64_t)c.Hkv * c.page_tokens * c.d; }

struct KvTablesParams {
  int32_t N, max_pages, num_free, num_pages, page_tokens;
  int32_t seqs_per_cta;
  int64_t T;
  const int32_t* kv_len;
  const int32_t* new_len;
  const int32_t* free_pages;
  int32_t* block_table;
  int32_t* cu_seqlens;
  int32_t* cu_kv;
  int32_t* kv_len_out;
  int64_t* positions;
  int64_t* slot_map;
  int32_t* pages_taken;
  int32_t* err;
};

struct KvAppendParams {
  KvCache c;
  int64_t T, k_stride, v_stride;
  const void* k;
  const void* v;
  const int64_t* slot_map;
  int32_t* err;
};

struct KvGatherParams {
  KvCache c;
  int32_t N, max_pages;
  int64_t T;
  const int32_t* cu_kv;
  const int32_t* block_table;
  void* k;
  void* v;
  int32_t* err;
};

struct AttnDecodeParams {
  KvCache c;
  int32_t N, max_pages, Hq, G, max_q, max_kv, max_pieces;
  int64_t T, q_stride;
  float scale_log2;   // scale * log2(e)
  const int32_t* cu;
  const int32_t* kv_len;
  const int32_t* block_table;
  const void* q;
  void* o;
  float* lse;
  float* part_o;      // [max_pieces][T * Hq][d] sums of p v (nullptr: one piece, written to o)
  float2* part_ml;    // [max_pieces][T * Hq] (m, l) of the pieces
  int32_t* err;
  int64_t wait_cycles;
};

struct AttnPrefillParams {
  int32_t N, Hq, Hkv, G, d, max_q, max_kv;
  int64_t Tq, Tk, q_stride, k_stride, v_stride;
  float scale_log2;
  const int32_t* cu_q;
  const int32_t* cu_kv;
  const void* q;
  const void* k;
  const void* v;
  void* o;
  float* lse;
  int32_t* err;
  int64_t wait_cycles;
  int32_t flat;       // the order of the row tiles (prefill_grid)
};

// Row tiles of a prefill, `rows` rows each, as blocks (times kv heads), in one of
// two orders.  Even: every sequence's last tile, then the ones before, and so on,
// as many as max_q allows the longest, so that those with the most keys start
// first.  Flat: sequence after sequence, s at the places from cu_q[s] G / rows + s
// on, which are as many as its tiles or one more, whatever max_q is.  A place
// without a tile costs the tensor-core kernel, a CTA an SM, more than the search
// for a place and the worse order, so it takes the order with fewer places
// (24 heads, 4 kv heads, d = 256, even and flat: 24 prompts of 1 to 600 tokens
// after up to 2,000 keys 207 and 187 us; 24 of 500 under a bound of 4,000, 210
// and 147; one of 4,000 and 60 of 50, 366 and 180; 256 of 64, which are even's,
// 32 heads, 8, d = 128, 165 and 190).  The fp32 kernel's empty blocks cost less:
// flat from `times` = 8 (4 heads, 2, d = 32, 24 prompts of 500 under a bound of
// 500: 107 and 122; of 4,000: 119 and 121; of all rows: 156 and 123).
inline int64_t prefill_grid(AttnPrefillParams& p, int rows, int times) {
  const int64_t even = ((int64_t)p.max_q * p.G + rows - 1) / rows * p.N, flat = p.Tq * p.G / rows + p.N;
  p.flat = even > times * flat;
  return (p.flat ? flat : even) * p.Hkv;
}

// Keys of a decode sequence are cut into even pieces by its own length and
// number of (row, head of the group) pairs alone, so a row's sums are formed in
// the same order whatever batch it is in.  About 256 keys spread a short
// context over more SMs; 512 keep a few rows' outputs (4 d bytes each for a
// piece, written and read once) under 3 % of the keys' bytes at 6 rows; a
// draft's take 1,024, and 2,048 from 8,192 keys on (16 drafts of 16 rows over
// 2,048 to 32,768 keys: 262 us with 1,024, 226 with 2,048); beyond 38,912
// tokens 76 pieces a head are one CTA on each of the 152 SMs for two kv heads.
// Over 4 bits, half the keys' bytes, a few rows' pieces are of 1,024 keys from 2,048
// on, so that the outputs' share is the same.  There the kernel of a few rows has three
// CTAs on an SM at d = 256, and 114 pieces a head are theirs for four kv heads (one
// sequence of 229,376 tokens: 75 us with 76, 66 with 112, before the join).  One or
// two kv heads leave three quarters or half of those places empty: the cut does not
// go by the number of heads.
constexpr int kMaxPieces = 76, kMaxPieces4 = 114;
constexpr int kDtNarrow = 16;   // (row, head of the group) pairs up to which a sequence counts as a few rows
template <int MOST = kMaxPieces>
__host__ __device__ inline int decode_piece_target(int tiles, int rows, int bits) {   // pieces aimed at
  const int per = rows > kDtNarrow ? (tiles <= 16 ? 4 : tiles <= 64 ? 8 : 16) : tiles <= 16 ? 2 : bits == 8 ? 4 : 8;
  const int n = (tiles + per / 2) / per;
  return n < 1 ? 1 : n > MOST ? MOST : n;
}
template <int MOST = kMaxPieces>
__host__ __device__ inline int decode_piece_tokens(int L, int rows, int bits) {
  const int tiles = L < 1 ? 1 : (int)(((int64_t)L + 127) / 128), n = decode_piece_target<MOST>(tiles, rows, bits);
  return (tiles + n - 1) / n * 128;
}
template <int MOST = kMaxPieces>
__host__ __device__ inline int decode_pieces(int L, int rows, int bits) {
  const int c = decode_piece_tokens<MOST>(L, rows, bits);
  return L < 1 ? 1 : (int)(((int64_t)L + c - 1) / c);
}
// At least the pieces of any length up to L and any number of rows.
__host__ __device__ inline int decode_max_pieces(int L, int bits) {
  const int tiles = (int)(((int64_t)(L < 1 ? 1 : L) + 127) / 128);
  int most = 1;
  for (int rows = 1; rows <= kDtNarrow + 1; rows += kDtNarrow)
    for (int at = 16; at <= 128; at *= 2) {   // (up to 16 or 64 tiles, from where pieces are longer)
      const int t = tiles < at || at == 128 ? tiles : at;
      const int n = bits == 8 ? decode_piece_target<kMaxPieces>(t, rows, bits) : decode_piece_target<kMaxPieces4>(t, rows, bits);
      most = n > most ? n : most;
    }
  return most;
}

// In place of a row's sum (never negative) in a piece that was not finished.
constexpr float kLostPiece = -1.f;

cudaError_t launch_kv_tables(const KvTablesParams& p, cudaStream_t st);
cudaError_t launch_kv_append(const KvAppendParams& p, int dtype, cudaStream_t st);
cudaError_t launch_kv_gather(const KvGatherParams& p, int dtype, cudaStream_t st);
cudaError_t launch_kv4_append(const KvAppendParams& p, int dtype, cudaStream_t st);
cudaError_t launch_kv4_gather(const KvGatherParams& p, int dtype, cudaStream_t st);
cudaError_t launch_attn_decode(const AttnDecodeParams& p, int dtype, cudaStream_t st);
cudaError_t launch_attn_prefill(const AttnPrefillParams& p, int dtype, cudaStream_t st);
// The tensor-core decode (bf16, d a multiple of 32): the pieces, without the join.
bool attn_decode_tc_supported(const AttnDecodeParams& p, int dtype);
cudaError_t launch_attn_decode_tc(const AttnDecodeParams& p, cudaStream_t st);
// The decode over the 4-bit cache: the pieces, without the join.
constexpr int kD4Few = 8;   // (row, head of the group) pairs up to which bf16 sequences take the kernel of a few rows
cudaError_t launch_attn_decode4_tc(const AttnDecodeParams& p, int dtype, cudaStream_t st);
cudaError_t launch_attn_decode4_few(const AttnDecodeParams& p, int sms, bool follows, cudaStream_t st);
cudaError_t launch_attn_draft_tc(const AttnDecodeParams& p, int sms, bool overlap, cudaStream_t st);
// The tensor-core prefill: bf16, d = 64, 128 or 256, at least one key row.
bool attn_prefill_tc_supported(const AttnPrefillParams& p, int dtype);
cudaError_t launch_attn_prefill_tc(const AttnPrefillParams& p, cudaStream_t st);

}  // namespace gdn

#ifdef __CUDACC__
#include <cuda_fp16.h>

namespace gdn {

// Eight consecutive elements of a row, as loaded.
template <typename T> struct Row8;
template <> struct Row8<__nv_bfloat16> {
  uint4 w;
  __device__ void zero() { w = make_uint4(0, 0, 0, 0); }
  __device__ void load(const void* p) { w = *reinterpret_cast<const uint4*>(p); }
  __device__ float get(int i) const {
    const uint32_t x = (&w.x)[i >> 1];
    return __uint_as_float(i & 1 ? x & 0xffff0000u : x << 16);
  }
};
template <> struct Row8<float> {
  float4 a, b;
  __device__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ void load(const void* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ float get(int i) const { return i < 4 ? (&a.x)[i] : (&b.x)[i - 4]; }
};

// ---- e4m3 ----------------------------------------------------------------------
// Two fp32 values to e4m3, nearest even, saturating (lo in the low byte); NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}
// Two e4m3 codes (the low 16 bits of w) to fp32.
__device__ __forceinline__ float2 e4m3_f32x2(uint32_t w) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)w));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}
__device__ __forceinline__ void e4m3_f32x16(const uint4& v, float (&f)[16]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = e4m3_f32x2(w[i]), b = e4m3_f32x2(w[i] >> 16);
    f[4 * i] = a.x, f[4 * i + 1] = a.y, f[4 * i + 2] = b.x, f[4 * i + 3] = b.y;
  }
}

// ---- a prefill's row tiles ---------------------------------------------------------
// Block -> sequence, kv head, and which of the sequence's tiles, counted from its last.
__device__ __forceinline__ void prefill_place(const AttnPrefillParams& p, int rows, int block, int& s, int& h, int& back) {
  const int groups = p.N * p.Hkv;
  back = block / groups;
  const int pr = block - back * groups;
  s = pr / p.Hkv;
  h = pr - s * p.Hkv;
  if (!p.flat) return;
  const int i = back * p.N + s;   // block / Hkv
  auto first = [&](int k) { return (int64_t)p.cu_q[k] * p.G / rows + k; };
  int lo = 0, hi = p.N;   // the last s with first(s) <= i
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first(mid) <= i) lo = mid;
    else hi = mid;
  }
  s = lo;
  back = (int)(i - first(lo));
}

// ---- cache addressing ------------------------------------------------------------
__device__ __forceinline__ const uint8_t* kv_k_block(const KvCache& c, int page, int h, int b) {
  return reinterpret_cast<const uint8_t*>(c.base) + (int64_t)page * c.page_bytes +
         kv_block_index(c, h, b) * (c.d * kKvBlock);
}
__device__ __forceinline__ const uint8_t* kv_v_block(const KvCache& c, int page, int h, int b) {
  return kv_k_block(c, page, h, b) + kv_codes_bytes(c);
}
__device__ __forceinline__ const float* kv_k_scale(const KvCache& c, int page, int h, int b) {
  return reinterpret_cast<const float*>(c.base + (int64_t)page * c.page_bytes + 2 * kv_codes_bytes(c)) +
         kv_block_index(c, h, b);
}
__device__ __forceinline__ const float* kv_v_scale(const KvCache& c, int page, int h, int b) {
  return kv_k_scale(c, page, h, b) + (int64_t)c.Hkv * (c.page_tokens / kKvBlock);
}

}  // namespace gdn
#endif
