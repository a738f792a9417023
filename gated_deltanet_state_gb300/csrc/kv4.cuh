// kv4.cuh — the 4-bit form of the attention layers' cache (layout and rules:
// include/gdn.h): addresses, scales, codes.
#pragma once

#include "attn.h"

namespace gdn {

constexpr int kKv4Group = GDN_KV4_GROUP;   // channels of K that share a scale
constexpr uint32_t kKv4Nan = 255;          // the scale byte of NaN
constexpr float kKv4Most = 25088.f;        // the largest magnitude that no scale cuts off: 7 * 14 * 2^8

// Bytes of a block of 16 tokens of a head: K's codes (V's are as many), K's scales, V's scales.
__host__ __device__ inline int kv4_codes(int d) { return kKvBlock * d / 2; }
__host__ __device__ inline int kv4_k_scales(int d) { return kKvBlock * (d / kKv4Group); }

}  // namespace gdn

#ifdef __CUDACC__
namespace gdn {

__device__ __forceinline__ uint8_t* kv4_page(const KvCache& c, int page) {
  return reinterpret_cast<uint8_t*>(c.base) + (int64_t)page * c.page_bytes;
}
__device__ __forceinline__ uint8_t* kv4_k_block(const KvCache& c, int page, int h, int b) {
  return kv4_page(c, page) + kv_block_index(c, h, b) * kv4_codes(c.d);
}
__device__ __forceinline__ uint8_t* kv4_v_block(const KvCache& c, int page, int h, int b) {
  return kv4_k_block(c, page, h, b) + kv_codes_bytes(c) / 2;
}
__device__ __forceinline__ uint8_t* kv4_k_scale(const KvCache& c, int page, int h, int b) {
  return kv4_page(c, page) + kv_codes_bytes(c) + kv_block_index(c, h, b) * kv4_k_scales(c.d);
}
__device__ __forceinline__ uint8_t* kv4_v_scale(const KvCache& c, int page, int h, int b) {
  return kv4_page(c, page) + kv_codes_bytes(c) + (int64_t)c.Hkv * c.page_tokens * (c.d / kKv4Group) +
         kv_block_index(c, h, b) * kKvBlock;
}

// Value of a scale byte: (8 + b % 8) 2^(b / 8 - 23), whose fp32 bits are the byte
// next to an exponent of 107; its bf16 bits the upper half of those (4
// significant bits: exact).  As a number, also where the byte stands for NaN.
__device__ __forceinline__ float kv4_number(uint32_t b) { return __uint_as_float((b << 20) + (107u << 23)); }
__device__ __forceinline__ float kv4_scale(uint32_t b) { return b == kKv4Nan ? __int_as_float(0x7fffffff) : kv4_number(b); }
__device__ __forceinline__ uint32_t kv4_scale_bf16(uint32_t b) { return b == kKv4Nan ? 0x7fffu : (b << 4) + (107u << 7); }

// The least byte whose scale times 7 (exact: 7 bits) reaches a magnitude, given by its bits.
__device__ __forceinline__ uint32_t kv4_byte(uint32_t amax_bits) {
  const float amax = __uint_as_float(amax_bits), y = amax * (1.f / 7.f);
  int b = ((int)__float_as_uint(y) - (107 << 23) + 0xfffff) >> 20;
  b = max(0, min(254, b));
  // (the quotient's rounding can be off by one step at a scale's own value)
  if (b > 0 && 7.f * kv4_scale(b - 1) >= amax) --b;
  if (b < 254 && 7.f * kv4_scale(b) < amax) ++b;
  return b;
}

// Four words of each of four lanes (lane % 4 = q), transposed: word i of lane q
// goes to word q of lane i.
__device__ __forceinline__ void kv4_transpose(uint32_t (&w)[4], int q) {
  const bool odd = q & 1, up = q & 2;
  uint32_t a = __shfl_xor_sync(0xffffffffu, odd ? w[0] : w[1], 1), b = __shfl_xor_sync(0xffffffffu, odd ? w[2] : w[3], 1);
  if (odd) w[0] = a, w[2] = b;
  else w[1] = a, w[3] = b;
  a = __shfl_xor_sync(0xffffffffu, up ? w[0] : w[2], 2), b = __shfl_xor_sync(0xffffffffu, up ? w[1] : w[3], 2);
  if (up) w[0] = a, w[1] = b;
  else w[2] = a, w[3] = b;
}

// Two neighbouring elements of a word of eight, already shifted to bits 0 .. 3 and
// 16 .. 19, as bf16 of 128 + n: the codes become the mantissas' last bits.  (One
// instruction, where the compiler makes two of (w & a) | b with constants.)
__device__ __forceinline__ uint32_t kv4_pair(uint32_t w) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(w), "r"(0x000f000fu), "r"(0x43004300u));
  return r;
}
// (128 + n) s - 136 s = (n - 8) s: exact, since 136 s has 17 times s's 4 bits,
// 8 at most, and the product is not rounded on its way.
__device__ __forceinline__ uint32_t kv4_fma(uint32_t a, uint32_t s, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(s), "r"(c));
  return r;
}
// -136 s of a pair of scales in bf16.
__device__ __forceinline__ uint32_t kv4_offset(uint32_t s) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(s), "r"(0xc308c308u));
  return r;
}

// The eight elements of a word in f16: pairs 0 and 2 as n - 8, pairs 1 and 3, whose
// codes stay four bits further up, as 16 (n - 8), all exact.  The codes become the
// last bits of 1024 + n (or 16 n), from which 1024 + 8 (or 16 * 8) is taken.  (As
// subnormals, (n - 8) 2^-24, they take as long, but the tensor cores line a product's
// terms up by the operands' exponent fields, so that terms next to a large weight's
// lost bits even where that one's code is 0: fp32 rows with a key of 0.999 of the
// softmax were off by 1.4e-4 of sum w |v| in such channels.)
template <uint32_t MASK, uint32_t LESS>
__device__ __forceinline__ uint32_t kv4_half(uint32_t w) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(w), "r"(MASK), "r"(0x64006400u));
  asm("add.rn.f16x2 %0, %0, %1;" : "+r"(r) : "r"(LESS));
  return r;
}
__device__ __forceinline__ void kv4_halves(uint32_t w, uint32_t (&y)[4]) {
  const uint32_t v = w >> 8;
  y[0] = kv4_half<0x000f000fu, 0xe408e408u>(w), y[1] = kv4_half<0x00f000f0u, 0xe480e480u>(w);
  y[2] = kv4_half<0x000f000fu, 0xe408e408u>(v), y[3] = kv4_half<0x00f000f0u, 0xe480e480u>(v);
}

}  // namespace gdn
#endif
