// attn_api.cu — the exported C ABI of the attention layers (include/gdn.h):
// host-side validation, then the internal launchers.
#include <cmath>

#include "attn.h"

using namespace gdn;

namespace {

constexpr int32_t kMaxSeqs = 65535;   // grid y / z limit used for sequences
// Keys of a sequence: the kernels count in tiles of up to 512 keys in 32 bits,
// past the last key by less than two of them.
constexpr int32_t kMaxKeys = 0x7fffffff - 1023;

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
gdn_status cuda_status(cudaError_t e) { return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }
int elem_bytes(const gdn_attn_desc* d) { return d->dtype == GDN_BF16 ? 2 : 4; }

gdn_status check_desc(const gdn_attn_desc* d) {
  if (!d || d->num_q_heads <= 0 || d->num_kv_heads <= 0 || d->head_dim <= 0 || d->page_tokens <= 0)
    return GDN_ERR_INVALID_ARG;
  if (d->dtype != GDN_F32 && d->dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
  if (!(d->scale > 0.0f) || !std::isfinite(d->scale) || d->reserved != 0) return GDN_ERR_INVALID_ARG;
  if (d->head_dim % 16 != 0 || d->head_dim > 256 || d->page_tokens % GDN_KV_BLOCK != 0 ||
      d->page_tokens > (1 << 24) || d->num_q_heads % d->num_kv_heads != 0 || d->num_q_heads > 1024)
    return GDN_ERR_UNSUPPORTED_SHAPE;
  return GDN_OK;
}

gdn_status check_pool(const gdn_attn_desc* d, const gdn_pool* pool) {
  if (!pool || !pool->base || pool->num_pages <= 0) return GDN_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(pool->base) % 256 != 0 || pool->page_bytes % 256 != 0) return GDN_ERR_INVALID_ARG;
  if (pool->page_bytes < gdn_kv_page_bytes(d)) return GDN_ERR_INVALID_ARG;
  return GDN_OK;
}

KvCache make_cache(const gdn_attn_desc* d, const gdn_pool* pool) {
  return KvCache{static_cast<char*>(pool->base), pool->page_bytes, pool->num_pages, d->page_tokens, d->num_kv_heads,
                 d->head_dim};
}

// Rows of `heads` heads, `stride` elements apart, each 16-byte aligned.
gdn_status check_rows(const gdn_attn_desc* d, const void* p, int64_t stride, int heads) {
  if (!p || !aligned16(p)) return GDN_ERR_INVALID_ARG;
  if (stride < (int64_t)heads * d->head_dim || stride * elem_bytes(d) % 16 != 0) return GDN_ERR_INVALID_ARG;
  return GDN_OK;
}

// Decode workspace: the pieces' outputs, then their statistics.
size_t part_o_bytes(const gdn_attn_desc* d, int64_t T, int pieces) {
  const size_t b = (size_t)T * d->num_q_heads * pieces * d->head_dim * sizeof(float);
  return (b + 255) / 256 * 256;
}

}  // namespace

extern "C" {

int64_t gdn_kv_page_bytes(const gdn_attn_desc* d) {
  if (check_desc(d) != GDN_OK) return -1;
  const int64_t per = 2 * (int64_t)d->head_dim * GDN_KV_BLOCK + 2 * (int64_t)sizeof(float);   // a block, K and V
  return (d->num_kv_heads * (int64_t)(d->page_tokens / GDN_KV_BLOCK) * per + 255) / 256 * 256;
}

gdn_status gdn_kv_tables(const gdn_attn_desc* desc, const gdn_kv_tables_args* a, void* stream) {
  const gdn_status st = check_desc(desc);
  if (st != GDN_OK) return st;
  if (!a || a->num_seqs < 0 || a->num_seqs > kMaxSeqs || a->max_pages < 0 || a->num_free < 0 || a->num_pages <= 0 ||
      a->total_tokens < 0 || a->total_tokens > 0x7fffffff)
    return GDN_ERR_INVALID_ARG;
  if (a->num_seqs == 0) return GDN_OK;
  if (!a->kv_len || !a->new_len || (a->num_free > 0 && !a->free_pages) || (a->max_pages > 0 && !a->block_table) ||
      !a->cu_seqlens || !a->cu_kv || !a->kv_len_out || a->kv_len_out == a->kv_len || a->kv_len_out == a->new_len ||
      !a->pages_taken || !a->dev_error || (a->total_tokens > 0 && (!a->positions || !a->slot_map)))
    return GDN_ERR_INVALID_ARG;
  KvTablesParams p{};
  p.N = a->num_seqs;
  p.max_pages = a->max_pages;
  p.num_free = a->num_free;
  p.num_pages = a->num_pages;
  p.page_tokens = desc->page_tokens;
  p.T = a->total_tokens;
  p.kv_len = a->kv_len;
  p.new_len = a->new_len;
  p.free_pages = a->free_pages;
  p.block_table = a->block_table;
  p.cu_seqlens = a->cu_seqlens;
  p.cu_kv = a->cu_kv;
  p.kv_len_out = a->kv_len_out;
  p.positions = a->positions;
  p.slot_map = a->slot_map;
  p.pages_taken = a->pages_taken;
  p.err = a->dev_error;
  return cuda_status(launch_kv_tables(p, static_cast<cudaStream_t>(stream)));
}

gdn_status gdn_kv_append(const gdn_attn_desc* desc, const gdn_pool* pool, const gdn_kv_append_args* a, void* stream) {
  gdn_status st = check_desc(desc);
  if (st == GDN_OK) st = check_pool(desc, pool);
  if (st != GDN_OK) return st;
  if (!a || a->total_tokens < 0 || a->total_tokens > 0x7fffffff) return GDN_ERR_INVALID_ARG;
  if (a->total_tokens == 0) return GDN_OK;
  if (!a->slot_map || !a->dev_error || desc->num_kv_heads > kMaxSeqs) return GDN_ERR_INVALID_ARG;
  st = check_rows(desc, a->k, a->k_stride, desc->num_kv_heads);
  if (st == GDN_OK) st = check_rows(desc, a->v, a->v_stride, desc->num_kv_heads);
  if (st != GDN_OK) return st;
  const KvAppendParams p{make_cache(desc, pool), a->total_tokens, a->k_stride, a->v_stride, a->k, a->v, a->slot_map,
                         a->dev_error};
  return cuda_status(launch_kv_append(p, desc->dtype, static_cast<cudaStream_t>(stream)));
}

gdn_status gdn_kv_gather(const gdn_attn_desc* desc, const gdn_pool* pool, const gdn_kv_gather_args* a, void* stream) {
  gdn_status st = check_desc(desc);
  if (st == GDN_OK) st = check_pool(desc, pool);
  if (st != GDN_OK) return st;
  if (!a || a->num_seqs < 0 || a->num_seqs > kMaxSeqs || a->max_pages < 0 || a->total_tokens < 0 ||
      a->total_tokens > 0x7fffffff)
    return GDN_ERR_INVALID_ARG;
  if (a->num_seqs == 0 || a->total_tokens == 0) return GDN_OK;
  if (!a->cu_kv || (a->max_pages > 0 && !a->block_table) || !a->k || !a->v || !a->dev_error || !aligned16(a->k) ||
      !aligned16(a->v))
    return GDN_ERR_INVALID_ARG;
  const KvGatherParams p{make_cache(desc, pool), a->num_seqs, a->max_pages, a->total_tokens, a->cu_kv, a->block_table,
                         a->k, a->v, a->dev_error};
  return cuda_status(launch_kv_gather(p, desc->dtype, static_cast<cudaStream_t>(stream)));
}

size_t gdn_attn_decode_workspace_size(const gdn_attn_desc* desc, int32_t num_seqs, int64_t total_tokens,
                                      int32_t max_kv_len) {
  if (check_desc(desc) != GDN_OK || num_seqs < 0 || total_tokens < 0 || max_kv_len < 0) return 0;
  const int pieces = decode_max_pieces(max_kv_len);
  if (pieces == 1) return 256;
  return part_o_bytes(desc, total_tokens, pieces) +
         ((size_t)total_tokens * desc->num_q_heads * pieces * sizeof(float2) + 255) / 256 * 256;
}

gdn_status gdn_attn_decode(const gdn_attn_desc* desc, const gdn_pool* pool, const gdn_attn_decode_args* a,
                           void* workspace, size_t workspace_bytes, void* stream) {
  gdn_status st = check_desc(desc);
  if (st == GDN_OK) st = check_pool(desc, pool);
  if (st != GDN_OK) return st;
  if (!a || a->num_seqs < 0 || a->num_seqs > kMaxSeqs || a->max_pages < 0 || a->total_tokens < 0 ||
      a->total_tokens > 0x7fffffff || a->max_kv_len < 0 || a->max_q_len < 1 || a->max_q_len > GDN_ATTN_DECODE_ROWS)
    return GDN_ERR_INVALID_ARG;
  if (a->num_seqs == 0 || a->total_tokens == 0) return GDN_OK;
  if (!a->cu_seqlens || !a->kv_len || (a->max_pages > 0 && !a->block_table) || !a->o || !a->dev_error ||
      !aligned16(a->o))
    return GDN_ERR_INVALID_ARG;
  st = check_rows(desc, a->q, a->q_stride, desc->num_q_heads);
  if (st != GDN_OK) return st;
  const int pieces = decode_max_pieces(a->max_kv_len);
  const size_t need = gdn_attn_decode_workspace_size(desc, a->num_seqs, a->total_tokens, a->max_kv_len);
  if (pieces > 1 && (!workspace || workspace_bytes < need || !aligned16(workspace))) return GDN_ERR_WORKSPACE;
  AttnDecodeParams p{};
  p.c = make_cache(desc, pool);
  p.N = a->num_seqs;
  p.max_pages = a->max_pages;
  p.Hq = desc->num_q_heads;
  p.G = desc->num_q_heads / desc->num_kv_heads;
  p.max_q = a->max_q_len;
  p.max_kv = a->max_kv_len < kMaxKeys ? a->max_kv_len : kMaxKeys;
  p.max_pieces = pieces;
  p.T = a->total_tokens;
  p.q_stride = a->q_stride;
  p.scale_log2 = desc->scale * 1.44269504088896341f;
  p.cu = a->cu_seqlens;
  p.kv_len = a->kv_len;
  p.block_table = a->block_table;
  p.q = a->q;
  p.o = a->o;
  p.lse = a->lse;
  if (pieces > 1) {
    p.part_o = static_cast<float*>(workspace);
    p.part_ml = reinterpret_cast<float2*>(static_cast<char*>(workspace) + part_o_bytes(desc, a->total_tokens, pieces));
  }
  p.err = a->dev_error;
  p.wait_cycles = a->wait_cycles;
  return cuda_status(launch_attn_decode(p, desc->dtype, static_cast<cudaStream_t>(stream)));
}

gdn_status gdn_attn_prefill(const gdn_attn_desc* desc, const gdn_attn_prefill_args* a, void* stream) {
  gdn_status st = check_desc(desc);
  if (st != GDN_OK) return st;
  if (!a || a->num_seqs < 0 || a->num_seqs > kMaxSeqs || a->total_q < 0 || a->total_q > 0x7fffffff ||
      a->total_kv < 0 || a->total_kv > 0x7fffffff || a->max_q_len < 0 || a->max_kv_len < 0 || a->reserved != 0)
    return GDN_ERR_INVALID_ARG;
  if (a->num_seqs == 0 || a->total_q == 0) return GDN_OK;
  if (!a->cu_seqlens || !a->cu_kv || !a->o || !a->dev_error || !aligned16(a->o)) return GDN_ERR_INVALID_ARG;
  st = check_rows(desc, a->q, a->q_stride, desc->num_q_heads);
  if (st == GDN_OK && a->total_kv > 0) st = check_rows(desc, a->k, a->k_stride, desc->num_kv_heads);
  if (st == GDN_OK && a->total_kv > 0) st = check_rows(desc, a->v, a->v_stride, desc->num_kv_heads);
  if (st != GDN_OK) return st;
  AttnPrefillParams p{};
  p.N = a->num_seqs;
  p.Hq = desc->num_q_heads;
  p.Hkv = desc->num_kv_heads;
  p.G = desc->num_q_heads / desc->num_kv_heads;
  p.d = desc->head_dim;
  p.max_q = a->max_q_len > 0 ? a->max_q_len : (int32_t)a->total_q;
  p.max_kv = a->max_kv_len > 0 ? a->max_kv_len : (int32_t)a->total_kv;
  if (p.max_kv > kMaxKeys) p.max_kv = kMaxKeys;
  p.Tq = a->total_q;
  p.Tk = a->total_kv;
  p.q_stride = a->q_stride;
  p.k_stride = a->k_stride;
  p.v_stride = a->v_stride;
  p.scale_log2 = desc->scale * 1.44269504088896341f;
  p.cu_q = a->cu_seqlens;
  p.cu_kv = a->cu_kv;
  p.q = a->q;
  p.k = a->k;
  p.v = a->v;
  p.o = a->o;
  p.lse = a->lse;
  p.err = a->dev_error;
  p.wait_cycles = a->wait_cycles;
  return cuda_status(launch_attn_prefill(p, desc->dtype, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
