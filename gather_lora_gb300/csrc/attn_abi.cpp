// C ABI of the cache and attention calls (include/gather_lora.h): argument checks
// on the host before any CUDA call, then one launch.
#include "../../include/gather_lora.h"

#include <cuda_runtime.h>

#include <cmath>

#include "abi_common.h"
#include "attn_types.h"

namespace {

using glora::aligned16;
using glora::cuda_fail;
using glora::fail;
using glora::ok;

int check_head_dim(int32_t d) {
  return d == 64 || d == 128 ? LORA_OK : fail(LORA_ERR_SIZE, "head_dim %d is not 64 or 128", d);
}

int check_heads(int32_t q_heads, int32_t kv_heads) {
  if (kv_heads < 1 || kv_heads > LORA_MAX_HEADS)
    return fail(LORA_ERR_SIZE, "kv_heads %d outside [1, %d]", kv_heads, LORA_MAX_HEADS);
  if (q_heads < 1 || q_heads > LORA_MAX_HEADS || q_heads % kv_heads)
    return fail(LORA_ERR_SIZE, "q_heads %d is not a multiple of kv_heads %d in [1, %d]", q_heads, kv_heads, LORA_MAX_HEADS);
  return LORA_OK;
}

int check_rows(const char* what, int64_t stride, int64_t width) {
  if (stride < width) return fail(LORA_ERR_STRIDE, "%s row stride %lld < %lld", what, (long long)stride, (long long)width);
  if (stride % 8) return fail(LORA_ERR_ALIGN, "%s row stride %lld is not a multiple of 8", what, (long long)stride);
  return LORA_OK;
}

int check_scale(float scale) {
  return std::isfinite(scale) && scale > 0.f ? LORA_OK : fail(LORA_ERR_SIZE, "scale %g is not positive and finite", (double)scale);
}

// log2 of v (>= 1), or -1 if v is no power of two.
int log2_or(int32_t v) {
  if (v & (v - 1)) return -1;
  int s = 0;
  while ((int64_t{1} << s) < v) ++s;
  return s;
}

// The cache's description, checked; `c` gets the kernels' view of it.
int check_cache(const lora_kv_cache* cache, glora::KvView& c) {
  if (!cache) return fail(LORA_ERR_NULL, "cache is NULL");
  if (cache->format < LORA_KV_BF16 || cache->format > LORA_KV_INT8)
    return fail(LORA_ERR_SIZE, "cache format %d outside [%d, %d]", cache->format, LORA_KV_BF16, LORA_KV_INT8);
  if (int rc = check_head_dim(cache->head_dim)) return rc;
  if (int rc = check_heads(cache->kv_heads, cache->kv_heads)) return rc;
  if (cache->num_pages < 0) return fail(LORA_ERR_SIZE, "num_pages %d < 0", cache->num_pages);
  if (cache->page_size < 1) return fail(LORA_ERR_SIZE, "page_size %d < 1", cache->page_size);
  const bool coded = cache->format != LORA_KV_BF16;
  if (cache->num_pages > 0 && (!cache->k_pages || !cache->v_pages || (coded && (!cache->k_scale || !cache->v_scale))))
    return fail(LORA_ERR_NULL, "a required cache pointer is NULL (k_pages, v_pages%s)", coded ? ", k_scale, v_scale" : "");
  if (!aligned16(cache->k_pages) || !aligned16(cache->v_pages))
    return fail(LORA_ERR_ALIGN, "k_pages and v_pages must be 16-byte aligned");
  if (coded && ((reinterpret_cast<uintptr_t>(cache->k_scale) | reinterpret_cast<uintptr_t>(cache->v_scale)) & 3u))
    return fail(LORA_ERR_ALIGN, "k_scale and v_scale must be 4-byte aligned");
  const int64_t bytes = coded ? 1 : 2;
  const int64_t strides[3] = {cache->page_stride, cache->head_stride, cache->token_stride};
  const int64_t counts[3] = {cache->num_pages, cache->kv_heads, cache->page_size};
  for (int i = 0; i < 3; ++i) {
    static const char* const names[3] = {"page", "head", "token"};
    if (strides[i] * bytes % 16) return fail(LORA_ERR_ALIGN, "cache %s stride %lld is not a multiple of 16 bytes", names[i], (long long)strides[i]);
    if (counts[i] > 1 && strides[i] < cache->head_dim)
      return fail(LORA_ERR_STRIDE, "cache %s stride %lld < head_dim %d", names[i], (long long)strides[i], cache->head_dim);
  }
  c.k = static_cast<unsigned char*>(cache->k_pages);
  c.v = static_cast<unsigned char*>(cache->v_pages);
  c.ks = cache->k_scale;
  c.vs = cache->v_scale;
  c.page_bytes = cache->page_stride * bytes;
  c.head_bytes = cache->head_stride * bytes;
  c.token_bytes = cache->token_stride * bytes;
  c.num_pages = cache->num_pages;
  c.kv_heads = cache->kv_heads;
  c.page_size = cache->page_size;
  return LORA_OK;
}

// What lora_kv_write and lora_kv_read share.
int kv_rows(const void* k, int64_t k_row_stride, const void* v, int64_t v_row_stride, const int64_t* slots, int32_t n,
            const lora_kv_cache* cache, glora::KvRowsArgs& a) {
  if (n < 0 || n > LORA_MAX_KV_ROWS) return fail(LORA_ERR_SIZE, "n %d outside [0, %d]", n, LORA_MAX_KV_ROWS);
  if (int rc = check_cache(cache, a.c)) return rc;
  const int64_t width = static_cast<int64_t>(cache->kv_heads) * cache->head_dim;
  if (int rc = check_rows("k", k_row_stride, width)) return rc;
  if (int rc = check_rows("v", v_row_stride, width)) return rc;
  if (n == 0) return LORA_OK;
  if (!k || !v || !slots) return fail(LORA_ERR_NULL, "a required pointer is NULL (k, v, slots)");
  if (!aligned16(k) || !aligned16(v)) return fail(LORA_ERR_ALIGN, "k and v must be 16-byte aligned");
  a.k_stride = k_row_stride;
  a.v_stride = v_row_stride;
  a.slots = reinterpret_cast<const long long*>(slots);
  a.n = n;
  a.head_dim = cache->head_dim;
  a.format = cache->format;
  a.page_shift = log2_or(cache->page_size);
  a.heads_magic = static_cast<uint32_t>(((1ull << 32) + cache->kv_heads - 1) / cache->kv_heads);
  return LORA_OK;
}

}  // namespace

extern "C" {

int lora_kv_write(const lora_bf16_t* k, int64_t k_row_stride, const lora_bf16_t* v, int64_t v_row_stride,
                  const int64_t* slots, int32_t n, const lora_kv_cache* cache, void* stream) {
  glora::KvRowsArgs a{};
  if (int rc = kv_rows(k, k_row_stride, v, v_row_stride, slots, n, cache, a)) return rc;
  if (n == 0) return ok();
  a.k = k;
  a.v = v;
  const int rc = glora::launch_kv_write(a, stream);
  return rc ? cuda_fail(rc, "lora_kv_write launch") : ok();
}

int lora_kv_read(lora_bf16_t* k_out, int64_t k_row_stride, lora_bf16_t* v_out, int64_t v_row_stride,
                 const int64_t* slots, int32_t n, const lora_kv_cache* cache, void* stream) {
  glora::KvRowsArgs a{};
  if (int rc = kv_rows(k_out, k_row_stride, v_out, v_row_stride, slots, n, cache, a)) return rc;
  if (n == 0) return ok();
  a.k_out = k_out;
  a.v_out = v_out;
  const int rc = glora::launch_kv_read(a, stream);
  return rc ? cuda_fail(rc, "lora_kv_read launch") : ok();
}

int lora_attn_decode(const lora_bf16_t* q, int64_t q_row_stride, lora_bf16_t* out, int64_t out_row_stride,
                     int32_t batch, int32_t q_heads, float scale, const lora_kv_cache* cache,
                     const int32_t* block_table, int64_t table_stride, int32_t max_pages,
                     const int32_t* seq_lens, float* lse, void* workspace, int64_t workspace_bytes,
                     void* stream) {
  glora::DecodeArgs a{};
  if (batch < 0 || batch > LORA_MAX_SEQS) return fail(LORA_ERR_SIZE, "batch %d outside [0, %d]", batch, LORA_MAX_SEQS);
  if (int rc = check_cache(cache, a.c)) return rc;
  if (int rc = check_heads(q_heads, cache->kv_heads)) return rc;
  if (int rc = check_scale(scale)) return rc;
  if (max_pages < 0) return fail(LORA_ERR_SIZE, "max_pages %d < 0", max_pages);
  if (static_cast<int64_t>(max_pages) * cache->page_size > LORA_MAX_SEQ_TOKENS)
    return fail(LORA_ERR_SIZE, "max_pages %d x page_size %d passes %d tokens", max_pages, cache->page_size, LORA_MAX_SEQ_TOKENS);
  const int64_t width = static_cast<int64_t>(q_heads) * cache->head_dim;
  if (int rc = check_rows("q", q_row_stride, width)) return rc;
  if (int rc = check_rows("out", out_row_stride, width)) return rc;
  if (table_stride < max_pages) return fail(LORA_ERR_STRIDE, "table_stride %lld < max_pages %d", (long long)table_stride, max_pages);
  if (workspace_bytes < LORA_ATTN_WORKSPACE)
    return fail(LORA_ERR_SIZE, "workspace of %lld bytes, %d are needed", (long long)workspace_bytes, LORA_ATTN_WORKSPACE);
  if (batch == 0) return ok();
  if (!q || !out || !seq_lens || !workspace || (max_pages > 0 && !block_table))
    return fail(LORA_ERR_NULL, "a required pointer is NULL (q, out, block_table, seq_lens, workspace)");
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace))
    return fail(LORA_ERR_ALIGN, "q, out and workspace must be 16-byte aligned");
  a.q = q;
  a.q_stride = q_row_stride;
  a.out = out;
  a.out_stride = out_row_stride;
  a.table = block_table;
  a.table_stride = table_stride;
  a.max_pages = max_pages;
  a.lens = seq_lens;
  a.lse = lse;
  a.workspace = workspace;
  a.batch = batch;
  a.q_heads = q_heads;
  a.head_dim = cache->head_dim;
  a.format = cache->format;
  a.page_shift = log2_or(cache->page_size);
  a.scale = scale;
  const int rc = glora::launch_decode(a, stream);
  return rc ? cuda_fail(rc, "lora_attn_decode launch") : ok();
}

int lora_attn_prefill(const lora_bf16_t* q, int64_t q_row_stride, const lora_bf16_t* k, int64_t k_row_stride,
                      const lora_bf16_t* v, int64_t v_row_stride, lora_bf16_t* out, int64_t out_row_stride,
                      const int32_t* cu_q, const int32_t* cu_k, int32_t batch, int32_t total_q,
                      int32_t total_k, int32_t q_heads, int32_t kv_heads, int32_t head_dim, float scale,
                      float* lse, void* stream) {
  if (batch < 0 || batch > LORA_MAX_SEQS) return fail(LORA_ERR_SIZE, "batch %d outside [0, %d]", batch, LORA_MAX_SEQS);
  if (total_q < 0 || total_q > LORA_MAX_KV_ROWS || total_k < 0 || total_k > LORA_MAX_KV_ROWS)
    return fail(LORA_ERR_SIZE, "total_q %d or total_k %d outside [0, %d]", total_q, total_k, LORA_MAX_KV_ROWS);
  if (int rc = check_head_dim(head_dim)) return rc;
  if (int rc = check_heads(q_heads, kv_heads)) return rc;
  if (int rc = check_scale(scale)) return rc;
  const int64_t q_width = static_cast<int64_t>(q_heads) * head_dim, k_width = static_cast<int64_t>(kv_heads) * head_dim;
  if (int rc = check_rows("q", q_row_stride, q_width)) return rc;
  if (int rc = check_rows("k", k_row_stride, k_width)) return rc;
  if (int rc = check_rows("v", v_row_stride, k_width)) return rc;
  if (int rc = check_rows("out", out_row_stride, q_width)) return rc;
  if (batch == 0 || total_q == 0) return ok();
  if (!q || !out || !cu_q || !cu_k || (total_k > 0 && (!k || !v)))
    return fail(LORA_ERR_NULL, "a required pointer is NULL (q, k, v, out, cu_q, cu_k)");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out))
    return fail(LORA_ERR_ALIGN, "q, k, v and out must be 16-byte aligned");
  glora::PrefillArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.out = out;
  a.q_stride = q_row_stride;
  a.k_stride = k_row_stride;
  a.v_stride = v_row_stride;
  a.out_stride = out_row_stride;
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.batch = batch;
  a.total_q = total_q;
  a.total_k = total_k;
  a.q_heads = q_heads;
  a.kv_heads = kv_heads;
  a.head_dim = head_dim;
  a.scale = scale;
  a.lse = lse;
  // Heads of a group in equal blocks of at most 128 (one block up to 128), as many whole tokens as fit 128 rows.
  const int group = q_heads / kv_heads, blocks = (group + 127) / 128;
  a.head_block = (group + blocks - 1) / blocks;
  a.tile_tokens = 128 / a.head_block;
  const uint64_t qd[3] = {static_cast<uint64_t>(head_dim), static_cast<uint64_t>(q_heads), static_cast<uint64_t>(total_q)};
  const uint64_t qs[2] = {static_cast<uint64_t>(head_dim) * 2, static_cast<uint64_t>(q_row_stride) * 2};
  const uint32_t qb[3] = {64, static_cast<uint32_t>(a.head_block), static_cast<uint32_t>(a.tile_tokens)};
  // (without any key nothing is loaded through the K and V maps: they describe one row of q then)
  const uint64_t kd[2] = {static_cast<uint64_t>(total_k ? k_width : head_dim), static_cast<uint64_t>(total_k ? total_k : 1)};
  const uint64_t ks = static_cast<uint64_t>(k_row_stride) * 2, vs = static_cast<uint64_t>(v_row_stride) * 2;
  const uint32_t kb[2] = {64, 128};
  int rc;
  if ((rc = glora::encode_bf16_map(&a.map_q, q, 3, qd, qs, qb, CU_TENSOR_MAP_SWIZZLE_128B, "q")) ||
      (rc = glora::encode_bf16_map(&a.map_k, total_k ? k : q, 2, kd, &ks, kb, CU_TENSOR_MAP_SWIZZLE_128B, "k")) ||
      (rc = glora::encode_bf16_map(&a.map_v, total_k ? v : q, 2, kd, &vs, kb, CU_TENSOR_MAP_SWIZZLE_128B, "v")))
    return rc;
  rc = glora::launch_prefill(a, stream);
  return rc ? cuda_fail(rc, "lora_attn_prefill launch") : ok();
}

}  // extern "C"
