// C ABI of the cache and attention calls (include/gather_lora.h): argument checks
// on the host before any CUDA call, then one launch.
#include "../../include/gather_lora.h"

#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

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

// TMA boxes over the cache's pages, where their size and strides allow: slots in eights (the swizzle's period), every stride a
// multiple of the one before it. Otherwise a.box_tokens stays 0.
int page_boxes(const lora_kv_cache* cache, glora::ChunkArgs& a) {
  a.box_tokens = 0;
  if (cache->num_pages == 0 || cache->page_size % 8) return LORA_OK;
  int tokens = 8;
  while (tokens < 128 && cache->page_size % (2 * tokens) == 0) tokens *= 2;
  const bool bf16 = cache->format == LORA_KV_BF16;
  const int64_t row = static_cast<int64_t>(cache->head_dim) * (bf16 ? 2 : 1);
  // (a dimension of one may have any stride: it gets the one that follows from those inside it)
  const bool inside = cache->kv_heads > 1 && a.c.head_bytes < a.c.token_bytes;
  const int64_t count[2] = {inside ? cache->kv_heads : cache->page_size, inside ? cache->page_size : cache->kv_heads};
  int64_t stride[3] = {inside ? a.c.head_bytes : a.c.token_bytes, inside ? a.c.token_bytes : a.c.head_bytes, a.c.page_bytes};
  if (count[1] == 1) stride[1] = stride[0] * count[0];
  if (cache->num_pages == 1) stride[2] = stride[1] * count[1];
  if (stride[0] < row || stride[1] % stride[0] || stride[1] < stride[0] * count[0] || stride[2] % stride[1] ||
      stride[2] < stride[1] * count[1] || stride[2] >= (int64_t{1} << 40))
    return LORA_OK;
  const uint64_t dims[4] = {static_cast<uint64_t>(cache->head_dim), static_cast<uint64_t>(count[0]), static_cast<uint64_t>(count[1]),
                            static_cast<uint64_t>(cache->num_pages)};
  const uint64_t strides[3] = {static_cast<uint64_t>(stride[0]), static_cast<uint64_t>(stride[1]), static_cast<uint64_t>(stride[2])};
  const uint32_t t = static_cast<uint32_t>(tokens), inner = bf16 ? 64 : static_cast<uint32_t>(cache->head_dim);
  const uint32_t box[4] = {inner, inside ? 1 : t, inside ? t : 1, 1};
  if (int rc = glora::encode_page_map(&a.map_k, a.c.k, bf16, dims, strides, box, "k_pages")) return rc;
  if (int rc = glora::encode_page_map(&a.map_v, a.c.v, bf16, dims, strides, box, "v_pages")) return rc;
  a.box_tokens = tokens;
  a.heads_inside = inside;
  return LORA_OK;
}

// Heads of a group in equal blocks of at most 128 (one block up to 128), as many whole tokens as fit 128 rows.
void row_tiles(int group, int& head_block, int& tile_tokens) {
  const int blocks = (group + 127) / 128;
  head_block = (group + blocks - 1) / blocks;
  tile_tokens = 128 / head_block;
}

int check_table(int32_t max_pages, int64_t table_stride, const lora_kv_cache* cache) {
  if (max_pages < 0) return fail(LORA_ERR_SIZE, "max_pages %d < 0", max_pages);
  if (static_cast<int64_t>(max_pages) * cache->page_size > LORA_MAX_SEQ_TOKENS)
    return fail(LORA_ERR_SIZE, "max_pages %d x page_size %d passes %d tokens", max_pages, cache->page_size, LORA_MAX_SEQ_TOKENS);
  if (table_stride < max_pages) return fail(LORA_ERR_STRIDE, "table_stride %lld < max_pages %d", (long long)table_stride, max_pages);
  return LORA_OK;
}

int check_window(int32_t window, int32_t sinks) {
  if (window < 1) return fail(LORA_ERR_SIZE, "window %d < 1", window);
  return sinks >= 0 ? LORA_OK : fail(LORA_ERR_SIZE, "sinks %d < 0", sinks);
}

// freq / (2 pi) less its whole part in units of 2^-64, to the nearest, |freq| < 2^64: the product of freq's 53 bits with the first 192
// of 1 / (2 pi) as integers (Machin's formula gives them). What is cut off moves it by less than 2^-64 units more.
uint64_t turns_of(double freq) {
  static const uint64_t inv_2pi[3] = {0x28be60db9391054aull, 0x7f09d5f47d4d3770ull, 0x36d8a5664f10e410ull};
  int e = 0;
  const uint64_t m = static_cast<uint64_t>(std::ldexp(std::frexp(std::fabs(freq), &e), 53));   // |freq| = m 2^(e - 53)
  uint64_t p[4] = {};                                   // m / (2 pi) in units of 2^-192, low word first
  for (int i = 0; i < 3; ++i) {
    const unsigned __int128 t = static_cast<unsigned __int128>(m) * inv_2pi[2 - i] + p[i];
    p[i] = static_cast<uint64_t>(t);
    p[i + 1] = static_cast<uint64_t>(t >> 64);
  }
  const int shift = 128 - (e - 53);                     // >= 117: units of 2^-64 begin at this bit of p
  auto word = [&](int w) { return w < 4 ? p[w] : uint64_t{0}; };
  auto bits = [&](int at) {                             // 64 bits of p from bit `at`
    const int w = at / 64, off = at % 64;
    return off ? word(w) >> off | word(w + 1) << (64 - off) : word(w);
  };
  const uint64_t t = bits(shift) + (bits(shift - 1) & 1);
  return freq < 0 ? 0 - t : t;
}

// What lora_qk_rope and lora_kv_append share: the rotation, positions and norms, and a pair of q rows.
int rope_args(const lora_bf16_t* q, int64_t q_row_stride, lora_bf16_t* q_out, int64_t q_out_row_stride, int32_t n, int32_t q_heads,
              const lora_rope* rope, const int32_t* positions, int64_t position_stride, const lora_bf16_t* q_norm,
              const lora_bf16_t* k_norm, float eps, glora::RopeArgs& a) {
  if (n < 0 || n > LORA_MAX_KV_ROWS) return fail(LORA_ERR_SIZE, "n %d outside [0, %d]", n, LORA_MAX_KV_ROWS);
  if (q_heads < 0 || q_heads > LORA_MAX_HEADS) return fail(LORA_ERR_SIZE, "q_heads %d outside [0, %d]", q_heads, LORA_MAX_HEADS);
  if (!rope) return fail(LORA_ERR_NULL, "rope is NULL");
  if (int rc = check_head_dim(rope->head_dim)) return rc;
  if (rope->rotary_dim < 0 || rope->rotary_dim > rope->head_dim || rope->rotary_dim % 8)
    return fail(LORA_ERR_SIZE, "rotary_dim %d is not a multiple of 8 in [0, %d]", rope->rotary_dim, rope->head_dim);
  if (rope->axes < 1 || rope->axes > LORA_MAX_ROPE_AXES)
    return fail(LORA_ERR_SIZE, "axes %d outside [1, %d]", rope->axes, LORA_MAX_ROPE_AXES);
  for (int j = 0; j < rope->rotary_dim / 2; ++j)
    if (rope->axis[j] >= rope->axes) return fail(LORA_ERR_SIZE, "axis %d of pair %d is not below axes %d", rope->axis[j], j, rope->axes);
  if (rope->rotary_dim && position_stride < n) return fail(LORA_ERR_STRIDE, "position_stride %lld < n %d", (long long)position_stride, n);
  if ((q_norm || k_norm) && !(std::isfinite(eps) && eps >= 0.f)) return fail(LORA_ERR_SIZE, "eps %g is not finite and >= 0", (double)eps);
  if (q_heads) {
    const int64_t width = static_cast<int64_t>(q_heads) * rope->head_dim;
    if (int rc = check_rows("q", q_row_stride, width)) return rc;
    if (int rc = check_rows("q_out", q_out_row_stride, width)) return rc;
  }
  if (n > 0 && q_heads && (!q || !q_out)) return fail(LORA_ERR_NULL, "a required pointer is NULL (q, q_out)");
  if (n > 0 && rope->rotary_dim && !positions) return fail(LORA_ERR_NULL, "positions is NULL");
  if (q_heads && (!aligned16(q) || !aligned16(q_out))) return fail(LORA_ERR_ALIGN, "q and q_out must be 16-byte aligned");
  if (!aligned16(q_norm) || !aligned16(k_norm)) return fail(LORA_ERR_ALIGN, "q_norm and k_norm must be 16-byte aligned");
  std::memcpy(a.rope.turns, rope->turns, sizeof a.rope.turns);
  std::memcpy(a.rope.axis, rope->axis, sizeof a.rope.axis);
  a.rope.rotary = rope->rotary_dim;
  a.rope.axes = rope->axes;
  a.rope.interleaved = rope->interleaved != 0;
  a.q = q;
  a.q_stride = q_row_stride;
  a.q_out = q_out;
  a.q_out_stride = q_out_row_stride;
  a.positions = positions;
  a.position_stride = position_stride;
  a.q_norm = q_norm;
  a.k_norm = k_norm;
  a.eps = eps;
  a.n = n;
  a.q_heads = q_heads;
  a.head_dim = rope->head_dim;
  return LORA_OK;
}

// What lora_attn_decode and lora_attn_decode_window share: `a` checked and filled in (batch > 0 if `a.batch` is).
int decode_args(const lora_bf16_t* q, int64_t q_row_stride, lora_bf16_t* out, int64_t out_row_stride, int32_t batch,
                int32_t q_heads, float scale, const lora_kv_cache* cache, const int32_t* block_table, int64_t table_stride,
                int32_t max_pages, const int32_t* seq_lens, float* lse, void* workspace, int64_t workspace_bytes,
                glora::DecodeArgs& a) {
  if (batch < 0 || batch > LORA_MAX_SEQS) return fail(LORA_ERR_SIZE, "batch %d outside [0, %d]", batch, LORA_MAX_SEQS);
  if (int rc = check_cache(cache, a.c)) return rc;
  if (int rc = check_heads(q_heads, cache->kv_heads)) return rc;
  if (int rc = check_scale(scale)) return rc;
  if (int rc = check_table(max_pages, table_stride, cache)) return rc;
  const int64_t width = static_cast<int64_t>(q_heads) * cache->head_dim;
  if (int rc = check_rows("q", q_row_stride, width)) return rc;
  if (int rc = check_rows("out", out_row_stride, width)) return rc;
  if (workspace_bytes < LORA_ATTN_WORKSPACE)
    return fail(LORA_ERR_SIZE, "workspace of %lld bytes, %d are needed", (long long)workspace_bytes, LORA_ATTN_WORKSPACE);
  if (batch == 0) return LORA_OK;
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
  if (int rc = decode_args(q, q_row_stride, out, out_row_stride, batch, q_heads, scale, cache, block_table, table_stride, max_pages,
                           seq_lens, lse, workspace, workspace_bytes, a)) return rc;
  if (batch == 0) return ok();
  const int rc = glora::launch_decode(a, stream);
  return rc ? cuda_fail(rc, "lora_attn_decode launch") : ok();
}

int lora_attn_decode_window(const lora_bf16_t* q, int64_t q_row_stride, lora_bf16_t* out, int64_t out_row_stride,
                            int32_t batch, int32_t q_heads, float scale, const lora_kv_cache* cache,
                            const int32_t* block_table, int64_t table_stride, int32_t max_pages,
                            const int32_t* seq_lens, int32_t window, int32_t sinks, float* lse,
                            void* workspace, int64_t workspace_bytes, void* stream) {
  glora::DecodeArgs a{};
  if (int rc = check_window(window, sinks)) return rc;
  if (int rc = decode_args(q, q_row_stride, out, out_row_stride, batch, q_heads, scale, cache, block_table, table_stride, max_pages,
                           seq_lens, lse, workspace, workspace_bytes, a)) return rc;
  if (batch == 0) return ok();
  a.window = window;
  a.sinks = sinks;
  // A window that holds all that the block table can name hides nothing.
  const bool all = window >= static_cast<int64_t>(max_pages) * cache->page_size;
  const int rc = all ? glora::launch_decode(a, stream) : glora::launch_decode_window(a, stream);
  return rc ? cuda_fail(rc, "lora_attn_decode_window launch") : ok();
}

int lora_attn_chunk(const lora_bf16_t* q, int64_t q_row_stride, lora_bf16_t* out, int64_t out_row_stride,
                    const int32_t* cu_q, int32_t batch, int32_t total_q, int32_t q_heads, float scale,
                    const lora_kv_cache* cache, const int32_t* block_table, int64_t table_stride,
                    int32_t max_pages, const int32_t* seq_lens, int32_t window, int32_t sinks, float* lse,
                    void* workspace, int64_t workspace_bytes, void* stream) {
  glora::ChunkArgs a{};
  if (batch < 0 || batch > LORA_MAX_SEQS) return fail(LORA_ERR_SIZE, "batch %d outside [0, %d]", batch, LORA_MAX_SEQS);
  if (total_q < 0 || total_q > LORA_MAX_KV_ROWS) return fail(LORA_ERR_SIZE, "total_q %d outside [0, %d]", total_q, LORA_MAX_KV_ROWS);
  if (int rc = check_cache(cache, a.c)) return rc;
  if (int rc = check_heads(q_heads, cache->kv_heads)) return rc;
  if (int rc = check_scale(scale)) return rc;
  if (int rc = check_window(window, sinks)) return rc;
  if (int rc = check_table(max_pages, table_stride, cache)) return rc;
  const int64_t width = static_cast<int64_t>(q_heads) * cache->head_dim;
  if (int rc = check_rows("q", q_row_stride, width)) return rc;
  if (int rc = check_rows("out", out_row_stride, width)) return rc;
  if (workspace_bytes < LORA_CHUNK_WORKSPACE)
    return fail(LORA_ERR_SIZE, "workspace of %lld bytes, %d are needed", (long long)workspace_bytes, LORA_CHUNK_WORKSPACE);
  if (batch == 0 || total_q == 0) return ok();
  if (!q || !out || !cu_q || !seq_lens || !workspace || (max_pages > 0 && !block_table))
    return fail(LORA_ERR_NULL, "a required pointer is NULL (q, out, cu_q, block_table, seq_lens, workspace)");
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace))
    return fail(LORA_ERR_ALIGN, "q, out and workspace must be 16-byte aligned");
  a.out = out;
  a.out_stride = out_row_stride;
  a.cu_q = cu_q;
  a.table = block_table;
  a.table_stride = table_stride;
  a.max_pages = max_pages;
  a.lens = seq_lens;
  a.lse = lse;
  a.workspace = workspace;
  a.batch = batch;
  a.total_q = total_q;
  a.q_heads = q_heads;
  a.head_dim = cache->head_dim;
  a.format = cache->format;
  a.page_shift = log2_or(cache->page_size);
  a.scale = scale;
  a.window = window;
  a.sinks = sinks;
  row_tiles(q_heads / cache->kv_heads, a.head_block, a.tile_tokens);
  const uint64_t qd[3] = {static_cast<uint64_t>(a.head_dim), static_cast<uint64_t>(q_heads), static_cast<uint64_t>(total_q)};
  const uint64_t qs[2] = {static_cast<uint64_t>(a.head_dim) * 2, static_cast<uint64_t>(q_row_stride) * 2};
  const uint32_t qb[3] = {64, static_cast<uint32_t>(a.head_block), static_cast<uint32_t>(a.tile_tokens)};
  if (int rc = glora::encode_bf16_map(&a.map_q, q, 3, qd, qs, qb, CU_TENSOR_MAP_SWIZZLE_128B, "q")) return rc;
  if (int rc = page_boxes(cache, a)) return rc;
  const int rc = glora::launch_chunk(a, stream);
  return rc ? cuda_fail(rc, "lora_attn_chunk launch") : ok();
}

int lora_rope_init(lora_rope* rope, int32_t head_dim, int32_t rotary_dim, const double* freqs, const uint8_t* axis,
                   int32_t axes, int32_t interleaved) {
  if (!rope) return fail(LORA_ERR_NULL, "rope is NULL");
  if (int rc = check_head_dim(head_dim)) return rc;
  if (rotary_dim < 0 || rotary_dim > head_dim || rotary_dim % 8)
    return fail(LORA_ERR_SIZE, "rotary_dim %d is not a multiple of 8 in [0, %d]", rotary_dim, head_dim);
  if (axes < 1 || axes > LORA_MAX_ROPE_AXES) return fail(LORA_ERR_SIZE, "axes %d outside [1, %d]", axes, LORA_MAX_ROPE_AXES);
  if (rotary_dim && !freqs) return fail(LORA_ERR_NULL, "freqs is NULL");
  lora_rope r{};
  for (int j = 0; j < rotary_dim / 2; ++j) {
    if (!(std::fabs(freqs[j]) < 0x1p64)) return fail(LORA_ERR_SIZE, "freqs[%d] %g is not below 2^64 in magnitude", j, freqs[j]);
    if (axis && axis[j] >= axes) return fail(LORA_ERR_SIZE, "axis %d of pair %d is not below axes %d", axis[j], j, axes);
    r.turns[j] = turns_of(freqs[j]);
    r.axis[j] = axis ? axis[j] : 0;
  }
  r.head_dim = head_dim;
  r.rotary_dim = rotary_dim;
  r.axes = axes;
  r.interleaved = interleaved != 0;
  *rope = r;
  return ok();
}

int lora_qk_rope(const lora_bf16_t* q, int64_t q_row_stride, lora_bf16_t* q_out, int64_t q_out_row_stride,
                 const lora_bf16_t* k, int64_t k_row_stride, lora_bf16_t* k_out, int64_t k_out_row_stride,
                 int32_t n, int32_t q_heads, int32_t kv_heads, const lora_rope* rope,
                 const int32_t* positions, int64_t position_stride, const lora_bf16_t* q_norm,
                 const lora_bf16_t* k_norm, float eps, void* stream) {
  glora::RopeArgs a{};
  if (kv_heads < 0 || kv_heads > LORA_MAX_HEADS || (q_heads == 0 && kv_heads == 0))
    return fail(LORA_ERR_SIZE, "kv_heads %d outside [0, %d], or no heads at all", kv_heads, LORA_MAX_HEADS);
  if (int rc = rope_args(q, q_row_stride, q_out, q_out_row_stride, n, q_heads, rope, positions, position_stride, q_norm, k_norm, eps, a)) return rc;
  if (kv_heads) {
    const int64_t width = static_cast<int64_t>(kv_heads) * rope->head_dim;
    if (int rc = check_rows("k", k_row_stride, width)) return rc;
    if (int rc = check_rows("k_out", k_out_row_stride, width)) return rc;
    if (n > 0 && (!k || !k_out)) return fail(LORA_ERR_NULL, "a required pointer is NULL (k, k_out)");
    if (!aligned16(k) || !aligned16(k_out)) return fail(LORA_ERR_ALIGN, "k and k_out must be 16-byte aligned");
  }
  if (n == 0) return ok();
  a.k = k;
  a.k_stride = k_row_stride;
  a.k_out = k_out;
  a.k_out_stride = k_out_row_stride;
  a.kv_heads = kv_heads;
  a.format = glora::kRopeRows;
  const int rc = glora::launch_rope(a, stream);
  return rc ? cuda_fail(rc, "lora_qk_rope launch") : ok();
}

int lora_kv_append(const lora_bf16_t* q, int64_t q_row_stride, lora_bf16_t* q_out, int64_t q_out_row_stride,
                   int32_t q_heads, const lora_bf16_t* k, int64_t k_row_stride, const lora_bf16_t* v,
                   int64_t v_row_stride, const int64_t* slots, int32_t n, const lora_kv_cache* cache,
                   const lora_rope* rope, const int32_t* positions, int64_t position_stride,
                   const lora_bf16_t* q_norm, const lora_bf16_t* k_norm, float eps, void* stream) {
  glora::RopeArgs a{};
  glora::KvRowsArgs rows{};
  if (int rc = kv_rows(k, k_row_stride, v, v_row_stride, slots, n, cache, rows)) return rc;
  if (int rc = rope_args(q, q_row_stride, q_out, q_out_row_stride, n, q_heads, rope, positions, position_stride, q_norm, k_norm, eps, a)) return rc;
  if (rope->head_dim != cache->head_dim)
    return fail(LORA_ERR_SIZE, "the rotation is for head_dim %d, the cache has %d", rope->head_dim, cache->head_dim);
  if (n == 0) return ok();
  a.c = rows.c;
  a.k = k;
  a.k_stride = k_row_stride;
  a.v = v;
  a.v_stride = v_row_stride;
  a.slots = rows.slots;
  a.kv_heads = cache->kv_heads;
  a.format = cache->format;
  a.page_shift = rows.page_shift;
  const int rc = glora::launch_rope(a, stream);
  return rc ? cuda_fail(rc, "lora_kv_append launch") : ok();
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
  row_tiles(q_heads / kv_heads, a.head_block, a.tile_tokens);
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
