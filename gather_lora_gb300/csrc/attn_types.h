// Argument blocks of the cache and attention kernels, shared by the host
// launcher (attn_abi.cpp) and the kernels.
#pragma once

#include <stdint.h>

#include "dense_types.h"   // TensorMapBytes

namespace glora {

enum KvFormat { kKvBf16 = 0, kKvE4m3 = 1, kKvInt8 = 2 };

// The paged cache as the kernels see it (lora_kv_cache; strides in bytes).
struct KvView {
  unsigned char* k;
  unsigned char* v;
  float* ks;                 // [num_pages, kv_heads, page_size] (8-bit formats)
  float* vs;
  long long page_bytes, head_bytes, token_bytes;
  int num_pages, kv_heads, page_size;
};

struct KvRowsArgs {
  KvView c;
  const uint16_t* k;         // write: the rows to store; read: NULL
  const uint16_t* v;
  uint16_t* k_out;           // read: the rows to fill; write: NULL
  uint16_t* v_out;
  long long k_stride, v_stride;
  const long long* slots;
  int n, head_dim, format;
  int page_shift;            // log2 of page_size, or -1: not a power of two
  uint32_t heads_magic;      // ceil(2^32 / kv_heads): x / kv_heads = hi(x * magic) for x * kv_heads < 2^32, kv_heads > 1
};

struct DecodeArgs {
  KvView c;
  const uint16_t* q;
  long long q_stride;
  uint16_t* out;
  long long out_stride;
  const int32_t* table;
  long long table_stride;
  int max_pages;
  const int32_t* lens;
  float* lse;
  void* workspace;
  int batch, q_heads, head_dim, format;
  int page_shift;            // log2 of page_size, or -1: not a power of two
  float scale;
};

struct PrefillArgs {
  TensorMapBytes map_q;      // q as [total_q, q_heads, head_dim], box {64, head_block, tile_tokens}, 128-byte swizzle
  TensorMapBytes map_k;      // k [total_k, kv_heads * head_dim], box {64, 128}, 128-byte swizzle
  TensorMapBytes map_v;
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* out;
  long long q_stride, k_stride, v_stride, out_stride;
  const int32_t* cu_q;
  const int32_t* cu_k;
  int batch, total_q, total_k, q_heads, kv_heads, head_dim;
  int head_block;            // query heads of a row tile: the group's, in blocks of at most 128
  int tile_tokens;           // tokens of a row tile: 128 / head_block
  float scale;
  float* lse;
};

// Launchers. Return 0 or a cudaError_t value.
int launch_kv_write(const KvRowsArgs& a, void* stream);
int launch_kv_read(const KvRowsArgs& a, void* stream);
int launch_decode(const DecodeArgs& a, void* stream);
int launch_prefill(const PrefillArgs& a, void* stream);
// OR of the prefill kernel's device status bits since the last clear (synchronizes `stream`).
int read_prefill_status(void* stream, uint32_t* out, int clear);

}  // namespace glora
