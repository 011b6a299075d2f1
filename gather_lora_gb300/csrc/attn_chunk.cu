// Attention of chunks of new tokens over the paged cache (sm_103a).
//
// Row i of a sequence's n rows stands at position p = L - n + i of its L cached tokens and sees the tokens t <= p with
// t > p - window or t < sinks:
//   z_t = scale (q_i . k_t),   out_i = sum_t softmax(z)_t v_t.
//
// One warp a row and head, a token at a time, everything in fp32: running maximum, sum and result.
#include "attn_common.cuh"

namespace glora {

namespace {

constexpr int kChunkWarps = 8;

}  // namespace

template <int FMT, int D>
__global__ void __launch_bounds__(kChunkWarps * 32) chunk_kernel(const ChunkArgs p) {
  constexpr int E = D / 32;            // consecutive dimensions of a lane
  pdl_wait_then_release();
  const int lane = threadIdx.x & 31, b = blockIdx.y;
  const int q0 = __ldg(p.cu_q + b), q1 = __ldg(p.cu_q + b + 1);
  if (q0 < 0 || q1 > p.total_q || q1 <= q0) return;
  const int n = q1 - q0, G = p.q_heads / p.c.kv_heads;
  const long long most = static_cast<long long>(p.max_pages) * p.c.page_size;
  const int len = static_cast<int>(min(static_cast<long long>(max(__ldg(p.lens + b), 0)), most));
  const float sl2 = p.scale * kLog2e;
  for (long long unit = static_cast<long long>(blockIdx.x) * kChunkWarps + threadIdx.x / 32; unit < static_cast<long long>(n) * p.q_heads;
       unit += static_cast<long long>(gridDim.x) * kChunkWarps) {
    const int i = static_cast<int>(unit / p.q_heads), h = static_cast<int>(unit - static_cast<long long>(i) * p.q_heads), kvh = h / G;
    const long long row = q0 + i;
    float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      q[e] = bf16_bits_to_f32(p.q[row * p.q_stride + h * D + lane * E + e]) * sl2;
      o[e] = 0.f;
    }
    const int pos = len - n + i, low = max(0, pos - min(p.window - 1, pos));
    auto value = [&](const unsigned char* at, int e, const float* scales, long long si) {
      if constexpr (FMT == kKvBf16) return bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(at)[lane * E + e]);
      float f[4];
      codes_to_f32<FMT>(at[lane * E + e], f);
      return f[0] * scales[si];
    };
    for (int t = 0; t <= pos; ++t) {
      if (t >= p.sinks && t < low) t = low;
      const int entry = p.page_shift >= 0 ? t >> p.page_shift : t / p.c.page_size, slot = t - entry * p.c.page_size;
      const int page = __ldg(p.table + b * p.table_stride + entry);
      if (page < 0 || page >= p.c.num_pages) continue;
      const long long off = page * p.c.page_bytes + kvh * p.c.head_bytes + slot * p.c.token_bytes, si = scale_index(p.c, page, kvh, slot);
      float z = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) z += q[e] * value(p.c.k + off, e, p.c.ks, si);
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) z += __shfl_xor_sync(0xffffffffu, z, x);
      const float mn = fmaxf(m, z), ref = mn == -INFINITY ? 0.f : mn, keep = exp2_fast(m - ref), w = exp2_fast(z - ref);
      m = mn;
      l = l * keep + w;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = o[e] * keep + w * value(p.c.v + off, e, p.c.vs, si);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int e = 0; e < E; ++e) p.out[row * p.out_stride + h * D + lane * E + e] = f32_to_bf16_bits(o[e] * inv);
    if (p.lse && lane == 0) p.lse[row * p.q_heads + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
  }
}

namespace {

template <int FMT>
int launch_format(const ChunkArgs& a, void* stream) {
  const unsigned per = static_cast<unsigned>(152 * 8 / a.batch + 1);
  if (a.head_dim == 128) chunk_kernel<FMT, 128><<<dim3(per, a.batch), kChunkWarps * 32, 0, static_cast<cudaStream_t>(stream)>>>(a);
  else chunk_kernel<FMT, 64><<<dim3(per, a.batch), kChunkWarps * 32, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return static_cast<int>(cudaGetLastError());
}

}  // namespace

int launch_chunk(const ChunkArgs& a, void* stream) {
  switch (a.format) {
    case kKvBf16: return launch_format<kKvBf16>(a, stream);
    case kKvE4m3: return launch_format<kKvE4m3>(a, stream);
    default: return launch_format<kKvInt8>(a, stream);
  }
}

}  // namespace glora
