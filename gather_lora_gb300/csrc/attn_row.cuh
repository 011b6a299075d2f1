// One query row's attention by one warp, key by key (sm_103a): the plain form of
// the running softmax. Lane l holds dimensions [l * D / 32, + D / 32). With
// z = (q . k) * scale * log2(e), running maximum m, l = sum 2^(z - m) and
// acc = sum 2^(z - m) v, a new key with a larger z first multiplies l and acc by
// 2^(m_old - m_new).
#pragma once

#include "attn_common.cuh"

namespace glora {

template <int D>
struct RowState {
  static constexpr int E = D / 32;
  float q[E], acc[E];
  float m, l;

  // q: the row's BF16 values; each is multiplied by `factor` (scale * log2 e).
  __device__ __forceinline__ void begin(const uint16_t* row, float factor, int lane) {
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      q[e] = bf16_bits_to_f32(row[lane * E + e]) * factor;
      acc[e] = 0.f;
    }
  }
  __device__ __forceinline__ void add(const float (&k)[E], const float (&v)[E]) {
    float z = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) z += q[e] * k[e];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    if (z == -INFINITY) return;   // weight zero (only infinite inputs give it)
    const float mn = fmaxf(m, z);   // a NaN score leaves m and makes the weight NaN
    const float keep = exp2_fast(m - mn), w = exp2_fast(z - mn);
    l = l * keep + w;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * keep + w * v[e];
    m = mn;
  }
};

// E BF16 values at p as f32.
template <int E>
__device__ __forceinline__ void load_bf16(const uint16_t* p, float (&f)[E]) {
#pragma unroll
  for (int e = 0; e < E; ++e) f[e] = bf16_bits_to_f32(p[e]);
}

}  // namespace glora
