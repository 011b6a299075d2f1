// Device helpers of the cache and attention kernels: 16-byte global accesses,
// the 8-bit cache formats, base-2 exponentials.
#pragma once

#include <cuda_fp8.h>

#include "attn_types.h"
#include "common.cuh"

namespace glora {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// 2^x by the special-function unit (2^-inf = 0).
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// The pair m with the largest magnitudes of 8 BF16 values taken in.
__device__ __forceinline__ uint32_t abs_max2(uint32_t m, const uint4& x) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  __nv_bfloat162 r = *reinterpret_cast<const __nv_bfloat162*>(&m);
#pragma unroll
  for (int i = 0; i < 4; ++i) r = __hmax2_nan(r, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[i])));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// Of a pair of largest magnitudes: neither is an infinity or NaN.
__device__ __forceinline__ bool all_finite(uint32_t m) { return (m & 0xffffu) < 0x7f80u && (m >> 16) < 0x7f80u; }
// A BF16 pair with what is not finite set to zero.
__device__ __forceinline__ uint32_t finite_or_zero(uint32_t x) {
  if ((x & 0x7f80u) == 0x7f80u) x &= 0xffff0000u;
  if ((x & 0x7f800000u) == 0x7f800000u) x &= 0xffffu;
  return x;
}

// Four E4M3 codes -> two pairs of f16 (low byte first). Every E4M3 value is exact in f16.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t c, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(c));
}

__device__ __forceinline__ float2 f16x2_to_f32(uint32_t h) {
  const __half2 v = *reinterpret_cast<const __half2*>(&h);
  return __half22float2(v);
}

// Largest magnitude an 8-bit code stands for.
template <int FMT>
__device__ __forceinline__ constexpr float kv_qmax() {
  return FMT == kKvE4m3 ? 448.f : 127.f;
}

// Element offset of (page, head, slot) in the scale arrays.
__device__ __forceinline__ long long scale_index(const KvView& c, int page, int head, int slot) {
  return (static_cast<long long>(page) * c.kv_heads + head) * c.page_size + slot;
}

// Four codes of an 8-bit format as f32.
template <int FMT>
__device__ __forceinline__ void codes_to_f32(uint32_t c, float (&f)[4]) {
  if constexpr (FMT == kKvE4m3) {
    uint32_t lo, hi;
    e4m3x4_to_f16(c, lo, hi);
    const float2 a = f16x2_to_f32(lo), b = f16x2_to_f32(hi);
    f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
  } else {
    c ^= 0x80808080u;   // 0x4b000000 | (code + 128) is the number 2^23 + 128 + code
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(__byte_perm(c, 0x4b000000u, 0x7440 | i)) - 8388736.f;
  }
}

}  // namespace glora
