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

// Pairs of fp32 operations in one instruction, and the maximum of three.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
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

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Codes (b0, b1, b2, b3) -> f16 pairs (b0, b1) and (b2, b3).
template <int FMT>
__device__ __forceinline__ void codes_to_f16(uint32_t c, uint32_t& lo, uint32_t& hi) {
  if constexpr (FMT == kKvE4m3) {
    e4m3x4_to_f16(c, lo, hi);
  } else {   // 0x6400 | (code + 128) is the f16 number 1152 + code
    c ^= 0x80808080u;
    const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    uint32_t l = __byte_perm(c, 0x64646464u, 0x4140), h = __byte_perm(c, 0x64646464u, 0x4342);
    const __half2 a = __hsub2(*reinterpret_cast<__half2*>(&l), off), b = __hsub2(*reinterpret_cast<__half2*>(&h), off);
    lo = *reinterpret_cast<const uint32_t*>(&a);
    hi = *reinterpret_cast<const uint32_t*>(&b);
  }
}

__device__ __forceinline__ float2 f16x2_to_f32(uint32_t h) {
  const __half2 v = *reinterpret_cast<const __half2*>(&h);
  return __half22float2(v);
}

// Asynchronous copies of 16 and 4 bytes, of which the first `bytes` are read and the others set to zero; waiting for all but N groups.
__device__ __forceinline__ void cp_async16_n(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4_n(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait_n() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* map, int c0, int c1, int c2, uint32_t bar) {
  asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n"
               ::"r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
               : "memory");
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

// Page and slot of a cache-wide slot number; false outside the cache. page_shift: log2 of page_size, or -1.
__device__ __forceinline__ bool locate(const KvView& c, int page_shift, long long at, int& page, int& slot) {
  if (at < 0 || at >= static_cast<long long>(c.num_pages) * c.page_size) return false;
  if (page_shift >= 0) {
    page = static_cast<int>(at >> page_shift);
    slot = static_cast<int>(at) & (c.page_size - 1);
  } else if ((at >> 32) == 0) {   // 32-bit division where it is enough
    const uint32_t q = static_cast<uint32_t>(at) / static_cast<uint32_t>(c.page_size);
    page = static_cast<int>(q);
    slot = static_cast<int>(static_cast<uint32_t>(at) - q * static_cast<uint32_t>(c.page_size));
  } else {
    page = static_cast<int>(at / c.page_size);
    slot = static_cast<int>(at - static_cast<long long>(page) * c.page_size);
  }
  return true;
}

constexpr float kZeroRow = 7.888609052210118e-31f;   // 2^-100: a row whose magnitudes are below it is stored as zeros

// Four values times `inv`, rounded to codes.
template <int FMT>
__device__ __forceinline__ uint32_t quantise4(const float (&x)[4], float inv) {
  float f[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = __fmul_rn(x[j], inv);
  if constexpr (FMT == kKvE4m3) {
    uint32_t code;
    asm("{\n .reg .b16 l, h;\n cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n"
        " mov.b32 %0, {l, h};\n}\n"
        : "=r"(code)
        : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]));
    return code;
  } else {   // at most 127 (1 + 2^-23) in magnitude: 1.5 * 2^23 + f holds the rounded integer in its low byte
    uint32_t t[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) t[j] = __float_as_uint(__fadd_rn(f[j], 12582912.f));
    return __byte_perm(__byte_perm(t[0], t[1], 0x0040), __byte_perm(t[2], t[3], 0x0040), 0x5410);
  }
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
