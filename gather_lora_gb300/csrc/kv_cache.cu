// The paged key-value cache written and read back (sm_103a).
//
// write: for every row i and key-value head h, the head_dim values of k and of v
// go to the cache slot slots[i]; in the 8-bit formats with one f32 scale each:
//   a = max |x|,  scale = a / Q,  code = round(x * (Q / a)),  Q = 448 or 127.
// read: x = bf16(code * scale).
//
// Both move every byte once and compute almost nothing: HBM bandwidth bounds them, latency at a few
// rows. A thread holds 8 values (16 bytes of BF16) of a K row and the same 8 of the V row, so the slot is
// divided into page and slot once for both; the 8 or 16 threads of a head row find its largest magnitude by
// shuffles. Large calls give a thread kMany such pieces, whose loads are all in flight before the first is
// used (with one, the wait for the slot number left half of the memory system idle). The write's four
// divisions a row go to four threads and its maxima to packed BF16: it was bound by issue, 315 instructions a
// warp and piece, 85 us in the case below.
//
// Measured on a GB300: 65536 tokens of 8 x 128 in E4M3 written in 67.7 us and read back in 65.4, 6.0 and 6.2
// TB/s; 32 tokens of 4 x 128 in 1.7 and 1.5 us.
#include "attn_common.cuh"

namespace glora {

namespace {

constexpr int kRowThreads = 256;
constexpr int kMany = 4;          // pieces of a thread in large calls

// Larger of two BF16 pairs, NaN if either is.
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
  const __nv_bfloat162 m = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&m);
}
__device__ __forceinline__ uint32_t abs_max8(const uint4& x) {
  constexpr uint32_t abs = 0x7fff7fffu;
  return max2_nan(max2_nan(x.x & abs, x.y & abs), max2_nan(x.z & abs, x.w & abs));
}

// The 8 BF16 values in `x` times `inv`, rounded to codes.
template <int FMT>
__device__ __forceinline__ uint2 quantise8(const uint4& x, float inv) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t code[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float f[4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      f[2 * j] = __uint_as_float(w[2 * h + j] << 16);
      f[2 * j + 1] = __uint_as_float(w[2 * h + j] & 0xffff0000u);
    }
    code[h] = quantise4<FMT>(f, inv);
  }
  return make_uint2(code[0], code[1]);
}

}  // namespace

// Row and head of this thread's piece j: head rows in order, heads fastest, kRowThreads * U / TPR of them a block.
template <int TPR, int U>
__device__ __forceinline__ int piece(const KvRowsArgs& p, int j, int& head) {
  constexpr uint32_t UNITS = kRowThreads * U / TPR;
  const uint32_t kvh = static_cast<uint32_t>(p.c.kv_heads), q = blockIdx.x / kvh, r = blockIdx.x - q * kvh;
  const uint32_t at = r * UNITS + j * (kRowThreads / TPR) + threadIdx.x / TPR;   // < 2^17
  const uint32_t row = kvh == 1 ? at : __umulhi(at, p.heads_magic);
  head = static_cast<int>(at - row * kvh);
  return static_cast<int>(q * UNITS + row);
}

template <int FMT, int D, int U>
__global__ void __launch_bounds__(kRowThreads) kv_write_kernel(const KvRowsArgs p) {
  constexpr int TPR = D / 8;   // threads of a head row
  const int part = threadIdx.x % TPR;
  pdl_wait_then_release();
  uint4 x[U][2];
  long long at[U];
  int row[U], head[U];
#pragma unroll
  for (int j = 0; j < U; ++j) {
    row[j] = piece<TPR, U>(p, j, head[j]);
    x[j][0] = x[j][1] = make_uint4(0, 0, 0, 0);
    at[j] = -1;
    if (row[j] < p.n) {
      const int col = head[j] * D + part * 8;
      at[j] = __ldg(p.slots + row[j]);
      x[j][0] = __ldg(reinterpret_cast<const uint4*>(p.k + row[j] * p.k_stride + col));
      x[j][1] = __ldg(reinterpret_cast<const uint4*>(p.v + row[j] * p.v_stride + col));
    }
  }
#pragma unroll
  for (int j = 0; j < U; ++j) {
    int page = 0, slot = 0;
    const bool live = locate(p.c, p.page_shift, at[j], page, slot);
    const long long to = page * p.c.page_bytes + head[j] * p.c.head_bytes + slot * p.c.token_bytes;
    if constexpr (FMT == kKvBf16) {
      if (live) {
        *reinterpret_cast<uint4*>(p.c.k + to + part * 16) = x[j][0];
        *reinterpret_cast<uint4*>(p.c.v + to + part * 16) = x[j][1];
      }
    } else {
      // Largest magnitudes of the K row (low half) and the V row (high half).
      const uint32_t mk = abs_max8(x[j][0]), mv = abs_max8(x[j][1]);
      uint32_t m = max2_nan(__byte_perm(mk, mv, 0x5410), __byte_perm(mk, mv, 0x7632));
#pragma unroll
      for (int o = TPR / 2; o > 0; o >>= 1) m = max2_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
      // The four divisions of a row by four threads: Q / a of K and of V, a / Q of K and of V.
      const uint32_t mine = (part & 1) ? m >> 16 : m & 0xffffu;
      const float amax = __uint_as_float(mine << 16);
      const bool finite = mine < 0x7f80u;
      const float quot = finite && amax >= kZeroRow ? ((part & 2) ? __fdiv_rn(amax, kv_qmax<FMT>()) : __fdiv_rn(kv_qmax<FMT>(), amax)) : 0.f;
      const float ik = __shfl_sync(0xffffffffu, quot, 0, TPR), iv = __shfl_sync(0xffffffffu, quot, 1, TPR);
      if (live) {
        // (a row that is not finite, or all but zero, has codes of zero)
        const uint2 zero = make_uint2(0u, 0u);
        *reinterpret_cast<uint2*>(p.c.k + to + part * 8) = ik != 0.f ? quantise8<FMT>(x[j][0], ik) : zero;
        *reinterpret_cast<uint2*>(p.c.v + to + part * 8) = iv != 0.f ? quantise8<FMT>(x[j][1], iv) : zero;
        if ((part & ~1) == 2)
          (part == 2 ? p.c.ks : p.c.vs)[scale_index(p.c, page, head[j], slot)] = finite ? quot : __int_as_float(0x7fffffff);
      }
    }
  }
}

template <int FMT, int D, int U>
__global__ void __launch_bounds__(kRowThreads) kv_read_kernel(const KvRowsArgs p) {
  constexpr int TPR = D / 8;
  const int part = threadIdx.x % TPR;
  pdl_wait_then_release();
  long long at[U];
  int row[U], head[U];
#pragma unroll
  for (int j = 0; j < U; ++j) {
    row[j] = piece<TPR, U>(p, j, head[j]);
    at[j] = row[j] < p.n ? __ldg(p.slots + row[j]) : -1;
  }
  uint4 x[U][2];       // BF16 values, or 8 codes in the first two words
  float s[U][2];
#pragma unroll
  for (int j = 0; j < U; ++j) {
    int page = 0, slot = 0;
    const bool live = locate(p.c, p.page_shift, at[j], page, slot);
    const long long from0 = page * p.c.page_bytes + head[j] * p.c.head_bytes + slot * p.c.token_bytes;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      x[j][h] = make_uint4(0, 0, 0, 0);
      s[j][h] = 0.f;
      if (!live) continue;
      const unsigned char* from = (h ? p.c.v : p.c.k) + from0;
      if constexpr (FMT == kKvBf16) {
        x[j][h] = __ldg(reinterpret_cast<const uint4*>(from + part * 16));
      } else {
        const uint2 code = __ldg(reinterpret_cast<const uint2*>(from + part * 8));
        x[j][h].x = code.x;
        x[j][h].y = code.y;
        s[j][h] = __ldg((h ? p.c.vs : p.c.ks) + scale_index(p.c, page, head[j], slot));
      }
    }
  }
#pragma unroll
  for (int j = 0; j < U; ++j) {
    if (row[j] >= p.n) continue;
    const int col = head[j] * D + part * 8;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint4 v = x[j][h];
      if constexpr (FMT != kKvBf16) {
        float f[4], g[4];
        codes_to_f32<FMT>(v.x, f);
        codes_to_f32<FMT>(v.y, g);
        const float sc = s[j][h];
        v = make_uint4(pack_bf16x2(f[0] * sc, f[1] * sc), pack_bf16x2(f[2] * sc, f[3] * sc),
                       pack_bf16x2(g[0] * sc, g[1] * sc), pack_bf16x2(g[2] * sc, g[3] * sc));
      }
      *reinterpret_cast<uint4*>((h ? p.v_out + row[j] * p.v_stride : p.k_out + row[j] * p.k_stride) + col) = v;
    }
  }
}

namespace {

template <class K>
int launch_rows(K kernel, int pieces, const KvRowsArgs& a, void* stream) {
  const long long units = static_cast<long long>(a.n) * a.c.kv_heads, per = kRowThreads * pieces / (a.head_dim / 8);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((units + per - 1) / per), 1, 1);
  cfg.blockDim = dim3(kRowThreads, 1, 1);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return static_cast<int>(cudaLaunchKernelEx(&cfg, kernel, a));
}

// One piece a thread while the call is too small to fill the GPU's 152 x 2048 threads twice, else kMany.
bool many(const KvRowsArgs& a) { return static_cast<long long>(a.n) * a.c.kv_heads * (a.head_dim / 8) >= 2LL * 152 * 2048; }

template <int FMT, int D>
int launch_write(const KvRowsArgs& a, void* stream) {
  return many(a) ? launch_rows(kv_write_kernel<FMT, D, kMany>, kMany, a, stream) : launch_rows(kv_write_kernel<FMT, D, 1>, 1, a, stream);
}
template <int FMT, int D>
int launch_read(const KvRowsArgs& a, void* stream) {
  return many(a) ? launch_rows(kv_read_kernel<FMT, D, kMany>, kMany, a, stream) : launch_rows(kv_read_kernel<FMT, D, 1>, 1, a, stream);
}

}  // namespace

int launch_kv_write(const KvRowsArgs& a, void* stream) {
  const bool wide = a.head_dim == 128;
  switch (a.format) {
    case kKvBf16: return wide ? launch_write<kKvBf16, 128>(a, stream) : launch_write<kKvBf16, 64>(a, stream);
    case kKvE4m3: return wide ? launch_write<kKvE4m3, 128>(a, stream) : launch_write<kKvE4m3, 64>(a, stream);
    default: return wide ? launch_write<kKvInt8, 128>(a, stream) : launch_write<kKvInt8, 64>(a, stream);
  }
}

int launch_kv_read(const KvRowsArgs& a, void* stream) {
  const bool wide = a.head_dim == 128;
  switch (a.format) {
    case kKvBf16: return wide ? launch_read<kKvBf16, 128>(a, stream) : launch_read<kKvBf16, 64>(a, stream);
    case kKvE4m3: return wide ? launch_read<kKvE4m3, 128>(a, stream) : launch_read<kKvE4m3, 64>(a, stream);
    default: return wide ? launch_read<kKvInt8, 128>(a, stream) : launch_read<kKvInt8, 64>(a, stream);
  }
}

}  // namespace glora
