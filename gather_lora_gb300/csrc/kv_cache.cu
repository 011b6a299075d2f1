// The paged key-value cache written and read back (sm_103a).
//
// write: for every row i and key-value head h, the head_dim values of k and of v
// go to the cache slot slots[i]; in the 8-bit formats with one f32 scale each:
//   a = max |x|,  scale = a / Q,  code = round(x * (Q / a)),  Q = 448 or 127.
// read: x = bf16(code * scale).
//
// Both move every byte once and compute almost nothing: HBM bandwidth bounds
// them, latency at a few rows. One thread holds 8 values (16 bytes of BF16) of a
// K row and the same 8 of the V row, so the slot is divided into page and slot
// once for both and two independent loads are in flight; the 8 or 16 threads of
// a head row find its largest magnitude by shuffles.
#include "attn_common.cuh"

namespace glora {

namespace {

constexpr int kRowThreads = 256;
constexpr float kZeroRow = 7.888609052210118e-31f;   // 2^-100: below it a row is stored as zeros

// Page and slot of slots[i]; false outside the cache.
__device__ __forceinline__ bool locate(const KvView& c, long long at, int& page, int& slot) {
  if (at < 0 || at >= static_cast<long long>(c.num_pages) * c.page_size) return false;
  if ((at >> 32) == 0) {   // 32-bit division where it is enough
    const uint32_t p = static_cast<uint32_t>(at) / static_cast<uint32_t>(c.page_size);
    page = static_cast<int>(p);
    slot = static_cast<int>(static_cast<uint32_t>(at) - p * static_cast<uint32_t>(c.page_size));
  } else {
    page = static_cast<int>(at / c.page_size);
    slot = static_cast<int>(at - static_cast<long long>(page) * c.page_size);
  }
  return true;
}

// The 8 BF16 values in `x` as codes; `a` is the bit pattern of the row's largest
// magnitude. The scale goes to *scale_out.
template <int FMT>
__device__ __forceinline__ uint2 quantise8(const uint4& x, uint32_t a, float* scale_out) {
  const float amax = bf16_bits_to_f32(static_cast<uint16_t>(a));
  const bool finite = a < 0x7f80u, keep = finite && amax >= kZeroRow;
  const float inv = keep ? __fdiv_rn(kv_qmax<FMT>(), amax) : 0.f;
  *scale_out = !finite ? __int_as_float(0x7fffffff) : keep ? __fdiv_rn(amax, kv_qmax<FMT>()) : 0.f;
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t code[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float f[4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      f[2 * j] = __uint_as_float(w[2 * h + j] << 16) * inv;
      f[2 * j + 1] = __uint_as_float(w[2 * h + j] & 0xffff0000u) * inv;
    }
    if constexpr (FMT == kKvE4m3) {
      uint32_t c;
      asm("{\n .reg .b16 l, h;\n cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n"
          " mov.b32 %0, {l, h};\n}\n"
          : "=r"(c)
          : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]));
      code[h] = c;
    } else {
      uint32_t c = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int q = max(-127, min(127, __float2int_rn(f[j])));
        c |= static_cast<uint32_t>(q & 0xff) << (8 * j);
      }
      code[h] = c;
    }
  }
  // (a row that is not finite holds NaN or infinity times zero here: its codes are zeros)
  return finite ? make_uint2(code[0], code[1]) : make_uint2(0u, 0u);
}

__device__ __forceinline__ uint32_t abs_max2(uint32_t m, uint32_t pair) {
  return max(m, max(pair & 0x7fffu, (pair >> 16) & 0x7fffu));
}

}  // namespace

template <int FMT, int D>
__global__ void __launch_bounds__(kRowThreads) kv_write_kernel(const KvRowsArgs p) {
  constexpr int TPR = D / 8;   // threads of a head row
  pdl_wait_then_release();
  const long long unit = (static_cast<long long>(blockIdx.x) * kRowThreads + threadIdx.x) / TPR;
  const int part = threadIdx.x % TPR;
  const long long row = unit / p.c.kv_heads;
  const int head = static_cast<int>(unit - row * p.c.kv_heads);
  int page = 0, slot = 0;
  const bool live = row < p.n && locate(p.c, p.slots[row], page, slot);
  uint4 x[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
  if (live) {
    const int col = head * D + part * 8;
    x[0] = *reinterpret_cast<const uint4*>(p.k + row * p.k_stride + col);
    x[1] = *reinterpret_cast<const uint4*>(p.v + row * p.v_stride + col);
  }
  const long long at = page * p.c.page_bytes + head * p.c.head_bytes + slot * p.c.token_bytes;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    unsigned char* to = (j ? p.c.v : p.c.k) + at;
    if constexpr (FMT == kKvBf16) {
      if (live) *reinterpret_cast<uint4*>(to + part * 16) = x[j];
    } else {
      uint32_t a = abs_max2(abs_max2(abs_max2(abs_max2(0u, x[j].x), x[j].y), x[j].z), x[j].w);
#pragma unroll
      for (int o = TPR / 2; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
      float scale;
      const uint2 code = quantise8<FMT>(x[j], a, &scale);
      if (live) {
        *reinterpret_cast<uint2*>(to + part * 8) = code;
        if (part == 0) (j ? p.c.vs : p.c.ks)[scale_index(p.c, page, head, slot)] = scale;
      }
    }
  }
}

template <int FMT, int D>
__global__ void __launch_bounds__(kRowThreads) kv_read_kernel(const KvRowsArgs p) {
  constexpr int TPR = D / 8;
  pdl_wait_then_release();
  const long long unit = (static_cast<long long>(blockIdx.x) * kRowThreads + threadIdx.x) / TPR;
  const int part = threadIdx.x % TPR;
  const long long row = unit / p.c.kv_heads;
  const int head = static_cast<int>(unit - row * p.c.kv_heads);
  if (row >= p.n) return;
  int page = 0, slot = 0;
  const bool live = locate(p.c, p.slots[row], page, slot);
  const long long at = page * p.c.page_bytes + head * p.c.head_bytes + slot * p.c.token_bytes;
  uint4 x[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    x[j] = make_uint4(0, 0, 0, 0);
    if (!live) continue;
    const unsigned char* from = (j ? p.c.v : p.c.k) + at;
    if constexpr (FMT == kKvBf16) {
      x[j] = *reinterpret_cast<const uint4*>(from + part * 16);
    } else {
      const uint2 code = *reinterpret_cast<const uint2*>(from + part * 8);
      const float s = (j ? p.c.vs : p.c.ks)[scale_index(p.c, page, head, slot)];
      float f[4], g[4];
      codes_to_f32<FMT>(code.x, f);
      codes_to_f32<FMT>(code.y, g);
      x[j] = make_uint4(pack_bf16x2(f[0] * s, f[1] * s), pack_bf16x2(f[2] * s, f[3] * s),
                        pack_bf16x2(g[0] * s, g[1] * s), pack_bf16x2(g[2] * s, g[3] * s));
    }
  }
  const int col = head * D + part * 8;
  *reinterpret_cast<uint4*>(p.k_out + row * p.k_stride + col) = x[0];
  *reinterpret_cast<uint4*>(p.v_out + row * p.v_stride + col) = x[1];
}

namespace {

template <class K>
int launch_rows(K kernel, const KvRowsArgs& a, void* stream) {
  const long long threads = static_cast<long long>(a.n) * a.c.kv_heads * (a.head_dim / 8);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((threads + kRowThreads - 1) / kRowThreads), 1, 1);
  cfg.blockDim = dim3(kRowThreads, 1, 1);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return static_cast<int>(cudaLaunchKernelEx(&cfg, kernel, a));
}

}  // namespace

int launch_kv_write(const KvRowsArgs& a, void* stream) {
  const bool wide = a.head_dim == 128;
  switch (a.format) {
    case kKvBf16: return wide ? launch_rows(kv_write_kernel<kKvBf16, 128>, a, stream) : launch_rows(kv_write_kernel<kKvBf16, 64>, a, stream);
    case kKvE4m3: return wide ? launch_rows(kv_write_kernel<kKvE4m3, 128>, a, stream) : launch_rows(kv_write_kernel<kKvE4m3, 64>, a, stream);
    default: return wide ? launch_rows(kv_write_kernel<kKvInt8, 128>, a, stream) : launch_rows(kv_write_kernel<kKvInt8, 64>, a, stream);
  }
}

int launch_kv_read(const KvRowsArgs& a, void* stream) {
  const bool wide = a.head_dim == 128;
  switch (a.format) {
    case kKvBf16: return wide ? launch_rows(kv_read_kernel<kKvBf16, 128>, a, stream) : launch_rows(kv_read_kernel<kKvBf16, 64>, a, stream);
    case kKvE4m3: return wide ? launch_rows(kv_read_kernel<kKvE4m3, 128>, a, stream) : launch_rows(kv_read_kernel<kKvE4m3, 64>, a, stream);
    default: return wide ? launch_rows(kv_read_kernel<kKvInt8, 128>, a, stream) : launch_rows(kv_read_kernel<kKvInt8, 64>, a, stream);
  }
}

}  // namespace glora
