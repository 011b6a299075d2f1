// Attention of one new token per sequence over the paged cache (sm_103a).
#include "attn_row.cuh"

namespace glora {

namespace {

constexpr int kDecodeWarps = 4;

template <int FMT, int E>
__device__ __forceinline__ void load_cached(const unsigned char* row, float s, int lane, float (&f)[E]) {
  if constexpr (FMT == kKvBf16) {
    load_bf16<E>(reinterpret_cast<const uint16_t*>(row) + lane * E, f);
  } else {
    uint32_t c = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) c |= static_cast<uint32_t>(row[lane * E + e]) << (8 * e);
    float g[4];
    codes_to_f32<FMT>(c, g);
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = g[e] * s;
  }
}

}  // namespace

// One CTA per (sequence, query head): its warps take the tokens in turn, each with
// its own running softmax, and join through shared memory.
template <int FMT, int D>
__global__ void __launch_bounds__(kDecodeWarps * 32) decode_row_kernel(const DecodeArgs p) {
  constexpr int E = D / 32;
  pdl_wait_then_release();
  const int b = blockIdx.x / p.q_heads, h = blockIdx.x - b * p.q_heads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kvh = h / (p.q_heads / p.c.kv_heads);
  const long long most = static_cast<long long>(p.max_pages) * p.c.page_size;
  const int len = static_cast<int>(min(static_cast<long long>(max(p.lens[b], 0)), most));
  RowState<D> st;
  st.begin(p.q + b * p.q_stride + h * D, p.scale * kLog2e, lane);
  for (int t = warp; t < len; t += kDecodeWarps) {
    const int page = p.table[b * p.table_stride + t / p.c.page_size], slot = t % p.c.page_size;
    if (page < 0 || page >= p.c.num_pages) continue;
    const long long at = page * p.c.page_bytes + kvh * p.c.head_bytes + slot * p.c.token_bytes;
    float ks = 1.f, vs = 1.f;
    if constexpr (FMT != kKvBf16) {
      const long long si = scale_index(p.c, page, kvh, slot);
      ks = p.c.ks[si];
      vs = p.c.vs[si];
    }
    float k[E], v[E];
    load_cached<FMT, E>(p.c.k + at, ks, lane, k);
    load_cached<FMT, E>(p.c.v + at, vs, lane, v);
    st.add(k, v);
  }
  __shared__ float sm[kDecodeWarps], sl[kDecodeWarps], so[kDecodeWarps][D];
  if (lane == 0) {
    sm[warp] = st.m;
    sl[warp] = st.l;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) so[warp][lane * E + e] = st.acc[e];
  __syncthreads();
  float m = -INFINITY, l = 0.f;
  for (int w = 0; w < kDecodeWarps; ++w) m = fmaxf(m, sm[w]);
  float f[kDecodeWarps];
  for (int w = 0; w < kDecodeWarps; ++w) {
    f[w] = (sm[w] == -INFINITY && sl[w] == 0.f) ? 0.f : exp2_fast(sm[w] - m);
    l += f[w] * sl[w];
  }
  for (int d = threadIdx.x; d < D; d += kDecodeWarps * 32) {
    float o = 0.f;
    for (int w = 0; w < kDecodeWarps; ++w) o += f[w] * so[w][d];
    p.out[b * p.out_stride + h * D + d] = f32_to_bf16_bits(l == 0.f ? 0.f : o / l);
  }
  if (p.lse && threadIdx.x == 0) p.lse[static_cast<long long>(b) * p.q_heads + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

namespace {

template <int FMT>
int launch_format(const DecodeArgs& a, void* stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(a.batch) * a.q_heads, 1, 1);
  cfg.blockDim = dim3(kDecodeWarps * 32, 1, 1);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return static_cast<int>(a.head_dim == 128 ? cudaLaunchKernelEx(&cfg, decode_row_kernel<FMT, 128>, a)
                                            : cudaLaunchKernelEx(&cfg, decode_row_kernel<FMT, 64>, a));
}

}  // namespace

int launch_decode(const DecodeArgs& a, void* stream) {
  switch (a.format) {
    case kKvBf16: return launch_format<kKvBf16>(a, stream);
    case kKvE4m3: return launch_format<kKvE4m3>(a, stream);
    default: return launch_format<kKvInt8>(a, stream);
  }
}

}  // namespace glora
