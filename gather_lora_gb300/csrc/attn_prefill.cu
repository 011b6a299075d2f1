// Causal attention over packed sequences of different lengths (sm_103a).
#include "attn_row.cuh"

namespace glora {

namespace {

constexpr int kRowWarps = 4;

// The sequence that holds query row r (cu_q non-decreasing), or -1.
__device__ __forceinline__ int sequence_of(const PrefillArgs& p, int r) {
  int lo = 0, hi = p.batch;   // the last b with cu_q[b] <= r
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (p.cu_q[mid + 1] <= r) lo = mid + 1; else hi = mid;
  }
  return lo < p.batch && p.cu_q[lo] <= r && r < p.cu_q[lo + 1] ? lo : -1;
}

}  // namespace

// One warp per (query row, query head).
template <int D>
__global__ void __launch_bounds__(kRowWarps * 32) prefill_row_kernel(const PrefillArgs p) {
  constexpr int E = D / 32;
  pdl_wait_then_release();
  const long long unit = static_cast<long long>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int r = static_cast<int>(unit / p.q_heads), h = static_cast<int>(unit - static_cast<long long>(r) * p.q_heads);
  if (r >= p.total_q) return;
  const int b = sequence_of(p, r);
  if (b < 0) return;
  const int q0 = p.cu_q[b], q1 = p.cu_q[b + 1], k0 = p.cu_k[b], k1 = p.cu_k[b + 1];
  if (q0 < 0 || q1 > p.total_q || k0 < 0 || k1 < k0 || k1 > p.total_k) return;
  const int seen = min(k1 - k0, (r - q0) + (k1 - k0) - (q1 - q0) + 1);
  const int kvh = h / (p.q_heads / p.kv_heads);
  RowState<D> st;
  st.begin(p.q + r * p.q_stride + h * D, p.scale * kLog2e, lane);
  for (int j = 0; j < seen; ++j) {
    float k[E], v[E];
    load_bf16<E>(p.k + (k0 + j) * p.k_stride + kvh * D + lane * E, k);
    load_bf16<E>(p.v + (k0 + j) * p.v_stride + kvh * D + lane * E, v);
    st.add(k, v);
  }
  const float inv = st.l == 0.f ? 0.f : 1.f / st.l;
#pragma unroll
  for (int e = 0; e < E; ++e) p.out[r * p.out_stride + h * D + lane * E + e] = f32_to_bf16_bits(st.l == 0.f ? 0.f : st.acc[e] * inv);
  if (p.lse && lane == 0) p.lse[static_cast<long long>(r) * p.q_heads + h] = st.l == 0.f ? -INFINITY : (st.m + log2f(st.l)) * kLn2;
}

int launch_prefill(const PrefillArgs& a, void* stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((static_cast<long long>(a.total_q) * a.q_heads + kRowWarps - 1) / kRowWarps), 1, 1);
  cfg.blockDim = dim3(kRowWarps * 32, 1, 1);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return static_cast<int>(a.head_dim == 128 ? cudaLaunchKernelEx(&cfg, prefill_row_kernel<128>, a)
                                            : cudaLaunchKernelEx(&cfg, prefill_row_kernel<64>, a));
}

}  // namespace glora
