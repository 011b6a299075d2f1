// Queries and keys normed per head and rotated by their positions, into rows or on the way into the
// paged cache (sm_103a).
//
//   x <- x * rsqrt(mean(x^2) + eps) * w          per head (optional)
//   (y0, y1) = (x0 cos a - x1 sin a, x1 cos a + x0 sin a),   a = position[axis_j] * freq_j, pair j
//   cache: k after that, v as it is: scale = a (1 / Q), code = round(y (Q (1 / a))), a = max |y|, Q = 448 or 127
//
// Every value is read and written once, with some 12 operations on it between: HBM bandwidth bounds it, latency at a
// few rows. All of a value's work is done in fp32 registers and rounded once.
//
// Angles. A position turns pair j by position * turns_j, in units of 2^-64 of a full turn: the 64-bit product drops
// whole turns by wrapping around, exactly, and its upper 32 bits are the angle in [-pi, pi), off by at most the 2^-32 of a turn cut off and
// the position times the table's rounding, 2^31 * 2^-65 turns. The special-function unit's sine and cosine are then within 2^-21 absolutely, a
// 2^12th of what rounding the result to BF16 costs.
//
// Layout. A team of D / 8 lanes holds a head row, 8 values a lane: four pairs, so that no lane needs another's values for
// the rotation (halves apart: elements 4 i .. and rotary_dim / 2 + 4 i ..; neighbours: 8 i .. 8 i + 7), and the rows' sums and
// maxima take 3 or 4 shuffles. A team takes kHeads heads of one token, in the order q, k, v: their loads are in flight
// together and the lane's four sines and cosines serve all of them; the teams of a warp take the same heads of consecutive tokens,
// so that a warp does not go through what is done for queries, keys and values one after another. Calls too small to fill the
// GPU with that take one head a team.
//
// Measured on a GB300 (copy rate 6.8 TB/s): 16411 rows of 28 + 4 heads of 128 in 45 us (6.0 TB/s); appended with 8 key-value heads,
// 20011 rows of 32 heads of 128 in BF16 82 us (6.0 TB/s; heads side by side in a warp instead of tokens 89), in E4M3 97 (4.7), 40009
// rows of 32 heads of 64 in INT8 93 (4.9). HBM bounds the 16-bit forms, the 8-bit ones instruction issue (INT8: 74% of it, 21
// instructions a value). A fourth block an SM is worth its registers in INT8 (99 -> 93), not in E4M3 (spills, 97 -> 99) or BF16
// (82 -> 85). With norms the 20011 rows take 97 us in BF16 (5.1 TB/s), 116 in E4M3, 118 in INT8. A few rows are latency: the host's time for
// the call and two trips to memory.
#include "attn_common.cuh"

namespace glora {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kHeads = 4;           // heads of a team at a time in large calls

__device__ __forceinline__ void unpack4(const uint2& v, float (&f)[4]) {
  f[0] = __uint_as_float(v.x << 16);
  f[1] = __uint_as_float(v.x & 0xffff0000u);
  f[2] = __uint_as_float(v.y << 16);
  f[3] = __uint_as_float(v.y & 0xffff0000u);
}
__device__ __forceinline__ uint2 pack4(const float (&f)[4]) { return make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3])); }

// Tokens of a unit, and units that a block has in hand at a time: with several heads a team, the teams of a warp take the same heads
// of consecutive tokens.
template <int D, int U>
struct RopeUnits {
  static constexpr int tokens = U > 1 ? 32 / (D / 8) : 1, takers = kRopeThreads / (U > 1 ? 32 : D / 8);
};

}  // namespace

// FMT: the cache's format, or kRopeRows. INTER: pairs are neighbours. U: heads of a team at a time.
template <int FMT, int D, bool INTER, int U>
__global__ void __launch_bounds__(kRopeThreads, FMT == kKvInt8 && U > 1 ? 4 : 0) rope_kernel(const __grid_constant__ RopeArgs p) {
  constexpr int TPR = D / 8, TOKS = RopeUnits<D, U>::tokens, TAKERS = RopeUnits<D, U>::takers;
  __shared__ __align__(16) unsigned long long s_turns[64];
  __shared__ __align__(4) unsigned char s_axis[64];
  const int tid = threadIdx.x, i = tid % TPR;
  if (tid < 64) {
    s_turns[tid] = p.rope.turns[tid];
    s_axis[tid] = p.rope.axis[tid];
  }
  __syncthreads();

  const int rot = p.rope.rotary, half = rot / 2;
  const bool turns = 8 * i < rot;                    // (rotary_dim is a multiple of 8: all of a lane's pairs or none)
  const int lo = INTER || !turns ? 8 * i : 4 * i, hi = INTER || !turns ? 8 * i + 4 : half + 4 * i;   // the lane's elements: four from each
  const int heads = p.q_heads + p.kv_heads * (FMT == kRopeRows ? 1 : 2), groups = (heads + U - 1) / U;

  // Units: (TOKS tokens, U of their heads).
  const int who = TOKS > 1 ? __shfl_sync(0xffffffffu, tid >> 5, 0) : tid / TPR;
  const long long unit = static_cast<long long>(blockIdx.x) * TAKERS + who, stride = static_cast<long long>(gridDim.x) * TAKERS;
  const int step_tok = static_cast<int>(stride / groups), step_grp = static_cast<int>(stride - static_cast<long long>(step_tok) * groups);
  long long tok = unit / groups;
  int grp = static_cast<int>(unit - tok * groups);
  tok = tok * TOKS + (TOKS > 1 ? (tid & 31) / TPR : 0);

  pdl_wait_then_release();

  // Teams of a warp stay together: the shuffles below need all of its lanes.
  const long long first_of_warp = TOKS > 1 ? unit : static_cast<long long>(blockIdx.x) * TAKERS + (tid & ~31) / TPR;
  const long long units = static_cast<long long>((p.n + TOKS - 1) / TOKS) * groups;
  for (long long w = first_of_warp; w < units; w += stride) {
    const bool live = tok < p.n;
    uint2 x[U][2];
    int kind[U];                                     // 0: q, 1: k, 2: v, 3: none
    int head[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      int h = grp * U + u;
      kind[u] = live && h < heads ? 0 : 3;
      const uint16_t* from = p.q + tok * p.q_stride;
      if (h >= p.q_heads && kind[u] == 0) {
        h -= p.q_heads;
        kind[u] = 1;
        from = p.k + tok * p.k_stride;
        if (FMT != kRopeRows && h >= p.kv_heads) {
          h -= p.kv_heads;
          kind[u] = 2;
          from = p.v + tok * p.v_stride;
        }
      }
      head[u] = h;
      x[u][0] = x[u][1] = make_uint2(0, 0);
      if (kind[u] != 3) {
        x[u][0] = *reinterpret_cast<const uint2*>(from + h * D + lo);
        x[u][1] = *reinterpret_cast<const uint2*>(from + h * D + hi);
      }
    }
    long long at = -1;
    if constexpr (FMT != kRopeRows)
      if (live && grp * U + U > p.q_heads) at = __ldg(p.slots + tok);
    // Sine and cosine of the lane's four pairs.
    float sn[4], cs[4];
    if (live && turns && grp * U < p.q_heads + p.kv_heads) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int pos = __ldg(p.positions + s_axis[4 * i + j] * p.position_stride + tok);
        const unsigned long long a = s_turns[4 * i + j] * static_cast<unsigned long long>(static_cast<long long>(pos));
        const float t = static_cast<float>(static_cast<int>(a >> 32)) * 1.4629180792671596e-9f;   // 2 pi 2^-32
        sn[j] = __sinf(t);
        cs[j] = __cosf(t);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) sn[j] = 0.f, cs[j] = 1.f;
    }
    int page = 0, slot = 0;
    bool stored = false;
    if constexpr (FMT != kRopeRows) stored = locate(p.c, p.page_shift, at, page, slot);

#pragma unroll
    for (int u = 0; u < U; ++u) {
      float f[4], g[4];
      unpack4(x[u][0], f);
      unpack4(x[u][1], g);
      if (kind[u] < 2) {
        const uint16_t* const norm = kind[u] == 0 ? p.q_norm : p.k_norm;
        if (norm) {                                  // (the same for the whole team)
          float sum = 0.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) sum = __fmaf_rn(f[j], f[j], __fmaf_rn(g[j], g[j], sum));
          const uint32_t team = TPR == 32 ? 0xffffffffu : ((1u << TPR) - 1) << ((tid & 31) & ~(TPR - 1));
#pragma unroll
          for (int o = TPR / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(team, sum, o);
          const float r = rsqrtf(__fmaf_rn(sum, 1.f / D, p.eps));
          float a[4], b[4];
          unpack4(__ldg(reinterpret_cast<const uint2*>(norm + lo)), a);
          unpack4(__ldg(reinterpret_cast<const uint2*>(norm + hi)), b);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            f[j] *= r * a[j];
            g[j] *= r * b[j];
          }
        }
        if (turns) {
          if constexpr (INTER) {
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
              const float f0 = f[j], g0 = g[j];
              f[j] = f0 * cs[j / 2] - f[j + 1] * sn[j / 2];
              f[j + 1] = f[j + 1] * cs[j / 2] + f0 * sn[j / 2];
              g[j] = g0 * cs[2 + j / 2] - g[j + 1] * sn[2 + j / 2];
              g[j + 1] = g[j + 1] * cs[2 + j / 2] + g0 * sn[2 + j / 2];
            }
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float f0 = f[j];
              f[j] = f0 * cs[j] - g[j] * sn[j];
              g[j] = g[j] * cs[j] + f0 * sn[j];
            }
          }
        }
      }
      if (kind[u] == 0 || (FMT == kRopeRows && kind[u] == 1)) {
        uint16_t* const to = (kind[u] == 0 ? p.q_out + tok * p.q_out_stride : p.k_out + tok * p.k_out_stride) + head[u] * D;
        *reinterpret_cast<uint2*>(to + lo) = pack4(f);
        *reinterpret_cast<uint2*>(to + hi) = pack4(g);
      }
      if constexpr (FMT != kRopeRows) {
        if (kind[u] == 1 || kind[u] == 2) {
          unsigned char* const to = (kind[u] == 1 ? p.c.k : p.c.v) + page * p.c.page_bytes + head[u] * p.c.head_bytes + slot * p.c.token_bytes;
          if constexpr (FMT == kKvBf16) {
            if (stored) {
              *reinterpret_cast<uint2*>(to + 2 * lo) = pack4(f);
              *reinterpret_cast<uint2*>(to + 2 * hi) = pack4(g);
            }
          } else {
            // Largest magnitude, as bits: NaN and infinities are above every number.
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) m = max(m, max(__float_as_uint(f[j]) & 0x7fffffffu, __float_as_uint(g[j]) & 0x7fffffffu));
            const uint32_t team = TPR == 32 ? 0xffffffffu : ((1u << TPR) - 1) << ((tid & 31) & ~(TPR - 1));
#pragma unroll
            for (int o = TPR / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(team, m, o));
            const bool finite = m < 0x7f800000u;
            const float amax = __uint_as_float(m);
            // The divisions Q / a and a / Q as a reciprocal and products: every lane has the factor, without a division.
            const float inv = finite && amax >= kZeroRow ? __fmul_rn(kv_qmax<FMT>(), __frcp_rn(amax)) : 0.f;
            if (stored) {
              *reinterpret_cast<uint32_t*>(to + lo) = inv != 0.f ? quantise4<FMT>(f, inv) : 0u;   // (not finite, or all but zero: codes of zero)
              *reinterpret_cast<uint32_t*>(to + hi) = inv != 0.f ? quantise4<FMT>(g, inv) : 0u;
              if (i == 0)
                (kind[u] == 1 ? p.c.ks : p.c.vs)[scale_index(p.c, page, head[u], slot)] =
                    !finite ? __int_as_float(0x7fffffff) : inv != 0.f ? __fmul_rn(amax, 1.f / kv_qmax<FMT>()) : 0.f;
            }
          }
        }
      }
    }
    tok += static_cast<long long>(step_tok) * TOKS;
    grp += step_grp;
    if (grp >= groups) {
      grp -= groups;
      tok += TOKS;
    }
  }
}

namespace {

template <int FMT, int D, bool INTER, int U>
int launch_units(const RopeArgs& a, void* stream) {
  constexpr int TOKS = RopeUnits<D, U>::tokens, TAKERS = RopeUnits<D, U>::takers;
  const long long heads = a.q_heads + a.kv_heads * (FMT == kRopeRows ? 1LL : 2LL), units = (heads + U - 1) / U * ((a.n + TOKS - 1) / TOKS);
  const long long blocks = (units + TAKERS - 1) / TAKERS;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks < 152 * 8 * 4 ? blocks : 152 * 8 * 4), 1, 1);
  cfg.blockDim = dim3(kRopeThreads, 1, 1);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return static_cast<int>(cudaLaunchKernelEx(&cfg, rope_kernel<FMT, D, INTER, U>, a));
}

template <int FMT, int D, bool INTER>
int launch_one(const RopeArgs& a, void* stream) {
  // kHeads heads a team once that still gives every SM its 2048 threads.
  const long long lanes = (a.q_heads + a.kv_heads * (FMT == kRopeRows ? 1LL : 2LL)) * a.n * (D / 8);
  return lanes >= 152LL * 2048 * kHeads ? launch_units<FMT, D, INTER, kHeads>(a, stream) : launch_units<FMT, D, INTER, 1>(a, stream);
}

template <int FMT>
int launch_format(const RopeArgs& a, void* stream) {
  if (a.head_dim == 128) return a.rope.interleaved ? launch_one<FMT, 128, true>(a, stream) : launch_one<FMT, 128, false>(a, stream);
  return a.rope.interleaved ? launch_one<FMT, 64, true>(a, stream) : launch_one<FMT, 64, false>(a, stream);
}

}  // namespace

int launch_rope(const RopeArgs& a, void* stream) {
  switch (a.format) {
    case kRopeRows: return launch_format<kRopeRows>(a, stream);
    case kKvBf16: return launch_format<kKvBf16>(a, stream);
    case kKvE4m3: return launch_format<kKvE4m3>(a, stream);
    default: return launch_format<kKvInt8>(a, stream);
  }
}

}  // namespace glora
