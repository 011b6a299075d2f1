// Attention of one new token per sequence over the paged cache (sm_103a).
//
// For sequence b and the G query heads that share key-value head h:
//   z[g, t] = scale (q_g . k_t),  out_g = sum_t softmax(z_g)_t v_t.
// With up to 16 query heads a group every cached byte is read once per call (2 G multiply-adds per element), so
// HBM bandwidth bounds the kernel; what it needs is enough bytes in flight on every SM and an even share of the
// batch's tokens for each, whatever the lengths are. Larger groups read it once for each block of 16 heads. The 8-bit formats are bound by instruction issue before
// that: 840 a warp and 8 KB tile (E4M3), 470 in BF16, with two warps a scheduler (registers).
//
// Measured on a GB300: 128 contexts to 16384 (8 key-value heads of 128, BF16) 733 us, 6.9 TB/s; 32 to 4096
// 58.8 us, 5.8 TB/s; 64 to 8191 (4 heads, E4M3) 65.7 us, 5.3 TB/s; 5 to 100003 (16 heads of 64, INT8) 128 us,
// 4.8 TB/s; one of 100000 with one key-value head (BF16, 304 parts in 19 groups) 20.4 us; one of 700 tokens 9.2 us,
// all latency: plan 1.2, first loads 1, tile 0.6, join 3.
//
// Split. The work unit is a tile of kTile tokens of one segment: a segment is (sequence, key-value
// head, block of 16 query heads). All tiles of the batch, segment after segment, are cut into equal
// contiguous ranges, one per CTA (two CTAs per SM; fewer CTAs when there would be less than one tile
// for each warp); ends that fall into a segment of at most kWhole tiles move to its nearer end, as
// joining its parts takes longer than the few tiles. A range is walked piece by piece (a piece: its part of one segment). A piece that is
// a whole segment is finished by its CTA; otherwise the CTA stores (maximum, sum, unnormalised output)
// in the workspace and the last CTA of the segment to arrive joins them in CTA order, so the bits never
// depend on who was last. Segments over many CTAs join in two levels (kJoinGroup).
//
// Tile. A warp streams its own tiles (every kDecWarps-th of a piece) through a ring of kStages 8 KB stages of
// cp.async copies that runs on across pieces; the CTA's warps join once per piece. On the tensor cores
// (mma.sync m16n8k16) the 16 rows of A are the query heads, so the scores' accumulator layout is the
// layout of A in the product with V. Running maximum m and sum l per row as usual.
//
// 8-bit formats. K's codes become f16 pairs in registers (exact: E4M3 and integers to 127 fit f16's 11
// bits; Q is scaled by a power of two into f16's range). V's become TF32, exact too, with the weights: K's scale
// multiplies the score but V's the weight, p_t s_t, so weights may span any range (TF32 has fp32's) and even
// a single token's must not be rounded to 8 bits (BF16 weights measured 1.5 times the error of rounding the
// result alone, and more instructions: the codes come out of their conversions in fp32). A lane's 4
// consecutive code bytes of K are 4 consecutive dimensions, so the dimensions of Q are dealt to the MMA's k
// index in that order; V is read transposed as byte pairs and split into even and odd dimensions.
//
// Rounding to fewer bits: softmax weights before they multiply V, to BF16 (BF16 cache: the tensor cores take
// operands of one type) or TF32 (8-bit); sums and statistics are fp32; the output rounds once to BF16.
#include "attn_common.cuh"

namespace glora {

namespace {

constexpr int kDecWarps = 4;
constexpr int kDecThreads = kDecWarps * 32;
constexpr int kStages = 3;
constexpr int kHalfStage = 4096;                 // bytes of K (and of V) in a stage
constexpr int kCtasPerSm = 2;
constexpr int kJoinGroup = 16;                   // partial results in a group of the first level, in flight together in a join
constexpr int kMaxCtas = 512;                    // counters in the workspace
constexpr int kJoinMost = kMaxCtas / kJoinGroup; // parts of one join: the groups of a segment over all CTAs
static_assert(kMaxCtas % kJoinGroup == 0 && kJoinMost >= kJoinGroup, "a join holds a whole group, and all groups of a segment");
constexpr int kWhole = 2 * kDecWarps;            // segments of at most this many tiles are not divided
constexpr int kRows = 16;                        // query heads of a segment

// Workspace: counters [3][kMaxCtas] (a segment's first join group, by its first CTA; its other groups, by
// theirs: that CTA may also start the next segment; its groups together), then 2 slots per CTA of m[16],
// l[16], O[16][D].
constexpr int kCounterBytes = 3 * kMaxCtas * 4;
template <int D>
constexpr int kSlotFloats = 2 * kRows + kRows * D;
static_assert(kCounterBytes + 2LL * kMaxCtas * kSlotFloats<128> * 4 <= (16 << 20), "workspace");

template <int FMT, int D>
struct Tile {
  static constexpr int row_bytes = D * (FMT == kKvBf16 ? 2 : 1);
  static constexpr int chunks = row_bytes / 16;               // 16-byte chunks of a token's row
  static constexpr int tokens = kHalfStage / row_bytes;       // 16, 32 or 64
  static constexpr int per_lane = (tokens + 31) / 32;         // tokens whose page a lane looks up
  static constexpr int scale_bytes = FMT == kKvBf16 ? 0 : 2 * tokens * 4;
  static constexpr int stage_bytes = 2 * kHalfStage + scale_bytes;
  // Shared address of chunk c of token row t: chunks permuted by the row so that the 8 rows of a
  // matrix load fall into different banks.
  static __device__ __forceinline__ uint32_t at(int t, int c) {
    return t * row_bytes + ((c ^ (chunks >= 8 ? (t & 7) : ((t >> 1) & 3))) << 4);
  }
};

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
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

// Four codes -> fp32 (low byte first), by way of f16: its unpacking runs beside the ALU (INT8, 5 contexts to 100003, 144.9 -> 140.9 us).
template <int FMT>
__device__ __forceinline__ void codes_to_tf32(uint32_t c, uint32_t (&v)[4]) {
  uint32_t lo, hi;
  codes_to_f16<FMT>(c, lo, hi);
  const float2 x = f16x2_to_f32(lo), y = f16x2_to_f32(hi);
  v[0] = __float_as_uint(x.x);
  v[1] = __float_as_uint(x.y);
  v[2] = __float_as_uint(y.x);
  v[3] = __float_as_uint(y.y);
}
// fp32 rounded to TF32's 11 significant bits.
__device__ __forceinline__ uint32_t to_tf32(float f) {
  uint32_t r;
  asm("cvt.rna.tf32.f32 %0, %1;\n" : "=r"(r) : "f"(f));
  return r;
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

// The batch's segments in order: where a walk stands, and how it goes on.
struct Walk {
  int b, sub;          // sequence; key-value head * blocks + block of 16 query heads
  int tiles;           // tiles of sequence b
  int len;
};

template <int TOK>
__device__ __forceinline__ int tiles_of(const DecodeArgs& p, int b, int& len) {
  const long long most = static_cast<long long>(p.max_pages) * p.c.page_size;
  len = static_cast<int>(min(static_cast<long long>(max(p.lens[b], 0)), most));
  return (len - 1) / TOK + (len > 0 ? 1 : 0);
}

// a * b / d, in 32 bits where the product fits (a 64-bit division is a call of a hundred instructions).
__device__ __forceinline__ long long mul_div(long long a, long long b, long long d) {
  const unsigned long long ab = static_cast<unsigned long long>(a) * static_cast<unsigned long long>(b);
  if (((ab | static_cast<unsigned long long>(d)) >> 32) == 0) return static_cast<uint32_t>(ab) / static_cast<uint32_t>(d);
  return static_cast<long long>(ab / static_cast<unsigned long long>(d));
}

// Next segment that has tiles (the caller knows there is one).
template <int TOK>
__device__ __forceinline__ void next_segment(const DecodeArgs& p, int subs, Walk& w) {
  if (++w.sub < subs) return;
  w.sub = 0;
  do ++w.b, w.tiles = tiles_of<TOK>(p, w.b, w.len);
  while (w.tiles == 0);
}

}  // namespace

// HALF: at most 8 query heads share a key-value head (the lower 8 rows of a tile are unused).
template <int FMT, int D, bool HALF>
__global__ void __launch_bounds__(kDecThreads, kCtasPerSm) decode_kernel(const DecodeArgs p) {
  using T = Tile<FMT, D>;
  constexpr int TOK = T::tokens, NT = TOK / 8, KS = D / 16, R = HALF ? 1 : 2;
  constexpr int PL = T::per_lane;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ long long s_sum[kDecWarps], s_u[2];
  __shared__ int s_b, s_sub, s_tiles, s_len, s_tile0, s_last;
  __shared__ float s_m[kDecWarps][kRows], s_l[kDecWarps][kRows];
  __shared__ float s_jm[kJoinMost * kRows], s_jl[kJoinMost * kRows];
  __shared__ uint64_t s_live[kDecWarps][kStages];     // valid tokens of each stage
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, qd = lane & 3;
  float* const s_o = reinterpret_cast<float*>(smem + kDecWarps * kStages * T::stage_bytes);   // two buffers of D / 8 / R accumulator tiles

  pdl_wait_then_release();

  const int G = p.q_heads / p.c.kv_heads, blocks = (G + kRows - 1) / kRows, subs = p.c.kv_heads * blocks;
  // Sequences without tokens: zeros.
  auto zero_empty = [&]() {
    for (int b = blockIdx.x; b < p.batch; b += gridDim.x) {
      int len;
      if (tiles_of<TOK>(p, b, len) > 0) continue;
      for (int i = tid; i < p.q_heads * D / 8; i += kDecThreads)
        *reinterpret_cast<uint4*>(p.out + b * p.out_stride + i * 8) = make_uint4(0, 0, 0, 0);
      if (p.lse)
        for (int i = tid; i < p.q_heads; i += kDecThreads) p.lse[static_cast<long long>(b) * p.q_heads + i] = -INFINITY;
    }
  };

  // The batch's tiles, and this CTA's range [u0, u1) of them.
  const int per = (p.batch + kDecThreads - 1) / kDecThreads, b0 = min(tid * per, p.batch), b1 = min(b0 + per, p.batch);
  long long mine = 0, before, total = 0;
  for (int b = b0; b < b1; ++b) {
    int len;
    mine += tiles_of<TOK>(p, b, len);
  }
  before = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += t;
  }
  if (lane == 31) s_sum[warp] = before;
  before -= mine;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kDecWarps; ++w) {
    if (w < warp) before += s_sum[w];
    total += s_sum[w];
  }
  before *= subs;
  mine *= subs;
  total *= subs;
  const long long n = min(static_cast<long long>(gridDim.x), (total + kDecWarps - 1) / kDecWarps);   // CTAs with work
  const int c = blockIdx.x;
  if (c >= n) {
    zero_empty();
    return;
  }
  // Ends of the range: equal shares, moved to the nearer end of a segment of at most kWhole tiles.
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    long long u = mul_div(c + e, total, n);
    if (u < before || u >= before + mine) continue;   // another thread's sequences hold it
    long long at = before;
    for (int b = b0; b < b1; ++b) {
      int len;
      const int t = tiles_of<TOK>(p, b, len);
      const long long span = static_cast<long long>(t) * subs;
      if (u < at + span) {
        const int sub = static_cast<int>(mul_div(u - at, 1, t));
        int tile = static_cast<int>(u - at - static_cast<long long>(sub) * t);
        if (t <= kWhole) {
          const int to = 2 * tile < t ? 0 : t;
          u += to - tile;
          tile = to;
        }
        s_u[e] = u;
        if (e == 0) {
          s_b = b;
          s_tiles = t;
          s_len = len;
          s_sub = sub;
          s_tile0 = tile;
        }
        break;
      }
      at += span;
    }
  }
  __syncthreads();
  const long long u0 = s_u[0], u1 = c + 1 < n ? s_u[1] : total;
  if (u0 >= u1) {
    zero_empty();
    return;
  }
  Walk start{s_b, s_sub, s_tiles, s_len};
  int start_tile = s_tile0;
  if (start_tile == start.tiles) {
    next_segment<TOK>(p, subs, start);
    start_tile = 0;
  }

  const uint32_t ring = smem_u32(smem) + warp * kStages * T::stage_bytes;
  const unsigned char* const ring_ptr = smem + warp * kStages * T::stage_bytes;

  // Q of a segment as A fragments (raw BF16 pairs): loaded ahead of the copies, and for the next piece before
  // the join of the one before.
  uint32_t qa[KS][2 * R];
  auto load_q = [&](const Walk& at) {
    const int head = at.sub / blocks, first = head * G + (at.sub - head * blocks) * kRows, rows = min(kRows, head * G + G - first);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int row = g + 8 * r;
      const uint16_t* q = p.q + at.b * p.q_stride + (first + row) * D;
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int d = FMT == kKvBf16 ? k * 16 + j * 8 + qd * 2 : k * 16 + qd * 4 + j * 2;
          qa[k][j * R + r] = row < rows ? __ldg(reinterpret_cast<const uint32_t*>(q + d)) : 0u;
        }
    }
  };
  load_q(start);

  // ---- loads: a cursor over this warp's tiles, two tiles ahead of the copies in its page look-ups
  Walk lw = start;
  long long lu = u0;                       // first unit of the cursor's piece
  int lt0 = start_tile, lt1 = static_cast<int>(min(static_cast<long long>(lw.tiles), start_tile + (u1 - u0)));
  int lt = lt0 + warp;
  bool more = true;
  struct Ahead {                           // a tile to copy: its tokens' pages and slots, its head
    int page[PL], slot[PL], head;
    bool is;
  } next{}, after{};
  auto settle = [&]() {                    // to the next tile of this warp, or the end
    while (lt >= lt1) {
      lu += lt1 - lt0;
      if (lu >= u1) {
        more = false;
        return;
      }
      next_segment<TOK>(p, subs, lw);
      lt0 = 0;
      lt1 = static_cast<int>(min(static_cast<long long>(lw.tiles), u1 - lu));
      lt = warp;
    }
  };
  auto look_up = [&](Ahead& t) {            // the cursor's tile, then the cursor moves on
    t.is = more;
    if (!more) return;
    t.head = lw.sub / blocks;
#pragma unroll
    for (int j = 0; j < PL; ++j) {
      const int i = lane + 32 * j, at = lt * TOK + i;
      t.page[j] = -1;
      t.slot[j] = 0;
      if (i < TOK && at < lw.len) {
        const int e = p.page_shift >= 0 ? at >> p.page_shift : at / p.c.page_size;
        t.slot[j] = at - e * p.c.page_size;
        t.page[j] = __ldg(p.table + lw.b * p.table_stride + e);
      }
    }
    lt += kDecWarps;
    settle();
  };
  auto load = [&](int s) {                 // the next tile into stage s
    if (next.is) {
      const uint32_t st = ring + s * T::stage_bytes;
      const int head = next.head;
      long long off[PL];
      uint64_t live = 0;
#pragma unroll
      for (int j = 0; j < PL; ++j) {
        const int page = next.page[j], slot = next.slot[j];
        const bool ok = page >= 0 && page < p.c.num_pages;
        off[j] = ok ? page * p.c.page_bytes + head * p.c.head_bytes + slot * p.c.token_bytes : -1;
        live |= static_cast<uint64_t>(__ballot_sync(0xffffffffu, ok)) << (32 * j);
        if constexpr (FMT != kKvBf16) {
          const long long si = ok ? scale_index(p.c, page, head, slot) : 0;
          const uint32_t to = st + 2 * kHalfStage + (lane + 32 * j) * 4;
          cp_async4_n(to, p.c.ks + si, ok ? 4 : 0);
          cp_async4_n(to + TOK * 4, p.c.vs + si, ok ? 4 : 0);
        }
      }
      if (lane == 0) s_live[warp][s] = live;
      constexpr int RPI = 32 / T::chunks;  // token rows per copy instruction
#pragma unroll
      for (int i = 0; i < TOK / RPI; ++i) {
        const int t = i * RPI + lane / T::chunks, ch = lane % T::chunks;
        const long long o = __shfl_sync(0xffffffffu, off[(i * RPI) / 32], t & 31);
        const uint32_t to = st + T::at(t, ch);
        const long long from = (o < 0 ? 0 : o) + ch * 16;
        cp_async16_n(to, p.c.k + from, o < 0 ? 0 : 16);
        cp_async16_n(to + kHalfStage, p.c.v + from, o < 0 ? 0 : 16);
      }
      next = after;
      look_up(after);
    }
    cp_async_commit();
  };
  settle();
  look_up(next);
  look_up(after);
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) load(s);

  // ---- pieces
  Walk w = start;
  int ta = start_tile, it = 0;
  for (long long u = u0; u < u1;) {
    const int tb = static_cast<int>(min(static_cast<long long>(w.tiles), ta + (u1 - u)));
    const int head = w.sub / blocks, h0 = head * G + (w.sub - head * blocks) * kRows;
    const int rows = min(kRows, head * G + G - h0);

    // Scores come out in units of zscale (base-2 exponents).
    float zscale[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      zscale[r] = p.scale * kLog2e;
      if constexpr (FMT != kKvBf16) {      // BF16 -> f16, the row's largest magnitude at 2^14 .. 2^15
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t v = qa[k][j * R + r];
            top = max(top, max(v & 0x7fffu, (v >> 16) & 0x7fffu));
          }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // factor 2^(14 - e) of the exponent e; rows of zeros (or not finite) are taken as they are
        const int e = static_cast<int>(top >> 7) - 127;
        const int up = top == 0 || e == 128 ? 0 : max(-126, min(126, 14 - e));
        const float f = __int_as_float((127 + up) << 23);
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t v = qa[k][j * R + r];
            qa[k][j * R + r] = pack_f16x2(__uint_as_float(v << 16) * f, __uint_as_float(v & 0xffff0000u) * f);
          }
        zscale[r] *= __int_as_float((127 - up) << 23);
      }
    }

    constexpr int OT = HALF ? D / 16 : D / 8;
    float o[OT][4], m[R], l[R];
#pragma unroll
    for (int i = 0; i < OT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
    }

    for (int t = ta + warp; t < tb; t += kDecWarps, ++it) {
      const int s = it % kStages;
      cp_async_wait_n<kStages - 2>();
      __syncwarp();
      load((it + kStages - 1) % kStages);
      const uint32_t sk = ring + s * T::stage_bytes, sv = sk + kHalfStage;
      const float* const sc = reinterpret_cast<const float*>(ring_ptr + s * T::stage_bytes + 2 * kHalfStage);
      const uint64_t live = s_live[warp][s];

      // scores [16 heads][TOK tokens]
      float z[NT][4];
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        z[i][0] = z[i][1] = z[i][2] = z[i][3] = 0.f;
        if constexpr (FMT == kKvBf16) {
#pragma unroll
          for (int k = 0; k < KS; k += 2) {
            uint32_t b0, b1, b2, b3;
            ldsm_x4(sk + T::at(i * 8 + (lane & 7), k * 2 + (lane >> 3)), b0, b1, b2, b3);
            mma_k16(z[i], qa[k][0], HALF ? 0u : qa[k][R - 1], qa[k][R], HALF ? 0u : qa[k][2 * R - 1], b0, b1);
            mma_k16(z[i], qa[k + 1][0], HALF ? 0u : qa[k + 1][R - 1], qa[k + 1][R], HALF ? 0u : qa[k + 1][2 * R - 1], b2, b3);
          }
        } else {
#pragma unroll
          for (int k = 0; k < KS; k += 4) {
            uint32_t c[4];
            ldsm_x4(sk + T::at(i * 8 + (lane & 7), k + (lane >> 3)), c[0], c[1], c[2], c[3]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t b0, b1;
              codes_to_f16<FMT>(c[j], b0, b1);
              mma_f16(z[i], qa[k + j][0], HALF ? 0u : qa[k + j][R - 1], qa[k + j][R], HALF ? 0u : qa[k + j][2 * R - 1], b0, b1);
            }
          }
        }
      }
      // to base-2 exponents, masked; running maximum
      float mt[R];
#pragma unroll
      for (int r = 0; r < R; ++r) mt[r] = -INFINITY;
      const bool whole = live == (TOK == 64 ? ~0ull : (1ull << (TOK & 63)) - 1);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        float2 ks = make_float2(1.f, 1.f);
        if constexpr (FMT != kKvBf16) ks = *reinterpret_cast<const float2*>(sc + i * 8 + qd * 2);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          z[i][2 * r] *= zscale[r] * ks.x;
          z[i][2 * r + 1] *= zscale[r] * ks.y;
          if (!whole) {
            const uint32_t bits = static_cast<uint32_t>(live >> (i * 8 + qd * 2));
            if (!(bits & 1)) z[i][2 * r] = -INFINITY;
            if (!(bits & 2)) z[i][2 * r + 1] = -INFINITY;
          }
          mt[r] = fmaxf(mt[r], fmaxf(z[i][2 * r], z[i][2 * r + 1]));
        }
      }
      float keep[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float mn = fmaxf(m[r], quad_max(mt[r]));
        const float ref = mn == -INFINITY ? 0.f : mn;    // nothing seen so far: every weight is 0
        keep[r] = exp2_fast(m[r] - ref);
        m[r] = mn;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float w0 = exp2_fast(z[i][2 * r + j] - ref);
            sum += w0;
            z[i][2 * r + j] = FMT == kKvBf16 ? w0 : w0 * sc[TOK + i * 8 + qd * 2 + j];
          }
        l[r] = l[r] * keep[r] + sum;
      }
      if (__any_sync(0xffffffffu, keep[0] != 1.f || (!HALF && keep[R - 1] != 1.f))) {
        // (HALF: accumulator columns are heads 2 qd, 2 qd + 1, whose factors lanes 8 qd, 8 qd + 4 hold)
        float kx[2] = {keep[0], keep[R - 1]};
        if constexpr (HALF) {
          kx[0] = __shfl_sync(0xffffffffu, keep[0], qd * 8);
          kx[1] = __shfl_sync(0xffffffffu, keep[0], qd * 8 + 4);
        }
#pragma unroll
        for (int i = 0; i < OT; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[i][j] *= kx[HALF ? j & 1 : j >> 1];
      }
      // O += P V; with at most 8 heads O^T += V^T P^T instead, the same registers the other way round: dimensions
      // are the MMA's 16 rows and the heads its 8 columns, half as many MMAs and accumulators (E4M3 72.9 -> 66.2 us, INT8
      // 141 -> 126.6 in the cases above).
#pragma unroll
      for (int k = 0; k < TOK / 16; ++k) {
        if constexpr (FMT == kKvBf16) {
          const uint32_t a0 = pack_bf16x2(z[2 * k][0], z[2 * k][1]), a2 = pack_bf16x2(z[2 * k + 1][0], z[2 * k + 1][1]);
          const uint32_t a1 = HALF ? 0u : pack_bf16x2(z[2 * k][2], z[2 * k][3]);
          const uint32_t a3 = HALF ? 0u : pack_bf16x2(z[2 * k + 1][2], z[2 * k + 1][3]);
#pragma unroll
          for (int i = 0; i < D / 8; i += 2) {
            uint32_t b0, b1, b2, b3;
            ldsm_x4_t(sv + T::at(k * 16 + (lane & 15), i + (lane >> 4)), b0, b1, b2, b3);
            if constexpr (HALF) {
              mma_k16(o[i / 2], b0, b2, b1, b3, a0, a2);
            } else {
              mma_k16(o[i], a0, a1, a2, a3, b0, b1);
              mma_k16(o[i + 1], a0, a1, a2, a3, b2, b3);
            }
          }
        } else {
          // The MMA's k index q, q + 4 is token 2q, 2q + 1 of a group of 8: the scores' own layout.
          uint32_t a[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int x = 0; x < 4; ++x)      // (row g, g + 8) x (token 2q, 2q + 1)
              a[h][x] = HALF && (x & 1) ? 0u : to_tf32(z[2 * k + h][2 * (x & 1) + (x >> 1)]);
#pragma unroll
          for (int i = 0; i < D / 16; i += 2) {
            uint32_t c[4];                   // (tokens 0-7, 8-15) of 16-dimension blocks i and i + 1
            ldsm_x4_t(sv + T::at(k * 16 + (lane & 15), i + (lane >> 4)), c[0], c[1], c[2], c[3]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              // bytes of a register: token 2 qd: dimensions 2g, 2g + 1; token 2 qd + 1: the same
              uint32_t v[4];
              codes_to_tf32<FMT>(c[j], v);
              const uint32_t(&w)[4] = a[j & 1];
              if constexpr (HALF) {
                mma_tf32(o[i + (j >> 1)], v[0], v[1], v[2], v[3], w[0], w[2]);
              } else {
                mma_tf32(o[2 * (i + (j >> 1))], w[0], w[1], w[2], w[3], v[0], v[2]);
                mma_tf32(o[2 * (i + (j >> 1)) + 1], w[0], w[1], w[2], w[3], v[1], v[3]);
              }
            }
          }
        }
      }
    }
    u += tb - ta;
    Walk nw = w;
    if (u < u1) {
      next_segment<TOK>(p, subs, nw);
      load_q(nw);
    }

    // ---- join the warps: (m, l) of each row, then O in two steps through two buffers
#pragma unroll
    for (int r = 0; r < R; ++r) {
      l[r] = quad_sum(l[r]);
      if (qd == 0) {
        s_m[warp][g + 8 * r] = m[r];
        s_l[warp][g + 8 * r] = l[r];
      }
    }
    __syncthreads();
    // Joined maximum and sum of this lane's two accumulator rows (HALF: columns), and this warp's factor.
    float mj[2], lj[2];
    int own[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      own[r] = HALF ? 2 * qd + r : g + 8 * r;
      mj[r] = -INFINITY;
      lj[r] = 0.f;
#pragma unroll
      for (int x = 0; x < kDecWarps; ++x) mj[r] = fmaxf(mj[r], s_m[x][own[r]]);
      const float ref = mj[r] == -INFINITY ? 0.f : mj[r];
#pragma unroll
      for (int x = 0; x < kDecWarps; ++x) lj[r] += s_l[x][own[r]] * exp2_fast(s_m[x][own[r]] - ref);
      const float f = exp2_fast(s_m[warp][own[r]] - ref);
#pragma unroll
      for (int i = 0; i < OT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if ((HALF ? j & 1 : j >> 1) == r) o[i][j] *= f;
    }
    // (16 rows go through the buffers in two halves of the dimensions)
    constexpr int NB = D / 16;
    auto buffer = [&](int x, int i, int j) -> float& { return s_o[(x * NB * 4 + i * 4 + j) * 32 + lane]; };
#pragma unroll
    for (int h = 0; h < R; ++h) {
#pragma unroll
      for (int step = kDecWarps / 2; step > 0; step >>= 1) {
        if (warp >= step && warp < 2 * step)
#pragma unroll
          for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) buffer(warp - step, i, j) = o[h * NB + i][j];
        __syncthreads();
        if (warp < step)
#pragma unroll
          for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[h * NB + i][j] += buffer(warp, i, j);
        if (step > 1 || h + 1 < R) __syncthreads();
      }
    }

    // ---- the piece's result: from warp 0 to [rows][D] fp32 in shared memory, then all threads take it
    if (warp == 0) {
      __syncwarp();
#pragma unroll
      for (int i = 0; i < OT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int row = own[HALF ? j & 1 : j >> 1];
          // HALF: dimensions g, g + 8 of block i (8-bit: 2g, 2g + 1); else 8 i + 2 qd, + 1 (8-bit: blocks of 16 as
          // (even, odd) pairs)
          int d;
          if constexpr (HALF) d = FMT == kKvBf16 ? 16 * i + g + 8 * (j >> 1) : 16 * i + 2 * g + (j >> 1);
          else d = FMT == kKvBf16 ? 8 * i + 2 * qd + (j & 1) : 16 * (i >> 1) + 4 * qd + 2 * (j & 1) + (i & 1);
          s_o[row * D + d] = o[i][j];
        }
      if (HALF ? g == 0 : qd == 0)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          s_jm[own[r]] = mj[r];
          s_jl[own[r]] = lj[r];
        }
    }
    __syncthreads();
    const bool complete = ta == 0 && tb == w.tiles;
    if (complete) {
      for (int i = tid; i < rows * D / 4; i += kDecThreads) {
        const int row = i / (D / 4), d = (i - row * (D / 4)) * 4;
        const float4 v = *reinterpret_cast<const float4*>(s_o + row * D + d);
        const float lr = s_jl[row], f = lr == 0.f ? 0.f : 1.f / lr;
        *reinterpret_cast<uint2*>(p.out + w.b * p.out_stride + (h0 + row) * D + d) =
            make_uint2(pack_bf16x2(v.x * f, v.y * f), pack_bf16x2(v.z * f, v.w * f));
        if (p.lse && d == 0)
          p.lse[static_cast<long long>(w.b) * p.q_heads + h0 + row] = lr == 0.f ? -INFINITY : (s_jm[row] + log2f(lr)) * kLn2;
      }
    } else {
      int* const counters = static_cast<int*>(p.workspace);
      float* const slots = reinterpret_cast<float*>(static_cast<unsigned char*>(p.workspace) + kCounterBytes);
      constexpr int SF = kSlotFloats<D>;
      float* const to = slots + static_cast<long long>(2 * c + (ta == 0)) * SF;
      if (tid < rows) {
        to[tid] = s_jm[tid];
        to[kRows + tid] = s_jl[tid];
      }
      for (int i = tid; i < rows * D / 4; i += kDecThreads)
        *reinterpret_cast<float4*>(to + 2 * kRows + 4 * i) = *reinterpret_cast<const float4*>(s_o + 4 * i);
      // The segment's CTAs c0 .. c1, in groups of kJoinGroup; slot of CTA x: its part either starts
      // the segment (x == c0: slot 2 x + 1) or goes on with it (slot 2 x).
      const long long s0 = u - tb, s1 = s0 + w.tiles - 1;
      auto cta_of = [&](long long unit) {   // the last x with x * total / n <= unit: ((unit + 1) n - 1) / total
        const long long v = (unit + 1) * n - 1;
        return static_cast<int>(mul_div(v, 1, total));
      };
      const int c0 = cta_of(s0), c1 = cta_of(s1);
      const int groups = (c1 - c0) / kJoinGroup + 1, gi = (c - c0) / kJoinGroup;
      // Joins slots first, first + step, .. (at most kJoinMost); the result goes to the output, or in place into
      // slot `first`. A thread's loads of kJoinGroup parts are in flight together: one trip to L2 for a group, two
      // for the groups of a segment over more than kJoinGroup^2 CTAs.
      auto join = [&](int first_cta, int count, int step, bool last) {
        auto slot_of = [&](int x) { return slots + static_cast<long long>(2 * x + (x == c0)) * SF; };
        for (int i = tid; i < count * kRows; i += kDecThreads) {
          const float* const from = slot_of(first_cta + (i / kRows) * step) + i % kRows;
          s_jm[i] = i % kRows < rows ? __ldcg(from) : -INFINITY;
          s_jl[i] = i % kRows < rows ? __ldcg(from + kRows) : 0.f;
        }
        __syncthreads();
        // thread: 4 consecutive dimensions of one row at a time
        for (int i = tid; i < rows * D / 4; i += kDecThreads) {
          const int row = i / (D / 4), d = (i - row * (D / 4)) * 4;
          float mm = -INFINITY, ref = 0.f, ll = 0.f;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
          for (int x0 = 0; x0 < count; x0 += kJoinGroup) {
            float4 v[kJoinGroup];
#pragma unroll
            for (int x = 0; x < kJoinGroup; ++x) {
              v[x] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (x0 + x < count)
                v[x] = __ldcg(reinterpret_cast<const float4*>(slot_of(first_cta + (x0 + x) * step) + 2 * kRows + row * D + d));
            }
            if (x0 == 0) {   // (while the first loads are under way)
              for (int x = 0; x < count; ++x) mm = fmaxf(mm, s_jm[x * kRows + row]);
              ref = mm == -INFINITY ? 0.f : mm;
            }
#pragma unroll
            for (int x = 0; x < kJoinGroup; ++x) {
              if (x0 + x < count) {
                const float f = exp2_fast(s_jm[(x0 + x) * kRows + row] - ref);
                ll += s_jl[(x0 + x) * kRows + row] * f;
                acc.x += v[x].x * f;
                acc.y += v[x].y * f;
                acc.z += v[x].z * f;
                acc.w += v[x].w * f;
              }
            }
          }
          if (last) {
            const float f = ll == 0.f ? 0.f : 1.f / ll;
            *reinterpret_cast<uint2*>(p.out + w.b * p.out_stride + (h0 + row) * D + d) =
                make_uint2(pack_bf16x2(acc.x * f, acc.y * f), pack_bf16x2(acc.z * f, acc.w * f));
            if (p.lse && d == 0)
              p.lse[static_cast<long long>(w.b) * p.q_heads + h0 + row] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
          } else {
            float* const to = slot_of(first_cta);
            *reinterpret_cast<float4*>(to + 2 * kRows + row * D + d) = acc;
            if (d == 0) {   // (m and l were read before the barrier above)
              to[row] = mm;
              to[kRows + row] = ll;
            }
          }
        }
      };
      // Arrive at a counter; true in the CTA that is the last of `count`, which sets it back to 0.
      auto last_of = [&](int* counter, int count) {
        __syncthreads();
        if (tid == 0) {   // releases the CTA's writes before the barrier, acquires those of the CTAs before it
          int seen;
          asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;\n" : "=r"(seen) : "l"(counter) : "memory");
          s_last = seen == count - 1;
          if (s_last) *counter = 0;
        }
        __syncthreads();
        return s_last != 0;
      };
      const int first = c0 + gi * kJoinGroup, count = min(kJoinGroup, c1 - first + 1);
      if (last_of(counters + (gi ? kMaxCtas : 0) + first, count)) {
        join(first, count, 1, groups == 1);
        if (groups > 1 && last_of(counters + 2 * kMaxCtas + c0, groups)) join(c0, groups, kJoinGroup, true);
      }
    }
    w = nw;
    ta = 0;
    __syncthreads();
  }
  cp_async_wait_n<0>();
  zero_empty();
}

namespace {

template <int FMT, int D, bool HALF>
int launch_one(const DecodeArgs& a, void* stream) {
  using T = Tile<FMT, D>;
  constexpr int smem = kDecWarps * kStages * T::stage_bytes + (kDecWarps / 2) * (D / 8) * 2 * 32 * 4;
  const auto kernel = decode_kernel<FMT, D, HALF>;
  // (set on every call: the attribute belongs to the current device, like the launch)
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  int dev = 0, sms = 0;
  if (e == cudaSuccess) e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return static_cast<int>(e);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(sms * kCtasPerSm < kMaxCtas ? sms * kCtasPerSm : kMaxCtas), 1, 1);
  cfg.blockDim = dim3(kDecThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return static_cast<int>(cudaLaunchKernelEx(&cfg, kernel, a));
}

template <int FMT>
int launch_format(const DecodeArgs& a, void* stream) {
  const bool half = a.q_heads / a.c.kv_heads <= 8;
  if (a.head_dim == 128) return half ? launch_one<FMT, 128, true>(a, stream) : launch_one<FMT, 128, false>(a, stream);
  return half ? launch_one<FMT, 64, true>(a, stream) : launch_one<FMT, 64, false>(a, stream);
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
