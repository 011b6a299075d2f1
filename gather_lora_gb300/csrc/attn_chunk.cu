// Attention of chunks of new tokens over the paged cache (sm_103a).
//
// Row i of a sequence's n rows stands at position p = L - n + i of its L cached tokens and sees the tokens t <= p with
// t > p - window or t < sinks:
//   z_t = scale (q_i . k_t),   out_i = sum_t softmax(z)_t v_t.
//
// Both products run on tcgen05 (M = 128 rows, fp32 accumulators in tensor memory) with a running softmax between them,
// as in the prefill attention: rows of a tile are TT tokens x the G heads of a key-value head, a work item is two such row
// tiles of one sequence and key-value head, each owned by a softmax warpgroup (thread = row), and a key tile is 128 tokens.
//
// Split. The work unit is a key tile of an item. A window's tiles are numbered without the gap between the first
// tokens' and the window's. All units of the batch, item after item, are cut into equal contiguous ranges, one per CTA (one
// CTA per SM), so that any mix of long and short chunks and contexts takes equal time everywhere; ends within kSnap units of
// an item's end move there. A range is walked piece by piece (its part of one item). A piece that is a whole item is
// finished by its CTA; otherwise its rows' exponents, sums and O go to the workspace, and a second kernel joins an item's parts in
// CTA order: the bits never depend on who was last. (Joined by the item's last CTA to arrive, 16 rows after 1000 tokens took 36 us instead
// of 26, four packed chunks 252 instead of 238: one CTA's loads at the end of a range, and code that crowds the loops out of the
// instruction caches.)
//
// Roles of a CTA's 16 warps: 0-7 softmax, 8 issues the MMAs, 9 plans and loads Q (TMA), 11-15 bring K and V. Where the pages'
// size and strides allow (BOXED: sizes in eights), warp 11 looks the pages up, a lane four tokens, and issues TMA, a box a page,
// and warps 12-15 take what has landed over: codes are converted in place in their stage, V that some rows see and others do
// not is looked through. Otherwise the five warps take groups of 16 tokens in turn by cp.async (BF16) or through registers.
//
// 8-bit formats run in f16: the codes of both formats are exact in it, times their scale over a power of two that the tokens of a tile
// share (BOXED; else 16 tokens; a product rounded once, to 11 bits), so that the softmax meets scales once a tile. One a token is
// read from shared memory by every row, whose bandwidth the MMAs need: that is how tiles are taken whose scales are more than 2^12 apart or
// not finite, or that some rows of the item see and others do not. K's
// power of two multiplies the scores; V's the weight: to keep weights of any scale in f16's range the running reference is that of
// y_t = z_t + log2 of V's, the weight w = 2^(y - ref) multiplies V and the softmax's own sum is that of w over V's. Q is brought
// into f16's range by a power of two a row.
//
// Rounding to fewer bits: the weights (BF16 over a BF16 cache, else f16: the tensor cores' operand types; f16 ones lose bits below 2^-21 of a
// row's largest and are 0 below 2^-32, times V's codes below 2^15), K and V of 8 bits (once, to 11 bits), the result.
//
// Zero weight times what is not finite is NaN in an MMA. The loaders look through what some rows of the item see and others
// do not (its last tokens, and the first ones of its windows), set what is not finite in V to zero, and the softmax
// warps (or the join) add it to the stored rows that see it.
//
// Measured on a GB300 (cuBLAS bf16 1.9 PFLOP/s, copy 6.8 TB/s). Operations bound long chunks: four chunks of up to 1500 rows after 4000
// tokens, 32 heads of 128 over 8 in BF16, 236 us (floor 126; tensor pipe 47%: the chain of a key tile through softmax and MMA warp); 2048
// rows after 30000 over E4M3 1.10 ms (floor 0.55; 41%: that chain beside the conversion of the codes; over BF16 0.88). Bytes bound few rows: 32
// sequences of up to 6 rows after 8192 in BF16 124 us (floor 77; one warp looks up the pages of 16 tokens and issues their copies; of 64
// tokens 114), over E4M3 157. A window of 2048 over INT8 with heads of 64: 110 us (floor 10; 28% of the tiles are seen in part and
// scaled token by token, in a pass of their own, and an item costs as much as 2 tiles beside its 18 or so). 16 rows after 1000 tokens 22 us: the plan,
// the look-up, two launches of cold code. Without TMA (pages of 20 tokens) the first takes 328 us, the second 1.79 ms, few rows 161 over
// BF16 and 248 over E4M3.
#include <type_traits>

#include "attn_common.cuh"
#include "tc05.cuh"

namespace glora {

__device__ unsigned int g_chunk_status = 0;

namespace {

constexpr unsigned kChunkTimeoutBit = 0x2u;     // LORA_DEV_TIMEOUT
constexpr int kTile = 128;                      // rows of a tile, tokens of a key tile
constexpr int kSoftWarps = 8;
constexpr int kMmaWarp = 8, kPlanWarp = 9, kWatchWarp = 10, kLoadWarp = 11, kLoaders = 5, kTakers = 4;
constexpr int kChunkThreads = 512, kChunkWarps = kChunkThreads / 32;
constexpr int kPieces = 4;                      // depth of the ring of pieces
constexpr int kMeta = 4;                        // depth of the ring of tokens' masks and scales
constexpr int kGroup = 16, kGroups = kTile / kGroup;   // tokens of a loader's group; groups of a tile
constexpr int kLag = 3;                         // groups of copies that a loader has in flight behind the newest
constexpr int kStageBytes = 2048;               // staging of a warp's results: 32 rows of 64 bytes
constexpr float kGrow = 8.f;                    // the reference moves when the maximum grew by 2^8
constexpr float kTop = 7.f;                     // 8 bits: a weight at the reference is 2^7, at most 2^15
constexpr float kSumUnit = 6.103515625e-05f;    // 8 bits: 2^-14, so that weight / scale stays in range
constexpr int kMostCtas = 160;                  // slots in the workspace
constexpr int kSnap = 2;
constexpr int kItemCost = 2;                    // what an item costs besides its key tiles, in key tiles
constexpr int kMostSeqs = 8192;                 // LORA_MAX_SEQS
constexpr int kFewPairs = 8;                    // sequences of more row-tile pairs are summed by a warp

// Workspace: a head per CTA (the item that it begins and does not end, if any), then 2 slots per CTA (of the item that it goes on
// with, of the one it begins): exponent[256], sum[256], O[256][D], 4 words of flags. All written anew by every call.
constexpr int kHead = 128, kHeadBytes = 32768;
constexpr int kGone = 2;                        // in a slot's flags: its CTA has failed
template <int D>
constexpr int kSlotFloats = 2 * 2 * kTile + 2 * kTile * D + 4;
static_assert(kMostCtas * kHead <= kHeadBytes && kHeadBytes + 2LL * kMostCtas * kSlotFloats<128> * 4 <= (48 << 20), "workspace");

template <int D>
struct ChunkShape {
  static constexpr int tile_bytes = kTile * D * 2;              // Q row tile, K tile or V tile
  static constexpr int pairs = D == 128 ? 2 : 4;                // ring: stages of K and V
  // Tensor memory, all of it (its address is 0): score buffers of the row tiles at columns 0 and 128, O0 and O1 at the end.
  static constexpr uint32_t col_o = 512 - 2 * D;
  // Byte of 16-byte chunk c of row r: 64-column blocks, 128-byte swizzle.
  static __device__ __forceinline__ uint32_t at(int r, int c) { return (c >> 3) * (kTile * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4); }
};

struct ChunkMeta {           // of a key tile
  uint32_t live[4];          // tokens that are there and that some row sees
  // 8 bits, of 16 tokens (BOXED: the first, of all): scale log2(e) times K's power of two, log2 of V's, kSumUnit over V's, and
  // whether their scales are taken token by token instead (ab)
  float4 group[kGroups];
  float2 ab[kTile];          // scale log2(e) times the token's K scale, log2 of its V scale over 2^kRaise
  float iv[kTile];           // kSumUnit over that
  float ks[kTile], vs[kTile];   // (BOXED) the scales as they are
};

struct ChunkPiece {
  int valid;
  int b, row0;               // sequence; first query row
  int first, end;            // positions of its first token (may be negative) and of its last
  int kvh, h0, heads;
  int low, kept, skip;       // first token in any row's window; tiles from `kept` on stand `skip` further
  int ta, n, tiles;          // first tile, tiles; the item's
  int ni[2];                 // tiles of each row tile
  int c0, c1;                // the item's CTAs
};
static_assert(sizeof(ChunkPiece) <= kHead, "heads");

struct alignas(16) ChunkCtl {
  unsigned long long full[8], empty[8];              // K stages even, V stages odd
  unsigned long long landed[8];                      // (BOXED) full but for the look or the conversion
  unsigned long long meta_full[kMeta], meta_empty[kMeta];
  unsigned long long q_landed, q_full, q_empty;
  unsigned long long s_full[2][2], p_ready[2][2][2], o_done[2][2];   // [row tile][parity of its key tile] ([half])
  unsigned long long piece_full[kPieces], piece_empty[kPieces];
  unsigned long long drain, ended;
  ChunkPiece piece[kPieces];
  int bad[kPieces];                                  // something in V was set to zero
  float4 extremes[2][kTakers];                       // largest and least scales of a tile, by the converting warps
  uint32_t tmem;
  int failed, progress;
  // the plan
  long long warp_sum[kChunkWarps], total, sum[2], rem[2];
  int seq[2];
};

template <int D>
struct ChunkSmem {
  using Sh = ChunkShape<D>;
  static constexpr int q = 0, ring = 2 * Sh::tile_bytes, stage = ring + 2 * Sh::pairs * Sh::tile_bytes;
  static constexpr int meta = stage + kSoftWarps * kStageBytes;
  static constexpr int ctl = meta + kMeta * static_cast<int>(sizeof(ChunkMeta));
  static constexpr int bytes = ctl + static_cast<int>(sizeof(ChunkCtl));
  static_assert(sizeof(ChunkMeta) % 16 == 0 && bytes <= 232448, "shared memory");
  static_assert(kMostSeqs * 8 <= 2 * Sh::pairs * Sh::tile_bytes, "the plan's sums lie in the ring");
};

__device__ __forceinline__ bool failed(const ChunkCtl& c) { return *reinterpret_cast<const volatile int*>(&c.failed) != 0; }

// Bounded wait; true if the CTA has failed: warp 10 watches over all of them and says so when no key tile has been taken up
// for kWaitLimitCycles. Then all waits end at once. A piece is read only by who saw, behind the wait for it, that the CTA had not
// failed (piece_here), as only then it is known to be there; the others leave, and so do loops over its tiles. The planning warp publishes
// and overwrites nothing any more. What runs on until then stays in bounds; results are not stored, nor joined from what this CTA
// put into the workspace. (Small, as it is inlined at every wait: the roles' loops share the instruction caches.)
__device__ __forceinline__ bool wait(ChunkCtl& c, unsigned long long& bar, uint32_t parity) {
  const uint32_t b = smem_u32(&bar);
#pragma unroll 1
  while (!mbar_try_wait(b, parity, 100000))
    if (failed(c)) return true;
  return false;
}
// The whole warp: the next piece is there and is one (not the end).
__device__ __forceinline__ bool piece_here(ChunkCtl& c, int it) {
  wait(c, c.piece_full[it % kPieces], (it / kPieces) & 1);
  __syncwarp();
  return !__any_sync(0xffffffffu, failed(c)) && c.piece[it % kPieces].valid;
}
__device__ __forceinline__ bool passed(unsigned long long& bar, uint32_t parity) {
  uint32_t done;
  asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(done)
               : "r"(smem_u32(&bar)), "r"(parity)
               : "memory");
  return done != 0;
}

__device__ __forceinline__ void takers_sync() { asm volatile("bar.sync 1, %0;\n" ::"n"(kTakers * 32) : "memory"); }
// The same, and whether one of the warps has seen that the CTA failed: they stay together, as the others would wait at the next
// barrier for one that has left.
__device__ __forceinline__ bool takers_failed(const ChunkCtl& c) {
  uint32_t any;
  asm volatile("{\n .reg .pred f, a;\n setp.ne.u32 f, %1, 0;\n bar.red.or.pred a, 1, %2, f;\n selp.u32 %0, 1, 0, a;\n}\n"
               : "=r"(any)
               : "r"(static_cast<uint32_t>(failed(c))), "n"(kTakers * 32)
               : "memory");
  return any != 0;
}

// A scale over its group's power of two as f16 hi + lo (hi in the low half): 22 bits of it.
__device__ __forceinline__ uint32_t split_f16(float m) {
  const __half hi = __float2half_rn(m), lo = __float2half_rn(m - __half2float(hi));
  return static_cast<uint32_t>(__half_as_ushort(hi)) | static_cast<uint32_t>(__half_as_ushort(lo)) << 16;
}
// Eight codes times such a scale, rounded once.
template <int FMT>
__device__ __forceinline__ uint4 scaled8(uint32_t c0, uint32_t c1, uint32_t m) {
  uint32_t h[4];
  codes_to_f16<FMT>(c0, h[0], h[1]);
  codes_to_f16<FMT>(c1, h[2], h[3]);
  const uint32_t m0 = __byte_perm(m, m, 0x1010), m1 = __byte_perm(m, m, 0x3232);
  const __half2 hi = *reinterpret_cast<const __half2*>(&m0), lo = *reinterpret_cast<const __half2*>(&m1);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __half2 x = *reinterpret_cast<const __half2*>(&h[j]), r = __hfma2(x, hi, __hmul2(x, lo));
    h[j] = *reinterpret_cast<const uint32_t*>(&r);
  }
  return make_uint4(h[0], h[1], h[2], h[3]);
}
// Exponent of the power of two of a group whose largest scale is `most`: codes times scales are below 2^15 of it.
template <int FMT>
constexpr int kCodeBits = FMT == kKvE4m3 ? 9 : 7;          // codes are below 2 to that
template <int FMT>
__device__ __forceinline__ int group_exponent(float most) {
  return max(-120, (__float_as_int(most) >> 23) - 127 + 1 + kCodeBits<FMT> - 15);
}
__device__ __forceinline__ float exp2_int(int e) { return __int_as_float((127 + e) << 23); }
__device__ __forceinline__ float magnitude(float s) { return fabsf(s) < INFINITY ? fabsf(s) : INFINITY; }
// Scales of a tile (of 16 tokens) differ too much for one power of two, or one is not finite.
constexpr float kWide = 4096.f;
__device__ __forceinline__ bool wide(float most, float least) { return most > least * kWide || most == INFINITY; }
// What the softmax needs of a group. (One whose scales are all 0 only counts in the sums: 2^-64 keeps it from raising the reference.)
template <int FMT>
__device__ __forceinline__ float4 group_of(float most_k, float most_v, float sl2, bool exact) {
  const int ev = most_v == 0.f ? -64 : group_exponent<FMT>(most_v);
  return make_float4(most_k == 0.f ? sl2 : exp2_int(group_exponent<FMT>(most_k)) * sl2, static_cast<float>(ev), kSumUnit * exp2_int(-ev), exact);
}
// What the codes of a token with scale s are multiplied with.
template <int FMT>
__device__ __forceinline__ uint32_t scale_of(float s, float most) {
  return split_f16(most == 0.f ? 0.f : s * exp2_int(-group_exponent<FMT>(most)));
}
// Token by token: codes of K as they are, of V times 2^kRaise with the scale's sign (0: they only count in the sum; not finite: NaN, times 0
// too). With kRaise they lie below 2^15 as those of a group do, and a weight says as much of a token's part in the result: without it the
// weights beside a largest one that is taken token by token were 2^kRaise nearer to f16's least.
template <int FMT>
constexpr int kRaise = 15 - kCodeBits<FMT>;
constexpr uint32_t kOne = 0x3c00u;                         // (f16; adding to its exponent multiplies by powers of two)
template <int FMT>
__device__ __forceinline__ uint32_t sign_of(float s) {
  return s == 0.f ? 0u : !(fabsf(s) < INFINITY) ? 0x7e00u : kOne + (kRaise<FMT> << 10) + (s < 0.f ? 0x8000u : 0u);
}
// A V scale of 0 is 2^-64 to the weights (see above), and so is one that is not finite: the scores and their sum do not go by V. Below 2^-110,
// under what lora_kv_write stores, it is 2^-110.
__device__ __forceinline__ float magnitude_of(float v) {
  return v == 0.f || !(fabsf(v) < INFINITY) ? 5.421010862427522e-20f : fmaxf(fabsf(v), 7.703719777548943e-34f);
}
template <int FMT>
__device__ __forceinline__ float2 scales_of(float k, float v, float sl2) { return make_float2(k * sl2, log2f(magnitude_of(v)) - kRaise<FMT>); }
template <int FMT>
__device__ __forceinline__ float over_scale(float v) { return kSumUnit * (1 << kRaise<FMT>) / magnitude_of(v); }

// Chunks of V: whether all is finite, and with what is not set to zero.
template <bool CODED>
__device__ __forceinline__ bool chunk_finite(const uint4& x) {
  if (!CODED) return all_finite(abs_max2(0, x));
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  bool ok = true;
#pragma unroll
  for (int j = 0; j < 4; ++j) ok = ok && (w[j] & 0x7c00u) != 0x7c00u && (w[j] & 0x7c000000u) != 0x7c000000u;
  return ok;
}
template <bool CODED>
__device__ __forceinline__ uint4 chunk_or_zero(const uint4& x) {
  if (!CODED) return make_uint4(finite_or_zero(x.x), finite_or_zero(x.y), finite_or_zero(x.z), finite_or_zero(x.w));
  uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if ((w[j] & 0x7c00u) == 0x7c00u) w[j] &= 0xffff0000u;
    if ((w[j] & 0x7c000000u) == 0x7c000000u) w[j] &= 0xffffu;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* map, int c0, int c1, int c2, int c3, uint32_t bar) {
  asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];\n"
               ::"r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
               : "memory");
}

// ---- the plan ---------------------------------------------------------------

struct Seq {
  int q0, n, len;            // first row, rows (0: left out), cached tokens
};
__device__ __forceinline__ Seq sequence(const ChunkArgs& p, int b) {
  Seq s{};
  const int a0 = __ldg(p.cu_q + b), a1 = __ldg(p.cu_q + b + 1);
  if (a0 < 0 || a1 <= a0 || a1 > p.total_q) return s;
  s.q0 = a0;
  s.n = a1 - a0;
  const long long most = static_cast<long long>(p.max_pages) * p.c.page_size;
  s.len = static_cast<int>(min(static_cast<long long>(max(__ldg(p.lens + b), 0)), most));
  return s;
}

// What the rows at positions first .. end see between them, as key tiles.
struct Span {
  int low, kept, skip, tiles;
};
__device__ __forceinline__ Span span(const ChunkArgs& p, int first, int end) {
  Span s{};
  if (end < 0) return s;
  s.low = first >= p.window ? first - p.window + 1 : 0;
  const int sinks = min(p.sinks, s.low);
  s.kept = sinks / kTile + (sinks % kTile ? 1 : 0);
  s.skip = max(0, s.low / kTile - s.kept);
  s.tiles = end / kTile + 1 - s.skip;
  return s;
}
// Key tiles of row-tile pair x of a sequence (0 where all its rows stand before the first token); its units: kItemCost more.
__device__ __forceinline__ int pair_tiles(const ChunkArgs& p, const Seq& s, int step, int x) {
  const int t0 = x * step;
  return span(p, s.len - s.n + t0, s.len - s.n + min(t0 + step, s.n) - 1).tiles;
}

__device__ __forceinline__ int pair_units(const ChunkArgs& p, const Seq& s, int step, int x) {
  const int t = pair_tiles(p, s, step, x);
  return t ? t + kItemCost : 0;
}

// CTAs with work: at least this many units each.
constexpr int kLeast = 4;
__device__ __forceinline__ long long working(long long total, unsigned grid) {
  return min(static_cast<long long>(grid), (total + kLeast - 1) / kLeast);
}
// a / b of two numbers that are not negative, in 32 bits where they fit (a 64-bit division is a call of a hundred instructions).
__device__ __forceinline__ long long divide(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}
// Unit at which CTA c's range begins, before ends move.
__device__ __forceinline__ long long cut(long long c, long long total, long long n) { return divide(c * total, n); }

// Rows of an item up to the last that is somebody's.
__device__ __forceinline__ int rows_of(const ChunkArgs& p, const ChunkPiece& w) {
  const int tokens = w.end - w.first + 1, TT = p.tile_tokens, GB = p.head_block;
  return tokens > TT ? kTile + min(kTile, (tokens - TT) * GB) : min(kTile, tokens * GB);
}

// A row's stored weights stand for weight * 2^-exponent, their sum likewise (8 bits: times kSumUnit as well).
template <bool CODED>
__device__ __forceinline__ float log_sum(float exponent, float sum) {
  return sum == 0.f ? -INFINITY : (exponent + log2f(sum) + (CODED ? 14.f : 0.f)) * kLn2;
}
template <bool CODED>
__device__ __forceinline__ float inverse(float sum) {
  if (!CODED) return sum == 0.f ? 0.f : 1.f / sum;
  return sum == 0.f ? 0.f : sum > 1.f ? 1.f / sum * kSumUnit : 1.f / (sum / kSumUnit);
}

}  // namespace

// What was set to zero in V is added to the stored result rows of this warp that see it, as it is, since their weights are
// positive: per token of the warp, over the tokens that it sees and others of the item do not.
template <int FMT, int D>
__device__ __noinline__ void add_not_finite(const ChunkArgs& p, const ChunkPiece& w, int warp, int lane) {
  constexpr int E = D / 32;
  const int i = warp >> 2, r0 = (warp & 3) * 32, GB = p.head_block, TT = p.tile_tokens;
  const int32_t* const table = p.table + w.b * p.table_stride;
  for (int t_in = r0 / GB; t_in <= (r0 + 31) / GB && t_in < TT; ++t_in) {
    if (i * TT + t_in > w.end - w.first) break;
    const int pos = w.first + i * TT + t_in;
    if (pos < 0) continue;
    float s[E];
#pragma unroll
    for (int e = 0; e < E; ++e) s[e] = 0.f;
    // ends of the two ranges of such tokens: before the last row's window, and behind the first row
    const int low_end = min(pos, w.end - p.window);
    for (int part = 0; part < 2; ++part) {
      const int from = part ? max(max(w.first + 1, 0), low_end + 1) : max(0, pos - p.window + 1), to = part ? pos : low_end;
      for (int t = from; t <= to; ++t) {
        const bool sees = t > pos - p.window || t < p.sinks;
        const bool all_see = t <= w.first && (t > w.end - p.window || t < p.sinks);
        if (!sees || all_see) continue;
        const int entry = p.page_shift >= 0 ? t >> p.page_shift : t / p.c.page_size, page = __ldg(table + entry);
        if (page < 0 || page >= p.c.num_pages) continue;
        const unsigned char* const v = p.c.v + page * p.c.page_bytes + w.kvh * p.c.head_bytes + (t - entry * p.c.page_size) * p.c.token_bytes;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          if constexpr (FMT == kKvBf16) {
            const uint32_t x = reinterpret_cast<const uint16_t*>(v)[lane * E + e];
            if ((x & 0x7f80u) == 0x7f80u) s[e] += __uint_as_float(x << 16);
          } else {
            float f[4];
            codes_to_f32<FMT>(v[lane * E + e], f);
            const float x = f[0] * __ldg(p.c.vs + scale_index(p.c, page, w.kvh, t - entry * p.c.page_size));
            if (!(fabsf(x) < INFINITY)) s[e] = __int_as_float(0x7fffffff);
          }
        }
        bool all_nan = true;               // nothing more can change
#pragma unroll
        for (int e = 0; e < E; ++e) all_nan = all_nan && s[e] != s[e];
        if (__all_sync(0xffffffffu, all_nan)) {
          t = to;
          part = 1;
        }
      }
    }
    bool any = false;
#pragma unroll
    for (int e = 0; e < E; ++e) any = any || s[e] != 0.f;
    if (!__any_sync(0xffffffffu, any)) continue;
    for (int r = max(r0, t_in * GB); r < min(r0 + 32, t_in * GB + GB); ++r) {
      const int g = r - t_in * GB;
      if (g >= w.heads) break;
      uint16_t* const out = p.out + (static_cast<long long>(w.row0) + i * TT + t_in) * p.out_stride + (w.h0 + g) * D + lane * E;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        uint32_t* const at = reinterpret_cast<uint32_t*>(out + e);
        const uint32_t x = *at;
        *at = pack_bf16x2(__uint_as_float(x << 16) + s[e], __uint_as_float(x & 0xffff0000u) + s[e + 1]);
      }
    }
  }
}

template <int FMT, int D, bool BOXED>
__global__ void __launch_bounds__(kChunkThreads, 1) chunk_kernel(const __grid_constant__ ChunkArgs p) {
  using Sh = ChunkShape<D>;
  using Sm = ChunkSmem<D>;
  constexpr int NP = Sh::pairs;
  constexpr bool CODED = FMT != kKvBf16;
  extern __shared__ __align__(1024) unsigned char chunk_smem[];             // (aligned by its declaration, so that offsets are constants)
  unsigned char* const base = chunk_smem;
  const uint32_t q_s = smem_u32(chunk_smem) + Sm::q, ring = smem_u32(chunk_smem) + Sm::ring;
  ChunkMeta* const metas = reinterpret_cast<ChunkMeta*>(base + Sm::meta);
  ChunkCtl& c = *reinterpret_cast<ChunkCtl*>(base + Sm::ctl);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);    // (the same for the warp to the compiler, too)

  if (tid == 0) {
    for (int s = 0; s < 2 * NP; ++s) {
      mbar_init(smem_u32(&c.full[s]), !BOXED ? kGroups : CODED || (s & 1) ? kTakers : 1);
      mbar_init(smem_u32(&c.landed[s]), CODED && !(s & 1) ? 33 : 1);     // (K: each lane's scales as well)
      mbar_init(smem_u32(&c.empty[s]), 1);
    }
    for (int s = 0; s < kMeta; ++s) {
      mbar_init(smem_u32(&c.meta_full[s]), BOXED ? 1 + (CODED ? kTakers : 0) : kGroups);
      mbar_init(smem_u32(&c.meta_empty[s]), kSoftWarps);
    }
    mbar_init(smem_u32(&c.q_landed), 1);
    mbar_init(smem_u32(&c.q_full), CODED ? kSoftWarps : 1);
    mbar_init(smem_u32(&c.q_empty), 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&c.s_full[i >> 1][i & 1]), 1);
      mbar_init(smem_u32(&c.p_ready[i >> 1][i & 1][0]), 4);
      mbar_init(smem_u32(&c.p_ready[i >> 1][i & 1][1]), 4);
      mbar_init(smem_u32(&c.o_done[i >> 1][i & 1]), 1);
    }
    for (int i = 0; i < kPieces; ++i) {
      mbar_init(smem_u32(&c.piece_full[i]), 1);
      mbar_init(smem_u32(&c.piece_empty[i]), kSoftWarps + 1 + kLoaders);
    }
    mbar_init(smem_u32(&c.drain), 1);
    mbar_init(smem_u32(&c.ended), kSoftWarps);
    for (int i = 0; i < kPieces; ++i) c.piece[i].valid = 0;
    c.failed = 0;
    c.progress = 0;
    mbar_fence_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&c.tmem), 512);
    tmem_relinquish();
  }
  pdl_wait_then_release();

  // ---- the batch's units, and where this CTA's range begins and ends
  const int TT = p.tile_tokens, step = 2 * TT, GB = p.head_block;
  const int G = p.q_heads / p.c.kv_heads, blocks = (G + GB - 1) / GB, subs = p.c.kv_heads * blocks;
  {
    long long* const sums = reinterpret_cast<long long*>(base + Sm::ring);               // units of a sequence and key-value head
    const int per = (p.batch + kChunkThreads - 1) / kChunkThreads;
    const int b0 = min(tid * per, p.batch), b1 = min(b0 + per, p.batch);
    long long mine = 0;
    for (int k = 0; k < per; ++k) {
      const int b = b0 + k;
      Seq s{};
      if (b < b1) s = sequence(p, b);
      const int np = s.n > 0 ? (s.n - 1) / step + 1 : 0;
      long long sum = 0;
      if (np <= kFewPairs)
        for (int x = 0; x < np; ++x) sum += pair_units(p, s, step, x);
      uint32_t many = __ballot_sync(0xffffffffu, np > kFewPairs);
      while (many) {
        const int src = __ffs(many) - 1;
        many &= many - 1;
        Seq o;
        o.q0 = 0;
        o.n = __shfl_sync(0xffffffffu, s.n, src);
        o.len = __shfl_sync(0xffffffffu, s.len, src);
        const int onp = (o.n - 1) / step + 1;
        long long part = 0;
        for (int x = lane; x < onp; x += 32) part += pair_units(p, o, step, x);
#pragma unroll
        for (int y = 16; y > 0; y >>= 1) part += __shfl_xor_sync(0xffffffffu, part, y);
        if (lane == src) sum = part;
      }
      if (b < b1) sums[b] = sum;
      mine += sum;
    }
    mine *= subs;
    long long before = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += t;
    }
    if (lane == 31) c.warp_sum[warp] = before;
    before -= mine;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    long long total = 0;
    for (int w = 0; w < kChunkWarps; ++w) {
      if (w < warp) before += c.warp_sum[w];
      total += c.warp_sum[w];
    }
    const long long n = working(total, gridDim.x);
    if (tid == 0) c.total = total;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (blockIdx.x >= n) break;
      const long long u = cut(blockIdx.x + e, total, n);
      if (u < before || u >= before + mine) continue;                        // another thread's sequences hold it
      long long at = before;
      for (int b = b0; b < b1; ++b) {
        const long long all = sums[b] * subs;
        if (u < at + all) {
          c.seq[e] = b;
          c.sum[e] = sums[b];
          c.rem[e] = u - at;
          break;
        }
        at += all;
      }
    }
    fence_proxy_async_smem();            // the sums' bytes are TMA's next (each thread orders its own accesses before the barrier)
    __syncthreads();
  }
  if (tid == 0 && c.tmem != 0) *reinterpret_cast<volatile int*>(&c.failed) = 1;     // (never: all columns are this CTA's)
  const long long total = c.total, ctas = working(total, gridDim.x);
  const bool works = blockIdx.x < ctas;

  if (warp >= kSoftWarps) {
  if (warp == kPlanWarp) {
    // ===================== pieces, and the rows of Q ======================
    int b = 0, sub = 0, x = 0, tile = 0, tiles = 0;       // the item under the walk, and its next tile
    long long s0 = 0, u = 0, u1 = 0;                      // its first unit; the walk's position and end
    Seq s{};
    const int snap = static_cast<int>(min(static_cast<long long>(kSnap), divide(total, max(ctas, 1LL)) / 4));
    auto first_pair = [&]() { return max(0, (s.n - s.len) / step); };       // the first with a tile (s.len > 0)
    auto next_item = [&]() {                              // (there is one)
      s0 += kItemCost + tiles;
      if ((x + 1) * step < s.n) {
        ++x;
      } else {
        if (++sub == subs) {
          sub = 0;
          do s = sequence(p, ++b);
          while (s.n == 0 || s.len == 0);
        }
        x = first_pair();
      }
      tile = 0;
      tiles = pair_tiles(p, s, step, x);
    };
    if (works) {
      const Seq both[2] = {sequence(p, c.seq[0]), sequence(p, blockIdx.x + 1 < ctas ? c.seq[1] : c.seq[0])};
      // The item that holds a cut, by prefix sums over its sequence's pairs; 0: this CTA's first unit, 1: the next one's.
      for (int e = 1; e >= 0; --e) {
        const long long r = cut(blockIdx.x + e, total, ctas);
        if (r >= total) {
          u1 = total;
          continue;
        }
        b = c.seq[e];
        s = both[e];
        const long long su = c.sum[e];
        sub = static_cast<int>(divide(c.rem[e], su));
        const long long rest = c.rem[e] - sub * su;
        const int np = (s.n - 1) / step + 1;
        long long before = 0;
        for (int x0 = 0; x0 < np; x0 += 32) {
          const int mine = x0 + lane < np ? pair_units(p, s, step, x0 + lane) : 0;
          long long incl = mine;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += t;
          }
          const uint32_t hit = __ballot_sync(0xffffffffu, rest < before + incl);
          if (hit) {
            const int src = __ffs(hit) - 1;
            x = x0 + src;
            const int units = __shfl_sync(0xffffffffu, mine, src);
            tile = static_cast<int>(rest - before - (__shfl_sync(0xffffffffu, incl, src) - units));     // (in units so far)
            tiles = units - kItemCost;
            break;
          }
          before += __shfl_sync(0xffffffffu, incl, 31);
        }
        s0 = r - tile;
        tile -= kItemCost;
        if (tile <= snap) tile = 0;
        else if (tiles - tile <= snap) tile = tiles;
        const long long at = s0 + (tile ? kItemCost + tile : 0);
        if (e == 1) u1 = at;
        else u = at;
      }
      if (u < u1 && tile == tiles) next_item();
    }
    auto tiles_here = [&]() { return static_cast<int>(min(static_cast<long long>(tiles), u1 - s0 - kItemCost)) - tile; };   // of the item, in this range
    uint32_t loads = 0;
    for (int it = 0;; ++it) {
      const int sl = it % kPieces;
      // (a slot is written again only when all have left it; after a failure not at all, as some may still be reading)
      if (it >= kPieces) wait(c, c.piece_empty[sl], ((it / kPieces) - 1) & 1);
      __syncwarp();
      if (__any_sync(0xffffffffu, failed(c))) break;
      const bool go = u < u1;
      if (lane == 0) {
        ChunkPiece w{};
        w.valid = go;
        if (go) {
          const int t0 = x * step, t1 = min(t0 + step, s.n);
          w.b = b;
          w.row0 = s.q0 + t0;
          w.first = s.len - s.n + t0;
          w.end = s.len - s.n + t1 - 1;
          w.kvh = sub / blocks;
          w.h0 = w.kvh * G + (sub - w.kvh * blocks) * GB;
          w.heads = min(GB, w.kvh * G + G - w.h0);
          const Span v = span(p, w.first, w.end);
          w.low = v.low;
          w.kept = v.kept;
          w.skip = v.skip;
          w.tiles = tiles;
          w.ta = tile;
          w.n = tiles_here();
#pragma unroll
          for (int i = 0; i < 2; ++i) {                 // tiles that hold a token its last row may see
            const int last = w.first + min((i + 1) * TT, t1 - t0) - 1, any = i * TT < t1 - t0 && last >= 0;
            w.ni[i] = any ? max(0, min(w.ta + w.n, last / kTile + 1 - w.skip) - w.ta) : 0;
          }
          w.c0 = static_cast<int>(divide((s0 + kItemCost + snap + 1) * ctas + total - 1, total)) - 1;
          w.c1 = static_cast<int>(divide((s0 + kItemCost + tiles - snap) * ctas + total - 1, total)) - 1;
        }
        c.piece[sl] = w;
        *reinterpret_cast<volatile int*>(&c.bad[sl]) = 0;
        mbar_arrive(smem_u32(&c.piece_full[sl]));
      }
      __syncwarp();
      if (!go) break;
      const int t0 = x * step, tokens = min(step, s.n - t0), row0 = s.q0 + t0, kvh = sub / blocks, h0 = kvh * G + (sub - kvh * blocks) * GB;
      tile += tiles_here();
      u = s0 + kItemCost + tile;
      if (u < u1) next_item();
      // Q: rows of other sequences or heads that a box brings along are nobody's.
      if (loads > 0) wait(c, c.q_empty, (loads - 1) & 1);
      ++loads;
      __syncwarp();
      if (lane == 0 && !failed(c)) {
        const uint32_t bar = smem_u32(CODED ? &c.q_landed : &c.q_full);
        const int both = tokens > TT ? 2 : 1;
        mbar_arrive_expect_tx(bar, both * (D / 64) * GB * TT * 128);
        for (int y = 0; y < both * (D / 64); ++y) {
          const int i = y / (D / 64), a = y % (D / 64);
          tma_load_3d(q_s + i * Sh::tile_bytes + a * (kTile * 128), &p.map_q, a * 64, h0, row0 + i * TT, bar);
        }
      }
      __syncwarp();
    }
    if (lane == 0 && loads > 0 && failed(c)) mbar_wait_limit(smem_u32(CODED ? &c.q_landed : &c.q_full), (loads - 1) & 1, kDrainLimitCycles);
    __syncwarp();
  } else if (warp == kWatchWarp) {
    // ============================== watch =================================
    long long t0 = clock64();
    int seen = 0;
    while (!mbar_try_wait(smem_u32(&c.ended), 0, 1000000)) {
      const int now = *reinterpret_cast<volatile int*>(&c.progress);
      if (now != seen) {
        seen = now;
        t0 = clock64();
      } else if (clock64() - t0 > kWaitLimitCycles) {
        *reinterpret_cast<volatile int*>(&c.failed) = 1;
      }
      if (failed(c)) break;
    }
    __syncwarp();
  } else if (BOXED && warp == kLoadWarp) {
    // ==================== pages looked up, TMA of K and V ====================
    // A lane has 4 consecutive tokens of a tile (of one page: boxes are of 8 slots or more); the first lane of a box issues it. A
    // page that is not there is asked for behind the last: its rows are filled with zeros.
    const int BT = p.box_tokens;
    constexpr uint32_t bytes = CODED ? kTile * D : Sh::tile_bytes;
    uint32_t kt = 0, tiles = 0;          // key tiles of the pieces before; issued
    for (int it = 0;; ++it) {
      const int sl = it % kPieces;
      if (!piece_here(c, it)) break;
      const ChunkPiece& w = c.piece[sl];
      const int32_t* const table = p.table + w.b * p.table_stride;
      auto first_token = [&](int j) {
        const int t = w.ta + j;
        return (t < w.kept ? t : t + w.skip) * kTile;
      };
      int slot = 0, page = -1;           // of this lane's tokens of the tile to issue next
      auto look_up = [&](int j) {
        const int t = first_token(j) + lane * 4, box = t & ~(BT - 1);
        page = -1;
        if (box > w.end || (box + BT - 1 < w.low && box >= p.sinks)) return;      // (nobody sees any of the box)
        const int entry = p.page_shift >= 0 ? t >> p.page_shift : t / p.c.page_size;
        slot = t - entry * p.c.page_size;
        page = __ldg(table + entry);
      };
      look_up(0);
      for (int j = 0; j < w.n; ++j) {
        const uint32_t k = kt + j, ks = 2 * (k % NP);
        const int t = first_token(j) + lane * 4, my_slot = slot;
        const bool there = page >= 0 && page < p.c.num_pages;
        const int my_page = there ? page : p.c.num_pages;
        uint32_t seen = 0;
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (there && t + x <= w.end && (t + x >= w.low || t + x < p.sinks)) seen |= 1u << x;
        if (j + 1 < w.n) look_up(j + 1);
        ChunkMeta& m = metas[k % kMeta];
        if (k >= kMeta) wait(c, c.meta_empty[k % kMeta], ((k / kMeta) - 1) & 1);
        if (k >= NP) wait(c, c.empty[ks], ((k / NP) - 1) & 1);
        __syncwarp();
        // Copies first, then the masks and scales.
        auto copies = [&](uint32_t stage, const TensorMapBytes& map) {
          const uint32_t bar = smem_u32(!CODED && !(stage & 1) ? &c.full[stage] : &c.landed[stage]);
          if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
          __syncwarp();
          // (box by box by one lane: issued by the boxes' own lanes they took twice as long)
#pragma unroll 1
          for (int box = 0; box < kTile; box += BT) {
            const int at = __shfl_sync(0xffffffffu, my_slot, box / 4), of = __shfl_sync(0xffffffffu, my_page, box / 4);
            const int c1 = p.heads_inside ? w.kvh : at, c2 = p.heads_inside ? at : w.kvh;
            const uint32_t to = ring + stage * Sh::tile_bytes;
            if (elect_one()) {
              if constexpr (CODED) {
                tma_load_4d(to + Sh::tile_bytes / 2 + box * D, &map, 0, c1, c2, of, bar);
              } else {
#pragma unroll
                for (int a = 0; a < D / 64; ++a) tma_load_4d(to + a * (kTile * 128) + box * 128, &map, a * 64, c1, c2, of, bar);
              }
            }
            __syncwarp();
          }
        };
        if (__any_sync(0xffffffffu, failed(c))) break;
        if constexpr (CODED) {             // the scales (of tokens that are not there: 0) land with K's codes
          const long long si = there ? scale_index(p.c, my_page, w.kvh, my_slot) : 0;
          const uint32_t to = smem_u32(m.ks + lane * 4);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            cp_async4_n(to + x * 4, p.c.ks + si + x, there ? 4 : 0);
            cp_async4_n(to + kTile * 4 + x * 4, p.c.vs + si + x, there ? 4 : 0);
          }
          cp_async_arrive_noinc(smem_u32(&c.landed[ks]));
        }
        copies(ks, p.map_k);
        uint32_t live = seen << (4 * (lane & 7));
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) live |= __shfl_xor_sync(0xffffffffu, live, o);
        if ((lane & 7) == 0) m.live[lane >> 3] = live;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&c.meta_full[k % kMeta]));
        if (k >= NP) wait(c, c.empty[ks + 1], ((k / NP) - 1) & 1);
        __syncwarp();
        copies(ks + 1, p.map_v);
        tiles = k + 1;
      }
      kt += w.n;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&c.piece_empty[sl]));
    }
    if (lane == 0 && failed(c)) {        // let the copies in flight land
      for (uint32_t k = tiles > NP ? tiles - NP : 0; k <= tiles; ++k)
        for (int x = 0; x < 2; ++x) {
          const uint32_t st = 2 * (k % NP) + x;
          mbar_wait_limit(smem_u32(!CODED && !x ? &c.full[st] : &c.landed[st]), (k / NP) & 1, k < tiles ? kDrainLimitCycles : kDrainLimitCycles / 16);
        }
    }
    __syncwarp();
  } else if (BOXED && warp > kLoadWarp) {
    // ================= what has landed: converted, looked through =================
    // Warp q of the four has rows 32 q .. of every tile. 8 bits: a tile's codes lie in the upper half of its stage; at head_dim 128 a row's
    // are where the second half of its f16 goes, so that a warp's rows are its own; at 64 all four have read theirs before any writes.
    const int q = warp - kLoadWarp - 1;
    const float sl2 = p.scale * kLog2e;
    uint32_t kt = 0;
    for (int it = 0;; ++it) {
      const int sl = it % kPieces;
      const bool here = piece_here(c, it);
      if (CODED && takers_failed(c)) break;       // (else all four have the same piece, or the end)
      if (!here) break;
      const ChunkPiece& w = c.piece[sl];
      for (int j = 0; j < w.n; ++j) {
        const uint32_t k = kt + j;
        const int tile = w.ta + j, t0 = (tile < w.kept ? tile : tile + w.skip) * kTile + q * 32;
        const bool partly = !(t0 + 31 <= w.first && (t0 > w.end - p.window || t0 + 31 < p.sinks));   // some rows see some of it, others not
        auto part_seen = [&](int t) { return !(t <= w.first && (t > w.end - p.window || t < p.sinks)); };
        bool bad = false, gone = false;
        uint32_t mult_k = 0, mult_v = 0;
#pragma unroll 1
        for (int x = CODED ? 0 : 1; x < 2; ++x) {
          const uint32_t st = 2 * (k % NP) + x, at = ring + st * Sh::tile_bytes;
          [[maybe_unused]] const bool late = wait(c, c.landed[st], (k / NP) & 1);
          if constexpr (!CODED) {
            gone = __any_sync(0xffffffffu, late);
            if (gone) break;
          }
          __syncwarp();
          if constexpr (CODED) {
            if (x == 0) {                  // lane: the token of a row
              ChunkMeta& m = metas[k % kMeta];
              const int r = q * 32 + lane, tt = t0 - q * 32;
              const float sk = m.ks[r], sv = m.vs[r];
              float most_k = magnitude(sk), most_v = magnitude(sv);
              float least_k = most_k == 0.f ? INFINITY : most_k, least_v = most_v == 0.f ? INFINITY : most_v;
#pragma unroll
              for (int o = 1; o < 32; o <<= 1) {
                most_k = fmaxf(most_k, __shfl_xor_sync(0xffffffffu, most_k, o));
                most_v = fmaxf(most_v, __shfl_xor_sync(0xffffffffu, most_v, o));
                least_k = fminf(least_k, __shfl_xor_sync(0xffffffffu, least_k, o));
                least_v = fminf(least_v, __shfl_xor_sync(0xffffffffu, least_v, o));
              }
              float4* const of_warps = c.extremes[k & 1];        // (two in turn: nobody is two tiles ahead)
              if (lane == 0) of_warps[q] = make_float4(most_k, most_v, least_k, least_v);
              gone = takers_failed(c);
              if (gone) break;
#pragma unroll
              for (int y = 0; y < kTakers; ++y) {
                const float4 z = of_warps[y];
                most_k = fmaxf(most_k, z.x);
                most_v = fmaxf(most_v, z.y);
                least_k = fminf(least_k, z.z);
                least_v = fminf(least_v, z.w);
              }
              const bool exact = wide(most_k, least_k) || wide(most_v, least_v) ||
                                 !(tt + kTile - 1 <= w.first && (tt > w.end - p.window || tt + kTile - 1 < p.sinks));
              if (q == 0 && lane == 0) m.group[0] = group_of<FMT>(most_k, most_v, sl2, exact);
              if (exact) {
                m.ab[r] = scales_of<FMT>(sk, sv, sl2);
                m.iv[r] = over_scale<FMT>(sv);
              }
              mult_k = exact ? kOne : scale_of<FMT>(sk, most_k);
              mult_v = exact ? sign_of<FMT>(sv) : scale_of<FMT>(sv, most_v);
              __syncwarp();
              if (lane == 0) mbar_arrive(smem_u32(&c.meta_full[k % kMeta]));
            }
            const uint32_t mult = x ? mult_v : mult_k;
            constexpr int CH = D / 16, RPI = 32 / CH, NI = 32 / RPI;
            const int ch = lane % CH, r0 = q * 32 + lane / CH;
            const uint32_t from = at + Sh::tile_bytes / 2 + ch * 16;
            // The lane's two chunks of f16 in its first row (lanes of the upper half of a row store them in the other order: no bank
            // twice); in its i-th one RPI rows further, where rows four apart swap halves of the swizzle.
            const bool swap = CH == 8 && ch >= 4;
            const uint32_t to1 = at + Sh::at(r0, 2 * ch + swap), to2 = at + Sh::at(r0, 2 * ch + !swap);
            auto convert = [&](int i, const uint4& v) {
              const uint32_t m = __shfl_sync(0xffffffffu, mult, lane / CH + i * RPI), flip = RPI == 4 ? (i & 1) * 64 : 0;
              uint4 a = scaled8<FMT>(v.x, v.y, m), b = scaled8<FMT>(v.z, v.w, m);
              if (x && partly && part_seen(t0 - q * 32 + r0 + i * RPI) && !(chunk_finite<true>(a) && chunk_finite<true>(b))) {
                bad = true;
                a = chunk_or_zero<true>(a);
                b = chunk_or_zero<true>(b);
              }
              sts128((to1 ^ flip) + i * RPI * 128, swap ? b : a);
              sts128((to2 ^ flip) + i * RPI * 128, swap ? a : b);
            };
            if constexpr (D == 64) {
              uint4 v[NI];
#pragma unroll
              for (int i = 0; i < NI; ++i) v[i] = lds128(from + (r0 + i * RPI) * D);
              takers_sync();
#pragma unroll
              for (int i = 0; i < NI; ++i) convert(i, v[i]);
            } else {
              uint4 next = lds128(from + r0 * D);
#pragma unroll 2
              for (int i = 0; i < NI; ++i) {
                const uint4 v = next;
                if (i + 1 < NI) next = lds128(from + (r0 + (i + 1) * RPI) * D);
                __syncwarp();              // (all lanes have read these rows)
                convert(i, v);
              }
            }
            fence_proxy_async_smem();
          } else if (partly) {
            constexpr int CH = D / 8, RPI = 32 / CH;
            const int ch = lane % CH;
#pragma unroll 4
            for (int r = q * 32 + lane / CH; r < q * 32 + 32; r += RPI) {
              const uint32_t to = at + Sh::at(r, ch);
              const uint4 v = lds128(to);
              if (part_seen(t0 - q * 32 + r) && !chunk_finite<false>(v)) {
                bad = true;
                sts128(to, chunk_or_zero<false>(v));
              }
            }
            fence_proxy_async_smem();
          }
          if (x && partly && __any_sync(0xffffffffu, bad) && lane == 0) *reinterpret_cast<volatile int*>(&c.bad[sl]) = 1;
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(smem_u32(&c.full[st]));
          }
        }
        if (gone) break;
      }
      kt += w.n;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&c.piece_empty[sl]));
    }
  } else if (warp >= kLoadWarp) {
    // =========================== K and V tiles ============================
    // Groups of 16 tokens of K, then of V, tile by tile (K0 V0 K1 V1 ..), dealt to the warps in turn: every warp has one or two of
    // each tile.
    const int lw = warp - kLoadWarp;
    uint32_t kt = 0, gg = 0;             // key tiles and groups of the pieces before
    const float sl2 = p.scale * kLog2e;
    constexpr int CH = (CODED ? D : 2 * D) / 16, TPI = 32 / CH, NI = kGroup / TPI;   // 16-byte chunks of a token; tokens of an instruction; instructions
    const int ch = lane % CH, sub_t = lane / CH;
    for (int it = 0;; ++it) {
      const int sl = it % kPieces;
      if (!piece_here(c, it)) break;
      const ChunkPiece& w = c.piece[sl];
      const int32_t* const table = p.table + w.b * p.table_stride;
      const int groups = w.n * 2 * kGroups, ta = w.ta, kept = w.kept, skip = w.skip, end = w.end, low = w.low;
      const long long head_off = w.kvh * p.c.head_bytes;
      bool bad = false;
      // First token of group g of the piece.
      auto token0 = [&](int g) {
        const int t = ta + g / (2 * kGroups);
        return (t < kept ? t : t + skip) * kTile + (g % kGroups) * kGroup;
      };
      // Page of this lane's token (lanes 16 .. 31 as lanes 0 .. 15) and its slot; -1: nobody sees it.
      auto look_up = [&](int g, int& slot) {
        const int t = token0(g) + (lane & 15);
        slot = 0;
        if (t > end || (t < low && t >= p.sinks)) return -1;
        const int entry = p.page_shift >= 0 ? t >> p.page_shift : t / p.c.page_size;
        slot = t - entry * p.c.page_size;
        return __ldg(table + entry);
      };
      auto stage_of = [&](int g) { return 2 * ((kt + g / (2 * kGroups)) % NP) + (g / kGroups) % 2; };
      // Of a group: some of its tokens are seen by some rows and not by others.
      auto partly = [&](int g) {
        const int t = token0(g);
        return !(t + kGroup - 1 <= w.first && (t > end - p.window || t + kGroup - 1 < p.sinks));
      };
      auto part_seen = [&](int t) { return !(t <= w.first && (t > end - p.window || t < p.sinks)); };
      const int g0 = static_cast<int>((lw + kLoaders - gg % kLoaders) % kLoaders);   // this warp's first group
      // Group g's stage (K: and the masks of its tile) is free; false: it has to be waited for.
      auto ready = [&](int g, bool block) {
        const uint32_t k = kt + g / (2 * kGroups);
        unsigned long long& stage = c.empty[stage_of(g)];
        unsigned long long& meta = c.meta_empty[k % kMeta];
        const uint32_t ph = ((k / NP) - 1) & 1, mph = ((k / kMeta) - 1) & 1;
        const bool has = k >= NP, keys = k >= kMeta && (g / kGroups) % 2 == 0;
        if (block) {
          if (has) wait(c, stage, ph);
          if (keys) wait(c, meta, mph);
          return true;
        }
        return static_cast<bool>(__all_sync(0xffffffffu, (!has || passed(stage, ph)) && (!keys || passed(meta, mph))));
      };
      auto arrive = [&](int g) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if ((g / kGroups) % 2 == 0) mbar_arrive(smem_u32(&c.meta_full[(kt + g / (2 * kGroups)) % kMeta]));
          mbar_arrive(smem_u32(&c.full[stage_of(g)]));
        }
      };
      if constexpr (!CODED) {
        int next = g0;                   // the oldest group that has not been handed over
        auto hand_over = [&]() {         // its copies have landed
          if ((next / kGroups) % 2 && partly(next)) {
            const uint32_t at = ring + stage_of(next) * Sh::tile_bytes;
            const int t0 = token0(next), r0 = (next % kGroups) * kGroup;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
              const int t = i * TPI + sub_t;
              const uint32_t to = at + Sh::at(r0 + t, ch);
              const uint4 v = lds128(to);
              if (part_seen(t0 + t) && !chunk_finite<false>(v)) {
                bad = true;
                sts128(to, chunk_or_zero<false>(v));
              }
            }
            if (__any_sync(0xffffffffu, bad) && lane == 0) *reinterpret_cast<volatile int*>(&c.bad[sl]) = 1;
          }
          arrive(next);
          next += kLoaders;
        };
        int slot = 0, page = g0 < groups ? look_up(g0, slot) : -1;
        for (int g = g0; g < groups; g += kLoaders) {
          const bool there = page >= 0 && page < p.c.num_pages;
          const long long off = there ? page * p.c.page_bytes + head_off + slot * p.c.token_bytes : -1;
          const uint32_t live = __ballot_sync(0xffffffffu, there) & 0xffffu;
          if (g + kLoaders < groups) page = look_up(g + kLoaders, slot);     // (while this group is on its way)
          if (!ready(g, false)) {        // (what is in flight may be what it waits for)
            cp_async_wait_n<0>();
            while (next < g) hand_over();
            ready(g, true);
            if (__any_sync(0xffffffffu, failed(c))) break;
          }
          const bool keys = (g / kGroups) % 2 == 0;
          const unsigned char* const from = keys ? p.c.k : p.c.v;
          const uint32_t at = ring + stage_of(g) * Sh::tile_bytes;
          const int r0 = (g % kGroups) * kGroup;
          if (keys && lane == 0) reinterpret_cast<uint16_t*>(metas[(kt + g / (2 * kGroups)) % kMeta].live)[g % kGroups] = static_cast<uint16_t>(live);
#pragma unroll
          for (int i = 0; i < NI; ++i) {
            const int t = i * TPI + sub_t;
            const long long o = __shfl_sync(0xffffffffu, off, t);
            cp_async16_n(at + Sh::at(r0 + t, ch), from + (o < 0 ? 0 : o) + ch * 16, o < 0 ? 0 : 16);
          }
          cp_async_commit();
          if (next + kLag * kLoaders <= g) {
            cp_async_wait_n<kLag>();
            hand_over();
          }
        }
        cp_async_wait_n<0>();
        while (next < groups && !__any_sync(0xffffffffu, failed(c))) hand_over();
      } else {
        // A group's codes are loaded while the one before it is converted, its pages looked up one ahead of that.
        uint4 cur[NI], ahead[NI];
        float ks = 0.f, vs = 0.f;        // scales of the group loaded last (of both: K's and V's groups decide alike)
        bool there = false;
        int slot = 0, page = g0 < groups ? look_up(g0, slot) : -1;
        auto fetch = [&](int g) {        // the group whose page was looked up
          there = page >= 0 && page < p.c.num_pages;
          const long long off = there ? page * p.c.page_bytes + head_off + slot * p.c.token_bytes : -1;
          const bool keys = (g / kGroups) % 2 == 0;
          ks = vs = 0.f;
          if (there) {
            const long long si = scale_index(p.c, page, w.kvh, slot);
            ks = __ldg(p.c.ks + si);
            vs = __ldg(p.c.vs + si);
          }
          const unsigned char* const from = keys ? p.c.k : p.c.v;
#pragma unroll
          for (int i = 0; i < NI; ++i) {
            const long long o = __shfl_sync(0xffffffffu, off, i * TPI + sub_t);
            ahead[i] = make_uint4(0, 0, 0, 0);
            if (o >= 0) ahead[i] = __ldg(reinterpret_cast<const uint4*>(from + o + ch * 16));
          }
        };
        if (g0 < groups) fetch(g0);
        for (int g = g0; g < groups; g += kLoaders) {
#pragma unroll
          for (int i = 0; i < NI; ++i) cur[i] = ahead[i];
          const float k_scale = ks, v_scale = vs;
          const uint32_t live = __ballot_sync(0xffffffffu, there) & 0xffffu;
          if (g + kLoaders < groups) {
            page = look_up(g + kLoaders, slot);
            fetch(g + kLoaders);
          }
          ready(g, true);
          if (__any_sync(0xffffffffu, failed(c))) break;
          const bool keys = (g / kGroups) % 2 == 0;
          const uint32_t at = ring + stage_of(g) * Sh::tile_bytes;
          const int r0 = (g % kGroups) * kGroup, t0 = token0(g);
          // The group's powers of two (lanes 16 .. 31 as lanes 0 .. 15), a token's scale over them.
          float most_k = magnitude(k_scale), most_v = magnitude(v_scale);
          float least_k = most_k == 0.f ? INFINITY : most_k, least_v = most_v == 0.f ? INFINITY : most_v;
#pragma unroll
          for (int o = 1; o < kGroup; o <<= 1) {
            most_k = fmaxf(most_k, __shfl_xor_sync(0xffffffffu, most_k, o));
            most_v = fmaxf(most_v, __shfl_xor_sync(0xffffffffu, most_v, o));
            least_k = fminf(least_k, __shfl_xor_sync(0xffffffffu, least_k, o));
            least_v = fminf(least_v, __shfl_xor_sync(0xffffffffu, least_v, o));
          }
          const bool split = partly(g), exact = split || wide(most_k, least_k) || wide(most_v, least_v);
          if (keys) {
            ChunkMeta& m = metas[(kt + g / (2 * kGroups)) % kMeta];
            if (lane == 0) {
              reinterpret_cast<uint16_t*>(m.live)[g % kGroups] = static_cast<uint16_t>(live);
              m.group[g % kGroups] = group_of<FMT>(most_k, most_v, sl2, exact);
            }
            if (exact && lane < kGroup) {
              m.ab[r0 + lane] = scales_of<FMT>(k_scale, v_scale, sl2);
              m.iv[r0 + lane] = over_scale<FMT>(v_scale);
            }
          }
          const uint32_t mult = exact ? (keys ? kOne : sign_of<FMT>(v_scale)) : keys ? scale_of<FMT>(k_scale, most_k) : scale_of<FMT>(v_scale, most_v);
          const bool look = !keys && split;
#pragma unroll
          for (int i = 0; i < NI; ++i) {
            const int t = i * TPI + sub_t, r = r0 + t;
            const uint32_t m = __shfl_sync(0xffffffffu, mult, t);
            uint4 a = scaled8<FMT>(cur[i].x, cur[i].y, m), b = scaled8<FMT>(cur[i].z, cur[i].w, m);
            if (look && part_seen(t0 + t) && !(chunk_finite<true>(a) && chunk_finite<true>(b))) {
              bad = true;
              a = chunk_or_zero<true>(a);
              b = chunk_or_zero<true>(b);
            }
            const bool swap = CH == 8 && ch >= 4;
            sts128(at + Sh::at(r, 2 * ch + swap), swap ? b : a);
            sts128(at + Sh::at(r, 2 * ch + !swap), swap ? a : b);
          }
          if (look && __any_sync(0xffffffffu, bad) && lane == 0) *reinterpret_cast<volatile int*>(&c.bad[sl]) = 1;
          arrive(g);
        }
      }
      kt += w.n;
      gg += groups;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&c.piece_empty[sl]));
    }
    cp_async_wait_n<0>();
  } else if (warp == kMmaWarp) {
    // ============================ MMA issue ===============================
    // The warp takes every step together, lane 0 issues. The steps are compiled for each stage of the ring, so that descriptors and
    // addresses are constants: with run-time ones an MMA took 36 instructions and the warp was busy all the time. Step j, row
    // tile after row tile: P V of key tile j, then the scores of key tile j + 1.
    constexpr uint32_t type = CODED ? (1u << 7) | (1u << 10) : 0u;     // f16 instead of BF16
    constexpr uint32_t id_s = idesc_bf16_f32(kTile, kTile) & ~type;
    constexpr uint32_t id_o = (idesc_bf16_f32(kTile, D) & ~type) | (1u << 16);   // V: MN-major
    uint32_t kt = 0, pt[2] = {0, 0}, st[2] = {0, 0};   // key tiles of the pieces before; by row tile: P V, scores so far
    int loads = 0;
    bool dead = false;
    for (int it = 0;; ++it) {
      const int sl = it % kPieces;
      const bool valid = piece_here(c, it);
      const int n0 = __shfl_sync(0xffffffffu, c.piece[sl].ni[0], 0), n1 = __shfl_sync(0xffffffffu, c.piece[sl].ni[1], 0);
      const int n = __shfl_sync(0xffffffffu, c.piece[sl].n, 0);
      if (lane == 0) mbar_arrive(smem_u32(&c.piece_empty[sl]));
      __syncwarp();
      if (!valid) break;
      dead |= wait(c, c.q_full, loads & 1);
      ++loads;
      if (__any_sync(0xffffffffu, dead)) continue;
      for (int j = -1; j < n; ++j) {
        auto step_at = [&](auto slot) {
          constexpr int S = decltype(slot)::value, N = (S + 1) % NP;       // ring slots of key tiles j and j + 1
          const uint32_t k = kt + j;
          auto values = [&](auto row_tile) {           // O_i (+)= P_i V_j, as its halves of the keys come
            constexpr int i = decltype(row_tile)::value;
            const uint64_t va = smem_desc_mn128(ring + (2 * S + 1) * Sh::tile_bytes, kTile * 128, 1024);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              dead |= wait(c, c.p_ready[i][pt[i] & 1][half], (pt[i] >> 1) & 1);
              __syncwarp();
              tc_fence_after();
              const uint32_t done = smem_u32(&c.o_done[i][pt[i] & 1]);
              if (elect_one()) {
#pragma unroll
                for (int kk = half * (kTile / 32); kk < (half + 1) * (kTile / 32); ++kk)
                  umma_bf16_ts(Sh::col_o + i * D, i * kTile + kk * 8, va + kk * (2048 >> 4), id_o, kk != 0 || j != 0);
                if (half) umma_commit(done);
              }
              __syncwarp();
            }
            ++pt[i];
          };
          auto scores = [&](auto row_tile, bool release) {   // S_i = Q_i K_{j+1}^T; release: K's last use
            constexpr int i = decltype(row_tile)::value;
            const uint64_t qa = smem_desc(q_s + i * Sh::tile_bytes, 1024, Swz::k128), ka = smem_desc(ring + 2 * N * Sh::tile_bytes, 1024, Swz::k128);
            const uint32_t done = smem_u32(&c.s_full[i][st[i] & 1]);
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {            // (descriptors hold addresses in 16-byte units)
                constexpr uint64_t atom = (kTile * 128) >> 4;
                const uint64_t o = (kk >> 2) * atom + (kk & 3) * 2;
                umma_bf16(i * kTile, qa + o, ka + o, id_s, kk != 0);
              }
              umma_commit(done);
              if (release) {
                umma_commit(smem_u32(&c.empty[2 * N]));
                if (j + 2 == n) umma_commit(smem_u32(&c.q_empty));
              }
            }
            __syncwarp();
            ++st[i];
          };
          constexpr std::integral_constant<int, 0> r0{};
          constexpr std::integral_constant<int, 1> r1{};
          if (j >= 0) dead |= wait(c, c.full[2 * S + 1], (k / NP) & 1);
          if (j + 1 < n) dead |= wait(c, c.full[2 * N], ((k + 1) / NP) & 1);
          __syncwarp();
          tc_fence_after();
          if (j >= 0 && j < n0) values(r0);
          if (j + 1 < n0) scores(r0, j + 1 >= n1);
          if (j >= 0 && j < n1) values(r1);
          if (j >= 0 && elect_one()) umma_commit(smem_u32(&c.empty[2 * S + 1]));
          __syncwarp();
          if (j + 1 < n1) scores(r1, true);
          if (j + 1 < n && j + 1 >= n0 && j + 1 >= n1) {     // (a tile that no row of the piece needs)
            if (elect_one()) {
              umma_commit(smem_u32(&c.empty[2 * N]));
              if (j + 2 == n) umma_commit(smem_u32(&c.q_empty));
            }
            __syncwarp();
          }
        };
        if (lane == 0) *reinterpret_cast<volatile int*>(&c.progress) = static_cast<int>(kt + j + 2);
        const uint32_t slot = (kt + j) % NP;
        if (slot == 0) step_at(std::integral_constant<int, 0>{});
        else if (slot == 1) step_at(std::integral_constant<int, 1>{});
        else if (NP > 2 && slot == 2) step_at(std::integral_constant<int, 2 % NP>{});
        else if (NP > 2) step_at(std::integral_constant<int, 3 % NP>{});
        if (__any_sync(0xffffffffu, dead)) break;
      }
      kt += n;
    }
    if (failed(c)) {                     // let the MMAs in flight end
      __syncwarp();
      if (elect_one()) umma_commit(smem_u32(&c.drain));
      __syncwarp();
      mbar_wait_limit(smem_u32(&c.drain), 0, kDrainLimitCycles);
    }
    __syncwarp();
  }
  } else {
    // ============================= softmax ================================
    const int i = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t col_s = lane_base + i * kTile, col_o = lane_base + Sh::col_o + i * D;
    // (finite, so that any maximum passes a reference of -infinity by it, with the smallest scales too)
    const float sl2 = p.scale * kLog2e, grow = CODED ? kGrow : fminf(kGrow / sl2, 3.402823466e38f);
    const int t_in = row / GB, g = row - t_in * GB;
    const uint32_t stage = smem_u32(chunk_smem) + Sm::stage + warp * kStageBytes;
    bool dead = false, begun = false;    // (begun: an item that the next CTA goes on with)
    uint32_t t = 0, kt = 0;              // key tiles of this row tile so far; of the pieces before
    for (int it = 0;; ++it) {
      const int sl = it % kPieces;
      if (!piece_here(c, it)) break;
      const ChunkPiece& w = c.piece[sl];
      const int at_row = i * TT + t_in, n = w.ni[i];
      const bool live = t_in < TT && g < w.heads && at_row <= w.end - w.first;
      const int pos = w.first + min(at_row, w.end - w.first);      // (the rows behind stand there too: positions go up to 2^31 - 65)
      float qf = 1.f;                      // 8 bits: Q was divided by it
      if constexpr (CODED) {               // Q from BF16 to f16, the row's largest magnitude at 2^14 .. 2^15, by a power of two
        wait(c, c.q_landed, it & 1);
        __syncwarp();
        if (i == 0 || w.end - w.first + 1 > TT) {
          const uint32_t at = q_s + i * Sh::tile_bytes;
          uint32_t m2 = 0;
#pragma unroll 4
          for (int ch = 0; ch < D / 8; ++ch) m2 = abs_max2(m2, lds128(at + Sh::at(row, ch)));
          const uint32_t biggest = max(m2 & 0xffffu, m2 >> 16);
          const int e = static_cast<int>(biggest >> 7) - 127;
          const int up = biggest == 0 || e == 128 ? 0 : max(-126, min(126, 14 - e));
          const float f = exp2_int(up);
          qf = exp2_int(-up);
#pragma unroll 2
          for (int ch = 0; ch < D / 8; ++ch) {
            const uint4 v = lds128(at + Sh::at(row, ch));
            const uint32_t x4[4] = {v.x, v.y, v.z, v.w};
            uint32_t h[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) h[y] = pack_f16x2(__uint_as_float(x4[y] << 16) * f, __uint_as_float(x4[y] & 0xffff0000u) * f);
            sts128(at + Sh::at(row, ch), make_uint4(h[0], h[1], h[2], h[3]));
          }
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&c.q_full));
      }
      float ref = -INFINITY, l = 0.f;      // exponents are relative to ref (BF16: in units of raw scores, less kGrow)
      for (int j = 0; j < n; ++j, ++t) {
        const uint32_t k = kt + j;
        const ChunkMeta& m = metas[k % kMeta];
        dead |= wait(c, c.meta_full[k % kMeta], (k / kMeta) & 1);
        dead |= wait(c, c.s_full[i][t & 1], (t >> 1) & 1);
        __syncwarp();
        tc_fence_after();
        // What the row sees of the tile.
        const int tile = w.ta + j, t0 = (tile < w.kept ? tile : tile + w.skip) * kTile;
        const uint4 there = *reinterpret_cast<const uint4*>(m.live);
        const int hi = pos - t0, lo = hi - min(p.window - 1, max(pos, 0)), sk = p.sinks - t0;    // sees x <= hi with x >= lo or x < sk
        const bool whole = hi >= kTile - 1 && (lo <= 0 || sk >= kTile) && (there.x & there.y & there.z & there.w) == 0xffffffffu;
        const bool cuts = __any_sync(0xffffffffu, live && !whole);
        // Tiles that not all rows see whole, or with scales to be taken token by token, go through tensor memory once more first: what
        // is not seen to -infinity, y in the place of such scores. The loops behind that know nothing of it.
        uint32_t exact = 0;                // groups taken token by token
        // Factor of the scores, what is added to them, and the unit of the sum (8 bits: the tile's or the group's; the factor is never
        // 0, -infinity stays itself; what is y already is summed apart).
        float f_tile = sl2, add_tile = 0.f, unit_tile = 1.f;
        auto factor = [&](int g16, float& f, float& add, float& unit) {
          const float4 g4 = m.group[g16];
          const bool y = g4.w != 0.f;
          f = y ? 1.f : fmaxf(g4.x * qf, 1e-37f);
          add = y ? 0.f : g4.y;
          unit = y ? 0.f : g4.z;
        };
        if constexpr (CODED && BOXED) {
          factor(0, f_tile, add_tile, unit_tile);
          exact = unit_tile == 0.f ? (1u << kGroups) - 1 : 0;
        } else if constexpr (CODED) {
#pragma unroll 1
          for (int g16 = 0; g16 < kGroups; ++g16) exact |= static_cast<uint32_t>(m.group[g16].w != 0.f) << g16;
        }
        if (cuts || exact) {
          auto below = [&](int x) { return x <= 0 ? 0u : x >= 16 ? 0xffffu : (1u << x) - 1; };   // bits under x
#pragma unroll 1
          for (int g16 = 0; g16 < kGroups; ++g16) {
            const int at = g16 * 16;
            const uint32_t see = reinterpret_cast<const uint16_t*>(m.live)[g16] & below(min(hi, kTile) + 1 - at) & (~below(lo - at) | below(sk - at));
            if (!(exact >> g16 & 1) && __all_sync(0xffffffffu, see == 0xffffu || !live)) continue;
            uint32_t s[16];
            tmem_ld16(col_s + at, s);
            tmem_ld_wait();
            if (CODED && (exact >> g16 & 1)) {
#pragma unroll
              for (int e = 0; e < 16; e += 2) {
                const float4 ab = *reinterpret_cast<const float4*>(m.ab + at + e);
                s[e] = __float_as_uint(__fmaf_rn(__uint_as_float(s[e]) * qf, ab.x, ab.y));
                s[e + 1] = __float_as_uint(__fmaf_rn(__uint_as_float(s[e + 1]) * qf, ab.z, ab.w));
              }
            }
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (!((see >> e) & 1)) s[e] = 0xff800000u;
            tmem_st16(col_s + at, s);
          }
          tmem_st_wait();
        }
        // 16 columns at a time, the next 16 on their way from tensor memory. The loops are not unrolled further: the roles' loops
        // share the instruction caches, and unrolled once more these took 1.25 times as long.
        uint32_t sa[16], sb[16];
        float top = -INFINITY;
        auto most = [&](int g16, const uint32_t (&s)[16]) {
          float a = fmaxf(__uint_as_float(s[0]), __uint_as_float(s[15])), b = __uint_as_float(s[1]);
#pragma unroll
          for (int e = 2; e < 14; e += 4) {
            a = max3(a, __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
            b = max3(b, __uint_as_float(s[e + 2]), __uint_as_float(s[e + 3]));
          }
          a = max3(a, b, __uint_as_float(s[14]));
          if constexpr (CODED && !BOXED) {
            float f, add, unit;
            factor(g16, f, add, unit);
            a = __fmaf_rn(a, f, add);
          }
          top = fmaxf(top, a);
        };
        tmem_ld16(col_s, sa);
#pragma unroll 1
        for (int g16 = 0; g16 < kGroups; g16 += 2) {
          tmem_ld_wait();
          tmem_ld16(col_s + g16 * 16 + 16, sb);
          most(g16, sa);
          tmem_ld_wait();
          tmem_ld16(col_s + (g16 * 16 + 32) % kTile, sa);    // (at the end: the first 16 again)
          most(g16 + 1, sb);
        }
        if constexpr (CODED && BOXED) top = __fmaf_rn(top, f_tile, add_tile);
        if (j == 0) {
          ref = top;
        } else if (__any_sync(0xffffffffu, live && top > ref + grow)) {   // (rows of nobody hold anything: no say)
          const float nr = top > ref + grow ? top : ref;                  // (a row's bits do not go by its neighbours')
          const float f = nr == -INFINITY ? 1.f : exp2_fast(CODED ? ref - nr : (ref - nr) * sl2);
          ref = nr;
          l *= f;
          dead |= wait(c, c.o_done[i][(t - 1) & 1], ((t - 1) >> 1) & 1);
          __syncwarp();
          tc_fence_after();
#pragma unroll 1
          for (int q = 0; q < D / 16; ++q) {
            uint32_t o[16];
            tmem_ld16(col_o + q * 16, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st16(col_o + q * 16, o);
          }
        }
        // (nothing seen: every weight is 0)
        const float off = ref == -INFINITY ? 0.f : CODED ? kTop - ref : __fmaf_rn(-ref, sl2, -kGrow);
        uint64_t sum[2] = {0, 0};
        if (CODED && exact) {              // sums of weight / scale, token by token
#pragma unroll 1
          for (int g16 = 0; g16 < kGroups; ++g16) {
            if (!(exact >> g16 & 1)) continue;
            uint32_t s[16];
            tmem_ld16(col_s + g16 * 16, s);
            tmem_ld_wait();
            float each[2] = {0.f, 0.f};
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const float2 iv = *reinterpret_cast<const float2*>(m.iv + g16 * 16 + e);
              each[0] = __fmaf_rn(exp2_fast(__uint_as_float(s[e]) + off), iv.x, each[0]);
              each[1] = __fmaf_rn(exp2_fast(__uint_as_float(s[e + 1]) + off), iv.y, each[1]);
            }
            l += each[0] + each[1];
          }
        }
        uint32_t pk[16];                   // 32 columns
        auto weights = [&](int g16, auto which, const uint32_t (&s)[16]) {
          constexpr int h = decltype(which)::value;
          float f = f_tile, add = add_tile;
          [[maybe_unused]] float unit = 0.f;
          if constexpr (CODED && !BOXED) factor(g16, f, add, unit);
          add += off;
          const uint64_t fp = pair(f, f), addp = pair(add, add);
          uint64_t mine[2] = {0, 0};       // the group's sum
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 x = unpair(fma2(pair(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), fp, addp));
            const float w0 = exp2_fast(x.x), w1 = exp2_fast(x.y);
            uint64_t& to = CODED && !BOXED ? mine[e & 1] : sum[e & 1];
            to = add2(to, pair(w0, w1));
            pk[8 * h + e] = CODED ? pack_f16x2(w0, w1) : pack_bf16x2(w0, w1);
          }
          if constexpr (CODED && !BOXED) sum[h] = fma2(add2(mine[0], mine[1]), pair(unit, unit), sum[h]);
        };
#pragma unroll 1
        for (int g16 = 0; g16 < kGroups; g16 += 2) {
          tmem_ld_wait();
          tmem_ld16(col_s + g16 * 16 + 16, sb);
          weights(g16, std::integral_constant<int, 0>{}, sa);
          tmem_ld_wait();
          if (g16 + 2 < kGroups) tmem_ld16(col_s + g16 * 16 + 32, sa);
          weights(g16 + 1, std::integral_constant<int, 1>{}, sb);
          tmem_st16(col_s + g16 * 8, pk);  // (over scores that are in registers or done with)
          if (g16 & 2) {                   // half of the tile
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&c.p_ready[i][t & 1][g16 >> 2]));
          }
        }
        const float2 all = unpair(add2(sum[0], sum[1]));
        l += CODED && BOXED ? (all.x + all.y) * unit_tile : all.x + all.y;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&c.meta_empty[k % kMeta]));
        if ((j & 15) == 15 && __any_sync(0xffffffffu, dead)) break;
      }
      for (int j = n; j < w.n; ++j) {      // tiles that this row tile has no use for
        const uint32_t k = kt + j;
        const bool late = wait(c, c.meta_full[k % kMeta], (k / kMeta) & 1);
        if (__any_sync(0xffffffffu, late)) break;
        if (lane == 0) mbar_arrive(smem_u32(&c.meta_empty[k % kMeta]));
      }
      kt += w.n;
      if (n > 0) dead |= wait(c, c.o_done[i][(t - 1) & 1], ((t - 1) >> 1) & 1);
      __syncwarp();
      tc_fence_after();

      const float exponent = ref == -INFINITY ? -INFINITY : CODED ? ref - kTop : __fmaf_rn(ref, sl2, kGrow);
      const long long out_row = static_cast<long long>(w.row0) + i * TT + t_in;
      if (w.ta == 0 && w.n == w.tiles) {
        // The whole item: its rows, through shared memory so that a store instruction writes whole 64-byte pieces.
        uint16_t* const to = p.out + out_row * p.out_stride + (w.h0 + g) * D;
        const uint32_t lives = __ballot_sync(0xffffffffu, live);
        const float inv = n > 0 ? inverse<CODED>(l) : 0.f;
        const uint64_t invp = pair(inv, inv);
#pragma unroll 1
        for (int q = 0; q < D / 32; ++q) {
          uint32_t o[32];
          if (n > 0) {
            tmem_ld32(col_o + q * 32, o);
            tmem_ld_wait();
          }
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint32_t r[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const float2 v = unpair(mul2(pair(__uint_as_float(o[e + 2 * y]), __uint_as_float(o[e + 2 * y + 1])), invp));
              r[y] = n > 0 ? pack_bf16x2(v.x, v.y) : 0u;
            }
            sts128(stage + lane * 64 + (((e / 8) ^ ((lane >> 1) & 3)) << 4), make_uint4(r[0], r[1], r[2], r[3]));
          }
          __syncwarp();
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int r = y * 8 + lane / 4, ch = lane % 4;
            const uint4 v = lds128(stage + r * 64 + ((ch ^ ((r >> 1) & 3)) << 4));
            uint16_t* const at = reinterpret_cast<uint16_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(to), r));
            if (((lives >> r) & 1) && !failed(c)) *reinterpret_cast<uint4*>(at + q * 32 + ch * 8) = v;
          }
          __syncwarp();
        }
        tc_fence_before();
        if (p.lse && live && !failed(c)) p.lse[out_row * p.q_heads + w.h0 + g] = n > 0 ? log_sum<CODED>(exponent, l) : -INFINITY;
        if (*reinterpret_cast<volatile int*>(&c.bad[sl]) && !failed(c)) {
          __syncwarp();
          add_not_finite<FMT, D>(p, w, warp, lane);
        }
      } else {
        // A part: exponent, sum and O of its rows into this CTA's slot, and what item it is if it begins here.
        float* const slots = reinterpret_cast<float*>(static_cast<unsigned char*>(p.workspace) + kHeadBytes);
        constexpr int SF = kSlotFloats<D>, FLAG = SF - 4;
        const int me = blockIdx.x, rows = rows_of(p, w);
        float* const mine = slots + static_cast<long long>(2 * me + (w.ta == 0)) * SF;
        const int rr = i * kTile + row;
        if (rr < rows) {
          mine[rr] = n > 0 ? exponent : -INFINITY;
          mine[2 * kTile + rr] = n > 0 ? l : 0.f;
        }
        // Each row tile says for itself whether something in V was set to zero: it has waited for its last P V, before which that is
        // known of every tile that its rows see. (The other row tile's tiles may go on behind its own.)
        if (tid % (kSoftWarps / 2 * 32) == 0) mine[FLAG + i] = __int_as_float(*reinterpret_cast<volatile int*>(&c.bad[sl]));
        if (tid == 0 && w.ta == 0) begun = true;
        if (w.ta == 0 && tid < static_cast<int>(sizeof(ChunkPiece) / 4))
          reinterpret_cast<int*>(static_cast<unsigned char*>(p.workspace) + static_cast<long long>(me) * kHead)[tid] = reinterpret_cast<const int*>(&w)[tid];
        if (i * kTile + (warp & 3) * 32 < rows) {
#pragma unroll 1
          for (int q = 0; q < D / 16; ++q) {
            uint32_t o[16];
            if (n > 0) {
              tmem_ld16(col_o + q * 16, o);
              tmem_ld_wait();
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = 0u;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
              sts128(stage + lane * 64 + ((e ^ ((lane >> 1) & 3)) << 4), make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]));
            __syncwarp();
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const int r = y * 8 + lane / 4, ch = lane % 4, ra = i * kTile + (warp & 3) * 32 + r;
              const uint4 v = lds128(stage + r * 64 + ((ch ^ ((r >> 1) & 3)) << 4));
              if (ra < rows) *reinterpret_cast<uint4*>(mine + 4 * kTile + static_cast<long long>(ra) * D + q * 16 + ch * 4) = v;
            }
            __syncwarp();
          }
        }
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&c.piece_empty[sl]));
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&c.ended));
    if (tid == 0 && (!begun || failed(c))) *reinterpret_cast<int*>(static_cast<unsigned char*>(p.workspace) + static_cast<long long>(blockIdx.x) * kHead) = 0;   // (the head's `valid`)
    // Rows that stand before the first token, in whole pairs of row tiles (others are rows of an item): zeros.
    for (int b = blockIdx.x; b < p.batch; b += gridDim.x) {
      const Seq s = sequence(p, b);
      const int none = s.n == 0 ? 0 : s.len == 0 ? s.n : max(0, s.n - s.len) / step * step;
      for (int r = warp; r < none; r += kSoftWarps) {
        uint16_t* const to = p.out + (static_cast<long long>(s.q0) + r) * p.out_stride;
        for (int x = lane; x < p.q_heads * D / 8; x += 32) *reinterpret_cast<uint4*>(to + x * 8) = make_uint4(0, 0, 0, 0);
        if (p.lse)
          for (int x = lane; x < p.q_heads; x += 32) p.lse[(static_cast<long long>(s.q0) + r) * p.q_heads + x] = -INFINITY;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (tid == 0 && failed(c)) {           // items that this CTA has a part of are not joined
    atomicOr(&g_chunk_status, kChunkTimeoutBit);
    float* const slots = reinterpret_cast<float*>(static_cast<unsigned char*>(p.workspace) + kHeadBytes);
    for (int y = 2 * blockIdx.x; y < 2 * static_cast<int>(blockIdx.x) + 2; ++y)
      slots[static_cast<long long>(y) * kSlotFloats<D> + kSlotFloats<D> - 4] = __int_as_float(kGone);
  }
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(0, 512);
  }
}

// Joins the parts of the item that CTA blockIdx.x began, if others went on with it: rows 32 blockIdx.y .. of it.
template <int FMT, int D>
__global__ void __launch_bounds__(256) chunk_join_kernel(const __grid_constant__ ChunkArgs p) {
  constexpr bool CODED = FMT != kKvBf16;
  constexpr int SF = kSlotFloats<D>, FLAG = SF - 4, T = 32 * (D / 4) / 256, Y = 8 / T > 2 ? 8 / T : 2;
  __shared__ float s_top[32], s_inv[32];
  __shared__ int s_bad, s_gone;
  const int tid = threadIdx.x, r0 = blockIdx.y * 32;
  if (tid == 0) s_bad = s_gone = 0;
  pdl_wait_then_release();
  const ChunkPiece& w = *reinterpret_cast<const ChunkPiece*>(static_cast<const unsigned char*>(p.workspace) + static_cast<long long>(blockIdx.x) * kHead);
  if (!__ldcg(&w.valid)) return;
  const int rows = rows_of(p, w), tokens = w.end - w.first + 1, TT = p.tile_tokens, GB = p.head_block, count = w.c1 - w.c0 + 1;
  if (r0 >= rows) return;
  const float* const slots = reinterpret_cast<const float*>(static_cast<const unsigned char*>(p.workspace) + kHeadBytes) + static_cast<long long>(2 * w.c0) * SF;
  // (the item's first CTA has its part in the second of its slots)
  auto slot_of = [&](int y) { return slots + (y == 0 ? 1LL : 2LL * y) * SF; };
  __syncthreads();
  float e_all = -INFINITY, l_all = 0.f;
  if (tid < 32) {
    const int r = r0 + tid;
    if (r < rows) {
#pragma unroll 8
      for (int y = 0; y < count; ++y) e_all = fmaxf(e_all, __ldcg(slot_of(y) + r));
      const float from = e_all == -INFINITY ? 0.f : e_all;
#pragma unroll 8
      for (int y = 0; y < count; ++y) l_all += __ldcg(slot_of(y) + 2 * kTile + r) * exp2_fast(__ldcg(slot_of(y) + r) - from);
      s_top[tid] = from;
      s_inv[tid] = inverse<CODED>(l_all);
    }
  } else {
    for (int y = tid - 32; y < count; y += 224) {
      const int2 flags = __ldcg(reinterpret_cast<const int2*>(slot_of(y) + FLAG));
      if (((flags.x | flags.y) & 1) != 0) s_bad = 1;
      if (((flags.x | flags.y) & kGone) != 0) s_gone = 1;
    }
  }
  __syncthreads();
  if (s_gone) return;
  if (p.lse && tid < 32 && r0 + tid < rows) {
    const int r = r0 + tid, rt = r % kTile / GB, rg = r % kTile - rt * GB, tok = r / kTile * TT + rt;
    if (rt < TT && rg < w.heads && tok < tokens)
      p.lse[(static_cast<long long>(w.row0) + tok) * p.q_heads + w.h0 + rg] = log_sum<CODED>(e_all, l_all);
  }
  // A team of D / 4 lanes a row, 16 bytes a lane and part: T rows and Y parts of each thread in flight together.
  constexpr int LANES = D / 4, TEAMS = 256 / LANES;
  const int team = tid / LANES, d = tid % LANES * 4;
  float4 acc[T];
#pragma unroll
  for (int x = 0; x < T; ++x) acc[x] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int y0 = 0; y0 < count; y0 += Y) {
    float4 v[T][Y];
    float e[T][Y];
#pragma unroll
    for (int y = 0; y < Y; ++y)
#pragma unroll
      for (int x = 0; x < T; ++x) {
        const int r = r0 + team + x * TEAMS;
        e[x][y] = -INFINITY;
        v[x][y] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (y0 + y < count && r < rows) {
          e[x][y] = __ldcg(slot_of(y0 + y) + r);
          v[x][y] = __ldcg(reinterpret_cast<const float4*>(slot_of(y0 + y) + 4 * kTile + r * D + d));
        }
      }
#pragma unroll
    for (int y = 0; y < Y; ++y)
#pragma unroll
      for (int x = 0; x < T; ++x) {
        if (y0 + y >= count) continue;
        const float f = exp2_fast(e[x][y] - s_top[(team + x * TEAMS) & 31]);
        acc[x].x += v[x][y].x * f;
        acc[x].y += v[x][y].y * f;
        acc[x].z += v[x][y].z * f;
        acc[x].w += v[x][y].w * f;
      }
  }
#pragma unroll
  for (int x = 0; x < T; ++x) {
    const int at = team + x * TEAMS, r = r0 + at, rt = r % kTile / GB, rg = r % kTile - rt * GB, tok = r / kTile * TT + rt;
    if (r >= rows || rt >= TT || rg >= w.heads || tok >= tokens) continue;
    const float inv = s_inv[at];
    *reinterpret_cast<uint2*>(p.out + (static_cast<long long>(w.row0) + tok) * p.out_stride + (w.h0 + rg) * D + d) =
        make_uint2(pack_bf16x2(acc[x].x * inv, acc[x].y * inv), pack_bf16x2(acc[x].z * inv, acc[x].w * inv));
  }
  if (s_bad) {
    __syncthreads();
    if (tid < 32) add_not_finite<FMT, D>(p, w, blockIdx.y, tid);
  }
}

namespace {

template <int FMT, int D, bool BOXED>
int launch_one(const ChunkArgs& a, void* stream) {
  const auto kernel = chunk_kernel<FMT, D, BOXED>;
  // (set on every call: the attribute belongs to the current device, like the launch)
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, ChunkSmem<D>::bytes);
  int dev = 0, sms = 0;
  if (e == cudaSuccess) e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return static_cast<int>(e);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(sms < kMostCtas ? sms : kMostCtas), 1, 1);
  cfg.blockDim = dim3(kChunkThreads, 1, 1);
  cfg.dynamicSmemBytes = ChunkSmem<D>::bytes;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, a);
  if (e != cudaSuccess) return static_cast<int>(e);
  cfg.gridDim.y = 2 * kTile / 32;
  cfg.blockDim = dim3(256, 1, 1);
  cfg.dynamicSmemBytes = 0;
  return static_cast<int>(cudaLaunchKernelEx(&cfg, chunk_join_kernel<FMT, D>, a));
}

template <int FMT>
int launch_format(const ChunkArgs& a, void* stream) {
  if (a.head_dim == 128) return a.box_tokens ? launch_one<FMT, 128, true>(a, stream) : launch_one<FMT, 128, false>(a, stream);
  return a.box_tokens ? launch_one<FMT, 64, true>(a, stream) : launch_one<FMT, 64, false>(a, stream);
}

}  // namespace

int launch_chunk(const ChunkArgs& a, void* stream) {
  switch (a.format) {
    case kKvBf16: return launch_format<kKvBf16>(a, stream);
    case kKvE4m3: return launch_format<kKvE4m3>(a, stream);
    default: return launch_format<kKvInt8>(a, stream);
  }
}

int read_chunk_status(void* stream, uint32_t* out, int clear) {
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint32_t v = 0;
  cudaError_t err = cudaMemcpyFromSymbolAsync(&v, g_chunk_status, sizeof v, 0, cudaMemcpyDeviceToHost, s);
  if (err == cudaSuccess && clear) {
    static const uint32_t z = 0;
    err = cudaMemcpyToSymbolAsync(g_chunk_status, &z, sizeof z, 0, cudaMemcpyHostToDevice, s);
  }
  if (err == cudaSuccess) err = cudaStreamSynchronize(s);
  *out = v;
  return static_cast<int>(err);
}

}  // namespace glora
