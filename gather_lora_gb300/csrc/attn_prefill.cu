// Causal attention over packed sequences of different lengths (sm_103a).
//
//   z_ij = scale (q_i . k_j) for j <= i + Lk - Lq,   out_i = sum_j softmax(z_i)_j v_j
//
// Both products run on the fifth-generation tensor cores (tcgen05, M = 128, fp32 accumulators in tensor
// memory), with a running softmax between them: per 128 x 128 block of pairs 4 * 128^2 * D flops of MMA
// (1024 clocks of the SM's tensor pipe at D = 128, 512 at 64), 128^2 exponentials (512 clocks of the special
// function units) and as many multiply-adds, sums and maxima. Past a few hundred keys what bounds it is a
// warpgroup's chain per block: softmax 1300 clocks, then its P V and next Q K^T; two warpgroups hide most
// of each other's.
//
// Measured on a GB300 (32 heads over 4, head_dim 128): a prompt of 8192 345 us in a burst, 1.59 PFLOP/s, and
// 370 held under the 1400 W limit; 12 packed prompts to 1100 (32 over 8) 78 us; chunks of up to 513 rows after
// 6000 keys at head_dim 64 50 us; one prompt of 37 rows 6.9 us.
//
// Rows of a tile. The G query heads that share a key-value head read the same keys, so a 128-row tile
// holds TT = 128 / G tokens x G heads (row = token * G + head; one 3-D TMA box): short prompts and
// single-token chunks fill tiles G times as well, and one stream of K and V serves all heads of the group.
// A work item is two such row tiles of one sequence, key-value head and (G > 128) block of heads.
//
// CTA: one per SM, persistent over the items. Two warpgroups each own one row tile: thread = row, with its
// running reference and sum in registers. They alternate on the tensor pipe: while one does its softmax,
// the other's P V and the next Q K^T run. Warp 8 issues the MMAs, warp 9 picks the items and issues TMA: K and
// V tiles of 128 keys through one ring of stages, the next item's Q as soon as the last Q K^T has read the old.
// Warps 10 and 11 look through V tiles (below).
// Tensor memory: two (D = 128) or three (D = 64) score buffers of 128 columns, P as BF16 pairs over the first
// half of its scores, and O0, O1.
//
// Softmax: exponents are base 2. The reference that exponents are relative to follows the running maximum
// only when that has grown by more than 2^8 (one vote per warp): then l and O are multiplied by
// 2^(old - new); otherwise weights are kept as they are. Exponents are 8 less than the reference says, so
// weights stay at most 1 (O overflows only where sums of V itself would) and BF16 and fp32 hold them alike.
//
// Rounding to fewer bits: the weights to BF16 before P V (the tensor cores' operand type), the output once.
// Keys that a row does not see get weight zero, but zero times NaN or infinity in their V rows is NaN in
// an MMA. Only the last key tiles of an item (at most three) hold keys that some row does not see: warps 10 and 11
// look through the V of those, beside the scores' MMAs and the softmax. What is not finite they set to zero for
// the P V, and add to the result rows that do see it once those are stored: a price by the tile, whatever the
// length of the context (NaN throughout a prompt of 8192: 0.41 ms against 0.35). On clean data the look costs 12 packed
// prompts 75 -> 78 us, a prompt of 8192 1%; with the waits or the additions in the other warps' loops it was 80 to 91.
#include <cooperative_groups.h>

#include <type_traits>

#include "attn_common.cuh"
#include "tc05.cuh"

namespace cg = cooperative_groups;

namespace glora {

__device__ unsigned int g_prefill_status = 0;

namespace {

constexpr unsigned kPrefillTimeoutBit = 0x2u;   // LORA_DEV_TIMEOUT
constexpr int kTile = 128;                      // rows of a tile, keys of a tile
constexpr int kSoftmaxWarps = 8;
constexpr int kPreMmaWarp = 8, kPreTmaWarp = 9, kPreScanWarp = 10, kScanWarps = 2;
constexpr int kPreThreads = 384;
// Registers a thread: 168 at launch (65536 over 12 warps); the helper warpgroup gives 96 away, the softmax
// warpgroups hold a whole row of scores: 2 * 216 + 72 = 3 * 168.
constexpr int kHelperRegs = 72, kSoftmaxRegs = 216;
constexpr int kOutBytes = 4096;                 // staging of a warp's results: 32 rows x 64 columns
constexpr int kItems = 4;                       // depth of the item ring
constexpr int kJobs = 8;                        // V tiles to look through: at most 4 in the ring's stages, and the end
constexpr float kRescale = 8.f;                 // reference moves when the maximum grew by 2^8

template <int D>
struct PrefillShape {
  static constexpr int atoms = D / 64;                          // 64-column boxes of a tile
  static constexpr int tile_bytes = kTile * D * 2;              // Q row tile, K tile or V tile
  static constexpr int stages = D == 128 ? 4 : 8;
  static constexpr int bufs = D == 128 ? 2 : 3;                 // score buffers in tensor memory: what O0 and O1 leave
  static constexpr uint32_t col_o = 512 - 2 * D;                // columns: scores at 0, 128 (, 256), O0, O1 at the end
  // Score buffer of row tile i and key tile j.
  static __device__ __forceinline__ uint32_t buf(int i, int j) { return bufs == 2 ? i : (2u * j + i) % 3u; }
  static constexpr int smem = (2 + stages) * tile_bytes + kSoftmaxWarps * kOutBytes + 2048;   // + control, alignment
};

struct PrefillItem {
  int valid;
  int q0, k0;          // first query row of the item, first key row of its sequence
  int tok0, lq, lk;    // first token of the item in the sequence; the sequence's rows and keys
  int n[2];            // key tiles of each row tile (split: of this CTA's part of the keys)
  int shift;           // keys of the sequence before the first of them (0 unless split)
  int h0, heads, kvh;  // first query head, how many, key-value head
  int whole;           // keys that every row sees (of this CTA's part): key tiles from whole / 128 on are looked through
};

struct PrefillCtl {
  unsigned long long full[8], empty[8];   // (K tiles lie in even stages, V tiles in odd ones, whose `full` takes two arrivals)
  unsigned long long q_full, q_empty;
  unsigned long long s_full[2][2], p_ready[2][2][2], o_done[2][2];   // [row tile][parity of its key tile] ([half])
  unsigned long long item_full[kItems], item_empty[kItems];
  unsigned long long drain, next_full;
  unsigned long long landed[kJobs];    // the V tile of a job is there; `full` follows when it has been looked through
  uint4 next;                          // the answer to ask_next_block
  PrefillItem item[2 * kItems];        // (twice the ring's depth: an item can be read until its rows are stored)
  int2 job[kJobs];                     // a V tile to look through: (item, stage + 16 (first row + 256 if the item's last)); item -1: the end
  int stored[kSoftmaxWarps];           // items whose result rows the warp has stored
  int bad[kScanWarps];                 // (split) a part's V held values that are not finite, by halves of the columns
  uint32_t tmem;
  int failed;
};
static_assert(sizeof(PrefillCtl) <= 1024, "control block");

__device__ __forceinline__ bool failed(const PrefillCtl& c) { return *reinterpret_cast<const volatile int*>(&c.failed) != 0; }

// Bounded wait; true if it ran out. Once one has, all others of the CTA end at once, the roles leave their
// loops at the next point where their warp is together, nothing more is stored and no further item is taken
// (what runs on until then stays in bounds).
__device__ __forceinline__ bool pre_wait(PrefillCtl& c, unsigned long long& bar, uint32_t parity) {
  const uint32_t b = smem_u32(&bar);
  if (mbar_try_wait(b, parity, 100000)) return false;
  const long long t0 = clock64();
  while (!mbar_try_wait(b, parity, 100000)) {
    if (failed(c)) return true;
    if (clock64() - t0 > kWaitLimitCycles) {
      *reinterpret_cast<volatile int*>(&c.failed) = 1;
      atomicOr(&g_prefill_status, kPrefillTimeoutBit);
      return true;
    }
  }
  return false;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* map, int c0, int c1, int c2, uint32_t bar) {
  asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n"
               ::"r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
               : "memory");
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

// The grid's next block that has not started, taken over by this CTA: the answer (16 bytes at shared
// address `to`) arrives on mbarrier `bar`.
__device__ __forceinline__ void ask_next_block(uint32_t to, uint32_t bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];\n" ::"r"(to), "r"(bar)
               : "memory");
}
// Its blockIdx.x, or -1: no block was left.
__device__ __forceinline__ long long next_block(uint32_t from) {
  uint32_t x, got;
  asm volatile(
      "{\n .reg .b128 h;\n .reg .pred p;\n .reg .b32 y, z, w;\n"
      " ld.shared.b128 h, [%2];\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n"
      " selp.u32 %1, 1, 0, p;\n mov.u32 %0, 0;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, y, z, w}, h;\n}\n"
      : "=&r"(x), "=&r"(got)
      : "r"(from)
      : "memory");
  return got ? static_cast<long long>(x) : -1;
}

}  // namespace

// What was set to zero in half `half` of the columns of an item's V (its keys from w.whole on, rounded down to 8) is added to the
// stored result rows that see it, as it is, since their weights are positive. By a warp.
template <int D>
__device__ __forceinline__ void add_not_finite(const PrefillArgs& p, const PrefillItem& w, int half, int lane) {
  const int col = half * (D / 2) + 2 * lane;           // two columns a lane
  const bool mine = lane < D / 4;
  const uint16_t* const v = p.v + w.k0 * p.v_stride + w.kvh * D + col;
  float s0 = 0.f, s1 = 0.f;                            // of the keys so far; 0: nothing
  int k = w.whole & ~7;
  for (int tok = w.tok0; tok < min(w.tok0 + 2 * p.tile_tokens, w.lq); ++tok) {
    for (const int seen = min(w.lk, tok + 1 + w.lk - w.lq); k < seen; ++k) {
      const uint32_t x = mine ? __ldg(reinterpret_cast<const uint32_t*>(v + k * p.v_stride)) : 0u;
      if ((x & 0x7f80u) == 0x7f80u) s0 += __uint_as_float(x << 16);
      if ((x & 0x7f800000u) == 0x7f800000u) s1 += __uint_as_float(x & 0xffff0000u);
    }
    if (!__any_sync(0xffffffffu, s0 != 0.f || s1 != 0.f)) continue;
    uint16_t* const out = p.out + (w.q0 + tok - w.tok0) * p.out_stride + w.h0 * D + col;
#pragma unroll 4
    for (int g = 0; g < w.heads; ++g) {
      uint32_t* const at = reinterpret_cast<uint32_t*>(out + g * D);
      if (!mine) continue;
      const uint32_t x = *at;
      *at = pack_bf16x2(__uint_as_float(x << 16) + s0, __uint_as_float(x & 0xffff0000u) + s1);
    }
  }
}

// Sets what is not finite in half `half` of the columns of a V tile (rows first .. 127, first a multiple of 8) to zero, for
// the tensor cores; true if there was any. By a warp: 16-byte chunks, 8 of half a row by D = 128 (4 rows at a time),
// 4 by D = 64 (8 rows).
template <int D>
__device__ __forceinline__ bool zero_not_finite(uint32_t tile, int first, int half, int lane) {
  constexpr int across = D / 16, rows = 32 / across;
  const int r0 = lane / across, ch = lane % across + (D == 64 ? half * 4 : 0);
  const uint32_t from = tile + (D == 128 ? half * (kTile * 128) : 0) + r0 * 128;
  auto at = [&](int row) { return from + row * 128 + ((ch ^ ((row + r0) & 7)) << 4); };
  uint32_t m = 0;
#pragma unroll 2
  for (int row = first; row < kTile; row += rows) m = abs_max2(m, lds128(at(row)));
  if (!__any_sync(0xffffffffu, !all_finite(m))) return false;
  for (int row = first; row < kTile; row += rows) {
    const uint4 x = lds128(at(row));
    sts128(at(row), make_uint4(finite_or_zero(x.x), finite_or_zero(x.y), finite_or_zero(x.z), finite_or_zero(x.w)));
  }
  fence_proxy_async_smem();
  return true;
}

// How many items each softmax warp has stored: behind the rows themselves.
__device__ __forceinline__ void publish(int* at, int v) {
  asm volatile("st.release.cta.shared::cta.s32 [%0], %1;\n" ::"r"(smem_u32(at)), "r"(v) : "memory");
}
__device__ __forceinline__ int published(const int* at) {
  int v;
  asm volatile("ld.acquire.cta.shared::cta.s32 %0, [%1];\n" : "=r"(v) : "r"(smem_u32(at)) : "memory");
  return v;
}
// Wait (bounded) until all of them have stored `items` items.
__device__ __forceinline__ bool wait_stored(PrefillCtl& c, int items, int lane) {
  const long long t0 = clock64();
  while (!__all_sync(0xffffffffu, published(&c.stored[lane % kSoftmaxWarps]) >= items)) {
    if (__any_sync(0xffffffffu, failed(c))) return false;
    if (__any_sync(0xffffffffu, clock64() - t0 > kWaitLimitCycles)) {
      *reinterpret_cast<volatile int*>(&c.failed) = 1;
      atomicOr(&g_prefill_status, kPrefillTimeoutBit);
      return false;
    }
    __nanosleep(100);
  }
  return true;
}

// SPLIT: a cluster of CTAs takes one item, each an equal part of its key tiles, and joins through the others'
// shared memory; otherwise a CTA takes items one after the other.
template <int D, bool SPLIT>
__global__ void __launch_bounds__(kPreThreads, 1) prefill_kernel(const __grid_constant__ PrefillArgs p) {
  using Sh = PrefillShape<D>;
  constexpr int NS = Sh::stages;
  static_assert(NS % 2 == 0 && NS / 2 + 1 <= kJobs && NS <= 16 && 2 * kItems <= 16 && kScanWarps == 2, "jobs");
  extern __shared__ unsigned char prefill_smem_raw[];
  const uint32_t raw = smem_u32(prefill_smem_raw), pad = ((raw + 1023u) & ~1023u) - raw;
  const uint32_t q_s = raw + pad, ring = q_s + 2 * Sh::tile_bytes;
  const uint32_t out_s = ring + NS * Sh::tile_bytes;
  PrefillCtl& c = *reinterpret_cast<PrefillCtl*>(prefill_smem_raw + pad + (2 + NS) * Sh::tile_bytes + kSoftmaxWarps * kOutBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const cg::cluster_group cluster = cg::this_cluster();
  const int parts = SPLIT ? static_cast<int>(cluster.num_blocks()) : 1, part = SPLIT ? static_cast<int>(cluster.block_rank()) : 0;

  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(smem_u32(&c.full[s]), 1 + (s & 1));
      mbar_init(smem_u32(&c.empty[s]), 1);
    }
    mbar_init(smem_u32(&c.q_full), 1);
    mbar_init(smem_u32(&c.q_empty), 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&c.s_full[i >> 1][i & 1]), 1);
      mbar_init(smem_u32(&c.p_ready[i >> 1][i & 1][0]), 4);
      mbar_init(smem_u32(&c.p_ready[i >> 1][i & 1][1]), 4);
      mbar_init(smem_u32(&c.o_done[i >> 1][i & 1]), 1);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(smem_u32(&c.item_full[i]), 1);
      mbar_init(smem_u32(&c.item_empty[i]), kSoftmaxWarps + 1);
    }
    for (int i = 0; i < kJobs; ++i) mbar_init(smem_u32(&c.landed[i]), 1);
    mbar_init(smem_u32(&c.drain), 1);
    mbar_init(smem_u32(&c.next_full), 1);
    c.failed = 0;
    for (int i = 0; i < kSoftmaxWarps; ++i) c.stored[i] = 0;
    for (int i = 0; i < kScanWarps; ++i) c.bad[i] = 0;
    mbar_fence_init();
  }
  if (warp == kPreMmaWarp) {
    tmem_alloc(smem_u32(&c.tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem;

  pdl_wait_then_release();

  int met = 0;           // cluster barriers this thread has passed
  const int TT = p.tile_tokens, step = 2 * TT, GB = p.head_block;
  const int G = p.q_heads / p.kv_heads, blocks = (G + GB - 1) / GB, subs = p.kv_heads * blocks;

  if (warp >= kSoftmaxWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kHelperRegs));
  if (warp >= kPreScanWarp) {
    // ================ V tiles that not every row sees whole ================
    // Each warp takes half of the columns, from the first key on that not every row sees: what is not finite is set to
    // zero, then the tile is `full`. A job's barrier is used again only when its stage is, which is after that.
    const int half = warp - kPreScanWarp;
    bool bad = false;                    // in this item
    for (uint32_t job = 0;; ++job) {
      pre_wait(c, c.landed[job % kJobs], (job / kJobs) & 1);
      __syncwarp();
      const int it = __shfl_sync(0xffffffffu, failed(c) ? -1 : c.job[job % kJobs].x, 0);
      if (it < 0) break;
      const int what = __shfl_sync(0xffffffffu, c.job[job % kJobs].y, 0), vs = what & 15, first = ((what >> 4) & 127) & ~7;
      bad |= zero_not_finite<D>(ring + vs * Sh::tile_bytes, first, half, lane);
      const bool add = !SPLIT && bad && (what >> 12);
      PrefillItem w;
      if (add) w = c.item[it % (2 * kItems)];          // (its slot is safe until the tile is `full`)
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&c.full[vs]));
      if (add) {
        bad = false;
        if (wait_stored(c, it + 1, lane)) add_not_finite<D>(p, w, half, lane);
      }
    }
    if constexpr (SPLIT) {               // the first part is told, and adds them when all have stored their rows
      cluster.sync();
      met = 1;
      if (lane == 0 && bad && !failed(c)) *cluster.map_shared_rank(&c.bad[half], 0) = 1;
    }
  } else if (warp == kPreTmaWarp) {
    // ======================= items and TMA loads ==========================
    int b0 = 0, it = 0, items = 0;      // chunk of 32 sequences under search; items, those with keys
    uint32_t kv = 0;                    // ring tiles issued
    uint32_t jobs = 0, by_job = 0;      // V tiles given to the look; stages whose last tile was one
    long long base = 0;                 // row-tile pairs before sequence b0
    bool go = true;
    auto ask = [&]() {                  // (lane 0) the next item, once the current one's loads are nearly out
      fence_proxy_async_smem();
      mbar_arrive_expect_tx(smem_u32(&c.next_full), 16);
      ask_next_block(smem_u32(&c.next), smem_u32(&c.next_full));
    };
    for (long long idx = blockIdx.x / parts; go; ++it) {
      // Item idx (-1: none): sequences in order, within one its last rows (the most keys) first, heads fastest.
      const long long x = idx < 0 ? -1 : idx / subs;
      const int sub = idx < 0 ? 0 : static_cast<int>(idx - x * subs);
      int q0 = 0, lq = 0, k0 = 0, lk = 0, tile = -1;
      if (x < base) base = 0, b0 = 0;   // (blocks are handed out in rising order as a rule)
      while (idx >= 0 && b0 < p.batch) {
        const int b = b0 + lane;
        int a0 = 0, a1 = 0, e0 = 0, e1 = 0;
        if (b < p.batch) {
          a0 = __ldg(p.cu_q + b);
          a1 = __ldg(p.cu_q + b + 1);
          e0 = __ldg(p.cu_k + b);
          e1 = __ldg(p.cu_k + b + 1);
        }
        const bool good = a0 >= 0 && a1 > a0 && a1 <= p.total_q && e0 >= 0 && e1 >= e0 && e1 <= p.total_k;
        const int mine = good ? (a1 - a0 - 1) / step + 1 : 0;
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int t = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += t;
        }
        const long long lo = base + incl - mine;
        const uint32_t hit = __ballot_sync(0xffffffffu, x >= lo && x < lo + mine);
        if (hit) {
          const int src = __ffs(hit) - 1;
          q0 = __shfl_sync(0xffffffffu, a0, src);
          lq = __shfl_sync(0xffffffffu, a1 - a0, src);
          k0 = __shfl_sync(0xffffffffu, e0, src);
          lk = __shfl_sync(0xffffffffu, e1 - e0, src);
          tile = __shfl_sync(0xffffffffu, mine - 1 - static_cast<int>(x - lo), src);
          break;
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
        b0 += 32;
      }
      go = tile >= 0;
      if (lane == 0) {
        const int sl = it % kItems;
        if (it >= kItems) pre_wait(c, c.item_empty[sl], ((it / kItems) - 1) & 1);
        go = go && !failed(c);
        PrefillItem w;
        w.valid = go;
        w.tok0 = tile * step;
        w.q0 = q0 + w.tok0;
        w.lq = lq;
        w.lk = lk;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int first = w.tok0 + i * TT, last = min(first + TT, lq);       // the row tile's tokens
          const int keys = min(lk, last + lk - lq);
          w.n[i] = first < lq && keys > 0 ? (keys - 1) / kTile + 1 : 0;
        }
        if constexpr (SPLIT) {
          const long long all = max(w.n[0], w.n[1]);
          const int from = static_cast<int>(part * all / parts), to = static_cast<int>((part + 1) * all / parts);
          w.n[0] = max(0, min(w.n[0], to) - from);
          w.n[1] = max(0, min(w.n[1], to) - from);
          w.shift = from * kTile;
        } else {
          w.shift = 0;
        }
        w.k0 = k0 + w.shift;
        w.whole = max(0, min(lk, w.tok0 + 1 + lk - lq) - w.shift);   // (the first row sees the fewest)
        w.kvh = sub / blocks;
        w.h0 = w.kvh * G + (sub - w.kvh * blocks) * GB;
        w.heads = min(GB, w.kvh * G + G - w.h0);
        c.item[it % (2 * kItems)] = w;
        mbar_arrive(smem_u32(&c.item_full[sl]));
        const int n = max(w.n[0], w.n[1]);
        bool asked = !SPLIT && go && n == 0;
        if (asked) ask();
        if (go && n > 0) {
          if (items > 0) pre_wait(c, c.q_empty, (items - 1) & 1);
          ++items;
          const uint32_t qb = smem_u32(&c.q_full);
          mbar_arrive_expect_tx(qb, 2 * Sh::atoms * GB * TT * 128);
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int a = 0; a < Sh::atoms; ++a)
              tma_load_3d(q_s + i * Sh::tile_bytes + a * (kTile * 128), &p.map_q, a * 64, w.h0, w.q0 + i * TT, qb);
          for (int j = 0; j < 2 * n; ++j) {      // K0 V0 K1 V1 ..
            if (!SPLIT && j == 2 * n - 2) {
              ask();
              asked = true;
            }
            const uint32_t s = kv % NS;
            if (kv >= NS && pre_wait(c, c.empty[s], ((kv / NS) - 1) & 1)) break;
            ++kv;
            const bool look = (j & 1) && (j >> 1) >= w.whole / kTile;
            const uint32_t fb = smem_u32(look ? &c.landed[jobs % kJobs] : &c.full[s]), to = ring + s * Sh::tile_bytes;
            by_job &= ~(1u << s);
            if ((j & 1) && !look) mbar_arrive(fb);
            if (look) {
              const int row = (j >> 1) == w.whole / kTile ? w.whole % kTile : 0;
              c.job[jobs++ % kJobs] = make_int2(it, s + 16 * (row + (j == 2 * n - 1 ? 256 : 0)));
              by_job |= 1u << s;
            }
            mbar_arrive_expect_tx(fb, Sh::tile_bytes);
#pragma unroll
            for (int a = 0; a < Sh::atoms; ++a)
              tma_load_2d(to + a * (kTile * 128), (j & 1) ? &p.map_v : &p.map_k, w.kvh * D + a * 64, w.k0 + (j >> 1) * kTile, fb);
          }
        }
        if (asked) {
          pre_wait(c, c.next_full, it & 1);
          if (failed(c)) mbar_wait_limit(smem_u32(&c.next_full), it & 1, kDrainLimitCycles);
          idx = failed(c) ? -1 : next_block(smem_u32(&c.next));
        } else {
          idx = -1;
        }
      }
      idx = __shfl_sync(0xffffffffu, idx, 0);
      go = __shfl_sync(0xffffffffu, go, 0);
    }
    if (lane == 0) {                     // no more jobs
      c.job[jobs % kJobs].x = -1;
      mbar_arrive(smem_u32(&c.landed[jobs % kJobs]));
    }
    if (lane == 0 && failed(c)) {        // let the loads in flight land
      for (uint32_t k = kv > NS ? kv - NS : 0; k < kv; ++k) {
        if (!((by_job >> (k % NS)) & 1)) mbar_wait_limit(smem_u32(&c.full[k % NS]), (k / NS) & 1, kDrainLimitCycles);
      }
      for (uint32_t k = jobs > NS / 2 ? jobs - NS / 2 : 0; k < jobs; ++k)
        mbar_wait_limit(smem_u32(&c.landed[k % kJobs]), (k / kJobs) & 1, kDrainLimitCycles);
      if (items > 0) mbar_wait_limit(smem_u32(&c.q_full), (items - 1) & 1, kDrainLimitCycles);
    }
    __syncwarp();
  } else if (warp == kPreMmaWarp) {
    // ============================ MMA issue ===============================
    // The whole warp takes every step, one elected lane issues. Row tile i's scores of key tile j + 1 go out
    // after its P V of key tile j when there are two score buffers (one per row tile), so a warpgroup waits for
    // both; with three buffers they go out half a step earlier and are there when it is done with its weights.
    constexpr uint32_t id_s = idesc_bf16_f32(kTile, kTile);
    constexpr uint32_t id_o = idesc_bf16_f32(kTile, D) | (1u << 16);   // V: MN-major
    uint32_t kv = 0, st[2] = {0, 0}, pt[2] = {0, 0};   // ring tiles of the items before; key tiles by row tile: scores, P V
    int items = 0, n0 = 0, n1 = 0, n = 0;
    bool dead = false;
    auto scores = [&](auto row_tile, int j) {          // S_i = Q_i K_j^T
      constexpr int i = decltype(row_tile)::value;
      const uint32_t k = kv + 2 * j, ks = k % NS;
      if (Sh::bufs == 3 && (i == 0 || j >= n0)) {
        dead |= pre_wait(c, c.full[ks], (k / NS) & 1);    // the key tile's first use
        __syncwarp();
        tc_fence_after();
      }
      const uint64_t qa = smem_desc(q_s + i * Sh::tile_bytes, 1024, Swz::k128);
      const uint64_t ka = smem_desc(ring + ks * Sh::tile_bytes, 1024, Swz::k128);
      const uint32_t to = tmem + Sh::buf(i, j) * kTile;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {            // (descriptors hold addresses in 16-byte units)
        const uint64_t o = ((kk >> 2) * (kTile * 128) + (kk & 3) * 32) >> 4;
        umma_bf16_warp(to, qa + o, ka + o, id_s, kk != 0);
      }
      umma_commit_warp(smem_u32(&c.s_full[i][st[i] & 1]));
      ++st[i];
      if (i == 1 || j >= n1) {                         // and its last
        umma_commit_warp(smem_u32(&c.empty[ks]));
        if (j + 1 == n) umma_commit_warp(smem_u32(&c.q_empty));
      }
    };
    auto values = [&](auto row_tile, int j, uint32_t vs) {   // O_i (+)= P_i V_j, as its halves of the keys come
      constexpr int i = decltype(row_tile)::value;
      const uint64_t va = smem_desc_mn128(ring + vs * Sh::tile_bytes, kTile * 128, 1024);
      const uint32_t from = tmem + Sh::buf(i, j) * kTile;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (Sh::bufs == 2 || half == 0) {
          dead |= pre_wait(c, c.p_ready[i][pt[i] & 1][Sh::bufs == 2 ? half : 1], (pt[i] >> 1) & 1);
          __syncwarp();
          tc_fence_after();
        }
#pragma unroll
        for (int kk = half * (kTile / 32); kk < (half + 1) * (kTile / 32); ++kk)
          umma_bf16_ts_warp(tmem + Sh::col_o + i * D, from + kk * 8, va + kk * (2048 >> 4), id_o, kk != 0 || j != 0);
      }
      umma_commit_warp(smem_u32(&c.o_done[i][pt[i] & 1]));
      ++pt[i];
    };
    constexpr std::integral_constant<int, 0> r0{};
    constexpr std::integral_constant<int, 1> r1{};
    for (int it = 0;; ++it) {
      const int sl = it % kItems, si = it % (2 * kItems);
      pre_wait(c, c.item_full[sl], (it / kItems) & 1);
      __syncwarp();
      const bool valid = __shfl_sync(0xffffffffu, c.item[si].valid && !failed(c), 0);
      n0 = __shfl_sync(0xffffffffu, c.item[si].n[0], 0);
      n1 = __shfl_sync(0xffffffffu, c.item[si].n[1], 0);
      n = max(n0, n1);
      if (lane == 0) mbar_arrive(smem_u32(&c.item_empty[sl]));
      __syncwarp();
      if (!valid) break;
      if (n == 0) continue;
      pre_wait(c, c.q_full, items & 1);
      ++items;
      if constexpr (Sh::bufs == 2) {
        dead |= pre_wait(c, c.full[kv % NS], (kv / NS) & 1);
        __syncwarp();
        tc_fence_after();
      }
      if (n0 > 0) scores(r0, 0);
      if (n1 > 0) scores(r1, 0);
      if (Sh::bufs == 3 && n0 > 1) scores(r0, 1);
      for (int j = 0; j < n; ++j) {
        const uint32_t v = kv + 2 * j + 1, vs = v % NS;
        dead |= pre_wait(c, c.full[vs], (v / NS) & 1);
        if (Sh::bufs == 2 && j + 1 < n) dead |= pre_wait(c, c.full[(v + 1) % NS], ((v + 1) / NS) & 1);
        __syncwarp();
        if (j < n0) values(r0, j, vs);
        if (Sh::bufs == 2 ? j + 1 < n0 : j + 1 < n1) {
          if constexpr (Sh::bufs == 2) scores(r0, j + 1); else scores(r1, j + 1);
        }
        if (j < n1) values(r1, j, vs);
        umma_commit_warp(smem_u32(&c.empty[vs]));
        if (Sh::bufs == 2 ? j + 1 < n1 : j + 2 < n0) {
          if constexpr (Sh::bufs == 2) scores(r1, j + 1); else scores(r0, j + 2);
        }
        if (__any_sync(0xffffffffu, dead)) break;
      }
      kv += 2 * n;
    }
    if (failed(c)) {                     // let the MMAs in flight end
      __syncwarp();
      umma_commit_warp(smem_u32(&c.drain));
      mbar_wait_limit(smem_u32(&c.drain), 0, kDrainLimitCycles);
    }
    __syncwarp();
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kSoftmaxRegs));
    // ============================= softmax ================================
    const int i = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t col_o = lane_base + Sh::col_o + i * D;
    const float sl2 = p.scale * kLog2e, grow = kRescale / sl2;
    const int t_in = row / GB, g = row - t_in * GB;
    bool dead = false;
    uint32_t t = 0;                      // key tiles of this row tile so far, over the items
    for (int it = 0;; ++it) {
      const int sl = it % kItems;
      pre_wait(c, c.item_full[sl], (it / kItems) & 1);
      __syncwarp();
      const PrefillItem w = c.item[it % (2 * kItems)];
      const bool valid = __shfl_sync(0xffffffffu, w.valid && !failed(c), 0);
      if (lane == 0) mbar_arrive(smem_u32(&c.item_empty[sl]));
      if (!valid) break;
      const int tok = w.tok0 + i * TT + t_in, n = w.n[i];
      const bool live = t_in < TT && g < w.heads && tok < w.lq;
      const int lim = live ? max(0, min(w.lk, tok + 1 + w.lk - w.lq)) - w.shift : 0x7fffffff;   // keys the row sees, from the first tile on
      const int least = __reduce_min_sync(0xffffffffu, lim);
      uint32_t buf = Sh::buf(i, 0);
      float ref = -INFINITY, l = 0.f;      // exponents are relative to ref (in units of raw scores), less kRescale
      for (int j = 0; j < n; ++j, ++t) {
        const uint32_t col_s = lane_base + buf * kTile;
        if constexpr (Sh::bufs == 3) buf = buf == 0 ? 2 : buf - 1;   // (2 j + i) mod 3
        dead |= pre_wait(c, c.s_full[i][t & 1], (t >> 1) & 1);
        __syncwarp();
        tc_fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld32(col_s + q * 32, s[q]);
        tmem_ld_wait();
        const int seen = lim - j * kTile;
        if (least - j * kTile < kTile) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (q * 32 + e >= seen) s[q][e] = 0xff800000u;
        }
        float mx[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          mx[q] = __uint_as_float(s[q][0]);
#pragma unroll
          for (int e = 1; e < 31; e += 2) mx[q] = max3(mx[q], __uint_as_float(s[q][e]), __uint_as_float(s[q][e + 1]));
          mx[q] = fmaxf(mx[q], __uint_as_float(s[q][31]));
        }
        const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
        if (j == 0) {
          ref = top;
        } else if (__any_sync(0xffffffffu, live && top > ref + grow)) {   // (rows of nobody hold anything: no say)
          const float nr = fmaxf(ref, top);
          const float f = nr == -INFINITY ? 1.f : exp2_fast((ref - nr) * sl2);
          ref = nr;
          l *= f;
          // (with three score buffers the P V before may still run)
          pre_wait(c, c.o_done[i][(t - 1) & 1], ((t - 1) >> 1) & 1);
          __syncwarp();
          tc_fence_after();
#pragma unroll
          for (int q = 0; q < D / 32; ++q) {
            uint32_t o[32];
            tmem_ld32(col_o + q * 32, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st32(col_o + q * 32, o);
          }
        }
        const float off = ref == -INFINITY ? 0.f : __fmaf_rn(-ref, sl2, -kRescale);   // (nothing seen: every weight is 0)
        const uint64_t sl2p = pair(sl2, sl2), offp = pair(off, off);
        uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t pk[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const int q = 2 * h + (e >> 4), f = (e & 15) * 2;
            const float2 x = unpair(fma2(pair(__uint_as_float(s[q][f]), __uint_as_float(s[q][f + 1])), sl2p, offp));
            const float w0 = exp2_fast(x.x), w1 = exp2_fast(x.y);
            sum[e & 3] = add2(sum[e & 3], pair(w0, w1));
            pk[e] = pack_bf16x2(w0, w1);
          }
          tmem_st32(col_s + h * 32, pk);
          if (Sh::bufs == 2 || h == 1) {   // (with three score buffers nothing of this warpgroup waits for P V: one hand-over)
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&c.p_ready[i][t & 1][h]));
          }
        }
        const float2 all = unpair(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
        l += all.x + all.y;
        if ((j & 15) == 15 && __any_sync(0xffffffffu, dead)) break;
      }
      if constexpr (SPLIT) {
        // This part's reference and sum of the row, then the row's over all parts.
        if (n > 0) pre_wait(c, c.o_done[i][(t - 1) & 1], ((t - 1) >> 1) & 1);
        __syncwarp();
        float2* const stats = reinterpret_cast<float2*>(prefill_smem_raw + (out_s - raw)) + i * kTile + row;
        *stats = make_float2(n > 0 ? ref : -INFINITY, l);
        cluster.sync();
        float all_ref = -INFINITY, all_l = 0.f;
        for (int x = 0; x < parts; ++x) all_ref = fmaxf(all_ref, cluster.map_shared_rank(stats, x)->x);
        const float base_ref = all_ref == -INFINITY ? 0.f : all_ref;
        for (int x = 0; x < parts; ++x) {
          const float2 st = *cluster.map_shared_rank(stats, x);
          all_l += st.y * exp2_fast((st.x - base_ref) * sl2);
        }
        // This part's share of the result, fp32, over the key and value ring (nothing is in flight there any
        // more): row tile after row tile, 16-byte chunks permuted by the row.
        const float f = all_l == 0.f || n == 0 ? 0.f : exp2_fast((ref - base_ref) * sl2) / all_l;
        tc_fence_after();
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
          uint32_t o[32];
          if (n > 0) {
            tmem_ld32(col_o + q * 32, o);
            tmem_ld_wait();
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (n > 0)
              v = make_uint4(__float_as_uint(__uint_as_float(o[4 * e]) * f), __float_as_uint(__uint_as_float(o[4 * e + 1]) * f),
                             __float_as_uint(__uint_as_float(o[4 * e + 2]) * f), __float_as_uint(__uint_as_float(o[4 * e + 3]) * f));
            sts128(ring + ((i * kTile + row) * (D / 4) + ((q * 8 + e) ^ (row & (D / 4 - 1)))) * 16, v);
          }
        }
        tc_fence_before();
        if (p.lse && live && part == 0 && !failed(c))
          p.lse[static_cast<long long>(w.q0 + i * TT + t_in) * p.q_heads + w.h0 + g] =
              all_l == 0.f ? -INFINITY : (all_ref * sl2 + kRescale + log2f(all_l)) * kLn2;
        cluster.sync();
        // Rows part, part + parts, ..: the sum over the parts, a warp a row.
        constexpr int E = D / 32;
        const float* const mine = reinterpret_cast<const float*>(prefill_smem_raw + (ring - raw));
        for (int r = part + parts * warp; r < 2 * kTile; r += parts * kSoftmaxWarps) {
          const int x_in = (r & (kTile - 1)) / GB, gg = (r & (kTile - 1)) - x_in * GB, ri = r >> 7;
          const int tk = w.tok0 + ri * TT + x_in;
          if (x_in >= TT || gg >= w.heads || tk >= w.lq || failed(c)) continue;
          const int at = (r * (D / 4) + ((lane * E / 4) ^ (r & (D / 4 - 1)))) * 4 + lane * E % 4;
          float sum[E];
#pragma unroll
          for (int e = 0; e < E; ++e) sum[e] = 0.f;
#pragma unroll 4
          for (int x = 0; x < parts; ++x) {
            const float* const from = cluster.map_shared_rank(mine, x) + at;
            if constexpr (E == 4) {
              const float4 v = *reinterpret_cast<const float4*>(from);
              sum[0] += v.x; sum[1] += v.y; sum[2] += v.z; sum[3] += v.w;
            } else {
              const float2 v = *reinterpret_cast<const float2*>(from);
              sum[0] += v.x; sum[1] += v.y;
            }
          }
          uint32_t v[E / 2];
#pragma unroll
          for (int e = 0; e < E / 2; ++e) v[e] = pack_bf16x2(sum[2 * e], sum[2 * e + 1]);
          uint16_t* const out = p.out + (w.q0 + ri * TT + x_in) * p.out_stride + (w.h0 + gg) * D + lane * E;
          if constexpr (E == 4) *reinterpret_cast<uint2*>(out) = make_uint2(v[0], v[1]);
          else *reinterpret_cast<uint32_t*>(out) = v[0];
        }
        met = 2;
        continue;
      }
      // The row's result, through shared memory so that a store instruction writes 4 whole 128-byte lines
      // (one row per lane, 16 bytes each, wrote 32 and held up the SM's loads: 5000 clocks an item, now 1000).
      uint16_t* const to = p.out + static_cast<long long>(w.q0 + i * TT + t_in) * p.out_stride + (w.h0 + g) * D;
      const uint32_t lives = __ballot_sync(0xffffffffu, live);
      if (n > 0) {
        pre_wait(c, c.o_done[i][(t - 1) & 1], ((t - 1) >> 1) & 1);
        __syncwarp();
        if (__any_sync(0xffffffffu, failed(c))) break;
        tc_fence_after();
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const uint64_t invp = pair(inv, inv);
        const uint32_t stage = out_s + warp * kOutBytes;
#pragma unroll
        for (int half = 0; half < D / 64; ++half) {
          uint32_t o[2][32];
          tmem_ld32(col_o + half * 64, o[0]);
          tmem_ld32(col_o + half * 64 + 32, o[1]);
          tmem_ld_wait();
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              uint32_t r[4];
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const float2 v = unpair(mul2(pair(__uint_as_float(o[q][e + 2 * x]), __uint_as_float(o[q][e + 2 * x + 1])), invp));
                r[x] = pack_bf16x2(v.x, v.y);
              }
              sts128(stage + lane * 128 + (((q * 4 + e / 8) ^ (lane & 7)) << 4), make_uint4(r[0], r[1], r[2], r[3]));
            }
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int r = k * 4 + lane / 8, ch = lane % 8;
            const uint4 v = lds128(stage + r * 128 + ((ch ^ (r & 7)) << 4));
            uint16_t* const at = reinterpret_cast<uint16_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(to), r));
            if ((lives >> r) & 1) *reinterpret_cast<uint4*>(at + half * 64 + ch * 8) = v;
          }
          __syncwarp();
        }
        tc_fence_before();
      } else if (live) {
#pragma unroll
        for (int e = 0; e < D; e += 8) *reinterpret_cast<uint4*>(to + e) = make_uint4(0, 0, 0, 0);
      }
      const long long out_row = w.q0 + i * TT + t_in;
      if (p.lse && live) p.lse[out_row * p.q_heads + w.h0 + g] = l == 0.f ? -INFINITY : (ref * sl2 + kRescale + log2f(l)) * kLn2;
      __syncwarp();
      if (lane == 0) publish(&c.stored[warp], it + 1);
    }
  }

  if constexpr (SPLIT) {   // every thread of the cluster meets three times, whatever became of its item
    for (int x = met; x < 3; ++x) cluster.sync();
    if (part == 0 && warp >= kPreScanWarp && !failed(c)) {
      const int half = warp - kPreScanWarp;
      if (*const_cast<const volatile int*>(&c.bad[half])) add_not_finite<D>(p, c.item[0], half, lane);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kPreMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

namespace {

template <int D, bool SPLIT>
int launch_grid(const PrefillArgs& a, long long items, int parts, void* stream) {
  // (set on every call: the attribute belongs to the current device, like the launch)
  const auto kernel = prefill_kernel<D, SPLIT>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, PrefillShape<D>::smem);
  if (e != cudaSuccess) return static_cast<int>(e);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(items * parts), 1, 1);
  cfg.blockDim = dim3(kPreThreads, 1, 1);
  cfg.dynamicSmemBytes = PrefillShape<D>::smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(parts);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = SPLIT ? 2 : 1;
  return static_cast<int>(cudaLaunchKernelEx(&cfg, kernel, a));
}

template <int D>
int launch_one(const PrefillArgs& a, void* stream) {
  // At most this many items: a sequence adds one more than its whole pairs of row tiles.
  const long long subs = a.kv_heads * ((a.q_heads / a.kv_heads + a.head_block - 1) / a.head_block);
  const long long items = (a.total_q / (2 * a.tile_tokens) + static_cast<long long>(a.batch)) * subs;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return static_cast<int>(e);
  // Few items over long keys: split the keys over up to 8 CTAs while the GPU has SMs for them and each part
  // keeps at least two key tiles of the average sequence.
  const long long tiles = a.total_k / a.batch / kTile;
  int parts = 1;
  while (parts < 8 && items * parts * 2 <= sms && tiles >= 4 * parts) parts *= 2;
  return parts > 1 ? launch_grid<D, true>(a, items, parts, stream) : launch_grid<D, false>(a, items, 1, stream);
}

}  // namespace

int launch_prefill(const PrefillArgs& a, void* stream) {
  return a.head_dim == 128 ? launch_one<128>(a, stream) : launch_one<64>(a, stream);
}

int read_prefill_status(void* stream, uint32_t* out, int clear) {
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint32_t v = 0;
  cudaError_t err = cudaMemcpyFromSymbolAsync(&v, g_prefill_status, sizeof v, 0, cudaMemcpyDeviceToHost, s);
  if (err == cudaSuccess && clear) {
    static const uint32_t z = 0;
    err = cudaMemcpyToSymbolAsync(g_prefill_status, &z, sizeof z, 0, cudaMemcpyHostToDevice, s);
  }
  if (err == cudaSuccess) err = cudaStreamSynchronize(s);
  *out = v;
  return static_cast<int>(err);
}

}  // namespace glora
