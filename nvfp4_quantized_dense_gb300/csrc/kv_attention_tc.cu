// Causal attention over the paged NVFP4 cache for prefill-sized query tiles,
// on the tcgen05 tensor cores.  The mathematics is kv_attention.cu's.
//
// A unit is 256 query rows (query tokens times the heads that share a
// key/value head) of one sequence, as two tiles of 128 rows, against cached
// tiles of 128 tokens:
//   S_t = Q_t K^T   (A = Q_t and B = K from shared memory, fp32 in TMEM)
//   P_t = exp2(S_t * scale - reference) as f16, over S_t's own columns
//   O_t += P_t V    (A = P_t from TMEM, B = V^T from shared memory)
// The two tiles alternate on the tensor pipe: while one's softmax runs, the
// other's two products do.  All operands are f16 and exact but for P: a code
// times its scale has at most 6 significant bits, and a query row is scaled by
// a power of two (kv_attention.cu).
//
// Conversion.  A cached tile is 18 KB in HBM and 64 KB as f16, so four warps
// read the codes straight from global memory into registers (one tile ahead)
// and store f16 operand tiles; each serves both 128-row tiles.  K: a thread
// converts one token's row.  V: a thread takes 8 tokens of one 16-wide block,
// 64 contiguous bytes, pairs the nibbles of neighbouring tokens before the
// conversion, and so writes V^T rows of 8 tokens (16 bytes) with no exchange.
//
// Softmax.  One thread per row, so maxima and sums need no shuffles.  The
// reference of the exponentials follows the running maximum only when that
// has grown by more than kSlack (in powers of two; f16 has that much room
// above 2^kShift): the fp32 sums O and l are rescaled then, which is rare
// after the first tiles.
//
// Work split.  The batch's cached tiles lie on a line (query tile by query
// tile, each with the tokens that its rows see, head by head, and kUnitCost
// places ahead of each unit), cut into equal parts, one per CTA.  A shared
// unit is joined by the last part to arrive, warp by warp, from its own sums
// and the others' in the workspace, in the order of the parts.  Where there are
// no more units than CTAs and none stands out, each is a CTA's.
//
// Roles (512 threads, one CTA per SM): warps 0-3 and 4-7 the softmax of the
// two tiles (and their Q and O), warps 8-11 conversion, warp 12 the MMAs, warp 13
// the walk over the part's segments.
// Every wait is bounded.
//
// What bounds it (40 query heads on 8 key/value heads of 128).  A chunk of 2048
// queries behind 16,385 tokens: 501 us, 1.46 PFLOP/s, 76 % of the measured bf16
// burst rate and 86 % of the sustained one (at head_dim 64, half the products:
// 439 us); nine sequences of 70 to 4,099 with 1 to 701 queries: 84 us, 0.88
// PFLOP/s.  A unit's beginning takes 6,000 cycles
// (its queries' copies and conversion by 8 warps 4,500, the first scores 1,000)
// and its end 4,500, during which the tensor pipe waits; starting the next
// unit's queries under the last products gained nothing, for the same warps
// issue both.
// In the loop one group's chain is the bound: S 600 cycles, softmax 2100 (its
// loads and maxima 480, exponentials 1100, the P stores up to 640 while the
// other tile's products use tensor memory), P V 600, and S again; two groups
// alternate, so the tensor pipe works ~2400 of 3400 cycles a cached tile.  An
// S ahead of P V needs 128 columns of TMEM more than there are at head_dim 128
// (at 64 they are free, and not used).
// Tried and slower (the chunk, us, against 510): P announced in halves 569,
// two threads a row 796, unpaired float arithmetic 523 to 547, the cached bytes
// through a ring of bulk copies 610 (the operands' reads need the shared
// memory's bandwidth), L2 prefetches 546.
#include "common.cuh"
#include "internal.h"
#include "kv_attention_common.cuh"
#include "kv_layout.cuh"
#include "tc_ptx.cuh"

#include <type_traits>

namespace nvfp4 {
namespace {

constexpr int kThreads = 512;
constexpr int kConvWarp = 8, kMmaWarp = 12, kWalkWarp = 13;
constexpr int kSegSlots = 4;                 // segments announced ahead
constexpr int kTile = 128;                   // cached tokens of a step; rows of a query tile
constexpr int kRows = 2 * kTile;             // rows of a unit
constexpr int kMinTiles = 4;                 // cached tiles worth a CTA
constexpr int kUnitCost = 4;                 // what a unit's beginning and end cost, in tiles (11,000 cycles; a tile 3,400; 3 and 5 within 3 %)
constexpr int kMaxBatch = 1024;
constexpr float kShift = 14.0f, kSlack = 1.9f, kFar = 65536.0f;
constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr uint32_t kDrainPolls = 1u << 22, kPollNs = 20000;
constexpr int kSmsPlanned = 152;

template <int D>
struct TcCfg {
  using R = KvRecord<D>;
  static constexpr int Q_BYTES = kTile * D * 2;              // one tile of Q; one of K; one of V^T
  static constexpr int SUB = kTile * 128;                    // 64 elements of D for 128 rows (Q, K)
  static constexpr int VSUB = D * 128;                       // 64 tokens for D rows (V^T)
  static constexpr int K_AT = 2 * Q_BYTES, V_AT = K_AT + 2 * Q_BYTES;
  static constexpr int SMEM = V_AT + 2 * Q_BYTES + 1024;
  static constexpr uint32_t S_COL = 0, O_COL = 2 * kTile;    // TMEM columns
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr int PART_FLOATS = kRows * (D + 2);        // a partial result: m and l of the rows, then O
};

// A unit: the query tile `tile` of sequence b for one key/value head, and the
// cached tiles that its rows see.
struct Unit {
  int b, q0, qn, len, pos0;      // sequence: first query token, queries, cached tokens, first position
  int tiles;                     // query tiles of the sequence
  int tile, lo, count;           // query tile; its first cached tile and their number (at least one)
};

__device__ __forceinline__ void load_seq(const KvAttentionParams &a, int group, int b, Unit &u) {
  u.b = b;
  int q0 = b * (int)a.max_q, q1 = q0 + (int)a.max_q;
  if (a.cu_q) {
    q0 = min(max(__ldg(a.cu_q + b), 0), (int)a.tokens);
    q1 = min(max(__ldg(a.cu_q + b + 1), q0), (int)a.tokens);
  }
  u.q0 = q0;
  u.qn = min(q1 - q0, (int)a.max_q);
  u.len = min(max(__ldg(a.seq_lens + b), 0), (int)(a.max_pages * a.page_size));
  u.pos0 = u.len - u.qn;
  u.tiles = (int)(((int64_t)u.qn * group + kRows - 1) / kRows);
}

// Cached tiles [lo, lo + count) that query tile `tile` sees.
__device__ __forceinline__ void load_tile(const KvAttentionParams &a, int group, int tile, Unit &u) {
  u.tile = tile;
  const int row0 = tile * kRows, row1 = min(row0 + kRows, u.qn * group) - 1;
  const int first = u.pos0 + row0 / group, last = u.pos0 + row1 / group;
  u.lo = a.window > 0 ? max(first - (int)a.window + 1, 0) / kTile : 0;
  u.count = max((last < 0 ? 0 : last / kTile + 1) - u.lo, 1);
}

// Where this CTA begins on the line, found by one warp and read by all.
struct Start {
  int b, tile;
  int tile_at;         // where that query tile's units begin
};

// A segment, as the walking thread announces it to the other roles: `count`
// cached tiles from `first` on of one unit (0: no more segments).
struct Segment {
  int b, len, head, rows;
  int token, pos, rem; // of its first row: token, position, query head of the group
  int first, count;
  int seen;            // first token that any row of the unit sees
  int whole;           // the whole unit
  int p0, p1;          // else: the parts that share it
};

// Walks the part's segments.
template <int D>
struct Walk {
  const KvAttentionParams &a;
  int group, head_cost;
  int pos, end, tile_at;
  bool split, single;
  Unit u;
  // the current segment
  int head, first, count;        // head; first cached tile; number of cached tiles
  int unit0, unit1;              // the unit's places on the line
  bool whole;

  __device__ __forceinline__ Walk(const KvAttentionParams &p, int g, int cost, int begin, int e, bool sp, bool one,
                                  const Start &s)
      : a(p), group(g), head_cost(cost), pos(begin), end(e), tile_at(s.tile_at), split(sp), single(one) {
    load_seq(a, group, s.b, u);
    load_tile(a, group, s.tile, u);
  }
  __device__ __forceinline__ int places() const { return single ? 1 : u.count + head_cost; }     // of the current unit
  __device__ __forceinline__ bool next() {
    for (;;) {
      if (pos >= end) return false;
      int n = (int)a.kv_heads * places();
      while (pos >= tile_at + n) {
        tile_at += n;
        if (u.tile + 1 < u.tiles) {
          load_tile(a, group, u.tile + 1, u);
        } else {
          int b = u.b + 1;
          load_seq(a, group, b, u);
          while (u.tiles == 0) load_seq(a, group, ++b, u);
          load_tile(a, group, 0, u);
        }
        n = (int)a.kv_heads * places();
      }
      const int len = places();
      head = (pos - tile_at) / len;
      if (single) {                              // one unit, one place, one part
        first = u.lo, count = u.count, whole = true;
        ++pos;
        return true;
      }
      unit0 = tile_at + head * len + head_cost;      // its tiles are [unit0, unit1)
      unit1 = unit0 + u.count;
      if (pos < unit0) pos = unit0;
      if (pos >= end) return false;
      if (!split && pos != unit0) {                           // whole units belong to the part they begin in
        pos = unit1;
        continue;
      }
      const int stop = split && end < unit1 ? end : unit1;
      whole = pos == unit0 && stop == unit1;
      first = u.lo + pos - unit0;
      count = stop - pos;
      pos = unit1;
      return true;
    }
  }
  __device__ __forceinline__ int rows() const { return min(u.qn * group - u.tile * kRows, kRows); }
};

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// 16 bytes to shared memory; zeros where `there` is false.
__device__ __forceinline__ void cp_async16(uint32_t at, const void *src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at), "l"(src), "r"(there ? 16u : 0u) : "memory");
}
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ uint4 ld_shared16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

__device__ __forceinline__ bool mbar_try_wait_for(uint64_t *bar, uint32_t parity, uint32_t ns) {
  uint32_t ok;
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
      "selp.u32 %0, 1, 0, p;\n"
      "}"
      : "=r"(ok)
      : "r"(ptx::smem_u32(bar)), "r"(parity), "r"(ns)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ void st_shared16(uint32_t at, const uint32_t (&x)[4]) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3])
               : "memory");
}

// Registers move between the warpgroups: the launch's 512 x 128 become
// 2 x 128 x kSoftRegs + 128 x kConvRegs + 128 x kMmaRegs (the same sum).
constexpr int kSoftRegs = 184, kConvRegs = 96, kMmaRegs = 48;
static_assert(2 * kSoftRegs + kConvRegs + kMmaRegs == 4 * 128, "register shares");
template <int N>
__device__ __forceinline__ void grow_regs() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void shrink_regs() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    kv_attention_tc_kernel(const __grid_constant__ KvAttentionParams a, const bool split, int *status) {
  using C = TcCfg<D>;
  using R = KvRecord<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t s_qfull[2], s_sfull[2], s_pfull[2], s_ofull[2], s_kfull[2], s_kempty[2], s_vfull[2],
      s_vempty[2], s_drain;
  __shared__ uint32_t s_tmem;
  __shared__ uint8_t s_sc[2][kTile];             // exponents of the rows of Q
  __shared__ int s_abort;
  __shared__ uint32_t s_valid[4];                // by cached tile % 4: which records exist, two bits of a byte a conversion warp
  __shared__ int s_cost[kMaxBatch], s_units[kMaxBatch];    // of each sequence: cached tiles and units of a head
  __shared__ int s_longest[kThreads / 32];       // unit of a warp's sequences
  __shared__ Start s_start;
  __shared__ Segment s_seg[kSegSlots];
  __shared__ __align__(8) uint64_t s_segfull[kSegSlots], s_segempty[kSegSlots];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int group = (int)(a.q_heads / a.kv_heads);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&s_qfull[i], 4);
      ptx::mbar_init(&s_sfull[i], 1);
      ptx::mbar_init(&s_pfull[i], 4);
      ptx::mbar_init(&s_ofull[i], 1);
      ptx::mbar_init(&s_kfull[i], 4);
      ptx::mbar_init(&s_kempty[i], 1);
      ptx::mbar_init(&s_vfull[i], 4);
      ptx::mbar_init(&s_vempty[i], 1);
    }
    for (int i = 0; i < kSegSlots; ++i) {
      ptx::mbar_init(&s_segfull[i], 1);
      ptx::mbar_init(&s_segempty[i], kMmaWarp + 1);      // softmax and conversion warps, the MMA thread
    }
    ptx::mbar_init(&s_drain, 1);
    s_abort = 0;
    ptx::fence_barrier_init();
  }
  pdl_trigger();
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(&s_tmem, C::TMEM_COLS);
    ptx::tmem_relinquish();
  }
  pdl_wait();

  // ---- the line of cached tiles: a warp per sequence, a lane per query tile
  // (its length fits 31 bits: the launch sees to that)
  int longest = 0;
  for (int b = warp; b < (int)a.batch; b += kThreads / 32) {
    Unit u;
    load_seq(a, group, b, u);
    int n = 0;
    for (int t = lane; t < u.tiles; t += 32) {
      load_tile(a, group, t, u);
      n += u.count;
      longest = max(longest, u.count);
    }
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) s_cost[b] = n, s_units[b] = u.tiles;
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (lane == 0) s_longest[warp] = longest;
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = s_tmem;
  const int per = ((int)a.batch + 31) / 32, b_lo = min(lane * per, (int)a.batch), b_hi = min(b_lo + per, (int)a.batch);
  int cost = 0, units = 0;                       // every warp sums for itself
  for (int b = b_lo; b < b_hi; ++b) cost += s_cost[b], units += s_units[b];
  int upto = cost, upto_units = units;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, upto, o), y = __shfl_up_sync(0xffffffffu, upto_units, o);
    if (lane >= o) upto += x, upto_units += y;
  }
  const int heads = (int)a.kv_heads, part = (int)blockIdx.x;
  const int all = __shfl_sync(0xffffffffu, upto, 31) * heads, all_units = __shfl_sync(0xffffffffu, upto_units, 31) * heads;
  longest = __reduce_max_sync(0xffffffffu, s_longest[lane % (kThreads / 32)]);
  // No more units than CTAs and none much above the even share: a CTA each,
  // with nothing to join (512 queries of 40 heads on 8: 20 us, cut evenly 37).
  const bool single = all_units <= (int)gridDim.x && longest <= max(all / (int)gridDim.x + 4, 8);
  const int head_cost = min(kUnitCost, all / (int)gridDim.x);
  const int total = single ? all_units : all + head_cost * all_units;
  const bool has_work = single ? part < total : part * kMinTiles < total;
  const Line line(max(total, 1), single ? max(total, 1) : max(min((int)gridDim.x, (total + kMinTiles - 1) / kMinTiles), 1));
  const int begin = has_work ? line.at(part) : 0, end = has_work ? line.at(part + 1) : 0;
  if (has_work && warp == 0) {
    auto places = [&](int tiles, int n) { return single ? n : tiles + head_cost * n; };      // of n units
    const int my_end = places(upto, upto_units) * heads;
    int at = my_end - places(cost, units) * heads;
    int b = -1;
    if (begin >= at && begin < my_end)
      for (b = b_lo; b < b_hi; ++b) {
        const int n = places(s_cost[b], s_units[b]) * heads;
        if (begin < at + n) break;
        at += n;
      }
    const int src = __ffs(__ballot_sync(0xffffffffu, b >= 0)) - 1;
    b = __shfl_sync(0xffffffffu, b, src);
    at = __shfl_sync(0xffffffffu, at, src);
    Unit u;
    load_seq(a, group, b, u);
    for (int t0 = 0;; t0 += 32) {                // 32 query tiles at a time
      int n = 0;
      if (t0 + lane < u.tiles) {
        load_tile(a, group, t0 + lane, u);
        n = heads * places(u.count, 1);
      }
      int sum = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += x;
      }
      const uint32_t here = __ballot_sync(0xffffffffu, begin < at + sum && n > 0);
      if (here) {
        if (lane == __ffs(here) - 1) s_start = Start{b, t0 + lane, at + sum - n};
        break;
      }
      at += __shfl_sync(0xffffffffu, sum, 31);
      if (t0 + 32 >= u.tiles) break;             // (not reached)
    }
  }
  __syncthreads();

  const uint32_t limit = a.wait_limit;
  // (thirteen warps wait most of the time: a poll sleeps up to kPollNs in the
  // barrier unit instead of taking issue slots from those that work)
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    if (mbar_try_wait_for(bar, parity, kPollNs)) return true;
    uint64_t since = 0;
    for (uint32_t polls = 1;; ++polls) {
      if (mbar_try_wait_for(bar, parity, kPollNs)) return true;
      if (*const_cast<volatile int *>(&s_abort)) return false;
      if (limit) {
        if (polls >= limit) return false;
      } else {
        const uint64_t now = ptx::globaltimer();
        if (since == 0) since = now;
        else if (now - since > kTimeoutNs) return false;
      }
    }
  };
  auto give_up = [&]() {
    *const_cast<volatile int *>(&s_abort) = 1;
    atomicCAS(status, 0, (int)NVFP4_ERR_DEVICE_TIMEOUT);
  };
  bool mma_issued = false;

  if (!has_work) {
    // (falls through to the end)
  } else if (warp < kConvWarp) {
    grow_regs<kSoftRegs>();
    // ------------------------------------------------------------- softmax
    const int t = warp >> 2, row = (warp & 3) * 32 + lane;        // tile, its row
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lanes + C::S_COL + t * kTile, o_col = tmem + lanes + C::O_COL + t * D;
    // Rows of D 16-bit elements are staged in the Q tile's swizzled layout, a
    // warp's 32 rows by that warp alone: Q on its way in, the output on its
    // way out.  CPR 16-byte chunks a row, RPI rows a warp-wide access.
    constexpr int CPR = D / 8, RPI = 32 / CPR;
    const uint32_t stage = ptx::smem_u32(base) + t * C::Q_BYTES + (warp & 3) * 32 * 128;
    auto stage_at = [&](int r, int chunk) {
      return stage + (chunk >> 3) * C::SUB + r * 128 + (((chunk & 7) ^ (r & 7)) << 4);
    };
    // x / group for x < 2^22 / group, so for the sum of a remainder and a row of the tile
    const uint32_t per_group = ((1u << 22) + group - 1) / group;
    auto by_group = [&](int x) { return (int)((uint32_t)x * per_group >> 22); };
    const float qk0 = __ldg(a.qk_scale) * 1.4426950408889634f, qk = fabsf(qk0), vs = __ldg(a.v_scale);
    float *parts_at = reinterpret_cast<float *>(static_cast<uint8_t *>(a.workspace) + kCounterArea);
    uint32_t step = 0, seg = 0, tile_no = 0;     // of this tile: steps, segments; of the CTA: cached tiles
    for (uint32_t sn = 0;; ++sn) {
      if (__any_sync(0xffffffffu, !wait(&s_segfull[sn % kSegSlots], (sn / kSegSlots) & 1))) {
        give_up();
        break;
      }
      const Segment &w = s_seg[sn % kSegSlots];
      if (w.count == 0) break;
      bool ok = true;
      const bool active = t * kTile < w.rows;    // tile 1 of a short unit has no rows and takes no part
      const int win = (int)a.window;
      const bool have = t * kTile + row < w.rows;
      const int x = w.rem + t * kTile + row, k_row = by_group(x);       // tokens on from the segment's first
      const int hi = have ? w.pos + k_row : w.len - 1;
      // this warp's rows of the tile, from token token0, query head h0 of the group on
      const int rows_w = w.rows - t * kTile - (warp & 3) * 32, x_w = x - lane, k_w = by_group(x_w), h0 = x_w - k_w * group;
      const int token0 = w.token + k_w;
      float m = -INFINITY, l = 0.0f, sc = 0.0f;
      if (active) {
        // ---- Q: copied into the staging area as it is, then converted there
        // to f16 times a power of two per row; CPR lanes to a row.  (Loops, not
        // straight code: what runs once a segment is paced by its instruction
        // fetches.  The product with a power of two is exact in bf16.)
        const uint16_t *q_at = a.q + (int64_t)token0 * a.q_stride + w.head * group * D + lane % CPR * 8;
        const int64_t q_step = a.q_stride - group * D;
#pragma unroll 2
        for (int i = 0; i < CPR; ++i) {
          const int o = i * RPI + lane / CPR, h = h0 + o;         // (a row further: a head's elements; a group further: a token's)
          const uint16_t *src = q_at + h * D + by_group(h) * q_step;
          cp_async16(stage_at(o, lane % CPR), o < rows_w ? src : a.q, o < rows_w);
        }
        cp_async_wait();
        __syncwarp();
#pragma unroll 1
        for (int i0 = 0; i0 < CPR; i0 += 4) {    // four at a time, so that their latencies overlap
          uint4 raw[4];
          uint32_t top[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) raw[i] = ld_shared16(stage_at((i0 + i) * RPI + lane / CPR, lane % CPR));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t x[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
            top[i] = 0;                          // of the even and of the odd elements
#pragma unroll
            for (int k = 0; k < 4; ++k) top[i] = max_u16x2(top[i], x[k] & 0x7fff7fffu);
          }
#pragma unroll
          for (int d = CPR / 2; d > 0; d >>= 1)
#pragma unroll
            for (int i = 0; i < 4; ++i) top[i] = max_u16x2(top[i], __shfl_xor_sync(0xffffffffu, top[i], d));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int o = (i0 + i) * RPI + lane / CPR, e = min(max((int)(max(top[i] & 0xffffu, top[i] >> 16) >> 7), 15), 254);
            const float up = row_factor((uint32_t)(268 - e), qk0);
            const uint32_t x[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
            const __nv_bfloat162 up2 = __float2bfloat162_rn(up);
            uint32_t y[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const __nv_bfloat162 z = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&x[k]), up2);
              const uint32_t zz = *reinterpret_cast<const uint32_t *>(&z);
              y[k] = f16x2(bf16_lo(zz), bf16_hi(zz));
            }
            st_shared16(stage_at(o, lane % CPR), y);
            if (lane % CPR == 0) s_sc[t][(warp & 3) * 32 + o] = (uint8_t)e;
          }
        }
        ptx::fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&s_qfull[t]);
        sc = fmaxf(qk * __uint_as_float((uint32_t)max((int)s_sc[t][row] - 14, 1) << 23), 1.17549435e-38f);

        // columns of cached tile j that the row sees: [lo, end) - 128 j; tiles that any row of the tile sees part of only
        const int p0 = w.pos + by_group(w.rem + t * kTile), p1 = w.pos + by_group(w.rem + min((t + 1) * kTile, w.rows) - 1);
        const int base_t = w.first * kTile, count = w.count;
        const int end_c = min(hi + 1, w.len) - base_t, lo_c = win > 0 ? hi - win + 1 - base_t : -1;
        const int part_hi = min(p0 + 1, w.len) - base_t;
        const int part_lo = win > 0 ? p1 - win + 1 - base_t : -1;
        auto tiles = [&](auto far_rows) {
          for (int j = 0; j < count; ++j, ++step) {
            const bool got = wait(&s_sfull[t], step & 1);
            if (__any_sync(0xffffffffu, !got)) {
              give_up();
              return false;
            }
            ptx::tc_fence_after();
            const uint32_t valid = s_valid[(tile_no + j) & 3];
            const bool masked = valid != 0x03030303u || (j + 1) * kTile > part_hi || j * kTile < part_lo;
            // ---- the row's scores, all in registers, and their maximum
            uint32_t s[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) ptx::tmem_ld32(s_col + 32 * c, s[c]);
            ptx::tmem_wait_ld();
            if (masked) {
#pragma unroll
              for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                  const int col = 32 * c + i;
                  if (col >= end_c - j * kTile || col < lo_c - j * kTile || !((valid >> (c * 8 + (i >> 4))) & 1)) s[c][i] = 0xff800000u;
                }
            }
            float top4[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              top4[c] = __uint_as_float(s[c][0]);
#pragma unroll
              for (int i = 1; i + 1 < 32; i += 2)
                top4[c] = max3(top4[c], __uint_as_float(s[c][i]), __uint_as_float(s[c][i + 1]));
              top4[c] = fmaxf(top4[c], __uint_as_float(s[c][31]));
            }
            const float mx = fmaxf(max3(top4[0], top4[1], top4[2]), top4[3]);
            bool grow = false;
            float keep = 1.0f;
            if (j == 0) {
              m = mx;
            } else if ((mx - m) * sc > kSlack) {   // (infinite where m is -inf, NaN where both are)
              grow = true;
              keep = m == -INFINITY ? 0.0f : exp2_fast((m - mx) * sc);
              m = mx;
              l *= keep;
            }
            // ---- probabilities over the scores' own columns
            const float ref0 = m == -INFINITY ? 0.0f : __fmul_rn(m, sc);       // (the same roundings in both loops)
            float bias = __fadd_rn(kShift, -ref0);
            if constexpr (decltype(far_rows)::value) {
              const bool far = fabsf(ref0) >= kFar;
              const uint64_t minus = pack2(far ? -m : 0.0f, far ? -m : 0.0f);
              if (far) bias = kShift;
#pragma unroll
              for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                  float x0, x1;
                  unpack2(add2(pack2(__uint_as_float(s[c][i]), __uint_as_float(s[c][i + 1])), minus), x0, x1);
                  s[c][i] = __float_as_uint(x0), s[c][i + 1] = __float_as_uint(x1);
                }
            }
            const uint64_t sc2 = pack2(sc, sc), bias2 = pack2(bias, bias);
            uint64_t sum2[2] = {0, 0};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t p[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const uint64_t x = fma2(pack2(__uint_as_float(s[c][2 * i]), __uint_as_float(s[c][2 * i + 1])), sc2, bias2);
                float e0, e1;
                unpack2(x, e0, e1);
                e0 = exp2_fast(e0), e1 = exp2_fast(e1);
                sum2[i & 1] = add2(sum2[i & 1], pack2(e0, e1));
                p[i] = f16x2(e0, e1);
              }
              ptx::tmem_st16(s_col + 16 * c, p);
            }
            float l0, l1;
            unpack2(add2(sum2[0], sum2[1]), l0, l1);
            l += l0 + l1;
            if (__any_sync(0xffffffffu, grow)) {   // O follows the reference (last: the scores' registers are free now)
              const uint64_t keep2 = pack2(keep, keep);
              uint32_t o[D / 32][32];
#pragma unroll
              for (int c = 0; c < D / 32; ++c) ptx::tmem_ld32(o_col + 32 * c, o[c]);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < D / 32; ++c) {
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                  float x0, x1;
                  unpack2(mul2(pack2(__uint_as_float(o[c][i]), __uint_as_float(o[c][i + 1])), keep2), x0, x1);
                  o[c][i] = __float_as_uint(x0), o[c][i + 1] = __float_as_uint(x1);
                }
                ptx::tmem_st32(o_col + 32 * c, o[c]);
              }
            }
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&s_pfull[t]);
          }
          return true;
        };
        // s * sc + bias is off by the rounding of m * sc.  Rows where that could
        // be a good part of 1 take the difference s - m first, in a loop of
        // their own: scores are at most 2^15 * 2688 * D before sc, so a warp
        // without such a row knows it here (in one loop the chunk is 2 % slower).
        ok = __any_sync(0xffffffffu, sc * (88080384.0f * D) >= kFar) ? tiles(std::true_type{}) : tiles(std::false_type{});
      }
      tile_no += w.count;
      // ---- the unit's result, or this part's share of it.  A warp's rows are
      // joined by that warp of the part that arrives last, from its own sums
      // and what the others left in the workspace; a warp that sees all others
      // arrived need not write its own.
      const int p0 = w.p0, p1 = w.p1;
      const bool takes = active && rows_w > 0;
      auto place = [&](int q) { return parts_at + (int64_t)(2 * q + (q == p0 ? 1 : 0)) * C::PART_FLOATS; };
      uint32_t *counter = static_cast<uint32_t *>(a.workspace) + p0 * kConvWarp + warp, before = 0;
      if (takes && !w.whole && lane == 0)        // (on its way during the last products)
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(before) : "l"(counter) : "memory");
      if (active && ok) {
        const bool got = wait(&s_ofull[t], seg & 1);
        ++seg;
        if (__any_sync(0xffffffffu, !got)) {
          give_up();
          ok = false;
        }
      }
      const float ref = m == -INFINITY ? -INFINITY : m * sc;
      // eight elements of this thread's row, as bf16, to the staging area
      auto put8 = [&](int chunk, const float *x, float inv) {
        uint32_t y[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const __nv_bfloat162 z = __floats2bfloat162_rn(x[2 * k] * inv, x[2 * k + 1] * inv);
          y[k] = *reinterpret_cast<const uint32_t *>(&z);
        }
        st_shared16(stage_at(lane, chunk), y);
      };
      // the warp's rows from the staging area to the output, and their log-sum-exp
      auto write_rows = [&](float top, float sum) {
        uint16_t *out_at = a.out + ((int64_t)token0 * a.q_heads + w.head * group) * D + lane % CPR * 8;
        const int64_t out_step = (a.q_heads - group) * D;
        __syncwarp();
#pragma unroll 4
        for (int i = 0; i < CPR; ++i) {
          const int o = i * RPI + lane / CPR, h = h0 + o;
          if (o < rows_w) *reinterpret_cast<uint4 *>(out_at + h * D + by_group(h) * out_step) = ld_shared16(stage_at(o, lane % CPR));
        }
        if (a.lse && have)
          a.lse[(int64_t)(w.token + k_row) * a.q_heads + w.head * group + x - k_row * group] =
              sum == 0.0f ? -INFINITY : (top + (log2f(sum) - kShift)) * 0.6931471805599453f;   // (NaN where a query is)
      };
      if (takes && ok) {
        ptx::tc_fence_after();
        bool last = !w.whole && __shfl_sync(0xffffffffu, before, 0) == (uint32_t)(p1 - p0);
        if (w.whole) {
          const float inv = l == 0.0f ? 0.0f : vs / l;
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            ptx::tmem_ld32(o_col + c, o);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 4; ++i) put8(c / 8 + i, reinterpret_cast<const float *>(o) + 8 * i, inv);
          }
          write_rows(ref, l);
        } else if (!last) {
          // a partial result: m and l of the rows, then O as [D / 4][rows][4]
          float *mine = place(part) + t * kTile + row;
          __stcg(mine, ref);
          __stcg(mine + kRows, l);
          uint4 *dst = reinterpret_cast<uint4 *>(place(part) + 2 * kRows) + t * kTile + row;
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            ptx::tmem_ld32(o_col + c, o);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i)
              __stcg(dst + (c / 4 + i) * kRows, make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]));
          }
          __threadfence();
          __syncwarp();
          if (lane == 0)
            asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
          last = __shfl_sync(0xffffffffu, before, 0) == (uint32_t)(p1 - p0);
        }
        if (last) {
          __syncwarp();                          // lane 0's acquire comes before the other lanes' loads (a shuffle orders no memory)
          if (lane == 0) *counter = 0;
          // m and l of the parts, MB at a time, then O in blocks of CB 16-byte
          // chunks (the loads of a block are in flight together), in the
          // parts' order
          constexpr int MB = 4, CB = D == 128 ? 16 : 8, PB = D == 128 ? 1 : 2;
          float top = -INFINITY, sum = 0.0f;
#pragma unroll 1
          for (int q = p0; q <= p1; q += MB) {
            float mq[MB], lq[MB], t2 = top;
#pragma unroll
            for (int k = 0; k < MB; ++k) {
              const float *src = place(min(q + k, p1)) + t * kTile + row;
              mq[k] = ref, lq[k] = l;
              if (q + k != part) mq[k] = __ldcg(src), lq[k] = __ldcg(src + kRows);
            }
#pragma unroll
            for (int k = 0; k < MB; ++k) {
              if (q + k > p1) mq[k] = -INFINITY;
              t2 = fmaxf(t2, mq[k]);
            }
            const float zero = t2 == -INFINITY ? 0.0f : t2;
            sum *= exp2_fast(top - zero);
#pragma unroll
            for (int k = 0; k < MB; ++k) sum += q + k > p1 ? 0.0f : exp2_fast(mq[k] - zero) * lq[k];
            top = t2;
          }
          const float zero = top == -INFINITY ? 0.0f : top, inv = sum == 0.0f ? 0.0f : vs / sum;
#pragma unroll 1
          for (int c0 = 0; c0 < D / 4; c0 += CB) {
            float4 acc[CB];
#pragma unroll
            for (int i = 0; i < CB; ++i) acc[i] = make_float4(0, 0, 0, 0);
#pragma unroll 1
            for (int q = p0; q <= p1; q += PB) {
              float4 v[PB][CB];
              float mv[PB];
#pragma unroll
              for (int k = 0; k < PB; ++k) {
                mv[k] = q + k <= p1 ? ref : -INFINITY;
                if (q + k == part) {             // (still in tensor memory)
#pragma unroll
                  for (int i = 0; i < CB; i += 8) {
                    uint32_t o[32];
                    ptx::tmem_ld32(o_col + 4 * (c0 + i), o);
                    ptx::tmem_wait_ld();
#pragma unroll
                    for (int z = 0; z < 8; ++z)
                      v[k][i + z] = make_float4(__uint_as_float(o[4 * z]), __uint_as_float(o[4 * z + 1]),
                                                __uint_as_float(o[4 * z + 2]), __uint_as_float(o[4 * z + 3]));
                  }
                } else if (q + k <= p1) {
                  const float *src = place(q + k);
                  mv[k] = __ldcg(src + t * kTile + row);
                  const float4 *o = reinterpret_cast<const float4 *>(src + 2 * kRows) + c0 * kRows + t * kTile + row;
#pragma unroll
                  for (int i = 0; i < CB; ++i) v[k][i] = __ldcg(o + i * kRows);
                } else {
#pragma unroll
                  for (int i = 0; i < CB; ++i) v[k][i] = make_float4(0, 0, 0, 0);
                }
              }
#pragma unroll
              for (int k = 0; k < PB; ++k) {
                const float g = exp2_fast(mv[k] - zero);
#pragma unroll
                for (int i = 0; i < CB; ++i)
                  acc[i].x += g * v[k][i].x, acc[i].y += g * v[k][i].y, acc[i].z += g * v[k][i].z, acc[i].w += g * v[k][i].w;
              }
            }
#pragma unroll
            for (int i = 0; i < CB; i += 2) put8((c0 + i) / 2, reinterpret_cast<const float *>(&acc[i]), inv);
          }
          write_rows(top, sum);
        }
        ptx::tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&s_segempty[sn % kSegSlots]);
    }
  } else if (warp < kMmaWarp) {
    // ---------------------------------------------------------- conversion
    shrink_regs<kConvRegs>();
    const uint32_t sbase = ptx::smem_u32(base);
    const int ct = tid - kConvWarp * 32;                          // 0..127
    const int k_rec = ct >> 4, k_row = ct & 15;                   // K: token ct of the tile
    const int v_blk = ct >> 4, v_oct = ct & 15;                   // V: tokens 8 v_oct .. + 7 of block v_blk
    const bool v_on = v_blk < D / 16;
    constexpr int KW = D / 32;                                    // 16-byte words of a token's K codes
    const uint32_t rpp = (uint32_t)a.page_size / kKvGroup, step_pi = 8 / rpp, step_off = 8 % rpp;   // records of a page
    uint32_t n = 0;                                               // cached tiles so far
    bool ok = true;
    for (uint32_t sn = 0; ok; ++sn) {
      if (__any_sync(0xffffffffu, !wait(&s_segfull[sn % kSegSlots], (sn / kSegSlots) & 1))) {
        give_up();
        break;
      }
      const Segment w = s_seg[sn % kSegSlots];
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&s_segempty[sn % kSegSlots]);   // (copied)
      if (w.count == 0) break;
      const int32_t *table = a.block_table + (int64_t)w.b * a.max_pages;
      // This thread's K record and V record of the next tile to fetch: their
      // page's place in the table and place in the page, advanced by 8 records
      // a tile.  Table entries are loaded one tile before they are used, the
      // codes as soon as those of the tile before have been converted.
      struct Cursor {
        uint32_t pi, off;
        int rec, page;
      };
      auto look = [&](Cursor &c) { c.page = c.rec * kKvGroup < w.len ? __ldg(table + c.pi) : -1; };
      auto start = [&](int rec) {
        Cursor c;
        c.rec = rec, c.pi = (uint32_t)rec / rpp, c.off = (uint32_t)rec - c.pi * rpp;
        look(c);
        return c;
      };
      auto advance = [&](Cursor &c) {
        c.rec += 8, c.pi += step_pi, c.off += step_off;
        if (c.off >= rpp) c.off -= rpp, ++c.pi;
        look(c);
      };
      // a record that does not exist is read as record 0 of the cache with scales of 0
      auto locate = [&](const Cursor &c, bool &there) -> const uint8_t * {
        there = (uint32_t)c.page < (uint32_t)a.pages;
        return there ? a.cache + (((int64_t)c.page * a.kv_heads + w.head) * rpp + c.off) * R::BYTES : a.cache;
      };
      Cursor ck = start(w.first * 8 + k_rec), cv = start(w.first * 8 + (v_oct >> 1));
      uint4 kc[KW], vc[4];                       // codes and scales of the tile to convert next
      uint2 ksf = make_uint2(0, 0), vsf = make_uint2(0, 0);
      bool k_there, v_there;
      auto fetch_k = [&](bool more) {
        const uint8_t *p = locate(ck, k_there);
#pragma unroll
        for (int i = 0; i < KW; ++i) kc[i] = __ldg(reinterpret_cast<const uint4 *>(p + k_row * (D / 2)) + i);
        if constexpr (D == 128)
          ksf = __ldg(reinterpret_cast<const uint2 *>(p + R::K_SF + k_row * R::NB));
        else
          ksf.x = __ldg(reinterpret_cast<const uint32_t *>(p + R::K_SF + k_row * R::NB));
        if (more) advance(ck);
      };
      auto fetch_v = [&](bool more) {
        const uint8_t *p = locate(cv, v_there);
        if (v_on) {
          const int at = v_blk * kKvGroup + (v_oct & 1) * 8;
#pragma unroll
          for (int i = 0; i < 4; ++i) vc[i] = __ldg(reinterpret_cast<const uint4 *>(p + R::V_CODES + at * 8) + i);
          vsf = __ldg(reinterpret_cast<const uint2 *>(p + R::V_SF + at));
        }
        if (more) advance(cv);
      };
      fetch_k(w.count > 1);
      fetch_v(w.count > 1);
      for (int j = 0; j < w.count; ++j, ++n) {
        const int st = n & 1;
        const uint32_t ph = ((n >> 1) & 1) ^ 1u;
        // ---- K: row ct, D elements
        bool got = wait(&s_kempty[st], ph);
        if (__any_sync(0xffffffffu, !got)) {
          give_up();
          ok = false;
          break;
        }
        {
          const uint32_t there = __ballot_sync(0xffffffffu, k_there);    // two records a warp
          if (lane == 0)
            reinterpret_cast<uint8_t *>(&s_valid[n & 3])[warp & 3] = (uint8_t)((there & 1u) | ((there >> 15) & 2u));
          // 128-byte rows: chunk c of row r sits at c ^ (r & 7)
          const uint32_t ks = (sbase + C::K_AT + st * C::Q_BYTES + ct * 128) ^ ((uint32_t)(ct & 7) << 4);
          const uint32_t sw[2] = {k_there ? ksf.x : 0u, k_there ? ksf.y : 0u};
#pragma unroll
          for (int i = 0; i < KW; ++i) {                          // 32 elements: scales 2i, 2i + 1
            const uint32_t x[4] = {kc[i].x, kc[i].y, kc[i].z, kc[i].w};
            const uint32_t two = e4m3x2_to_f16x2((sw[i >> 1] >> (16 * (i & 1))) & 0xffffu);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t h[4];
              e2m1x8_to_f16x2(x[k], h);
              const uint32_t sf = __byte_perm(two, 0, k < 2 ? 0x1010 : 0x3232);
#pragma unroll
              for (int z = 0; z < 4; ++z) h[z] = hmul2_u32(h[z], sf);
              const int chunk = 4 * i + k;                        // 8 elements
              st_shared16((ks ^ ((chunk & 7) << 4)) + (chunk >> 3) * C::SUB, h);
            }
          }
        }
        ptx::fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&s_kfull[st]);
        if (j + 1 < w.count) fetch_k(j + 2 < w.count);
        // ---- V^T: rows 16 v_blk .. + 15, tokens 8 v_oct .. + 7
        got = wait(&s_vempty[st], ph);
        if (__any_sync(0xffffffffu, !got)) {
          give_up();
          ok = false;
          break;
        }
        if (v_on) {
          // tokens past the end and in front of every row's window count 0, whatever their scales hold
          const int at = (w.first + j) * kTile + 8 * v_oct, to = v_there ? w.len - at : 0, from = w.seen - at;
          const uint32_t sf[2] = {scales_within(vsf.x, from, to), scales_within(vsf.y, from - 4, to - 4)};
          uint32_t s2[4];
#pragma unroll
          for (int p = 0; p < 4; ++p) s2[p] = e4m3x2_to_f16x2((sf[p >> 1] >> (16 * (p & 1))) & 0xffffu);
          const uint32_t vt = (sbase + C::V_AT + st * C::Q_BYTES + (v_oct >> 3) * C::VSUB + v_blk * 16 * 128) ^
                              ((uint32_t)(v_oct & 7) << 4);
#pragma unroll
          for (int h = 0; h < 2; ++h) {                           // elements 8 h .. 8 h + 7 of the block
            uint32_t ev[4][4], od[4][4];                          // [token pair][element pair]
#pragma unroll
            for (int p = 0; p < 4; ++p) {
              const uint32_t w0 = h ? vc[p].y : vc[p].x, w1 = h ? vc[p].w : vc[p].z;
              e2m1x8_to_f16x2((w0 & 0x0f0f0f0fu) | ((w1 << 4) & 0xf0f0f0f0u), ev[p]);
              e2m1x8_to_f16x2(((w0 >> 4) & 0x0f0f0f0fu) | (w1 & 0xf0f0f0f0u), od[p]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              uint32_t y[4];
#pragma unroll
              for (int p = 0; p < 4; ++p) y[p] = hmul2_u32(i & 1 ? od[p][i >> 1] : ev[p][i >> 1], s2[p]);
              st_shared16((vt ^ (i << 4)) + (h * 8 + i) * 128, y);
            }
          }
        }
        ptx::fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&s_vfull[st]);
        if (j + 1 < w.count) fetch_v(j + 2 < w.count);
      }
    }
  } else {
    // ----------------------------------------------------------------- MMA
    shrink_regs<kMmaRegs>();
    if (warp == kMmaWarp) {
      // All lanes walk the loop and wait; one elected lane issues.  With the
      // loop uniform, addresses and descriptors stay in uniform registers, and
      // an MMA costs the warp a few issue slots (it shares them with softmax
      // and conversion warps).
      const bool lead = ptx::elect_one();
      // kind::f16: fp32 accumulator, f16 operands, K-major, N, M = 128
      constexpr uint32_t idesc_s = (1u << 4) | ((uint32_t)(kTile >> 3) << 17) | (8u << 24);
      constexpr uint32_t idesc_o = (1u << 4) | ((uint32_t)(D >> 3) << 17) | (8u << 24);
      const uint32_t sb = ptx::smem_u32(base);
      // Descriptors are built once; an MMA adds a constant (16-byte units) to
      // their address field: 64 cycles an MMA against 82 with each built anew.
      const uint64_t qd = ptx::smem_desc(sb, 16, 1024, 2), kd = ptx::smem_desc(sb + C::K_AT, 16, 1024, 2),
                     vd = ptx::smem_desc(sb + C::V_AT, 16, 1024, 2);
      auto wait_all = [&](uint64_t *bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)); };
      auto commit = [&](uint64_t *bar) {
        if (lead) ptx::tc_commit(bar);
      };
      auto issue_s = [&](int t, uint32_t n) {
        const uint64_t q = qd + (uint64_t)(t * (C::Q_BYTES >> 4)), k0 = kd + (uint64_t)((n & 1) * (C::Q_BYTES >> 4));
        const uint32_t acc = tmem + C::S_COL + t * kTile;
        if (lead) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint64_t at = (uint64_t)(((k >> 2) * C::SUB + (k & 3) * 32) >> 4);
            ptx::mma_bf16(acc, q + at, k0 + at, idesc_s, k > 0);
          }
          ptx::tc_commit(&s_sfull[t]);
        }
        mma_issued = true;
      };
      uint32_t n = 0, seg[2] = {0, 0}, step[2] = {0, 0};
      bool ok = true;
      for (uint32_t sn = 0; ok; ++sn) {
        ok = wait_all(&s_segfull[sn % kSegSlots], (sn / kSegSlots) & 1);
        if (!ok) break;
        const int count = s_seg[sn % kSegSlots].count, nt = s_seg[sn % kSegSlots].rows > kTile ? 2 : 1;
        __syncwarp();
        if (lead) ptx::mbar_arrive(&s_segempty[sn % kSegSlots]);
        if (count == 0) break;
        ok = wait_all(&s_kfull[n & 1], (n >> 1) & 1);
        for (int t = 0; t < nt && ok; ++t) {
          ok = wait_all(&s_qfull[t], seg[t] & 1);
          ++seg[t];
          if (!ok) break;
          ptx::tc_fence_after();
          issue_s(t, n);
          if (t == nt - 1) commit(&s_kempty[n & 1]);
        }
        // (what is waited for comes while a poll sleeps: with a limit of 1 the
        // first probabilities' wait gives up without one, S in flight, and the
        // other roles' by it)
        if (limit == 1) ok = false;
        for (int j = 0; j < count && ok; ++j, ++n) {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (t >= nt || !ok) break;
            if (t == 0) ok = wait_all(&s_vfull[n & 1], (n >> 1) & 1);
            if (ok) ok = wait_all(&s_pfull[t], step[t] & 1);
            ++step[t];
            if (!ok) break;
            ptx::tc_fence_after();
            const uint64_t v0 = vd + (uint64_t)((n & 1) * (C::Q_BYTES >> 4));
            const uint32_t acc = tmem + C::O_COL + t * D, pa = tmem + C::S_COL + t * kTile;
            if (lead) {
#pragma unroll
              for (int k = 0; k < kTile / 16; ++k)
                ptx::mma_f16_tmem_a(acc, pa + 8 * k, v0 + (uint64_t)(((k >> 2) * C::VSUB + (k & 3) * 32) >> 4), idesc_o,
                                    j > 0 || k > 0);
            }
            if (t == nt - 1) commit(&s_vempty[n & 1]);
            if (j + 1 < count) {
              if (t == 0) ok = wait_all(&s_kfull[(n + 1) & 1], ((n + 1) >> 1) & 1);
              if (!ok) break;
              ptx::tc_fence_after();
              issue_s(t, n + 1);
              if (t == nt - 1) commit(&s_kempty[(n + 1) & 1]);
            } else {
              commit(&s_ofull[t]);
            }
          }
        }
      }
      if (!ok) give_up();
      // everything issued has completed before TMEM and shared memory go
      if (mma_issued && lead) {
        ptx::tc_commit(&s_drain);
        for (uint32_t polls = 0; polls < kDrainPolls && !ptx::mbar_try_wait(&s_drain, 0); ++polls) {}
      }
      __syncwarp();
    }
    if (warp == kWalkWarp && lane == 0) {
      // ------------------------------------------------------------- walk
      Walk<D> w(a, group, head_cost, begin, end, split, single, s_start);
      for (uint32_t sn = 0;; ++sn) {
        const int i = sn % kSegSlots;
        if (!wait(&s_segempty[i], ((sn / kSegSlots) & 1) ^ 1u)) {
          give_up();
          break;
        }
        Segment g{};
        if (w.next()) {
          const int k = w.u.tile * kRows / group;
          g.b = w.u.b, g.len = w.u.len, g.head = w.head, g.rows = w.rows(), g.first = w.first, g.count = w.count;
          g.token = w.u.q0 + k, g.pos = w.u.pos0 + k, g.rem = w.u.tile * kRows - k * group;
          g.seen = a.window > 0 ? max(g.pos - (int)a.window + 1, 0) : 0;
          g.whole = w.whole;
          if (!w.whole) {
            g.p0 = line.part_of(w.unit0);
            g.p1 = line.part_of(w.unit1 - 1);
          }
        }
        s_seg[i] = g;
        ptx::mbar_arrive(&s_segfull[i]);
        if (g.count == 0) break;
      }
    }
    __syncwarp();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == kMmaWarp) ptx::tmem_dealloc(tmem, C::TMEM_COLS);
}

template <int D>
cudaError_t launch_tc_attention(const KvAttentionParams &a, cudaStream_t st) {
  using C = TcCfg<D>;
  auto kernel = kv_attention_tc_kernel<D>;
  static PerDeviceOnce once;
  if (cudaError_t e = once.run(
          [&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM); }))
    return e;
  const int64_t part_bytes = 2 * (int64_t)C::PART_FLOATS * 4;
  const int64_t room = a.ws_bytes > kCounterArea ? (int64_t)(a.ws_bytes - kCounterArea) / part_bytes : 0;
  const bool split = room >= kSmsPlanned;        // (with less than the room asked for no unit is split, on all CTAs)
  // A launch takes up to kMaxBatch sequences, and a line of 31 bits: larger batches go in slices.
  const double line = kv_attention_places(a.max_q, a.q_heads, a.kv_heads, a.head_dim, a.max_pages * a.page_size);
  const double fit = 2147483647.0 / line;
  if (fit < 1.0) return cudaErrorInvalidValue;               // (the entry point has seen to that)
  int64_t slice = a.batch < kMaxBatch ? a.batch : kMaxBatch;
  if (fit < (double)slice) slice = (int64_t)fit;
  for (int64_t b0 = 0; b0 < a.batch; b0 += slice) {
    const KvAttentionParams p = kv_attention_slice(a, b0, slice);
    int64_t most = num_sms();
    const double bound = line * (double)p.batch / kMinTiles + 1.0;
    if (bound < (double)most) most = (int64_t)bound;
    if (split && room < most) most = room;
    if (cudaError_t e = launch_pdl(kernel, dim3((unsigned)most), dim3(kThreads), C::SMEM, st, p, split, device_status_ptr()))
      return e;
  }
  return cudaSuccess;
}

}  // namespace

double kv_attention_tc_places(int64_t rows, int64_t kv_heads, int64_t tokens) {
  return (double)kv_heads * (double)((rows + kRows - 1) / kRows) * (double)((tokens + kTile - 1) / kTile + kUnitCost);
}

size_t kv_attention_tc_workspace_bytes(int64_t head_dim) {
  return kCounterArea + (size_t)kSmsPlanned * 2 * (size_t)kRows * (size_t)(head_dim + 2) * sizeof(float);
}

cudaError_t launch_kv_attention_tc(const KvAttentionParams &a, cudaStream_t st) {
  return a.head_dim == 64 ? launch_tc_attention<64>(a, st) : launch_tc_attention<128>(a, st);
}

}  // namespace nvfp4
