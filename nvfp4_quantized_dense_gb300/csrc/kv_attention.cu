// Causal attention of grouped query heads over the paged NVFP4 cache, for
// decode-sized query tiles.
//
// A query token i of a sequence (the sequence's last q_len tokens, already in
// the cache) stands at position p = len - q_len + i and sees the cached tokens
// t with t <= p and, with a window w > 0, t > p - w:
//   s_t = qk_scale * sum_d q_d * Kq[t, d],   m = max s,  l = sum exp(s_t - m)
//   out = v_scale / l * sum_t exp(s_t - m) * Vq[t, :],   lse = m + log l
// with Kq, Vq = E2M1 code * E4M3 scale.  A query that sees nothing gives 0 and
// lse = -inf.
//
// Tokens as the matrix instruction's rows.  The query heads that share a
// key/value head (times a few query tokens) are only 1 to 32 rows, so the
// products are taken transposed, with mma.m16n8k16:
//   S^T [16 tokens, 8 queries] = K [16, D] Q^T,   O^T [D, 8 queries] += V^T P^T
// The cached operand fills the 16-row side, the queries the 8-wide one: a
// padded row would cost conversions and products, a padded query column none
// of the first.  Which 16 tokens and which 16 elements share a k-step is free
// as long as both operands agree, and is chosen so that the cache's bytes go
// from shared memory to the fragments with no exchange between threads:
//   lane = 4 g + c.  K: lane (g, c) holds elements [c D/4, (c+1) D/4) of the
//   tokens of rows g and g + 8;  V: lane (g, c) holds elements [g D/8, (g+1)
//   D/8) of tokens 4c .. 4c+3 of a record;  so row r < 8 of S^T is token
//   4 (r/2) + r%2 of the record, and row r + 8 two tokens further.
// P^T is S^T's accumulator layout transposed: one movmatrix per 8x8 tile.
//
// Exactness.  Codes times scales have at most 6 significant bits and are exact
// in f16; a query row is scaled by a power of two that brings its largest
// magnitude into [2^14, 2^15), which makes its bf16 elements exact in f16 down
// to 2^-28 of that magnitude.  Products and sums are fp32, the probabilities
// enter as f16 times 2^kShift (kShift keeps the small ones of a long flat row
// normal: f16 is normal down to 2^-14, so down to 2^-28 of the largest).
//
// Work split.  A unit (sequence, key/value head, tile of query rows) is a row
// of 32-token steps.  With fewer units than CTAs, every CTA takes one piece of
// one unit, the pieces as even as the grid allows (8 steps at least; units of
// 16 and fewer stay whole).  With more units, or where whole pieces leave the
// longest most of a unit's end above the even share, the units lie on a
// line, with UNIT_COST places ahead of each for its beginning and end, and the
// line is cut into equal parts, one per CTA (24 sequences of 8192, 32 rows:
// 134 us, as pieces 204; 16 of 2048: 35, as pieces 36.  200 sequences of 1 to
// 4,000: 130 us with 12 places, 162 with 6, 150 with 24; all before the
// queries' move to shared memory).  Either way lengths may differ by any factor and
// stay balanced, and the plan needs nothing from the host but the grid, so a
// captured call follows the lengths on the device.  The CTAs that share a unit
// leave partial sums in the workspace, and the last of them to arrive adds
// them up in the order of the parts (the result does not depend on who is
// last).  In a CTA four warps take the steps in turn, each with its own ring of
// bulk copies (one per record: 16 tokens of one head, keys, values and scales
// together) and its own running maximum and sum, joined through shared memory
// at the end of the unit: no barrier between the warps inside a unit.
//
// What bounds it (8 key/value heads of 128):
//   4 sequences of 131,072 (604 MB): 120 us, 5.0 TB/s, 74 % of the copy rate.
//     Issue slots: 655 instructions a warp and step, 0.60 issued a cycle, the
//     ALU pipe 56 % busy (half of that are the E2M1 conversions, 2 cycles an
//     instruction).  The copies alone, the arithmetic left out, run at 92 %.
//     (5 query heads to each key/value head, as 8 rows.)
//   32 sequences of 1 to 8,190 tokens (38 MB): 19 us; 1 of 512: 7.7 us, of
//     which the launch, the plan, the first record's way from HBM and the join
//     are 5: latency, not a rate.
//   32 rows (16 sequences of 16,384, 4 query tokens by 8 heads): 137 us.  The
//     accumulators are 128 registers a thread, so two warps a scheduler run,
//     and they wait for themselves (0.4 instructions a cycle).  Two 16-row
//     tiles would convert everything twice.
// Four warps to a CTA and 4 CTAs an SM beat 8 and 16 warps a CTA (joins wait
// for more warps) and 5 CTAs at 96 registers (spills); two stages a warp beat
// three (shared memory is not the limit, but the first copies are later); from
// 16 rows on three do best.
#include "common.cuh"
#include "internal.h"
#include "kv_attention_common.cuh"
#include "kv_layout.cuh"
#include "tc_ptx.cuh"

namespace nvfp4 {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kStep = 32;                    // tokens of a step: two records
constexpr int kMinSteps = 8, kWhole = 16;    // steps of the smallest piece, of a unit not to be split (12: no gain)
constexpr float kShift = 14.0f;
constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr uint32_t kDrainPolls = 1u << 22;
constexpr int kSmsPlanned = 152;             // workspace sizing (the launch takes what fits)

// What a unit's beginning and end cost, in steps, by its groups of 8 rows.
constexpr int unit_cost(int groups) { return groups == 1 ? 8 : 12; }

template <int D, int NQ>
struct Cfg {
  using R = KvRecord<D>;
  static constexpr int ROWS = 8 * NQ;                       // query rows of a tile
  static constexpr int CTAS = (NQ == 1 ? 4 : NQ == 2 ? 3 : 2) + (D == 64 && NQ == 2);    // per SM, by registers
  static constexpr int STAGES = NQ == 1 ? 2 : 3;
  static constexpr int UNIT_COST = unit_cost(NQ);
  static constexpr int STAGE_BYTES = 2 * R::BYTES;
  static constexpr int RING_BYTES = kWarps * STAGES * STAGE_BYTES;
  static constexpr int JOIN_BYTES = kWarps * ROWS * (D + 2) * 4;
  static constexpr int Q_AT = RING_BYTES > JOIN_BYTES ? RING_BYTES : JOIN_BYTES;
  // The queries' fragments stay in registers, but for the largest tile: its
  // accumulators leave them no room, and read again from shared memory (each
  // lane its own) they cost less than the spills (24 sequences of 8192: 110 us
  // against 134).  At head_dim 64 there is room: 69 either way.
  static constexpr int Q_BYTES = D == 128 && NQ == 4 ? kWarps * ROWS * D * 2 : 0;
  static constexpr int SMEM = Q_AT + Q_BYTES;
  static constexpr int PART_FLOATS = ROWS * (D + 2);        // a partial result: m and l of the rows, then O
  static constexpr int PART_BYTES = PART_FLOATS * 4;
};

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same with no accumulator to start from.
__device__ __forceinline__ void mma16816_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
               : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// One sequence's share of the line of steps.
struct Seq {
  int q0, qn, len, pos0;      // first query token, queries, cached tokens, position of the first query
  int lo_step, steps;         // steps of a unit (at least one, so that empty rows are written)
  int tiles;                  // query tiles of a key/value head
};

template <int ROWS>
__device__ __forceinline__ Seq seq_of(const KvAttentionParams &a, int b, int group) {
  Seq s;
  int q0 = b * (int)a.max_q, q1 = q0 + (int)a.max_q;
  if (a.cu_q) {
    q0 = min(max(__ldg(a.cu_q + b), 0), (int)a.tokens);
    q1 = min(max(__ldg(a.cu_q + b + 1), q0), (int)a.tokens);
  }
  s.q0 = q0;
  s.qn = min(q1 - q0, (int)a.max_q);
  s.len = min(max(__ldg(a.seq_lens + b), 0), (int)(a.max_pages * a.page_size));
  s.pos0 = s.len - s.qn;
  const int lo = a.window > 0 ? max(s.pos0 - (int)a.window + 1, 0) : 0;
  s.lo_step = lo / kStep;
  s.steps = max((s.len + kStep - 1) / kStep - s.lo_step, 1);
  s.tiles = (int)(((int64_t)s.qn * group + ROWS - 1) / ROWS);
  return s;
}

// Pieces of a unit of n steps, of about 1 / inv_chunk each; a unit of a few
// steps is not worth joining.  (Floating point: integer divisions would be a
// good part of a short call.  Every CTA gets the same numbers.)
__device__ __forceinline__ int pieces_of(int n, float inv_chunk, bool split) {
  return !split || n <= kWhole ? 1 : 1 + (int)((float)(n - 1) * inv_chunk);
}
// x / d for x < 2^20 and small d, from 1 / d
__device__ __forceinline__ int div_small(int x, float inv) { return (int)(((float)x + 0.5f) * inv); }

template <int D, int NQ>
__global__ void __launch_bounds__(kThreads, Cfg<D, NQ>::CTAS)
    kv_attention_kernel(const __grid_constant__ KvAttentionParams a, const bool split, int *status) {
  using C = Cfg<D, NQ>;
  using R = KvRecord<D>;
  constexpr int ROWS = C::ROWS, KW = D / 32;      // KW: 32-bit words of a lane's K elements
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t s_full[kWarps][C::STAGES];
  __shared__ uint8_t s_valid[kWarps][C::STAGES];
  __shared__ int s_abort[kWarps];
  __shared__ uint32_t s_last;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int group = (int)(a.q_heads / a.kv_heads);
  // (a warp's ring is its own: no barrier with the others)
  if (lane < C::STAGES) ptx::mbar_init(&s_full[warp][lane], 1);
  if (lane == 0) s_abort[warp] = 0;
  ptx::fence_barrier_init();
  __syncwarp();
  pdl_trigger();
  pdl_wait();

  // ---- this CTA's part of the line of steps (its length fits 31 bits: the
  // launch sees to that).  Every warp finds it for itself, with no barrier:
  // lane i takes the sequences [i per, (i + 1) per).
  const int heads = (int)a.kv_heads, batch = (int)a.batch, grid = (int)gridDim.x, part = (int)blockIdx.x;
  const int per = (batch + 31) >> 5, b_lo = min(lane * per, batch), b_hi = min(b_lo + per, batch);
  Seq sq{};                                       // this lane's sequence, where it has one only
  int my_units = 0, my_steps = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    sq = seq_of<ROWS>(a, b, group);
    my_units += heads * sq.tiles;
    my_steps += heads * sq.tiles * sq.steps;
  }
  const int all_units = __reduce_add_sync(0xffffffffu, my_units), all_steps = __reduce_add_sync(0xffffffffu, my_steps);
  // Fewer units than CTAs: every CTA takes one piece of one unit, of at most
  // `chunk` steps (two ends of units in one CTA would cost it twice), unless
  // the pieces come out too uneven.  Else the units lie on the line with their
  // steps, and `head_cost` places ahead of them: what beginning and ending one
  // costs a CTA.
  bool pieces = all_units < grid;
  float inv_chunk = 0.0f;
  int head_cost = 0, mine = 0;                    // mine: places of this lane's sequences
  if (pieces) {
    // the even share if that fits the grid, else one that always does (a unit rounds up by less than one piece)
    inv_chunk = fminf(__fdividef((float)grid, (float)max(all_steps, 1)), 1.0f / kMinSteps);
    float longest = 0.0f;                         // piece, in steps
    for (int turn = 0;; ++turn) {
      mine = 0, longest = 0.0f;
      for (int b = b_lo; b < b_hi; ++b) {
        if (per > 1) sq = seq_of<ROWS>(a, b, group);
        const int n = pieces_of(sq.steps, inv_chunk, split);
        mine += heads * sq.tiles * n;
        if (sq.tiles > 0) longest = fmaxf(longest, __fdividef((float)sq.steps, (float)n));
      }
      if (turn || __reduce_add_sync(0xffffffffu, mine) <= grid) break;
      inv_chunk = fminf(__fdividef((float)(grid - all_units), 1.001f * (float)all_steps), 1.0f / kMinSteps);
    }
    // (the longest piece against the even share and most of a unit's end more)
    if (split && all_steps >= 4 * grid) {
      const float even = __fdividef((float)all_steps, (float)grid);
      pieces = !__any_sync(0xffffffffu, longest > fmaxf(even + 0.8f * C::UNIT_COST, (float)kWhole));
    }
  }
  if (!pieces) {
    head_cost = min(C::UNIT_COST, all_steps / grid);
    mine = my_steps + head_cost * my_units;
  }
  auto places = [&](int n) { return pieces ? pieces_of(n, inv_chunk, split) : n + head_cost; };   // of a unit of n steps
  int upto = mine;                                // places of the sequences up to and including this lane's
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += u;
  }
  const int total = __shfl_sync(0xffffffffu, upto, 31);
  if (part >= total) return;
  const Line line(pieces ? 1 : total, pieces ? 1 : grid);      // (pieces: places are parts)
  const int begin = pieces ? part : line.at(part), end = pieces ? part + 1 : line.at(part + 1);
  // the lane whose sequences hold the beginning; then the sequence, and where it begins on the line
  const int src = __ffs(__ballot_sync(0xffffffffu, begin < upto)) - 1;
  int seq_at = __shfl_sync(0xffffffffu, upto - mine, src), b = src * per;
  if (per == 1) {
    sq.q0 = __shfl_sync(0xffffffffu, sq.q0, src), sq.qn = __shfl_sync(0xffffffffu, sq.qn, src);
    sq.len = __shfl_sync(0xffffffffu, sq.len, src), sq.pos0 = __shfl_sync(0xffffffffu, sq.pos0, src);
    sq.lo_step = __shfl_sync(0xffffffffu, sq.lo_step, src), sq.steps = __shfl_sync(0xffffffffu, sq.steps, src);
    sq.tiles = __shfl_sync(0xffffffffu, sq.tiles, src);
  } else {
    sq = seq_of<ROWS>(a, b, group);
  }
  // a negative scale goes into q's sign, so that the largest raw score is the largest scaled one
  const float qk0 = __ldg(a.qk_scale) * 1.4426950408889634f, qk = fabsf(qk0), vs = __ldg(a.v_scale);
  const uint32_t rpp = (uint32_t)a.page_size / kKvGroup;     // records of a page
  const int rpp_shift = (rpp & (rpp - 1)) == 0 ? 31 - __clz(rpp) : -1;
  const float inv_group = __fdividef(1.0f, (float)group);    // (a unit has at most 64 rows)
  uint8_t *ring = smem + warp * C::STAGES * C::STAGE_BYTES;
  uint64_t *full = s_full[warp];
  uint4 *q_own = reinterpret_cast<uint4 *>(smem + C::Q_AT) + warp * (C::ROWS * D / 8) + lane;    // (Q_BYTES > 0)
  uint32_t put = 0, get = 0, phase = 0;           // stage to fill and to read next, and the latter's phase
  bool gave_up = false;
  const uint64_t policy = ptx::l2_policy_evict_normal();

  for (int pos = begin; pos < end;) {
    int len = places(sq.steps);
    while (pos >= seq_at + heads * sq.tiles * len) {
      seq_at += heads * sq.tiles * len;
      sq = seq_of<ROWS>(a, ++b, group);
      len = places(sq.steps);
    }
    const float inv_len = __fdividef(1.0f, (float)len), inv_tiles = __fdividef(1.0f, (float)sq.tiles);
    const int unit = pieces ? div_small(pos - seq_at, inv_len) : (pos - seq_at) / len;
    const int unit0 = seq_at + unit * len + head_cost, unit1 = seq_at + (unit + 1) * len;
    if (pos < unit0) pos = unit0;                 // its steps are [unit0, unit1), or its pieces
    if (pos >= end) break;
    const int head = div_small(unit, inv_tiles), tile = unit - head * sq.tiles;      // (at most 1024 heads of a few tiles)
    if (!split && pos != unit0) {                 // whole units only: this one belongs to the part it begins in
      pos = unit1;
      continue;
    }
    const int seg1 = split ? min(unit1, end) : unit1;
    auto step_at = [&](int x) {
      return !pieces ? x - unit0 : x == unit1 ? sq.steps : (int)((float)(x - unit0) * ((float)sq.steps * inv_len));
    };
    // rows of the tile: query row r -> (token q0 + r / group, head head * group + r % group)
    const int row0 = tile * ROWS, rows = min(sq.qn * group - row0, ROWS);
    const int first = sq.pos0 + div_small(row0, inv_group), last = sq.pos0 + div_small(row0 + rows - 1, inv_group);   // positions
    const int win = (int)a.window;
    const int seen = win > 0 ? max(first - win + 1, 0) : 0;      // first token that any row of the tile sees
    // the segment's steps that any row of the tile sees
    int st0 = sq.lo_step + step_at(pos), st1 = sq.lo_step + step_at(seg1);
    st1 = min(st1, last < 0 ? 0 : last / kStep + 1);
    st0 = max(st0, seen / kStep);

    // ---- the warp's steps: st0 + warp, + kWarps, ...  Lanes 2i, 2i+1 look up the
    // pages of the two records of step number base + i; `next` runs 16 steps ahead.
    const int count = max((st1 - st0 - warp + kWarps - 1) / kWarps, 0);
    const int32_t *table = a.block_table + (int64_t)b * a.max_pages;
    // ---- queries: lane (g, c) holds elements [c D/4, (c+1) D/4) of row 8 n + g
    uint32_t qf[NQ][D / 8];                       // (loaded ahead of the copies' addresses, converted after)
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int r = row0 + 8 * n + g, i = div_small(r, inv_group);
      const uint16_t *src = a.q + (int64_t)(sq.q0 + i) * a.q_stride + (int64_t)(head * group + r - i * group) * D + c * (D / 4);
#pragma unroll
      for (int i4 = 0; i4 < D / 32; ++i4) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r < row0 + rows) v = *reinterpret_cast<const uint4 *>(src + 8 * i4);
        qf[n][4 * i4] = v.x, qf[n][4 * i4 + 1] = v.y, qf[n][4 * i4 + 2] = v.z, qf[n][4 * i4 + 3] = v.w;
      }
    }
    auto lookup = [&](int base) -> int {          // number of the record in the cache, -1: none
      const int i = base + (lane >> 1);
      const uint32_t rec = (uint32_t)(st0 + warp + i * kWarps) * 2 + (lane & 1);
      if (i >= count || (int)rec * kKvGroup >= sq.len) return -1;
      const uint32_t pi = rpp_shift >= 0 ? rec >> rpp_shift : rec / rpp;
      const int page = __ldg(table + pi);
      if (page < 0 || page >= (int)a.pages) return -1;
      return (page * heads + head) * (int)rpp + (int)(rec - pi * rpp);
    };
    int here = lookup(0), next = count > 16 ? lookup(16) : -1;
    int issued = 0;
    auto issue = [&]() {                          // copies of step number `issued` into its stage
      const int at = __shfl_sync(0xffffffffu, here, 2 * (issued & 15) + (lane & 1));
      const uint32_t ok = __ballot_sync(0xffffffffu, at >= 0) & 3u;
      if (lane == 0) {
        s_valid[warp][put] = (uint8_t)ok;
        ptx::mbar_arrive_expect_tx(&full[put], __popc(ok) * R::BYTES);
      }
      __syncwarp();
      if (lane < 2 && at >= 0)
        ptx::bulk_load(ring + put * C::STAGE_BYTES + lane * R::BYTES, a.cache + (int64_t)at * R::BYTES, R::BYTES,
                       &full[put], policy);
      if (++put == C::STAGES) put = 0;
      if ((++issued & 15) == 0) {
        here = next;
        next = lookup(issued + 16);
      }
    };
    if (!gave_up)
      while (issued < count && issued < C::STAGES) issue();

    float sc[NQ][2];                              // scale of the scores of rows 8 n + 2c, + 1
    int hi[NQ][2];                                // last token that those rows see
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      uint32_t top = 0;                           // largest magnitude of the row, as bits
#pragma unroll
      for (int i = 0; i < D / 8; ++i) top = max(top, max(qf[n][i] & 0x7fffu, (qf[n][i] >> 16) & 0x7fffu));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // exponent field of the magnitude -> 2^(141 - e); subnormal and zero rows as the smallest normal one
      const int e = min(max((int)(top >> 7), 15), 254);
      const float up = row_factor((uint32_t)(127 + 141 - e), qk0);       // 2^126 .. 2^-113
#pragma unroll
      for (int i = 0; i < D / 8; ++i) qf[n][i] = f16x2(bf16_lo(qf[n][i]) * up, bf16_hi(qf[n][i]) * up);
      if constexpr (C::Q_BYTES > 0)
#pragma unroll
        for (int i = 0; i < KW; ++i)
          q_own[(n * KW + i) * 32] = make_uint4(qf[n][4 * i], qf[n][4 * i + 1], qf[n][4 * i + 2], qf[n][4 * i + 3]);
      const int e0 = __shfl_sync(0xffffffffu, e, 8 * c), e1 = __shfl_sync(0xffffffffu, e, 8 * c + 4);
      // 2^(e - 141) in two factors (e may be as low as 15: 2^-126, normal)
      // (positive even for a scale of 0: the maximum may be -inf)
      sc[n][0] = fmaxf(qk * __uint_as_float((uint32_t)max(e0 - 14, 1) << 23), 1.17549435e-38f);
      sc[n][1] = fmaxf(qk * __uint_as_float((uint32_t)max(e1 - 14, 1) << 23), 1.17549435e-38f);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int q = row0 + 8 * n + 2 * c + j;
        hi[n][j] = q < row0 + rows ? sq.pos0 + div_small(q, inv_group) : sq.len - 1;        // rows of no query see everything
      }
    }

    float o[NQ][D / 16][4];
    float m[NQ][2], l[NQ][2];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.0f;
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.0f;
    }

    // (the copies may be there before the first poll, or while it sleeps in the
    // barrier unit: a limit of 1 gives up without one)
    if (issued > 0 && a.wait_limit == 1) gave_up = true;
    int done = 0;
    for (; done < count && !gave_up; ++done) {
      if (!ptx::mbar_wait_bounded(&full[get], phase, a.wait_limit, kTimeoutNs, &s_abort[warp])) gave_up = true;
      if (__any_sync(0xffffffffu, gave_up)) {
        gave_up = true;
        break;
      }
      const uint32_t valid = s_valid[warp][get];
      const int t0 = (st0 + warp + done * kWarps) * kStep;
      const bool masked = valid != 3 || t0 + kStep - 1 > min(first, sq.len - 1) || (win > 0 && t0 <= last - win);
      const uint8_t *st = ring + get * C::STAGE_BYTES;

      // ---- scores
      float s[NQ][2][4];
#pragma unroll
      for (int rec = 0; rec < 2; ++rec) {
        const uint8_t *rp = st + rec * R::BYTES;
        const int tg = 4 * (g >> 1) + (g & 1);    // token of row g; row g + 8 is two further
        uint32_t w[2][KW], ks[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint8_t *kp = rp + (tg + 2 * h) * (D / 2) + c * (D / 8);
          if constexpr (D == 128) {
            const uint4 v = *reinterpret_cast<const uint4 *>(kp);
            w[h][0] = v.x, w[h][1] = v.y, w[h][2] = v.z, w[h][3] = v.w;
            ks[h] = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t *>(rp + R::K_SF + (tg + 2 * h) * R::NB + 2 * c));
          } else {
            const uint2 v = *reinterpret_cast<const uint2 *>(kp);
            w[h][0] = v.x, w[h][1] = v.y;
            ks[h] = e4m3x2_to_f16x2(rp[R::K_SF + (tg + 2 * h) * R::NB + c]);
          }
        }
#pragma unroll
        for (int j = 0; j < KW; ++j) {            // 8 elements of each row: two k-steps
          uint32_t x[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t sf = __byte_perm(ks[h], 0, j < 2 ? 0x1010 : 0x3232);
            e2m1x8_to_f16x2(w[h][j], x[h]);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[h][i] = hmul2_u32(x[h][i], sf);
          }
#pragma unroll
          for (int n = 0; n < NQ; ++n) {
            uint4 q = make_uint4(qf[n][4 * j], qf[n][4 * j + 1], qf[n][4 * j + 2], qf[n][4 * j + 3]);
            if constexpr (C::Q_BYTES > 0) q = q_own[(n * KW + j) * 32];
            if (j == 0)
              mma16816_zero(s[n][rec], x[0][0], x[1][0], x[0][1], x[1][1], q.x, q.y);
            else
              mma16816(s[n][rec], x[0][0], x[1][0], x[0][1], x[1][1], q.x, q.y);
            mma16816(s[n][rec], x[0][2], x[1][2], x[0][3], x[1][3], q.z, q.w);
          }
        }
      }
      if (masked) {
#pragma unroll
        for (int rec = 0; rec < 2; ++rec)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int t = t0 + rec * kKvGroup + 4 * (g >> 1) + (g & 1) + (i & 2);
#pragma unroll
            for (int n = 0; n < NQ; ++n)
              if (!((valid >> rec) & 1) || t > hi[n][i & 1] || t >= sq.len || (win > 0 && t <= hi[n][i & 1] - win))
                s[n][rec][i] = -INFINITY;
          }
      }

      // ---- running maximum and sum, probabilities
      uint32_t p[NQ][2][2];
      bool moved = false;
      float keep[NQ][2];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        float base[2];                            // what the exponentials refer to
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float top = fmaxf(fmaxf(s[n][0][j], s[n][0][j + 2]), fmaxf(s[n][1][j], s[n][1][j + 2]));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
          top = fmaxf(top, m[n][j]);
          base[j] = top == -INFINITY ? 0.0f : top;
          moved |= top != m[n][j];
          // (1 exactly where the maximum stays: the sum, unlike O, takes the factor at every step)
          keep[n][j] = exp2_fast((m[n][j] - base[j]) * sc[n][j]);
          m[n][j] = top;
        }
        // The difference first, then the scale: s * sc - base * sc would be off
        // by the product's rounding, without limit for large scores.  (Both
        // rows of a lane in one instruction.)
        const uint64_t minus = pack2(-base[0], -base[1]), sc2 = pack2(sc[n][0], sc[n][1]), shift2 = pack2(kShift, kShift);
        uint64_t sum2 = 0;
#pragma unroll
        for (int rec = 0; rec < 2; ++rec)
#pragma unroll
          for (int i = 0; i < 4; i += 2) {
            unpack2(fma2(add2(pack2(s[n][rec][i], s[n][rec][i + 1]), minus), sc2, shift2), s[n][rec][i], s[n][rec][i + 1]);
            s[n][rec][i] = exp2_fast(s[n][rec][i]), s[n][rec][i + 1] = exp2_fast(s[n][rec][i + 1]);
            sum2 = add2(sum2, pack2(s[n][rec][i], s[n][rec][i + 1]));
          }
        float sum[2];
        unpack2(sum2, sum[0], sum[1]);
#pragma unroll
        for (int j = 0; j < 2; ++j) l[n][j] = l[n][j] * keep[n][j] + sum[j];
      }
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int rec = 0; rec < 2; ++rec) {
          p[n][rec][0] = transpose8x8(f16x2(s[n][rec][0], s[n][rec][1]));
          p[n][rec][1] = transpose8x8(f16x2(s[n][rec][2], s[n][rec][3]));
        }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[n][i][j] *= keep[n][j & 1];
      }

      // ---- O^T += V^T P^T
#pragma unroll
      for (int rec = 0; rec < 2; ++rec) {
        const uint8_t *rp = st + rec * R::BYTES;
        uint32_t w[4][D / 64];                    // tokens 4c + i: this lane's D/8 elements
        uint32_t vsf;
        if constexpr (D == 128) {
          const uint4 *vp = reinterpret_cast<const uint4 *>(rp + R::V_CODES + (g * kKvGroup + 4 * c) * 8);
          const uint4 v0 = vp[0], v1 = vp[1];
          w[0][0] = v0.x, w[0][1] = v0.y, w[1][0] = v0.z, w[1][1] = v0.w;
          w[2][0] = v1.x, w[2][1] = v1.y, w[3][0] = v1.z, w[3][1] = v1.w;
          vsf = *reinterpret_cast<const uint32_t *>(rp + R::V_SF + g * kKvGroup + 4 * c);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i][0] = *reinterpret_cast<const uint32_t *>(rp + R::V_CODES + ((g >> 1) * kKvGroup + 4 * c + i) * 8 + (g & 1) * 4);
          vsf = *reinterpret_cast<const uint32_t *>(rp + R::V_SF + (g >> 1) * kKvGroup + 4 * c);
        }
        if (masked) {                             // past the end, and in front of every row's window
          const int at = t0 + rec * kKvGroup + 4 * c;
          vsf = scales_within(vsf, seen - at, ((valid >> rec) & 1) ? sq.len - at : 0);
        }
        const uint32_t s01 = e4m3x2_to_f16x2(vsf & 0xffffu), s23 = e4m3x2_to_f16x2(vsf >> 16);
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
          uint32_t e01[4], o01[4], e23[4], o23[4];      // even and odd elements, pairs of tokens
          e2m1x8_to_f16x2((w[0][j] & 0x0f0f0f0fu) | ((w[1][j] << 4) & 0xf0f0f0f0u), e01);
          e2m1x8_to_f16x2(((w[0][j] >> 4) & 0x0f0f0f0fu) | (w[1][j] & 0xf0f0f0f0u), o01);
          e2m1x8_to_f16x2((w[2][j] & 0x0f0f0f0fu) | ((w[3][j] << 4) & 0xf0f0f0f0u), e23);
          e2m1x8_to_f16x2(((w[2][j] >> 4) & 0x0f0f0f0fu) | (w[3][j] & 0xf0f0f0f0u), o23);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t a0 = hmul2_u32(e01[i], s01), a1 = hmul2_u32(o01[i], s01), a2 = hmul2_u32(e23[i], s23),
                           a3 = hmul2_u32(o23[i], s23);
#pragma unroll
            for (int n = 0; n < NQ; ++n) mma16816(o[n][4 * j + i], a0, a1, a2, a3, p[n][rec][0], p[n][rec][1]);
          }
        }
      }
      __syncwarp();                               // every lane has read the stage
      if (++get == C::STAGES) get = 0, phase ^= 1;
      if (issued < count) issue();
    }
    // copies still in flight (after a wait that gave up): wait for them, bounded, before the memory changes hands
    for (int i = done; i < issued; ++i) {
      for (uint32_t polls = 0; polls < kDrainPolls && !ptx::mbar_try_wait(&full[get], phase); ++polls) {}
      if (++get == C::STAGES) get = 0, phase ^= 1;
    }
    if (gave_up && lane == 0) *status = NVFP4_ERR_DEVICE_TIMEOUT;

    // ---- join the warps: [warp][row][D] sums, then m and l
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        l[n][j] += __shfl_xor_sync(0xffffffffu, l[n][j], 4);
        l[n][j] += __shfl_xor_sync(0xffffffffu, l[n][j], 8);
        l[n][j] += __shfl_xor_sync(0xffffffffu, l[n][j], 16);
      }
    float *join = reinterpret_cast<float *>(smem), *jm = join + kWarps * ROWS * D, *jl = jm + kWarps * ROWS;
    __syncthreads();                              // the rings are drained
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = 8 * n + 2 * c + j;
        float4 *dst = reinterpret_cast<float4 *>(join + (warp * ROWS + r) * D + g * (D / 8));
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
          dst[i] = make_float4(o[n][2 * i][j], o[n][2 * i][j + 2], o[n][2 * i + 1][j], o[n][2 * i + 1][j + 2]);
        if (g == 0) {
          jm[warp * ROWS + r] = m[n][j] == -INFINITY ? -INFINITY : m[n][j] * sc[n][j];
          jl[warp * ROWS + r] = l[n][j];
        }
      }
    __syncthreads();
    const bool whole = pos == unit0 && seg1 == unit1;
    // parts that share this unit, and this CTA's two places for partial results
    const int p0 = line.part_of(unit0), p1 = line.part_of(unit1 - 1);
    float *parts_at = reinterpret_cast<float *>(static_cast<uint8_t *>(a.workspace) + kCounterArea);
    auto place = [&](int q) { return parts_at + (int64_t)(2 * q + (q == p0 ? 1 : 0)) * C::PART_FLOATS; };
    auto write_out = [&](int r, int d, float4 acc, float top, float sum) {
      const int64_t token = sq.q0 + (row0 + r) / group;
      const int qh = head * group + (row0 + r) % group;
      const float inv = sum == 0.0f ? 0.0f : vs / sum;      // (a NaN in the query makes its row NaN)
      const __nv_bfloat162 x = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
      const __nv_bfloat162 y = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
      *reinterpret_cast<uint2 *>(a.out + (token * a.q_heads + qh) * D + d) =
          make_uint2(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y));
      if (a.lse && d == 0)
        a.lse[token * a.q_heads + qh] = sum == 0.0f ? -INFINITY : (top + (log2f(sum) - kShift)) * 0.6931471805599453f;
    };
    // the four warps' sums of one row, four elements at a time
    auto join_warps = [&](auto &&sink) {
      for (int i = tid; i < rows * (D / 4); i += kThreads) {
        const int r = i / (D / 4), d = i % (D / 4) * 4;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, jm[w * ROWS + r]);
        const float ref = top == -INFINITY ? 0.0f : top;
        float4 acc = make_float4(0, 0, 0, 0);
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float k = exp2_fast(jm[w * ROWS + r] - ref);
          const float4 v = *reinterpret_cast<const float4 *>(join + (w * ROWS + r) * D + d);
          sum += k * jl[w * ROWS + r];
          acc.x += k * v.x, acc.y += k * v.y, acc.z += k * v.z, acc.w += k * v.w;
        }
        sink(r, d, acc, top, sum);
      }
    };
    if (whole) {
      join_warps(write_out);
    } else {
      float *mine_at = place(part);
      join_warps([&](int r, int d, float4 acc, float top, float sum) {
        __stcg(reinterpret_cast<float4 *>(mine_at + 2 * ROWS + r * D + d), acc);
        if (d == 0) {
          __stcg(mine_at + r, top);
          __stcg(mine_at + ROWS + r, sum);
        }
      });
      // the last of the unit's parts to arrive joins them all, in their order
      __syncthreads();
      if (tid == 0) {
        uint32_t *counter = static_cast<uint32_t *>(a.workspace) + p0, before;
        asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
        s_last = before == (uint32_t)(p1 - p0);
        if (s_last) *counter = 0;
      }
      __syncthreads();
      if (s_last) {
        // (all of a batch's loads are in flight together: one after the other
        // they would cost a trip to L2 each)
        constexpr int ITEMS = (ROWS * D / 4 + kThreads - 1) / kThreads, BATCH = ITEMS < 16 ? 16 / ITEMS : 1;
        float4 acc[ITEMS];
        float top[ITEMS], sum[ITEMS];
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) acc[i] = make_float4(0, 0, 0, 0), top[i] = -INFINITY, sum[i] = 0.0f;
        for (int q0 = p0; q0 <= p1; q0 += BATCH) {
          float4 v[ITEMS][BATCH];
          float mq[ITEMS][BATCH], lq[ITEMS][BATCH];
#pragma unroll
          for (int i = 0; i < ITEMS; ++i)
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
              const int item = tid + i * kThreads, r = min(item / (D / 4), rows - 1), d = item % (D / 4) * 4;
              const float *src = place(min(q0 + k, p1));
              mq[i][k] = q0 + k <= p1 ? __ldcg(src + r) : -INFINITY;
              lq[i][k] = __ldcg(src + ROWS + r);
              v[i][k] = __ldcg(reinterpret_cast<const float4 *>(src + 2 * ROWS + r * D + d));
            }
#pragma unroll
          for (int i = 0; i < ITEMS; ++i)
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
              const float t2 = fmaxf(top[i], mq[i][k]), ref = t2 == -INFINITY ? 0.0f : t2;
              const float k0 = exp2_fast(top[i] - ref), k1 = exp2_fast(mq[i][k] - ref);
              top[i] = t2;
              sum[i] = sum[i] * k0 + lq[i][k] * k1;
              acc[i].x = acc[i].x * k0 + v[i][k].x * k1, acc[i].y = acc[i].y * k0 + v[i][k].y * k1;
              acc[i].z = acc[i].z * k0 + v[i][k].z * k1, acc[i].w = acc[i].w * k0 + v[i][k].w * k1;
            }
        }
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
          const int item = tid + i * kThreads, r = item / (D / 4), d = item % (D / 4) * 4;
          if (r < rows) write_out(r, d, acc[i], top[i], sum[i]);
        }
      }
    }
    ptx::fence_proxy_async_shared();
    __syncthreads();                              // the join area becomes the rings again
    pos = unit1;
  }
}

template <int D, int NQ>
size_t part_bytes() { return 2 * (size_t)Cfg<D, NQ>::PART_BYTES; }

template <int D, int NQ>
cudaError_t launch(const KvAttentionParams &a, cudaStream_t st) {
  using C = Cfg<D, NQ>;
  auto kernel = kv_attention_kernel<D, NQ>;
  static PerDeviceOnce once;
  if (cudaError_t e = once.run(
          [&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM); }))
    return e;
  // The kernel counts steps in 31 bits: a batch whose line could be longer is taken in slices.
  const double line = kv_attention_places(a.max_q, a.q_heads, a.kv_heads, a.head_dim, a.max_pages * a.page_size);
  const double fit = 2147483647.0 / line;
  if (fit < 1.0) return cudaErrorInvalidValue;               // (the entry point has seen to that)
  const int64_t slice = fit < (double)a.batch ? (int64_t)fit : a.batch;
  // With less than the room asked for no unit is split, on all CTAs: as many
  // CTAs as there is room for may be one.
  const int64_t room = a.ws_bytes > kCounterArea ? (int64_t)((a.ws_bytes - kCounterArea) / part_bytes<D, NQ>()) : 0;
  const bool split = room >= kSmsPlanned * C::CTAS;
  for (int64_t b0 = 0; b0 < a.batch; b0 += slice) {
    const KvAttentionParams p = kv_attention_slice(a, b0, slice);
    int64_t most = (int64_t)num_sms() * C::CTAS;
    const double bound = line * (double)p.batch / kMinSteps + 1.0;   // pieces, at most
    if (bound < (double)most) most = (int64_t)bound;
    if (split && room < most) most = room;
    if (cudaError_t e = launch_pdl(kernel, dim3((unsigned)most), dim3(kThreads), C::SMEM, st, p, split, device_status_ptr()))
      return e;
  }
  return cudaSuccess;
}

}  // namespace

KvAttentionParams kv_attention_slice(const KvAttentionParams &a, int64_t b0, int64_t n) {
  KvAttentionParams p = a;
  p.batch = a.batch - b0 < n ? a.batch - b0 : n;
  if (p.cu_q) {
    p.cu_q += b0;
  } else {
    p.q += b0 * a.max_q * a.q_stride;
    p.out += b0 * a.max_q * a.q_heads * a.head_dim;
    if (p.lse) p.lse += b0 * a.max_q * a.q_heads;
  }
  p.block_table += b0 * a.max_pages;
  p.seq_lens += b0;
  return p;
}

// Query rows of a key/value head above which the tcgen05 form runs.  Its tiles
// cost the same for 1 to 128 rows; here the cost grows with the rows.  Measured
// (us, here / there): head_dim 128, 16 sequences of 16384: 32 rows 136 / 180,
// 48 rows 205 / 181; of 2048: 31 / 34 and 39 / 34.  head_dim 64, 16 of 16384:
// 64 rows 160 / 166, 96 rows 234 / 166; of 2048: 31 / 30 and 42 / 30.  Single
// short sequences are faster here for longer (1 of 2048, 48 rows: 15 / 21), but
// the lengths are not known to the host.
static int64_t tc_rows(int64_t head_dim) { return head_dim == 128 ? 32 : 64; }

// Groups of 8 rows in a tile, for as few and as even tiles as there can be of
// up to 32 rows.  (What a tile costs grows with its rows: 24 sequences of 8192
// at head_dim 128 take 54, 69, 89 and 110 us with 8, 16, 24 and 32.)
static int tile_groups(int64_t rows) {
  const int64_t tiles = (rows + 31) / 32;
  return (int)((rows + 8 * tiles - 1) / (8 * tiles));
}

// One sequence's places on the line at most, as either form counts them.
double kv_attention_places(int64_t max_q, int64_t q_heads, int64_t kv_heads, int64_t head_dim, int64_t tokens) {
  const int64_t rows = max_q * (q_heads / kv_heads);
  if (rows > tc_rows(head_dim)) return kv_attention_tc_places(rows, kv_heads, tokens);
  return (double)kv_heads * (double)((rows + 31) / 32) * (double)((tokens + kStep - 1) / kStep + unit_cost(tile_groups(rows)));
}

size_t kv_attention_workspace_bytes(int64_t max_q, int64_t q_heads, int64_t kv_heads, int64_t head_dim) {
  const int64_t rows = max_q * (q_heads / kv_heads);
  if (rows > tc_rows(head_dim)) return kv_attention_tc_workspace_bytes(head_dim);
  const int nq = tile_groups(rows);
  const int64_t ctas = kSmsPlanned * ((nq == 1 ? 4 : nq == 2 ? 3 : 2) + (head_dim == 64 && nq == 2));
  return kCounterArea + (size_t)ctas * 2 * (size_t)(8 * nq) * (size_t)(head_dim + 2) * sizeof(float);
}

cudaError_t launch_kv_attention(const KvAttentionParams &a, cudaStream_t st) {
  const int64_t rows = a.max_q * (a.q_heads / a.kv_heads);
  if (rows > tc_rows(a.head_dim)) return launch_kv_attention_tc(a, st);
  switch (tile_groups(rows)) {
    case 1: return a.head_dim == 64 ? launch<64, 1>(a, st) : launch<128, 1>(a, st);
    case 2: return a.head_dim == 64 ? launch<64, 2>(a, st) : launch<128, 2>(a, st);
    case 3: return a.head_dim == 64 ? launch<64, 3>(a, st) : launch<128, 3>(a, st);
    default: return a.head_dim == 64 ? launch<64, 4>(a, st) : launch<128, 4>(a, st);
  }
}

}  // namespace nvfp4
