// Parameters and helpers shared by the 4-bit tree attention's kernels.
#pragma once

#include "q4.cuh"
#include "tsd_common.cuh"

namespace tsd {

struct Q4Attn {
  const uint16_t *q;
  const uint8_t *k, *v;
  const int32_t *table;
  int max_blocks, num_blocks;
  const int32_t *prefix_len, *n_nodes;
  const uint32_t *mask;  // null: node i sees nodes 0..i
  const int32_t *err;
  int B, N_max, Hq, Hkv, g, W, max_slots;
  float scale_log2;
  int rows;        // N_max * g, query rows of one kv head
  int rows_per_block, row_blocks;  // row_blocks blocks over them
  // Cutting up the key ranges.
  //   cluster > 0: a range's pieces are a thread-block cluster of that size
  //   planned: all ranges end to end, cut into equal parts, one a block (Q4Plan)
  //   else: pieces of `chunk` pages, `splits` of the longest range
  int cluster, planned;
  int splits, chunk;
  int slots, min_part;  // planned: blocks that run at a time; least part of one
  int range_cost, row_tiles;  // planned: a range's fixed cost; a unit's cost in a full row block
  int4 *plan;      // planned: per sequence (start, units, row blocks * 4 + cost of a unit in the last, part)
  float *part_o;   // [pieces][rows_per_block][D]: unnormalised fp32 outputs
  float2 *part_ml;  // [pieces][rows_per_block]: (reference in log2 units, sum), sum -1: bad page
  uint16_t *out;
  float *lse;
  int32_t *status;
  uint64_t wait_limit_ns;
  int test_stall;  // the many-row kernel waits for a barrier that nothing signals
};

// Lengths of sequence b; false when it is skipped (and then `bad` says whether
// its lengths are why).
__device__ __forceinline__ bool q4_seq(const Q4Attn &p, int b, int &P, int &nb, bool &bad) {
  bad = false;
  P = p.prefix_len[b];
  nb = p.n_nodes ? p.n_nodes[b] : p.N_max;
  if (p.err && p.err[b] != 0) return false;
  bad = nb < 1 || nb > p.N_max || P < 0 || (int64_t)P + nb > (int64_t)p.max_slots ||
        (int64_t)P + nb > (int64_t)p.max_blocks * kPage;
  return !bad;
}

// Visibility of the 16 slots of a page that starts at tail index j0 (slot -
// P; negative: prefix) for node i: bit s set when slot s is seen.
__device__ __forceinline__ uint32_t q4_visible(const Q4Attn &p, int b, int i, int j0, int nb) {
  if (j0 <= -kPage) return 0xFFFFu;
  uint32_t tail;  // bits of tail nodes from max(j0, 0) on
  const int first = max(j0, 0);
  if (p.mask) {
    const uint32_t *m = p.mask + ((size_t)b * p.N_max + i) * p.W;
    const int w = first >> 5;
    const uint32_t lo = w < p.W ? m[w] : 0u, hi = w + 1 < p.W ? m[w + 1] : 0u;
    tail = __funnelshift_r(lo, hi, first & 31);
  } else {
    const int n = i + 1 - first;  // nodes first..i
    tail = n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u;
  }
  const int left = nb - first;  // nodes of the tree from there on
  if (left < 32) tail &= left <= 0 ? 0u : (1u << left) - 1u;
  if (j0 < 0) tail = (tail << -j0) | ((1u << -j0) - 1u);
  return tail & 0xFFFFu;
}

// The exponent e for which 2^e brings amax to [2^13, 2^14); 0 for zero, inf or
// NaN.  It reaches 140, so 2^e is applied as two factors.
__device__ __forceinline__ int q4_exponent(float amax) {
  if (!(amax > 0.f) || !isfinite(amax)) return 0;
  return 13 - (((int)(__float_as_uint(amax) >> 23) & 0xFF) - 127);
}
// 2^e, |e| <= 126.
__device__ __forceinline__ float q4_pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// Output row of row r of kv head h of sequence b.
__device__ __forceinline__ size_t q4_out_row(const Q4Attn &p, int b, int h, int r) {
  return ((size_t)b * p.N_max + r / p.g) * p.Hq + h * p.g + r % p.g;
}

// First partial row of a uniformly cut piece.
__device__ __forceinline__ size_t q4_part_row(const Q4Attn &p, int b, int h, int rb, int split) {
  return ((((size_t)b * p.Hkv + h) * p.row_blocks + rb) * p.splits + split) * p.rows_per_block;
}

// The plan of a batch of up to 64 sequences.  Every (sequence, kv head, row block)
// has a key range of t units of 8 pages (128 keys).  A unit costs w, 1 or 2 (the
// many-row kernel's row tiles), and a range F more for its set-up, so unit u of a
// range begins at F + u w.  The ranges are laid end to end and cut into equal
// parts, as many as blocks run at a time, and a block takes the units that begin in
// its part: every block has the same work whatever the lengths, and only a range
// that a cut goes through leaves partial rows.  Every block computes the plan for
// itself (about a microsecond), which spares a kernel before this one.
constexpr int kPlanSeqs = 64;
constexpr int kPlanPieces = 64;  // pieces of one range at most
constexpr int kUnitPages = 8;

struct Q4Plan {
  int start[kPlanSeqs + 1];  // where each sequence begins
  int units[kPlanSeqs], rbs[kPlanSeqs], last_w[kPlanSeqs], P[kPlanSeqs], nb[kPlanSeqs];
  int part;  // length of a block's part
};

// One segment: pages [first, last) of a key range.
struct Q4Seg {
  int b, h, rb, P, nb;
  int first, last;
  bool direct;   // the whole range: rows go straight to the output
  size_t part;   // else the first partial row
};

// The plan, by warp 0; the block's other threads see it after its next barrier.
__device__ __forceinline__ void q4_plan(const Q4Attn &p, Q4Plan &sh) {
  const int lane = threadIdx.x & 31;
  int cnt[2], longest = 0;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int b = 2 * lane + e;
    int P = 0, nb = 0;
    bool bad = false;
    const bool ok = b < p.B && q4_seq(p, b, P, nb, bad);
    const int t = ok ? (P + nb + kUnitPages * kPage - 1) / (kUnitPages * kPage) : 0;
    const int rbs = ok ? (nb * p.g + p.rows_per_block - 1) / p.rows_per_block : 0;
    const int last_w = p.row_tiles > 1 && nb * p.g - (rbs - 1) * p.rows_per_block > p.rows_per_block / 2 ? 2 : 1;
    sh.units[b] = t;
    sh.rbs[b] = rbs;
    sh.last_w[b] = last_w;
    sh.P[b] = P;
    sh.nb[b] = nb;
    cnt[e] = rbs ? (rbs * p.range_cost + t * ((rbs - 1) * p.row_tiles + last_w)) * p.Hkv : 0;
    longest = max(longest, t * p.row_tiles + p.range_cost);
    if (blockIdx.x == 0 && bad && p.status) atomicOr(p.status, TSD_STATUS_BAD_LEN);
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
  int incl = cnt[0] + cnt[1];
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += y;
  }
  const int total = __shfl_sync(0xffffffffu, incl, 31);
  const int part = max(max((total + p.slots - 1) / p.slots, p.min_part),
                       (longest + kPlanPieces - 3) / (kPlanPieces - 2));
  const int first = incl - cnt[0] - cnt[1];
  sh.start[2 * lane] = first;
  sh.start[2 * lane + 1] = first + cnt[0];
  if (lane == 31) {
    sh.start[kPlanSeqs] = total;
    sh.part = part;
  }
  if (blockIdx.x == 0) {  // for the join
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int b = 2 * lane + e;
      if (b < p.B) p.plan[b] = make_int4(first + (e ? cnt[0] : 0), sh.units[b], sh.rbs[b] * 4 + sh.last_w[b], part);
    }
  }
}

// The next segment of this block; g counts along its part (start at blockIdx.x *
// part when planned, else at 0).  False: there is none.
__device__ __forceinline__ bool q4_next(const Q4Attn &p, const Q4Plan &sh, int &g, Q4Seg &s) {
  if (p.planned) {
    const int end = min(sh.start[kPlanSeqs], (int)(blockIdx.x + 1) * sh.part);
    while (g < end) {
      int b = 0;  // the last sequence that starts at or before g and is not empty
#pragma unroll
      for (int step = kPlanSeqs / 2; step; step >>= 1)
        if (sh.start[b + step] <= g) b += step;
      const int t = sh.units[b], last_w = sh.last_w[b], rbs = sh.rbs[b];
      const int full = p.range_cost + t * p.row_tiles;
      const int head = rbs * full - t * (p.row_tiles - last_w);
      const int local = g - sh.start[b];
      s.b = b;
      s.h = local / head;
      s.rb = min((local - s.h * head) / full, rbs - 1);
      const int w = s.rb == rbs - 1 ? last_w : p.row_tiles;
      const int x0 = local - s.h * head - s.rb * full;
      const int x1 = min(p.range_cost + t * w, x0 + end - g);
      g += x1 - x0;
      const int u0 = (max(x0 - p.range_cost, 0) + w - 1) / w, u1 = (max(x1 - p.range_cost, 0) + w - 1) / w;
      if (u0 >= u1) continue;
      s.P = sh.P[b];
      s.nb = sh.nb[b];
      s.first = u0 * kUnitPages;
      s.last = min((s.P + s.nb + kPage - 1) / kPage, u1 * kUnitPages);
      s.direct = u1 - u0 == t;
      // a cut leaves a block at most one range whose start it has but not its end,
      // and one whose start it has not
      s.part = ((size_t)blockIdx.x * 2 + (u0 == 0 ? 1 : 0)) * p.rows_per_block;
      return true;
    }
    return false;
  }
  if (g != 0) return false;
  g = 1;
  const int split = blockIdx.x % p.splits, hr = blockIdx.x / p.splits;
  s.b = blockIdx.y;
  s.h = hr / p.row_blocks;
  s.rb = hr % p.row_blocks;
  bool bad;
  const bool ok = q4_seq(p, s.b, s.P, s.nb, bad);
  if (bad && blockIdx.x == 0 && threadIdx.x == 0 && p.status) atomicOr(p.status, TSD_STATUS_BAD_LEN);
  if (!ok) s.nb = 0;  // (no valid row)
  const int pages = ok ? (s.P + s.nb + kPage - 1) / kPage : 0;
  // (even, so that a warp's two pages at a time are in one piece)
  const int chunk = p.cluster ? ((pages + p.splits - 1) / p.splits + 1) & ~1 : p.chunk;
  s.first = split * chunk;
  s.last = min(pages, s.first + chunk);
  s.direct = p.splits == 1;
  s.part = p.cluster ? 0 : q4_part_row(p, s.b, s.h, s.rb, split);
  return true;
}

// The many-row kernel (attention_q4_tc.cu); blocks: its grid when planned.
cudaError_t q4_tc_launch(const Q4Attn &p, int D, int blocks, cudaStream_t s);

}  // namespace tsd
