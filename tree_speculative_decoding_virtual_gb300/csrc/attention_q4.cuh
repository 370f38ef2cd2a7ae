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
  //   planned: pieces from the actual lengths (q4_item), one block each
  //   else: pieces of `chunk` pages, `splits` of the longest range
  int cluster, planned;
  int splits, chunk;
  int slots;       // blocks that run at a time
  int fixed;       // a block's set-up and end, in units of 8 pages
  int join_units;  // what a further piece costs in memory traffic, in 1/1024 unit per row block
  int4 *plan;      // planned: per sequence (first item, pieces, pages of a piece, row blocks)
  float *part_o;   // [blocks][rows_per_block][D]: unnormalised fp32 outputs
  float2 *part_ml;  // [blocks][rows_per_block]: (reference in log2 units, sum), sum -1: bad page
  uint16_t *out;
  float *lse;
  int32_t *status;
  uint64_t wait_limit_ns;
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

// First partial row of a uniformly cut piece (a planned one's: its block's).
__device__ __forceinline__ size_t q4_part_row(const Q4Attn &p, int b, int h, int rb, int split) {
  return ((((size_t)b * p.Hkv + h) * p.row_blocks + rb) * p.splits + split) * p.rows_per_block;
}

// A block's piece of work.
struct Q4Item {
  int b, h, rb;       // sequence, kv head, row block; b = -1: none
  int pieces, split;  // pieces of its key range, and which
  int chunk;          // pages of a piece
};

constexpr int kPlanSeqs = 64;    // sequences of a planned batch
constexpr int kPlanPieces = 32;  // pieces of one range at most
constexpr int kUnitPages = 8;    // ranges are cut at multiples of 8 pages

struct Q4PlanShared {
  int units[kPlanSeqs], mult[kPlanSeqs];  // of each sequence: key range, blocks per piece
  Q4Item item;
};

// The batch's plan and this block's item of it, by warp 0; the others learn it
// after the block's next barrier.  Candidate i cuts the longest range into i + 1
// pieces, of C units, and every other one into pieces of at most C; the plan is
// the candidate of least estimated time, with a = T / items the mean piece,
//   max(ceil(items / slots) (a + fixed), items / slots (a + fixed) + longest - a)
// plus the further pieces' traffic: whole waves for equal ranges, the last
// piece's excess for ragged ones.  Every block computes it (B <= 64: about a
// microsecond), which spares a kernel of its own before this one.
__device__ __forceinline__ void q4_plan_item(const Q4Attn &p, Q4PlanShared &sh, int k) {
  const int lane = threadIdx.x & 31;
  int units[2], mult[2], longest = 0;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int b = 2 * lane + e;
    int P, nb;
    bool bad;
    const bool ok = b < p.B && q4_seq(p, b, P, nb, bad);
    units[e] = ok ? (P + nb + kUnitPages * kPage - 1) / (kUnitPages * kPage) : 0;
    mult[e] = ok ? p.Hkv * ((nb * p.g + p.rows_per_block - 1) / p.rows_per_block) : 0;
    sh.units[b] = units[e];
    sh.mult[b] = mult[e];
    longest = max(longest, units[e]);
    if (k == 0 && b < p.B && !ok && bad && p.status) atomicOr(p.status, TSD_STATUS_BAD_LEN);
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
  __syncwarp();
  const int C = max(1, (longest + lane) / (lane + 1));  // this lane's candidate
  const float inv = 1.f / (float)C;
  int items = 0, extra = 0, total = 0;
  for (int b = 0; b < p.B; ++b) {
    const int t = sh.units[b], m = sh.mult[b], x = t + C - 1;
    int n = (int)((float)x * inv);
    n -= n * C > x ? 1 : 0;
    n += (n + 1) * C <= x ? 1 : 0;
    items += n * m;
    extra += n > 1 ? n * m : 0;
    total += t * m;
  }
  float est = 3.0e38f;
  if (items > 0 && (items <= (int)gridDim.x || lane == 0)) {
    const float mean = (float)total / (float)items, x = (float)items / (float)p.slots;
    est = fmaxf(ceilf(x) * (mean + p.fixed), x * (mean + p.fixed) + (float)C - mean);
    est += (float)extra * (float)p.join_units * (1.f / 1024.f);
  }
  const uint32_t key = __float_as_uint(est);  // (positive floats order as integers)
  const uint32_t least = __reduce_min_sync(0xffffffffu, key);
  const int who = __ffs(__ballot_sync(0xffffffffu, key == least)) - 1;
  const int best = __shfl_sync(0xffffffffu, C, who);
  // number the items: this lane's two sequences
  int n[2], cnt[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    n[e] = (units[e] + best - 1) / best;
    cnt[e] = n[e] * mult[e];
  }
  int incl = cnt[0] + cnt[1];
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += y;
  }
  if (lane == 31 && k >= incl) sh.item.b = -1;
  int first = incl - cnt[0] - cnt[1];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int b = 2 * lane + e;
    const int rbs = mult[e] / p.Hkv;
    const int chunk = n[e] > 0 ? (units[e] + n[e] - 1) / n[e] * kUnitPages : 0;
    if (k >= first && k < first + cnt[e]) {
      const int x = (k - first) / rbs;  // row blocks of a piece next to each other: they share its pages
      sh.item = Q4Item{b, x / n[e], (k - first) % rbs, n[e], x % n[e], chunk};
    }
    if (k == 0 && b < p.B) p.plan[b] = make_int4(first, n[e], chunk, rbs);
    first += cnt[e];
  }
}

// The many-row kernel (attention_q4_tc.cu); blocks: its grid when planned.
cudaError_t q4_tc_launch(const Q4Attn &p, int D, int blocks, cudaStream_t s);

}  // namespace tsd
