// Tree-masked attention for a batch whose sequences share prefixes: groups of
// sequences hold the same keys and values in their first S slots ("Speculative
// Decoding Hierárquico: Medusa, EAGLE-2 e Multi-Token Prediction", section on
// paged caches: blocks of a common prompt are shared), and these are read and
// multiplied once for the rows of the whole group.
//
// A softmax over a union of key sets is the weighted mean of the softmaxes over
// the parts, weights exp(lse): so the work is a list of units, each a set of query
// rows and one key range,
//   group g, kv head:     rows of all its trees x slots [0, S)
//   sequence b, kv head:  rows of its tree      x slots [S, P + n)
// in row blocks of 256, whose parts are joined at the end.
//
// Plan (one block, its own kernel): lengths are known to the device alone.  The
// units' key tiles (128 keys; cost 1, or 2 with more than 128 rows, and a fixed cost
// a unit) are laid end to end and cut into equal parts, one a block, so that every SM
// has the same work whatever the lengths, as long as there is enough of it: a part is no
// shorter than a set-up and two tiles, and a range has at most 64 (counted as if it had
// two row tiles), so one or two kv heads do not fill the GPU (4 tokens of 8 heads behind 131072
// slots of one kv head: 67 us, of two 77, of eight 122).  Trees are packed, so that padding nodes
// cost nothing.  Where there are blocks enough, no part spans two units (4 tokens behind
// 2048 slots: the attention 12 us, 19.5 with such parts).
//
// Block: the segments of its part in turn, each walked in 128-key tiles on the
// 5th-generation tensor cores:
//   warp 0       K tiles by TMA (2 stages), warp 2 V tiles
//   warp 1       owns TMEM; lane 0 issues every MMA
//   warp 3       tells it when V is there, after clearing what no row may see
//   warps 4-11   softmax of chain 0, warps 12-19 of chain 1: one TMEM lane (= one
//                query row) per thread, two threads a row (64 keys each)
// A chain is a row tile of 128 rows with its S (128 columns of TMEM; each thread's P, bf16,
// goes over the first half of its own scores, so that nothing but the reference ties
// the two threads of a row together) and O.  With more than 128 rows the chains are two row tiles
// that share every key tile; with fewer, chain c takes the key tiles j = c mod 2 of the
// same rows and the two are joined at the end.
//   S = Q K^T         M = 128, N = 128, bf16 in, fp32 accumulate
//   P = exp2(S c - m) bf16, over S
//   O += P V          A from TMEM, V MN-major
// The MMAs of a chain execute in issue order, S_{j+1} right behind P_j V_j, so the softmax
// that sees S_j complete may rescale O and overwrite S_j.  A row's reference m is the
// maximum of its chain's first tile, and moves when 64 keys' P sum above 2^60.
// Row sums add P before its rounding to bf16: the roundings are as often up as down,
// and the row's lse is that of the fp32 scores.  (The tensor core takes P in V's type.  Against
// 64 bits the outputs are off by 0.0023 of their size, by 0.0017 where nothing but they is rounded.)
//
// 0 times a NaN is one: V's rows outside the key range (the rest of a page, never
// written) are set to zero in shared memory, and so is a tree node's with a NaN or an
// infinity, for it may be hidden from some rows; the rows that do see it become NaN.
//
// What bounds it, and what it measured.  Long shared ranges with many rows: the two chains'
// MMAs and softmaxes (3500 cycles for a tile of 256 rows; 8 trees of 127 nodes, 64 heads,
// 32768 shared slots: 755 us, 1.5 PFLOP/s; a register split 104 / 64 and not 96 for all
// warps 850 -> 803, a row's threads tied by a barrier of two warps 803 -> 769).  Many
// short own ranges: the start and end of each (64 tokens behind 16384 slots: 77 us; 16
// trees of 16 to 31 nodes: 57 us).  These are the attention's; the plan takes 8 to 10, the join
// 8 to 40.  Beside tree_attn_fwd on the same tensors, cold and with all three kernels: 64 tokens 97
// and 568 us, 16 tokens behind 2048 slots 32 and 37, 4 behind 2048 30 and 22, behind 32768 58
// and 85; 8 trees of 127 nodes 790 and 935, 16 of 16 to 31 nodes 75 and 65.  Tried and slower: the next range's ids, queries and
// first tiles fetched ahead by warp 3 (791 to 902 us, 85 to 94 us; at the range's end no
// difference), all segments cut by the plan (it takes 20 instead of 7 us), a polynomial in
// place of half the exponentials.
//
// Every wait is bounded; on expiry the block flags TSD_STATUS_TIMEOUT, drains what it
// issued, frees its tensor memory and returns.

#include <cuda_bf16.h>

#include <cmath>

#include "cache_map.cuh"
#include "sm100_ptx.cuh"
#include "tsd_common.cuh"

namespace tsd {
namespace {

constexpr int kThreads = 640;
constexpr int kSoftmaxWarp = 4;     // the first softmax warp
constexpr int kBM = 128;            // rows of a row tile
constexpr int kRows = 256;          // rows of a row block
constexpr int kBN = 128;            // keys of a tile
constexpr int kTilePages = kBN / kPage;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemChain = 256, kTmemO = 128;
constexpr float kMaxSum = 0x1p60f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr uint64_t kDrainNs = 100000000ull;
constexpr int kMaxBatch = 1024;
constexpr int kPlanThreads = 1024, kSmallPlan = 256;  // of the plan; up to kSmallPlan sequences the fewer
constexpr int kPieces = 64;     // pieces of one key range at most
// A range's fixed cost in a row block of one or two row tiles, in key tiles of one: what
// its start and end take (loads of ids, queries and the first tiles one behind the other,
// masks, the finished rows: some 14k cycles of a range of three tiles with one row tile).
// Measured, 64 tokens / 16 trees / 8 trees of 127 nodes over 32768 slots: 8 and 20 75 / 55 /
// 746 us, 4 and 12 80 / 60 / 857, 12 and 28 82 / 62 / 748, 8 and 32 74 / 60 / 784.
constexpr int kRangeCost1 = 8, kRangeCost2 = 20;

// One row set and its key range, for every kv head.
struct Unit {
  long long start;     // where its cost begins
  long long row_base;  // query rows (times kv heads) of the units before
  int tiles, rows, rbs, last_w;  // rows of one kv head, their blocks, cost of a tile in the last
  int block_base;      // row blocks (times kv heads) of the units before
  int node0;           // first entry of the node map
  int table;           // sequence whose block table is read
  int lo, hi, P;       // key slots [lo, hi); from P on they are the tree's
  int nb;              // the tree's nodes (own ranges)
  int group;           // own ranges: the shared unit of the same rows, or -1
};
static_assert(sizeof(Unit) == 64, "");

struct Plan {
  long long total, part;
};

struct Seg;

struct Attn {
  const uint16_t *q, *k, *v;
  const int32_t *table;
  int max_blocks, num_blocks;
  const int32_t *prefix_len, *n_nodes;
  const uint32_t *mask;  // null: node i sees nodes 0..i
  const int32_t *err;
  const int32_t *first, *shared;
  int G, B, N_max, Hq, Hkv, g, W;
  float scale_log2;
  int blocks;
  int join_heads;  // heads of a block of the join, a multiple of 8
  Plan *plan;
  Unit *units;        // [G + B]: the groups', then the sequences'
  Seg *first_seg;     // [blocks]
  int2 *marks;        // by row block and kv head: first and last block of its key range
  int32_t *node_map;  // packed node -> b * N_max + i
  float2 *part_ml;    // (reference in log2 units, sum; sum -1: bad page)
  float *part_o;      // unnormalised fp32 outputs
  uint16_t *out;
  float *lse;
  int32_t *status;
  uint64_t wait_limit_ns;
  int test_stall;
};

// ---------------------------------------------------------------------------
// plan
// ---------------------------------------------------------------------------

// Exclusive sums over the block's threads, N at a time; `all` the sums of all.
template <int N>
__device__ __forceinline__ void block_scan(const long long (&x)[N], long long (*buf)[4], long long (&before)[N], long long (&all)[N]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long incl[N];
#pragma unroll
  for (int e = 0; e < N; ++e) {
    incl[e] = x[e];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl[e], off);
      if (lane >= off) incl[e] += y;
    }
  }
  __syncthreads();
  if (lane == 31)
#pragma unroll
    for (int e = 0; e < N; ++e) buf[warp][e] = incl[e];
  __syncthreads();
#pragma unroll
  for (int e = 0; e < N; ++e) {
    before[e] = incl[e] - x[e];
    all[e] = 0;
  }
  for (int w = 0; w < (int)blockDim.x / 32; ++w)
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const long long s = buf[w][e];
      if (w < warp) before[e] += s;
      all[e] += s;
    }
}

// A unit as the plan kernel left it (from L2: another launch may have used the place).
__device__ __forceinline__ Unit load_unit(const Unit *at) {
  union {
    int4 x[4];
    Unit u;
  } r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.x[i] = __ldcg(reinterpret_cast<const int4 *>(at) + i);
  return r.u;
}

// Cost of a unit's row block of w row tiles; `alone` > 0: what its parts of that many
// tiles take, with no set-up.
__device__ __forceinline__ long long block_cost(const Unit &u, int w, int alone) {
  const int tiles = u.tiles * w;
  return alone ? (long long)((tiles + alone - 1) / alone) * alone : (w == 2 ? kRangeCost2 : kRangeCost1) + tiles;
}
__device__ __forceinline__ long long unit_cost(const Unit &u, int Hkv, int alone) {
  return u.rbs ? (long long)Hkv * ((u.rbs - 1) * block_cost(u, 2, alone) + block_cost(u, u.last_w, alone)) : 0;
}

__device__ __forceinline__ void shape_unit(Unit &u, int nodes, int g) {
  const bool any = nodes > 0 && u.hi > u.lo;
  u.rows = nodes * g;
  u.rbs = any ? (u.rows + kRows - 1) / kRows : 0;
  u.tiles = any ? ((u.hi + kPage - 1) / kPage - u.lo / kPage + kTilePages - 1) / kTilePages : 0;
  u.last_w = u.rows - (u.rbs - 1) * kRows > kBM ? 2 : 1;
}

// A block's next piece of work: a run of key tiles for one row block of one kv head.
struct Seg {
  long long next;         // where the block goes on
  long long part;         // first partial row
  int rows, row0;         // the unit's rows of one kv head, the first of this row block
  int h, node0, table;
  int page, pages;        // first page of the range, its pages
  int lo, hi, P, nb;
  int n;                  // key tiles; 0: no more work
  int two;                // two row tiles (each with every key tile), or one row tile whose key
                          // tiles alternate between the chains
  int mark;               // where the join looks for the range's blocks; -1 - that: not the first piece
  int whole;              // 1: the range's last piece
  int pad;
};
static_assert(sizeof(Seg) == 80, "five 16-byte words");

// The segment at g of a unit that holds g, as far as `end`; false when none begins there
// (s.next is moved on).
__device__ __forceinline__ bool cut_segment(const Unit &u, long long g, long long end, int block, int alone, Seg &s) {
  const long long full = block_cost(u, 2, alone);
  const long long head = (u.rbs - 1) * full + block_cost(u, u.last_w, alone);
  const long long local = g - u.start;
  int rb;
  long long x0;
  if (local < 0x7FFFFFFF && head < 0x7FFFFFFF) {  // (a 64-bit division takes some 100 instructions)
    const uint32_t l = (uint32_t)local;
    s.h = (int)(l / (uint32_t)head);
    const uint32_t in_head = l - (uint32_t)s.h * (uint32_t)head;
    rb = min((int)(in_head / (uint32_t)full), u.rbs - 1);
    x0 = (long long)in_head - rb * full;
  } else {
    s.h = (int)(local / head);
    const long long in_head = local - s.h * head;
    rb = (int)min(in_head / full, (long long)(u.rbs - 1));
    x0 = in_head - rb * full;
  }
  const int w = rb == u.rbs - 1 ? u.last_w : 2, fixed = alone ? 0 : w == 2 ? kRangeCost2 : kRangeCost1;
  const long long x1 = min(block_cost(u, w, alone), x0 + end - g);
  s.next = g + x1 - x0;
  // (w is 1 or 2)
  const int u0 = (int)((max(x0 - fixed, 0ll) + w - 1) >> (w - 1));
  const int u1 = min((int)((max(x1 - fixed, 0ll) + w - 1) >> (w - 1)), u.tiles);
  if (u0 >= u1) return false;
  s.rows = u.rows;
  s.row0 = rb * kRows;
  s.node0 = u.node0;
  s.table = u.table;
  s.page = u.lo / kPage + u0 * kTilePages;
  s.pages = min((u.hi + kPage - 1) / kPage - s.page, (u1 - u0) * kTilePages);
  s.lo = u.lo;
  s.hi = u.hi;
  s.P = u.P;
  s.nb = u.nb;
  s.n = u1 - u0;
  s.two = u.rows - s.row0 > kBM;
  s.part = u.row_base + (long long)s.h * u.rows + s.row0 + (long long)block * kRows;
  s.mark = u.block_base + s.h * u.rbs + rb;
  if (u0 > 0) s.mark = -1 - s.mark;
  s.whole = u1 == u.tiles;
  return true;
}

__global__ void __launch_bounds__(kPlanThreads) shared_plan_kernel(const Attn p) {
  __shared__ int off[kMaxBatch + 1];   // packed nodes before sequence b
  __shared__ int first[kMaxBatch + 1], shared[kMaxBatch], members[kMaxBatch], rep[kMaxBatch];
  __shared__ long long starts[2 * kMaxBatch];
  __shared__ long long buf[kPlanThreads / 32][4];
  __shared__ int2 shape[2 * kSmallPlan];
  __shared__ int fits[kSmallPlan / 32];
  __shared__ int bad_groups;
  __shared__ long long longest;
  pdl_trigger();
  const int tid = threadIdx.x, B = p.B, G = p.G;  // (at least B threads, and G <= B)
  if (tid == 0) {
    bad_groups = 0;
    longest = 0;
  }
  pdl_wait();
  int P = 0, nb = 0, S = 0, gr = 0, err = 0;
  if (tid < B) {
    P = p.prefix_len[tid];
    nb = p.n_nodes ? p.n_nodes[tid] : p.N_max;
    err = p.err ? p.err[tid] : 0;
  }
  for (int i = tid; i <= G; i += blockDim.x) first[i] = p.first[i];
  if (tid < G) {
    shared[tid] = p.shared[tid];
    members[tid] = 0;
    rep[tid] = B;
  }
  __syncthreads();
  // the groups are runs of sequences, all of them in one
  if (tid < G && first[tid] > first[tid + 1]) bad_groups = 1;
  if (tid == 0 && (first[0] != 0 || first[G] != B)) bad_groups = 1;
  __syncthreads();
  const bool groups_ok = !bad_groups;
  bool ok = false;
  if (tid < B) {
    bool bad = !groups_ok;
    if (groups_ok) {  // the last group that begins at or before this sequence
      int hi = G - 1;
      while (gr < hi) {
        const int mid = (gr + hi + 1) >> 1;
        if (first[mid] <= tid) gr = mid; else hi = mid - 1;
      }
      S = shared[gr];
      bad = nb < 1 || nb > p.N_max || P < 0 || S < 0 || S > P ||
            (int64_t)P + nb > (int64_t)p.max_blocks * kPage;
    }
    const bool skip = err != 0;
    ok = !bad && !skip;
    if (bad && !skip && p.status) atomicOr(p.status, TSD_STATUS_BAD_LEN);
    if (ok) {
      atomicAdd(&members[gr], 1);
      atomicMin(&rep[gr], tid);
    }
  }
  long long nodes[1] = {ok ? nb : 0}, nodes_before[1], nodes_all[1];
  block_scan(nodes, buf, nodes_before, nodes_all);
  const int node0 = (int)nodes_before[0];
  if (tid < B) off[tid] = node0;
  if (tid == 0) off[B] = (int)nodes_all[0];
  __syncthreads();
  // a thread's two units: a group's shared range, a sequence's own
  Unit u[2] = {};
  if (tid < G && groups_ok) {
    const bool once = members[tid] > 1;  // (one sequence alone keeps its range whole)
    u[0].hi = u[0].P = once ? max(shared[tid], 0) : 0;
    u[0].node0 = off[first[tid]];
    u[0].table = min(rep[tid], B - 1);
    u[0].group = -1;
    shape_unit(u[0], off[first[tid + 1]] - off[first[tid]], p.g);
  }
  if (tid < B) {
    const bool split = ok && members[gr] > 1 && S > 0;
    u[1].lo = split ? S : 0;
    u[1].P = P;
    u[1].hi = ok ? P + nb : 0;
    u[1].node0 = node0;
    u[1].table = tid;
    u[1].nb = ok ? nb : 0;
    u[1].group = split ? gr : -1;
    shape_unit(u[1], u[1].nb, p.g);
  }
  // costs, and row blocks and rows (in one word: rows below 2^40, blocks below 2^23)
  auto packed = [&](const Unit &x) { return x.rbs ? ((long long)x.rbs << 40 | x.rows) * p.Hkv : 0; };
  constexpr long long kRowBits = (1ll << 40) - 1;
  long long total, row_blocks;
  {
    const long long x[4] = {unit_cost(u[0], p.Hkv, 0), unit_cost(u[1], p.Hkv, 0), packed(u[0]), packed(u[1])};
    long long before[4], all[4];
    block_scan(x, buf, before, all);
    u[0].start = before[0];
    u[1].start = all[0] + before[1];
    u[0].row_base = before[2] & kRowBits;
    u[1].row_base = (all[2] + before[3]) & kRowBits;
    u[0].block_base = (int)(before[2] >> 40);
    u[1].block_base = (int)((all[2] + before[3]) >> 40);
    total = all[0] + all[1];
    row_blocks = (all[2] + all[3]) >> 40;
  }
  const long long far = 2ll * max(u[0].tiles, u[1].tiles) + kRangeCost2;
  atomicMax((unsigned long long *)&longest, (unsigned long long)far);
  __syncthreads();
  // (a part shorter than a unit's set-up and two tiles is mostly set-up; longer ones leave
  // SMs idle: 4 tokens behind 2048 slots, laid end to end, take the attention 19.5 us, 21.6
  // with four tiles, 25.7 with ten)
  long long part = max((total + p.blocks - 1) / p.blocks, (long long)kRangeCost1 + 2);
  const long long least = (longest + kPieces - 3) / (kPieces - 2);
  part = max(part, least);
  // Few row blocks: each is cut into parts of its own, so that no block begins twice, if
  // there are blocks enough with parts that are not longer by more than half a
  // set-up.  Each warp tries another length.
  int alone = 0;
  if (row_blocks <= p.blocks && blockDim.x == kSmallPlan) {
    shape[tid] = make_int2(u[0].tiles, u[0].rbs * 2 + u[0].last_w - 2);
    shape[kSmallPlan + tid] = make_int2(u[1].tiles, u[1].rbs * 2 + u[1].last_w - 2);
    __syncthreads();
    const int lane = tid & 31, warp = tid >> 5, most = (int)min(part, 1ll << 20) + kRangeCost1 / 2;
    const int from = max((int)min(least, 1ll << 20), 2);
    const int len = from + warp * max((most - from + 6) / 7, 1);
    long long parts = 0;
    for (int i = lane; i < G + kSmallPlan && i < 2 * kSmallPlan; i += 32) {
      const int2 x = shape[i < G ? i : kSmallPlan + i - G];
      // (x.y: row tiles of all its row blocks)
      if (x.y > 0) parts += (x.y / 2) * ((2 * x.x + len - 1) / len) + (x.y & 1) * ((x.x + len - 1) / len);
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) parts += __shfl_xor_sync(0xffffffffu, parts, off);
    if (lane == 0) fits[warp] = len <= most && parts * p.Hkv <= p.blocks ? len : 0;
    __syncthreads();
    for (int w = kSmallPlan / 32 - 1; w >= 0; --w)
      if (fits[w]) alone = fits[w];
    if (alone) {
      part = alone;
      const long long x[2] = {unit_cost(u[0], p.Hkv, alone), unit_cost(u[1], p.Hkv, alone)};
      long long before[2], all[2];
      block_scan(x, buf, before, all);
      u[0].start = before[0];
      u[1].start = all[0] + before[1];
      total = all[0] + all[1];
    }
  }
  if (tid == 0) *p.plan = Plan{total, part};
  if (tid < G) {
    p.units[tid] = u[0];
    starts[tid] = u[0].start;
  }
  if (tid < B) {
    p.units[G + tid] = u[1];
    starts[G + tid] = u[1].start;
  }
  __syncthreads();
  // every block's first segment
  for (int k = tid; k < p.blocks; k += blockDim.x) {
    long long g = (long long)k * part;
    const long long end = min(total, g + part);
    Seg s;
    s.n = 0;
    while (g < end) {
      int at = 0, hi = G + B - 1;
      while (at < hi) {
        const int mid = (at + hi + 1) >> 1;
        if (starts[mid] <= g) at = mid; else hi = mid - 1;
      }
      if (cut_segment(load_unit(p.units + at), g, end, k, alone, s)) break;
      g = s.next;
      s.n = 0;
    }
    p.first_seg[k] = s;
  }
  for (int b = tid >> 5; b < B; b += blockDim.x / 32)
    for (int i = tid & 31; i < off[b + 1] - off[b]; i += 32) p.node_map[off[b] + i] = b * p.N_max + i;
}

// ---------------------------------------------------------------------------
// segments
// ---------------------------------------------------------------------------

// The block's next segment after `g`, in the part that ends at `end`; by a whole warp.
__device__ __forceinline__ void next_segment(const Attn &p, long long g, long long end, Seg &s) {
  const int lane = threadIdx.x & 31, count = p.G + p.B;
  while (g < end) {
    // the last unit that starts at or before g (it is not empty: those after share its
    // start or a later one)
    int at = 0, step = (count + 31) / 32;
    for (;;) {
      const int i = at + lane * step;
      const bool below = i < count && __ldcg(&p.units[i].start) <= g;
      const int last = 31 - __clz(__ballot_sync(0xffffffffu, below));
      at += last * step;
      if (step == 1) break;
      step = (step + 31) / 32;
    }
    if (cut_segment(load_unit(p.units + at), g, end, blockIdx.x, 0, s)) return;
    g = s.next;
  }
  s.n = 0;
}

template <int D>
struct Layout {
  static constexpr uint32_t kHalf = kBM * 128;         // one 64-column half of a tile
  static constexpr uint32_t kTile = kBM * D * 2;       // a Q, K or V tile
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kK = 2 * kTile;
  static constexpr uint32_t kV = kK + 2 * kTile;
  static constexpr uint32_t kBytes = kV + 2 * kTile;
  static constexpr uint32_t kAlloc = kBytes + 1024;    // alignment slack
  static_assert(kAlloc <= 220 * 1024, "shared memory");
};

struct Shared {
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t s_full[2], p_full[2], o_final[2], q_full, drain, never;
  float2 ml[kBM];           // chain 1's (reference, sum) when it shares chain 0's rows
  float half[2][2][kBM];    // by chain, thread of the row, row: exchange between the two
  uint8_t asks[2][2][kBM];  // likewise
  int stop[8][2];           // by pair of warps and tile parity: a wait ran out
  uint32_t poison[kMaxNodes / 32];  // tree nodes whose V has a NaN or an infinity
  int poisoned;
  uint32_t tmem_base;
  int abort, bad;
  long long end;   // of the block's part
  alignas(16) Seg seg;
  alignas(16) Seg ahead;  // the segment after the one in work
};
constexpr int kBarriers = 17;

__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
  using namespace sm100;
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
#pragma unroll 1
  for (int i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63) == 0 && global_timer_ns() - t0 > limit_ns) return false;
  }
}
// The same, and it gives up when another wait of the block ran out.
__device__ __forceinline__ bool tc_wait(uint64_t &bar, uint32_t parity, uint64_t limit, volatile int *abort) {
  using namespace sm100;
  if (mbar_try_wait(smem_addr(&bar), parity)) return true;
  const uint64_t t0 = global_timer_ns();
#pragma unroll 1
  for (int i = 1;; ++i) {
    if (mbar_try_wait(smem_addr(&bar), parity)) return true;
    if ((i & 63) != 0) continue;
    if (*abort) return false;
    if (global_timer_ns() - t0 > limit) {
      *abort = 1;
      return false;
    }
  }
}
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}
// Waits for this thread's TMEM loads; the registers are operands, so that no
// use of them can be scheduled before it.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
// Register split of the five warpgroups (96 a thread at launch, 480 in all).
template <int kRegs>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kRegs));
}
constexpr int kRegsLaunch = 96, kRegsIssue = 64, kRegsSoftmax = 104;
static_assert(kRegsIssue + 4 * kRegsSoftmax <= 5 * kRegsLaunch, "what the block was launched with");

// Barrier of the two warps that share a chain's quarter of 32 rows; returns whether any
// thread passed true.
__device__ __forceinline__ bool pair_any(int pair, bool x) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, 64, p;\n"
      " selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(1 + pair)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void pair_sync(int pair) {
  asm volatile("barrier.cta.sync %0, 64;\n" ::"r"(1 + pair) : "memory");
}
// Barrier of the four warps of both chains' same quarter.
__device__ __forceinline__ void quarter_sync(int quarter) {
  asm volatile("barrier.cta.sync %0, 128;\n" ::"r"(9 + quarter) : "memory");
}
__device__ __forceinline__ void mbar_inval(uint32_t bar) {
  asm volatile("mbarrier.inval.shared::cta.b64 [%0];\n" ::"r"(bar) : "memory");
}

// Visibility of the 32 key slots from s0 on for tree node i (own ranges; a shared
// range has no tree).  Out of line, once: few tiles need it.
__device__ __noinline__ uint32_t visible32(const Attn &p, const volatile Seg &sg, int i, int s0) {
  const int j0 = s0 - sg.P;
  uint32_t bits = 0xFFFFFFFFu;
  if (j0 > -32) {
    const int at = max(j0, 0), left = sg.nb - at;  // nodes of the tree from `at` on
    uint32_t tail = 0u;
    if (left > 0) {
      if (p.mask) {
        const uint32_t *m = p.mask + ((size_t)sg.table * p.N_max + i) * p.W;
        const int w = at >> 5;
        tail = __funnelshift_r(m[w], w + 1 < p.W ? m[w + 1] : 0u, at & 31);
      } else {
        const int n = i + 1 - at;  // nodes at..i
        tail = n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u;
      }
      if (left < 32) tail &= (1u << left) - 1u;
    }
    bits = j0 < 0 ? (tail << -j0) | ((1u << -j0) - 1u) : tail;
  }
  if (s0 < sg.lo) bits = sg.lo - s0 >= 32 ? 0u : bits & ~((1u << (sg.lo - s0)) - 1u);
  return bits;
}

// What the row may not see becomes -inf.
__device__ __forceinline__ void mask_scores(uint32_t vis, uint32_t (&s)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (!((vis >> i) & 1u)) s[i] = 0xFF800000u;
}

// Goes on to the segment ahead, and lays its barriers; every thread of the block calls
// it, after everything of the segment before has completed.  `fresh`: there was none.
__device__ __forceinline__ bool begin_segment(const Attn &p, Shared &sh, bool fresh, int tid) {
  using namespace sm100;
  tc_fence_before();
  __syncthreads();
  if (tid < 32) {
    if (tid < kBarriers && sh.ahead.n > 0) {
      // the barriers lie one after the other, from k_full to never
      const uint32_t bar = smem_addr(&sh.k_full[0] + tid);
      // p_full: the softmax warps, and what tells that V is there (with two row tiles
      // the first chain's alone)
      const int count = tid == 10 ? 9 : tid == 11 ? (sh.ahead.two ? 8 : 9) : tid == 14 ? 16 : 1;
      if (!fresh) mbar_inval(bar);
      mbar_init(bar, count);
      fence_mbar_init();
    }
    if (tid < kMaxNodes / 32) sh.poison[tid] = 0u;
    if (tid < 5) reinterpret_cast<int4 *>(&sh.seg)[tid] = reinterpret_cast<const int4 *>(&sh.ahead)[tid];
    if (tid == 0) {
      if (!fresh && sh.bad && p.status) atomicOr(p.status, TSD_STATUS_BAD_PAGE);
      sh.bad = 0;
      sh.poisoned = 0;
    }
  }
  __syncthreads();
  tc_fence_after();
  return sh.seg.n > 0;
}

// V tile j in shared memory as the MMAs may read it: rows outside the key range, and
// tree nodes with a NaN or an infinity, become zero.  By a whole warp.
template <int D>
__device__ __forceinline__ void clear_hidden(Shared &sh, const volatile Seg &sg, uint8_t *tile, int j, int lane) {
  const int s0 = sg.page * kPage + j * kBN, lo = sg.lo, hi = sg.hi, P = sg.P;
  if (s0 >= lo && s0 + kBN <= P) return;
  // A lane a row (a row's 128 bytes of a 64-column half lie together, in some order), its
  // chunks from its own place on, so that eight lanes touch all banks.
  for (int r0 = 0; r0 < kBN; r0 += 32) {
    const int r = r0 + lane, s = s0 + r;
    uint8_t *row = tile + r * 128;
    bool clear = s < lo || s >= hi;
    if (__any_sync(0xffffffffu, !clear && s >= P)) {
      uint32_t most = 0u;  // bf16 magnitudes order as integers
#pragma unroll
      for (int h = 0; h < D / 64; ++h)
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint4 v = *reinterpret_cast<const uint4 *>(row + h * Layout<D>::kHalf + ((c + lane) & 7) * 16);
          most = __vmaxu2(__vmaxu2(most, v.x & 0x7FFF7FFFu), v.y & 0x7FFF7FFFu);
          most = __vmaxu2(__vmaxu2(most, v.z & 0x7FFF7FFFu), v.w & 0x7FFF7FFFu);
        }
      const bool odd = !clear && s >= P && ((most & 0xFFFFu) >= 0x7F80u || (most >> 16) >= 0x7F80u);
      if (odd) {
        atomicOr(&sh.poison[(s - P) >> 5], 1u << ((s - P) & 31));
        sh.poisoned = 1;
      }
      clear = clear || odd;
    }
    if (clear) {
#pragma unroll
      for (int h = 0; h < D / 64; ++h)
#pragma unroll
        for (int c = 0; c < 8; ++c)
          *reinterpret_cast<uint4 *>(row + h * Layout<D>::kHalf + ((c + lane) & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  sm100::fence_proxy_async_smem();  // the tensor core reads the tile through the async proxy
  __syncwarp();
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
shared_attn_kernel(const Attn p, const __grid_constant__ CUtensorMap map_k1,
                   const __grid_constant__ CUtensorMap map_k8, const __grid_constant__ CUtensorMap map_v1,
                   const __grid_constant__ CUtensorMap map_v8) {
  using namespace sm100;
  using L = Layout<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared sh;
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *gbase = smem_raw + (base - raw);
  volatile int *abort = &sh.abort;
  const uint64_t lim = p.wait_limit_ns;
  if (tid == 0) {
    tma_prefetch_desc(&map_k1);
    tma_prefetch_desc(&map_k8);
    tma_prefetch_desc(&map_v1);
    tma_prefetch_desc(&map_v8);
    sh.abort = 0;
    sh.bad = 0;
    for (int i = 0; i < 16; ++i) sh.stop[i >> 1][i & 1] = 0;
  }
  if (warp == 1) tmem_alloc(smem_addr(&sh.tmem_base), kTmemCols);
  pdl_wait();
  if (tid < 5) reinterpret_cast<int4 *>(&sh.ahead)[tid] = __ldcg(reinterpret_cast<const int4 *>(p.first_seg + blockIdx.x) + tid);
  if (tid == 32) {
    const long long part = __ldcg(&p.plan->part), total = __ldcg(&p.plan->total);
    sh.end = min(total, (long long)(blockIdx.x + 1) * part);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;

  // The roles; each takes the block's segments in turn, all of them the same ones.
  const volatile Seg &sg = sh.seg;
  if (warp < kSoftmaxWarp) {
    regs_down<kRegsIssue>();
    for (bool fresh = true; begin_segment(p, sh, fresh, tid); fresh = false) {
    const int n = sg.n;
    const bool two = sg.two;
    const int chains = two || n > 1 ? 2 : 1;
    if (warp == 0 || warp == 2) {
      // ---- loaders: warp 0 K, warp 2 V; block ids 32 (four tiles) at a time ----
      const int v = warp >> 1;
      const CUtensorMap *m1 = v ? &map_v1 : &map_k1, *m8 = v ? &map_v8 : &map_k8;
      uint64_t *full = v ? sh.v_full : sh.k_full, *empty = v ? sh.v_empty : sh.k_empty;
      const uint32_t ring = base + (v ? L::kV : L::kK);
      const int pages = sg.pages, h = sg.h;
      const int32_t *trow = p.table + (size_t)sg.table * p.max_blocks + sg.page;
      auto read_ids = [&](int batch) {  // pages past the range: its last one (no row sees them)
        return __ldg(trow + min(batch * 32 + lane, pages - 1));
      };
      int ids = read_ids(0), ahead = read_ids(1), issued = 0;
      for (int j = 0; j < n; ++j) {
        if (j > 0 && (j & 3) == 0) {
          ids = ahead;
          ahead = read_ids((j >> 2) + 1);
        }
        int id = __shfl_sync(0xffffffffu, ids, (j & 3) * kTilePages + (lane & (kTilePages - 1)));
        if (id < 0 || id >= p.num_blocks) {
          sh.bad = 1;
          id = 0;
        }
        const int id0 = __shfl_sync(0xffffffffu, id, 0);
        const bool run = __all_sync(0xffffffffu, id == id0 + (lane & (kTilePages - 1)));
        const int st = j & 1;
        bool ok = true;
        if (j >= 2) ok = __all_sync(0xffffffffu, tc_wait(empty[st], ((j >> 1) - 1) & 1, lim, abort));
        if (!ok) break;
        const uint32_t bar = smem_addr(&full[st]);
        if (lane == 0) mbar_arrive_expect_tx(bar, L::kTile);
        __syncwarp();
        // a box for each 64-column half, or for each page of each
        const int half = lane >> 3, pg = lane & (kTilePages - 1);
        if (half < D / 64) {
          const uint32_t dst = ring + st * L::kTile + half * L::kHalf;
          if (!run) tma_load_4d(dst + pg * (kPage * 128), m1, half * 64, 0, h, id, bar);
          else if (pg == 0) tma_load_4d(dst, m8, half * 64, 0, h, id0, bar);
        }
        issued = j + 1;
      }
      // no copy is in flight when the block goes on
      for (int j = max(0, issued - 2); j < issued; ++j)
        wait_phase(smem_addr(&full[j & 1]), (j >> 1) & 1, kDrainNs);
    } else if (warp == 1) {
      // ---- MMA issue ----
      if (lane == 0) {
        constexpr uint32_t idS = idesc_bf16_f32(kBM, kBN, false, false);
        constexpr uint32_t idPV = idesc_bf16_f32(kBM, D, false, true);
        auto issue_s = [&](int c, int qt, int st) {
          const uint64_t qd = smem_desc_sw128(base + L::kQ + qt * L::kTile, 16, 1024);
          const uint64_t kd = smem_desc_sw128(base + L::kK + st * L::kTile, 16, 1024);
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            umma_bf16(tmem + c * kTmemChain, desc_add(qd, (kk >> 2) * L::kHalf + (kk & 3) * 32),
                      desc_add(kd, (kk >> 2) * L::kHalf + (kk & 3) * 32), idS, kk > 0);
          umma_commit(smem_addr(&sh.s_full[c]));
        };
        auto issue_pv = [&](int c, int st, bool accum, bool final) {
          const uint64_t vd = smem_desc_sw128(base + L::kV + st * L::kTile, L::kHalf, 1024);
          uint64_t v8[8];
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) v8[kk] = desc_add(vd, kk * 16 * 128);
          tc_fence_after();
          // (P of keys 0 .. 63 and 64 .. 127 lies over the first half of their scores each)
          const uint64_t va[4] = {v8[0], v8[1], v8[2], v8[3]}, vb[4] = {v8[4], v8[5], v8[6], v8[7]};
          umma4_ts(tmem + c * kTmemChain + kTmemO, tmem + c * kTmemChain, va, idPV, accum ? 1u : 0u);
          umma4_ts(tmem + c * kTmemChain + kTmemO, tmem + c * kTmemChain + 64, vb, idPV, 1u);
          if (final) umma_commit(smem_addr(&sh.o_final[c]));
        };
        bool ok = !p.test_stall || tc_wait(sh.never, 0, lim, abort);
        ok = ok && tc_wait(sh.q_full, 0, lim, abort);
        ok = ok && tc_wait(sh.k_full[0], 0, lim, abort);
        if (ok) issue_s(0, 0, 0);
        if (chains == 2) {
          if (!two) ok = ok && tc_wait(sh.k_full[1], 0, lim, abort);
          if (ok) issue_s(1, two ? 1 : 0, two ? 0 : 1);
        }
        if (two) {
          // This thread paces the tensor cores: its only wait in the loop is the one
          // for P, to which warp 3 adds once V_j and the next K are there.
          for (int j = 0; ok && j < n; ++j) {
            const int st = j & 1;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              ok = ok && tc_wait(sh.p_full[c], j & 1, lim, abort);
              if (!ok) break;
              issue_pv(c, st, j > 0, j == n - 1);
              if (j + 1 < n) issue_s(c, c, st ^ 1);
            }
          }
        } else {
          for (int j = 0; ok && j < n; ++j) {
            const int c = j & 1;
            ok = tc_wait(sh.p_full[c], (j >> 1) & 1, lim, abort);
            if (!ok) break;
            issue_pv(c, c, j > 1, j + 2 >= n);
            if (j + 2 < n) {
              ok = tc_wait(sh.k_full[c], ((j + 2) >> 1) & 1, lim, abort);
              if (ok) issue_s(c, 0, c);
            }
          }
        }
        if (!ok) *abort = 1;
        umma_commit(smem_addr(&sh.drain));
        wait_phase(smem_addr(&sh.drain), 0, kDrainNs);
      }
      __syncwarp();
    } else if (warp == 3) {
      // ---- phase j of p_full also means that V_j is in shared memory and cleared, and with
      // two row tiles that the K tile of the S behind P_j V_j is there.  (An arrival
      // counts toward the phase that is open: the one before has to be complete.  Each
      // barrier's phases are waited for one after the other.) ----
      bool ok = true;
      for (int j = 0; j < n; ++j) {
        const int c = two ? 0 : j & 1, u = two ? j : j >> 1;  // chain, its tile
        ok = tc_wait(sh.v_full[j & 1], (j >> 1) & 1, lim, abort);
        if (!__all_sync(0xffffffffu, ok)) break;
        clear_hidden<D>(sh, sg, gbase + L::kV + (j & 1) * L::kTile, j, lane);
        if (u > 0) ok = tc_wait(sh.p_full[c], (u - 1) & 1, lim, abort);
        // (P_{j-1} is there, so S_{j-1} was, and K_{j-1}: the phase before this one of its
        // barrier is complete.  K_{j+3} can not be there before this arrival.)
        if (two && j + 1 < n) ok = ok && tc_wait(sh.k_full[(j + 1) & 1], ((j + 1) >> 1) & 1, lim, abort);
        if (!__all_sync(0xffffffffu, ok)) break;
        if (lane == 0) mbar_arrive(smem_addr(&sh.p_full[c]));
      }
      __syncwarp();
      // the segment after this one, while the last tile is worked on
      Seg s;
      next_segment(p, sg.next, sh.end, s);
      if (lane == 0) {
        const int mark = sg.mark;
        if (mark >= 0) p.marks[mark].x = blockIdx.x;
        if (sg.whole) p.marks[mark >= 0 ? mark : -1 - mark].y = blockIdx.x;
        sh.ahead = s;
      }
      __syncwarp();
    }
    __syncwarp();
    }
  } else {
    regs_up<kRegsSoftmax>();
    for (bool fresh = true; begin_segment(p, sh, fresh, tid); fresh = false) {
      // ---- softmax ----
      const int n = sg.n;
      const bool two = sg.two;
      const int chains = two || n > 1 ? 2 : 1;
      const int c = (warp - kSoftmaxWarp) >> 3;           // chain
      const int half = ((warp - kSoftmaxWarp) >> 2) & 1;  // which 64 keys of a tile, and columns of O
      const int rt = two ? c : 0;                         // its row tile
      const int quarter = warp & 3, pair = c * 4 + quarter;
      const int rl = quarter * 32 + lane;                 // row within the tile
      const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
      const uint32_t tS = tmem + c * kTmemChain + lane_off, tO = tS + kTmemO;
      const int row = sg.row0 + rt * kBM + rl;
      // warps without a row only keep the others company
      const bool live = sg.row0 + rt * kBM + quarter * 32 < sg.rows;
      const bool rvalid = row < sg.rows;
      const int node = rvalid ? row / p.g : 0;

      if (two || c == 0) {  // half a Q row -> shared memory (128-byte swizzle); zeros past the rows
        uint8_t *dst = gbase + L::kQ + rt * L::kTile;
        const uint4 *src = nullptr;
        if (rvalid)
          src = reinterpret_cast<const uint4 *>(
                    p.q + ((size_t)__ldcg(p.node_map + sg.node0 + node) * p.Hq + sg.h * p.g + row % p.g) * D) +
                half * (D / 16);
        uint4 x[D / 16];
#pragma unroll
        for (int i = 0; i < D / 16; ++i) x[i] = rvalid ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const int ch = half * (D / 16) + i;  // 16-byte chunk of the row
          *reinterpret_cast<uint4 *>(dst + (ch >> 3) * L::kHalf + sw128_offset(rl, ch & 7)) = x[i];
        }
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&sh.q_full));

      float ref = 0.f, l = 0.f;  // the row's reference, this thread's part of its sum
      bool unset = true, ok = c < chains;
      const float mul = p.scale_log2;
      const unsigned long long mul2 = f2_pack(mul, mul);
      int u = 0;  // this chain's tiles
      // this thread's first key slot in tile j is 128 j + slot0
      const int slot0 = sg.page * kPage + half * 64, lo = sg.lo, tree_from = sg.P - 64;
      auto visible = [&](int s0) { return rvalid ? visible32(p, sg, node, s0) : 0xFFFFFFFFu; };
      for (int j = two ? 0 : c; ok && j < n; j += two ? 1 : 2, ++u) {
        const bool got = __all_sync(0xffffffffu, tc_wait(sh.s_full[c], u & 1, lim, abort));
        if (!got) sh.stop[pair][u & 1] = 1;
        tc_fence_after();
        if ((two ? c == 1 : true) && half == 0 && quarter == 0 && lane == 0) {
          // A commit follows every earlier MMA of its thread, so K_j and the V tile
          // that the P V in front of S_j read are free.
          mbar_arrive(smem_addr(&sh.k_empty[j & 1]));
          const int jv = two ? j - 1 : j - 2;
          if (jv >= 0) mbar_arrive(smem_addr(&sh.v_empty[jv & 1]));
        }
        const int s0 = j * kBN + slot0;
        const bool edge = s0 < lo || s0 > tree_from;
        unsigned long long acc0 = 0ull, acc1 = 0ull;
        uint32_t pk[32], seen = 0u;
        if (live) {
          // both loads before the one wait: a load's latency is some 250 cycles
          uint32_t x[2][32];
          tmem_ld32(tS + half * 64, x[0]);
          tmem_ld32(tS + half * 64 + 32, x[1]);
          tmem_wait_ld(x[0]);
          tmem_wait_ld(x[1]);
          if (edge) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t vis = visible(s0 + k * 32);
              seen |= vis;
              mask_scores(vis, x[k]);
            }
          }
          if (u == 0) {
            // the chain's first tile: the row's maximum over it is the reference
            float m = -INFINITY;
#pragma unroll
            for (int i = 0; i < 32; ++i) m = fmax3(m, __uint_as_float(x[0][i]), __uint_as_float(x[1][i]));
            sh.half[c][half][rl] = m;
            pair_sync(pair);
            m = __fmul_rn(fmaxf(sh.half[c][0][rl], sh.half[c][1][rl]), mul);
            if (m > -INFINITY) {
              ref = m;
              unset = false;
            }
          }
          const unsigned long long ref2 = f2_pack(-ref, -ref);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 t = f2_unpack(f2_fma(
                  f2_pack(__uint_as_float(x[k][2 * i]), __uint_as_float(x[k][2 * i + 1])), mul2, ref2));
              const float e0 = ex2_approx(t.x), e1 = ex2_approx(t.y);
              pk[k * 16 + i] = pack_bf16x2(e0, e1);
              if (i & 1) acc1 = f2_add(acc1, f2_pack(e0, e1));
              else acc0 = f2_add(acc0, f2_pack(e0, e1));
            }
          }
        }
        const float2 acc = f2_unpack(f2_add(acc0, acc1));
        float sum = acc.x + acc.y;
        // Rows that need more than that: no reference yet, or P out of range.
        const bool mine = live && ((unset && (!edge || seen != 0u)) || !(sum <= kMaxSum));
        if (__builtin_expect(pair_any(pair, mine || !got), 0)) {
          if (sh.stop[pair][u & 1]) {  // the same for both warps
            ok = false;
            break;
          }
          float m = -INFINITY;
          if (live) {
#pragma unroll 1
            for (int k = 0; k < 2; ++k) {
              uint32_t s[32];
              tmem_ld32(tS + half * 64 + k * 32, s);
              tmem_wait_ld(s);
              if (edge) mask_scores(visible(s0 + k * 32), s);
#pragma unroll
              for (int i = 0; i < 32; ++i) m = fmaxf(m, __fmul_rn(__uint_as_float(s[i]), mul));
            }
            // what the row's two threads know: its maximum, and whether either asked
            sh.half[c][half][rl] = m;
            sh.asks[c][half][rl] = mine;
          }
          pair_sync(pair);
          if (live) {
            const bool row_asks = mine || sh.asks[c][half ^ 1][rl];
            m = fmaxf(m, sh.half[c][half ^ 1][rl]);
            float f = 1.f;
            if (row_asks && m > -INFINITY && (unset || m > ref)) {
              // (nothing was added yet to a row without a reference)
              if (!unset) f = ex2_approx(ref - m);
              ref = m;
              unset = false;
              l *= f;
            }
            if (__any_sync(0xffffffffu, row_asks)) {
              float again = 0.f;
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                uint32_t s[32];
                tmem_ld32(tS + half * 64 + k * 32, s);
                tmem_wait_ld(s);
                if (edge) mask_scores(visible(s0 + k * 32), s);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  const float e0 = ex2_approx(__fsub_rn(__fmul_rn(__uint_as_float(s[2 * i]), mul), ref));
                  const float e1 = ex2_approx(__fsub_rn(__fmul_rn(__uint_as_float(s[2 * i + 1]), mul), ref));
                  again += e0 + e1;
                  pk[k * 16 + i] = row_asks ? pack_bf16x2(e0, e1) : pk[k * 16 + i];
                }
              }
              if (row_asks) sum = again;
            }
            if (u > 0 && __any_sync(0xffffffffu, f != 1.f)) {  // this thread's half of O
#pragma unroll 1
              for (int q = 0; q < D / 64; ++q) {
                uint32_t o[32];
                const uint32_t at = tO + half * (D / 2) + q * 32;
                tmem_ld32(at, o);
                tmem_wait_ld(o);
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                tmem_st32(at, o);
              }
            }
          }
        }
        if (live) {
          l += sum;
          tmem_st32(tS + half * 64, pk);  // (over its own scores)
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sh.p_full[c]));
      }

      // ---- epilogue: O of this chain is complete ----
      const bool joined = !two && chains == 2;
      if (ok) ok = __all_sync(0xffffffffu, tc_wait(sh.o_final[c], 0, lim, abort));
      // (the rows go over the K and V tiles, which the other chain's last MMAs may
      // still read)
      if (ok && chains == 2) ok = __all_sync(0xffffffffu, tc_wait(sh.o_final[c ^ 1], 0, lim, abort));
      tc_fence_after();
      pair_sync(pair);  // (what was exchanged before has been read)
      sh.half[c][half][rl] = l;
      pair_sync(pair);
      l += sh.half[c][half ^ 1][rl];
      float M = unset ? -INFINITY : ref;
      if (unset && l != l) M = 0.f;  // only NaN scores so far
      // K and V tiles are done with: chain 1's O when it shares chain 0's rows
      // (column-major, so that lanes do not collide), then the finished rows
      float *stage = reinterpret_cast<float *>(gbase + L::kK);
      const uint32_t rows_at = (two && c == 0 ? L::kK : L::kV);
      uint8_t *rows_out = gbase + rows_at;
      const int q0 = half * (D / 64);  // this thread's 32-column parts of O
      ok = ok && live;
      if (joined && c == 1) {
#pragma unroll 1
        for (int q = q0; ok && q < q0 + D / 64; ++q) {
          uint32_t o[32];
          tmem_ld32(tO + q * 32, o);
          tmem_wait_ld(o);
#pragma unroll
          for (int i = 0; i < 32; ++i) stage[(q * 32 + i) * kBM + rl] = __uint_as_float(o[i]);
        }
        if (half == 0) sh.ml[rl] = make_float2(M, l);
      }
      if (joined) quarter_sync(quarter);
      if (c < (two ? 2 : 1)) {
        float f0 = 1.f, f1 = 0.f;
        if (joined) {
          const float2 other = sh.ml[rl];
          const float top = fmaxf(M, other.x);
          f0 = M == -INFINITY ? 0.f : ex2_approx(M - top);
          f1 = other.x == -INFINITY ? 0.f : ex2_approx(other.x - top);
          l = f0 * l + f1 * other.y;
          M = top;
        }
        if (sh.poisoned && rvalid) {  // the row sees a node whose V has a NaN or an infinity
          bool sees = false;
          for (int w = 0; w < kMaxNodes / 32; ++w)
            sees = sees || (sh.poison[w] && (sh.poison[w] & visible32(p, sg, node, sg.P + 32 * w)));
          if (sees) {
            l = __uint_as_float(0x7FC00000u);
            M = M == -INFINITY ? 0.f : M;
          }
        }
#pragma unroll 1
        for (int q = q0; ok && q < q0 + D / 64; ++q) {
          uint32_t o[32];
          tmem_ld32(tO + q * 32, o);
          tmem_wait_ld(o);
          if (joined) {
            // (chain 1's O holds something for every row that it has a reference for)
            const float *theirs = stage + q * 32 * kBM + rl;
            if (__all_sync(0xffffffffu, f1 != 0.f)) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                o[i] = __float_as_uint(fmaf(f1, theirs[i * kBM], __uint_as_float(o[i]) * f0));
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float y = theirs[i * kBM];
                o[i] = __float_as_uint(fmaf(f1, f1 != 0.f ? y : 0.f, __uint_as_float(o[i]) * f0));
              }
            }
          }
          const float *v = reinterpret_cast<const float *>(o);
          // whole rows in shared memory, their 16-byte chunks swizzled by row
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<float4 *>(rows_out + rl * (D * 4) + (((q * 8 + i) ^ (rl & 7)) << 4)) =
                make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        }
        if (half == 0 && rvalid) p.part_ml[sg.part + rt * kBM + rl] = make_float2(M, sh.bad ? -1.f : l);
        fence_proxy_async_smem();
        pair_sync(pair);
        const int w = quarter * 2 + half;
        // 16 partial rows a warp, in one piece and as they lie
        const int rows = min(kBM / 8, sg.rows - sg.row0 - rt * kBM - w * (kBM / 8));
        if (lane == 0 && !*abort && rows > 0) {
          bulk_store(p.part_o + (sg.part + rt * kBM + w * (kBM / 8)) * D, base + rows_at + w * (kBM / 8) * (D * 4),
                     rows * D * 4);
          bulk_wait_read();
        }
      }
      fence_proxy_async_smem();  // (the next segment's tiles come over what was staged)
      __syncwarp();
    }
    if (lane == 0) bulk_wait();  // (the partial rows are written)
  }
  // (the last begin_segment ended with a barrier)
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
  if (tid == 0 && p.status && sh.abort) atomicOr(p.status, TSD_STATUS_TIMEOUT);
}

// ---------------------------------------------------------------------------
// join
// ---------------------------------------------------------------------------

// Where a row's partial rows of one unit are.
struct Pieces {
  long long row;  // partial row of a piece in block 0
  int k0, n;      // first block, pieces
};

// Blocks (node, some heads): its warps take the heads in turn.  A row's pieces of the shared and of
// the own range are weighed by their sums and added up.
template <int D>
__global__ void __launch_bounds__(256) shared_join_kernel(const Attn p) {
  using namespace sm100;
  constexpr int kPer = D / 32;  // columns of a lane
  constexpr int kAhead = 4;     // pieces read before the first is used
  __shared__ alignas(16) Unit unit[2];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x / p.N_max, i = blockIdx.x % p.N_max;
  if (warp == 0) {
    if (lane < 4) reinterpret_cast<int4 *>(&unit[0])[lane] = __ldcg(reinterpret_cast<const int4 *>(p.units + p.G + b) + lane);
    __syncwarp();
    const int group = unit[0].group;
    if (group >= 0 && lane < 4)
      reinterpret_cast<int4 *>(&unit[1])[lane] = __ldcg(reinterpret_cast<const int4 *>(p.units + group) + lane);
  }
  __syncthreads();
  const Unit &own = unit[0], &shd = unit[1];
  const bool on = i < own.nb, split = own.group >= 0;
  const int heads = p.join_heads;  // of this block
  for (int hq = blockIdx.y * heads + warp; hq < min(p.Hq, (int)(blockIdx.y + 1) * heads); hq += 8) {
    const int64_t x = (int64_t)blockIdx.x * p.Hq + hq;
    const int h = hq / p.g;
    Pieces set[2] = {};
    int rl[2] = {};  // place in the row tile, modulo 8
    if (on) {
      const int r = i * p.g + hq % p.g, rs = split ? (own.node0 - shd.node0) * p.g + r : 0;
      const int2 m0 = __ldcg(p.marks + own.block_base + h * own.rbs + r / kRows);
      set[0] = Pieces{own.row_base + (long long)h * own.rows + r, m0.x, m0.y - m0.x + 1};
      rl[0] = r & 7;
      if (split) {
        const int2 m1 = __ldcg(p.marks + shd.block_base + h * shd.rbs + rs / kRows);
        set[1] = Pieces{shd.row_base + (long long)h * shd.rows + rs, m1.x, m1.y - m1.x + 1};
        rl[1] = rs & 7;
      }
    }
    const int n = set[0].n + set[1].n;
    auto part_row = [&](int s) -> size_t {
      const Pieces &y = s < set[0].n ? set[0] : set[1];
      return (size_t)(y.row + (long long)(y.k0 + s - (s < set[0].n ? 0 : set[0].n)) * kRows);
    };
    // lane l holds the (reference, sum) of pieces l, l + 32, ...: at most 128
    float2 ml[4];
    float a[kPer] = {}, M = -INFINITY;
    float v[kAhead][kPer];
    auto load = [&](int s0) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int s = s0 + j;
        if (s >= n) break;
        // (a partial row's 16-byte chunks are swizzled by its place in the row tile, which
        // spreads the stores over the banks)
        const int phase = s < set[0].n ? rl[0] : rl[1];
        const float *src = p.part_o + part_row(s) * D + ((lane * kPer / 4) ^ phase) * 4 + lane * kPer % 4;
        if constexpr (kPer == 4) {
          const float4 y = __ldcg(reinterpret_cast<const float4 *>(src));
          v[j][0] = y.x;
          v[j][1] = y.y;
          v[j][2] = y.z;
          v[j][3] = y.w;
        } else {
          const float2 y = __ldcg(reinterpret_cast<const float2 *>(src));
          v[j][0] = y.x;
          v[j][1] = y.y;
        }
      }
    };
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      ml[e] = make_float2(-INFINITY, 0.f);
      if (lane + 32 * e < n) ml[e] = __ldcg(&p.part_ml[part_row(lane + 32 * e)]);
    }
    load(0);  // (before the weights are known)
    bool bad = false;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      bad = bad || ml[e].y == -1.f;
      M = fmaxf(M, ml[e].x);
    }
    bad = __any_sync(0xffffffffu, bad);
#pragma unroll
    for (int off = 16; off; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    float f[4], sum = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[e] = ml[e].x == -INFINITY ? 0.f : ex2_approx(ml[e].x - M);
      sum += f[e] * ml[e].y;
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    const bool empty = n == 0 || bad || sum == 0.f;
    for (int s0 = 0; s0 < n;) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int s = s0 + j;
        if (s >= n) break;
        const float mine = s < 64 ? (s < 32 ? f[0] : f[1]) : (s < 96 ? f[2] : f[3]);
        const float fs = __shfl_sync(0xffffffffu, mine, s & 31);
        // (a piece in which the row saw nothing has no row)
#pragma unroll
        for (int c = 0; c < kPer; ++c) a[c] += fs != 0.f ? fs * v[j][c] : 0.f;
      }
      s0 += kAhead;
      if (s0 < n) load(s0);
    }
    const float inv = empty ? 0.f : 1.f / sum;
    uint32_t w[kPer / 2];
#pragma unroll
    for (int c = 0; c < kPer / 2; ++c) w[c] = empty ? 0u : pack_bf16x2(a[2 * c] * inv, a[2 * c + 1] * inv);
    uint16_t *dst = p.out + x * D + lane * kPer;
    if constexpr (kPer == 4)
      *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
    else
      *reinterpret_cast<uint32_t *>(dst) = w[0];
    if (lane == 0 && p.lse) p.lse[x] = empty ? -INFINITY : (M + log2f(sum)) * kLn2;
  }
}

struct Sizes {
  size_t units, segs, marks, nodes, ml, o, bytes;
  size_t rows;  // partial rows
};

Sizes sizes(int B, int N_max, int Hq, int Hkv, int D, int G) {
  Sizes z;
  z.rows = 2 * (size_t)B * N_max * Hq + (size_t)sm_count() * kRows;
  z.units = align_up(sizeof(Plan), 256);
  z.segs = z.units + align_up((size_t)(G + B) * sizeof(Unit), 256);
  z.marks = z.segs + align_up((size_t)sm_count() * sizeof(Seg), 256);
  // row blocks: full ones of all rows, shared and own, and a last one of each unit
  const size_t row_blocks = (size_t)Hkv * (2 * ((size_t)B * N_max * (Hq / Hkv) / kRows) + G + B);
  z.nodes = z.marks + align_up(row_blocks * sizeof(int2), 256);
  z.ml = z.nodes + align_up((size_t)B * N_max * sizeof(int32_t), 256);
  z.o = z.ml + align_up(z.rows * sizeof(float2), 256);
  z.bytes = z.o + z.rows * D * sizeof(float);
  return z;
}

int check(int B, int N_max, int Hq, int Hkv, int D, int G) {
  if (B < 0 || N_max < 1 || Hq < 1 || Hkv < 1 || G < 0) return TSD_ERR_ARG;
  if (D != 64 && D != 128) return TSD_ERR_LIMIT;
  if (N_max > kMaxNodes || Hq % Hkv != 0 || Hq / Hkv > 16 || B > kMaxBatch ||
      (int64_t)(B > 0 ? B : 1) * Hkv > 65535)
    return TSD_ERR_LIMIT;
  if (B > 0 && (G < 1 || G > B)) return TSD_ERR_ARG;
  return TSD_OK;
}

// The register split draws on what the block was launched with: a build that gives a
// thread fewer registers must not run (it would wait forever).
template <int D>
bool ready() {
  static const bool enough = [] {
    cudaFuncAttributes a;
    return cudaFuncGetAttributes(&a, shared_attn_kernel<D>) == cudaSuccess && a.numRegs >= kRegsLaunch;
  }();
  return enough && set_smem((const void *)shared_attn_kernel<D>, Layout<D>::kAlloc);
}

template <int D>
int launch_all(const Attn &p, cudaStream_t s) {
  CUtensorMap k1, k8, v1, v8;
  if (!make_cache_map(&k1, p.k, p.num_blocks, p.Hkv, D, 1) ||
      !make_cache_map(&k8, p.k, p.num_blocks, p.Hkv, D, kTilePages) ||
      !make_cache_map(&v1, p.v, p.num_blocks, p.Hkv, D, 1) ||
      !make_cache_map(&v8, p.v, p.num_blocks, p.Hkv, D, kTilePages))
    return TSD_ERR_CUDA;
  if (!ready<D>()) return TSD_ERR_CUDA;
  const int threads = p.B <= kSmallPlan ? kSmallPlan : kPlanThreads;
  if (launch(shared_plan_kernel, dim3(1), dim3(threads), 0, s, p) != cudaSuccess) return TSD_ERR_CUDA;
  if (launch(shared_attn_kernel<D>, dim3(p.blocks), dim3(kThreads), Layout<D>::kAlloc, s, p, k1, k8, v1, v8) != cudaSuccess)
    return TSD_ERR_CUDA;
  const dim3 grid((unsigned)(p.B * p.N_max), (unsigned)((p.Hq + p.join_heads - 1) / p.join_heads));
  if (launch(shared_join_kernel<D>, grid, dim3(256), 0, s, p) != cudaSuccess)
    return TSD_ERR_CUDA;
  return TSD_OK;
}

}  // namespace
}  // namespace tsd

TSD_API size_t tsd_tree_attn_shared_workspace_bytes(int B, int N_max, int Hq, int Hkv, int D, int G) {
  using namespace tsd;
  if (B == 0 || check(B, N_max, Hq, Hkv, D, G) != TSD_OK) return 0;
  return sizes(B, N_max, Hq, Hkv, D, G).bytes;
}

TSD_API int tsd_tree_attn_fwd_shared(const uint16_t *q, const uint16_t *k_cache, const uint16_t *v_cache,
                                     const int32_t *block_table, int max_blocks, int num_blocks,
                                     const int32_t *prefix_len, const int32_t *n_nodes,
                                     const uint32_t *mask, const int32_t *err,
                                     const int32_t *group_first, const int32_t *shared_len, int G, int B,
                                     int N_max, int Hq, int Hkv, int D, float scale, uint16_t *out,
                                     float *lse, void *workspace, size_t ws_bytes, int32_t *status,
                                     tsd_stream_t stream) {
  using namespace tsd;
  const int rc = check(B, N_max, Hq, Hkv, D, G);
  if (rc != TSD_OK) return rc;
  if (max_blocks < 1 || num_blocks < 1 || !(scale > 0.f) || !std::isfinite(scale)) return TSD_ERR_ARG;
  if ((int64_t)num_blocks * Hkv * kPage > 0x7FFFFFFFll || (int64_t)max_blocks * kPage > 0x7FFFFFFFll)
    return TSD_ERR_LIMIT;
  if (B == 0) return TSD_OK;
  if (!q || !k_cache || !v_cache || !block_table || !prefix_len || !group_first || !shared_len || !out)
    return TSD_ERR_ARG;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16)) return TSD_ERR_ARG;
  const Sizes z = sizes(B, N_max, Hq, Hkv, D, G);
  if (!workspace || ws_bytes < z.bytes) return TSD_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return TSD_ERR_ARG;
  char *ws = static_cast<char *>(workspace);
  Attn p = {};
  p.q = q;
  p.k = k_cache;
  p.v = v_cache;
  p.table = block_table;
  p.max_blocks = max_blocks;
  p.num_blocks = num_blocks;
  p.prefix_len = prefix_len;
  p.n_nodes = n_nodes;
  p.mask = mask;
  p.err = err;
  p.first = group_first;
  p.shared = shared_len;
  p.G = G;
  p.B = B;
  p.N_max = N_max;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.g = Hq / Hkv;
  p.W = (N_max + 31) / 32;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.blocks = sm_count();
  // a warp takes more than one head where there are rows enough to fill the GPU without
  const int64_t turns = (int64_t)B * N_max * Hq / (64ll * p.blocks);
  p.join_heads = 8 * (int)(turns < 1 ? 1 : turns > 8 ? 8 : turns);
  p.plan = reinterpret_cast<Plan *>(ws);
  p.units = reinterpret_cast<Unit *>(ws + z.units);
  p.first_seg = reinterpret_cast<Seg *>(ws + z.segs);
  p.marks = reinterpret_cast<int2 *>(ws + z.marks);
  p.node_map = reinterpret_cast<int32_t *>(ws + z.nodes);
  p.part_ml = reinterpret_cast<float2 *>(ws + z.ml);
  p.part_o = reinterpret_cast<float *>(ws + z.o);
  p.out = out;
  p.lse = lse;
  p.status = status;
  p.wait_limit_ns = (uint64_t)option(TSD_OPT_WAIT_LIMIT_NS);
  p.test_stall = (int)option(TSD_OPT_TEST_STALL);
  return D == 128 ? launch_all<128>(p, as_cuda(stream)) : launch_all<64>(p, as_cuda(stream));
}
