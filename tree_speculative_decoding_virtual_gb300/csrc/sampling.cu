// Sampling with temperature, top-k, top-p and min-p from given random numbers, and
// the distribution that these filters leave ("Speculative Decoding Hierárquico:
// Medusa, EAGLE-2 e Multi-Token Prediction", modified rejection sampling: what is
// verified is the distribution that the tokens were drawn from).
//
// For a row x of V logits, m = max x:
//   d_i = (x_i - m) / T,  w_i = e^{d_i}
// ranked by (x descending, id ascending), and of the ranks r = 0, 1, ... are kept
//   top-k   r < k
//   top-p   sum of w over the ranks before r (of those left) < p times their sum
//   min-p   w_r >= min_p (the largest w is 1)
// which is always a prefix of the ranking: everything from one (logit, id) on.  A draw
// takes the first id, in id order, whose cumulative weight exceeds u times the sum
// of what is kept.
//
// A border that a sum decides moves with the sum's rounding, so weights are fp32 and
// their sums exact: fixed point of 2^-43, which no order of additions changes.
//
// One cluster of up to 8 CTAs a row; the row is read once and stays in shared memory,
// each warp with a run of consecutive ids.  A filter's border is found by
//   histogram  1024 bins of (m - x) / T, 32 a unit: counts for top-k, and for top-p
//              weights relative to the bin's (13 bits a weight: good to 1e-4) besides the
//              exact sum of all; the first CTA adds up the cluster's and finds the bin, or
//              the few bins, that must hold the border
//   list       what lies in them (a handful to some hundred) goes to the first CTA, with
//              the exact weight above them, and is ranked there
// When what lies in those bins and above fits the list (ordinary settings of top-k and
// top-p), the first CTA has all that can be kept, and finishes alone: both filters, min-p
// and the draws.  Bins that hold more than the list are cut into 1024 again; where that does
// not part them either (hundreds of equal logits), the border is found bit by bit.
#include <cuda_bf16.h>

#include <cmath>
#include <type_traits>

#include "sm100_ptx.cuh"
#include "tsd_common.cuh"

namespace tsd {
namespace {

constexpr int kSpThreads = 256;
constexpr int kSpWarps = kSpThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxVocab = 262144;
constexpr int kMaxDraws = 64;
constexpr int kBins = 1024;
constexpr int kThreadBins = kBins / kSpThreads;
constexpr int kList = 512;
constexpr float kCountScale = 16.f, kWideScale = 0.25f, kWeightScale = 32.f;  // bins a unit at first
constexpr int kLevels = 3;          // times bins are cut again at most
constexpr float kShare = 8192.f;    // a bin's own weight (262144 of them fit 32 bits)
constexpr float kShareError = 1e-4f;  // (a logit's share is off by 2^-14, sums and exponentials by less)
enum { kSample, kLogits, kProbs };

struct SpArgs {
  const void *logits;
  const int32_t *rows;
  const float *u;
  const float *temperature, *top_p, *min_p;
  const int32_t *top_k;
  int64_t num_rows;
  int R, V, draws;
  int per_param;  // consecutive rows that share an entry of the parameters
  int per_warp;   // logits of a warp's run
  int32_t *tokens;
  float *logprob, *out;
  int32_t *status;
};

// What is kept: everything down to logit x, of those equal to it the ids up to id.
struct Border {
  float x = -INFINITY;
  int id = -1;
  __device__ __forceinline__ bool has(float y, int i) const { return y > x || (y == x && i <= id); }
};

// Bins of a logit's distance from the maximum, from `from` on, `scale` a unit.  Top-k's
// distance is m - x (its border has nothing to do with T), top-p's (m - x) / T.
struct Bins {
  float from, scale;
};

enum { kNone, kWiden, kZoom, kCollect, kGather, kBitwise };  // what follows a histogram

struct Verdict {
  int what, lo, hi;  // the border is in bins lo..hi
};

struct SpShared {
  union {
    alignas(16) uint32_t hist[kBins];
    struct {
      unsigned long long list[kList];    // (ordered logit, ~id)
      unsigned long long weight[kList];  // fixed point
    };
  };
  float wmax[kSpWarps];
  int wcount[kSpWarps];
  long long wsum[kSpWarps];
  float scan[kSpWarps];
  float need, room, skipped;
  long long at[kMaxDraws];
  float max;
  // added up in the first CTA
  unsigned long long sum_all, sum_near, sum_above;
  int count_all, count_above, listed;
  // exchanged by the bitwise search and the draws (two places, by turn)
  int count[2];
  long long sum[2];
  // the first CTA's findings
  Verdict verdict;
  float border_x;
  int border_id;
  long long total;
  float in_border, up_to;  // how many logits the bins hold
  int mine;
  bool failed;
};

__device__ __forceinline__ uint32_t ordered(float x) {  // no NaN; both zeros alike
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint32_t peer(const void *p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(sm100::smem_addr(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ uint32_t ld_peer32(const void *p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];\n" : "=r"(v) : "r"(peer(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ unsigned long long ld_peer64(const void *p, uint32_t rank) {
  unsigned long long v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];\n" : "=l"(v) : "r"(peer(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ uint4 ld_peer128(const void *p, uint32_t rank) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(peer(p, rank))
               : "memory");
  return v;
}
// Into the first CTA's shared memory.
__device__ __forceinline__ void add_first32(void *p, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;\n" ::"r"(peer(p, 0)), "r"(v) : "memory");
}
__device__ __forceinline__ void add_first64(void *p, unsigned long long v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u64 [%0], %1;\n" ::"r"(peer(p, 0)), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t take_first32(void *p, uint32_t v) {
  uint32_t r;
  asm volatile("atom.relaxed.cluster.shared::cluster.add.u32 %0, [%1], %2;\n" : "=r"(r) : "r"(peer(p, 0)), "r"(v) : "memory");
  return r;
}
__device__ __forceinline__ void st_first64(void *p, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;\n" ::"r"(peer(p, 0)), "l"(v) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  sm100::cluster_arrive();
  sm100::cluster_wait();
}

// A sum of weights in [0, 1], exact to 2^-43 a weight: the weight's multiple of 2^-20
// and its rest's multiple of 2^-43, read off the last places of sums with 8 and
// with 1.5 * 2^-20.
struct Fixed {
  uint32_t hi = 0u;
  int lo = 0;
  __device__ __forceinline__ void add(float w) {
    const float a = __fadd_rn(w, 8.f);
    const float b = __fadd_rn(__fsub_rn(w, __fsub_rn(a, 8.f)), 0x1.8p-20f);
    hi += __float_as_uint(a) - 0x41000000u;
    lo += (int)(__float_as_uint(b) - 0x35C00000u);
  }
  // two at a time, on packed pairs
  __device__ __forceinline__ void add2(float w0, float w1) {
    using namespace sm100;
    const unsigned long long w = f2_pack(w0, w1), a = f2_add(w, f2_pack(8.f, 8.f));
    const unsigned long long rest = f2_fma(f2_add(a, f2_pack(-8.f, -8.f)), f2_pack(-1.f, -1.f), w);
    const float2 x = f2_unpack(a), y = f2_unpack(f2_add(rest, f2_pack(0x1.8p-20f, 0x1.8p-20f)));
    hi += __float_as_uint(x.x) + __float_as_uint(x.y) - 0x82000000u;
    lo += (int)(__float_as_uint(y.x) + __float_as_uint(y.y) - 0x6B800000u);
  }
  __device__ __forceinline__ long long value() const { return ((long long)hi << 23) + lo; }
};
constexpr float kUnit = 0x1p-43f;

__device__ __forceinline__ long long fixed(float w) {
  Fixed f;
  f.add(w);
  return f.value();
}
__device__ __forceinline__ long long warp_sum(long long x) {
#pragma unroll
  for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

// The logits of one lane's vector: 4 fp32 or 8 bf16 of a warp's run.
template <bool kBf16>
struct SpVec {
  static constexpr int kN = kBf16 ? 8 : 4;
  float x[kN];
  __device__ __forceinline__ void read(const uint4 *at) {
    const uint4 v = *at;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (kBf16) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      } else {
        x[i] = __uint_as_float(w[i]);
      }
    }
  }
};

// A warp's run of the row in shared memory, and what its logits mean.
template <bool kBf16>
struct Run {
  static constexpr int kN = SpVec<kBf16>::kN;
  const uint4 *at;  // this lane's vectors, 32 apart
  int steps, id;    // id of this lane's first logit; 32 * kN further a step
  float m, inv_t;
  uint32_t rank, ranks;

  __device__ __forceinline__ float scaled(float x) const { return __fmul_rn(__fsub_rn(x, m), inv_t); }
  // Calls f(logits, id of the first) for every vector of this lane that holds a logit of
  // `from` or more.
  template <class F>
  __device__ __forceinline__ void each_vec(float from, F f) const {
#pragma unroll 2
    for (int s = 0; s < steps; ++s) {
      SpVec<kBf16> v;
      v.read(at + s * 32);
      float most = fmaxf(v.x[0], v.x[1]);
#pragma unroll
      for (int i = 2; i < kN; i += 2) most = sm100::fmax3(most, v.x[i], v.x[i + 1]);
      if (most >= from) f(v.x, id + s * (32 * kN));
    }
  }
  // Calls f(logit, id) for every logit of `from` or more (and some others).
  template <class F>
  __device__ __forceinline__ void each(float from, F f) const {
    each_vec(from, [&](const float (&x)[kN], int first) {
#pragma unroll
      for (int i = 0; i < kN; ++i) f(x[i], first + i);
    });
  }
};

// The bin of a distance: -1 above the bins, kBins below them.  The same rounding for
// every logit, so that a larger logit is never in a later bin; y - kRound is the bin.
constexpr float kRound = 12582912.f;  // 1.5 * 2^23
__device__ __forceinline__ int bin_of(float distance, const Bins &b, float &rest) {
  const float at = fminf(fmaxf(__fmul_rn(__fsub_rn(distance, b.from), b.scale), -1.f), (float)kBins);
  const float y = __fadd_rn(at, kRound);
  rest = __fsub_rn(at, __fsub_rn(y, kRound));
  return (int)(__float_as_uint(y) - 0x4B400000u);
}
// A logit that is no larger than any of bin `last` (two bins and some rounding lower).
__device__ __forceinline__ float logit_of(const Bins &b, int last, float m, float inv_unit) {
  const float far = b.from + (float)(last + 2) / b.scale;
  return m - far * inv_unit * 1.00001f - fabsf(m) * 0x1p-21f;
}

// Count and weight over the block, in every thread.
__device__ __forceinline__ long long block_total(SpShared &sh, int &count, long long mine) {
  const int warp = threadIdx.x >> 5;
  const long long sum = warp_sum(mine);
  count = __reduce_add_sync(0xffffffffu, count);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) {
    sh.wsum[warp] = sum;
    sh.wcount[warp] = count;
  }
  __syncthreads();
  long long t = 0;
  count = 0;
#pragma unroll
  for (int w = 0; w < kSpWarps; ++w) {
    t += sh.wsum[w];
    count += sh.wcount[w];
  }
  return t;
}

// The same over the cluster; `turn` is which of the two places is used.
__device__ __forceinline__ long long cluster_total(SpShared &sh, int &turn, uint32_t ranks, int &count, long long mine) {
  const long long t = block_total(sh, count, mine);
  if (threadIdx.x == 0) {
    sh.sum[turn] = t;
    sh.count[turn] = count;
  }
  cluster_sync();
  long long all = 0;
  count = 0;
  for (uint32_t p = 0; p < ranks; ++p) {
    all += (long long)ld_peer64(&sh.sum[turn], p);
    count += (int)ld_peer32(&sh.count[turn], p);
  }
  turn ^= 1;
  return all;
}

// The border of what is kept, bit by bit: the highest one above which there are `k`
// logits, or (k = 0) a share p of the weight above `kept`.  50 passes: for hundreds of equal
// logits at the border.
template <bool kBf16>
__device__ __noinline__ Border bitwise_border(SpShared &sh, const Run<kBf16> &run, int &turn, const Border kept, int k, float p) {
  // (ordered logit, kMaxVocab - 1 - id) and above
  auto above = [&](uint32_t hi, uint32_t lo, int &count) -> long long {
    Fixed f;
    int c = 0;
    run.each(-INFINITY, [&](float x, int id) {
      const uint32_t o = ordered(x);
      const bool in = kept.has(x, id) && (o > hi || (o == hi && (uint32_t)(kMaxVocab - 1 - id) >= lo));
      c += in;
      if (in && k == 0) f.add(expf(run.scaled(x)));
    });
    count = c;
    return cluster_total(sh, turn, run.ranks, count, f.value());
  };
  int n;
  long long least = 0;
  if (k == 0) {
    const double want = (double)p * (double)above(0u, 0u, n);
    least = want > 1.0 ? (long long)ceil(want) : 1;
  }
  uint32_t hi = 0u, lo = 0u;
#pragma unroll 1
  for (int bit = 49; bit >= 0; --bit) {
    const uint32_t h = hi | (bit >= 18 ? 1u << (bit - 18) : 0u), l = lo | (bit < 18 ? 1u << bit : 0u);
    const long long sum = above(h, l, n);
    if (k ? n >= k : sum >= least) {
      hi = h;
      lo = l;
    }
  }
  Border b;
  b.x = unordered(hi);
  b.id = kMaxVocab - 1 - (int)lo;
  return b;
}

// First CTA: the bins that hold the border, from the cluster's histograms.
// Counts, and the first level of top-p from its end: `need` more from the bins' top
// on, or at most `room` left behind the border (the exact sum less the share wanted: what
// is left is small, and known better by itself than as a difference); `skipped`: the weight
// that was not binned.
__device__ __forceinline__ void find_bins(SpShared &sh, const Bins bins, bool by_count, float need, float room,
                                          bool from_end, float skipped, uint32_t ranks, int level, int V) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  static_assert(kThreadBins == 4, "");
  uint32_t h[4] = {0u, 0u, 0u, 0u};
  for (uint32_t p = 0; p < ranks; ++p) {
    const uint4 x = ld_peer128(&sh.hist[tid * 4], p);
    h[0] += x.x;
    h[1] += x.y;
    h[2] += x.z;
    h[3] += x.w;
  }
  float v[4], mine = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float at = bins.from + (float)(tid * 4 + i) / bins.scale;
    v[i] = by_count ? (float)h[i] : (float)h[i] * (expf(-at) * (1.f / kShare));
    mine += v[i];
  }
  float upto = mine;  // from the end when that is what counts
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const float y = from_end ? __shfl_down_sync(0xffffffffu, upto, off) : __shfl_up_sync(0xffffffffu, upto, off);
    if (from_end ? lane + off < 32 : lane >= off) upto += y;
  }
  if (lane == (from_end ? 0 : 31)) sh.scan[warp] = upto;
  if (tid == 0) {
    sh.verdict.lo = sh.verdict.hi = kBins;
    sh.in_border = sh.up_to = 0.f;
  }
  __syncthreads();
  float sum = upto - mine;
  if (from_end) room -= skipped;
#pragma unroll
  for (int w = 0; w < kSpWarps; ++w)
    if (from_end ? w > warp : w < warp) sum += sh.scan[w];
  const float e = by_count ? 0.f : kShareError, beyond = (float)V * 1.3e-14f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = from_end ? 3 - i : i;
    if (!from_end) sum += v[j];
    // from the end, `sum` is what bins after j hold
    const bool may = from_end ? sum * (1.f - e) <= room : sum * (1.f + e) >= need;
    const bool must = from_end ? sum * (1.f + e) + beyond <= room : sum * (1.f - e) >= need;
    if (from_end) sum += v[j];
    if (may) atomicMin(&sh.verdict.lo, tid * 4 + j);
    if (must) atomicMin(&sh.verdict.hi, tid * 4 + j);
  }
  __syncthreads();
  const int lo = sh.verdict.lo, hi = min(sh.verdict.hi, kBins - 1);
  float in = 0.f, up = 0.f;  // how many logits; from shares at most 2% too many
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int b = tid * 4 + i;
    const float n = by_count ? (float)h[i] : (float)h[i] * (1.02f / kShare);
    if (b >= lo && b <= hi) in += n;
    if (b <= hi) up += n;
  }
  if (in > 0.f) atomicAdd(&sh.in_border, in);
  if (up > 0.f) atomicAdd(&sh.up_to, up);
  __syncthreads();
  if (tid == 0) {
    sh.verdict.hi = hi;
    sh.verdict.what = lo == kBins                              ? (by_count && bins.scale == kCountScale ? kWiden : kBitwise)
                      : level == 0 && sh.up_to <= (float)kList ? kGather
                      : sh.in_border <= (float)kList           ? kCollect
                      : level < kLevels                        ? kZoom
                                                               : kBitwise;
  }
}

template <bool kBf16, int kMode>
__global__ void __launch_bounds__(kSpThreads, 3) sampling_kernel(const SpArgs a) {
  using namespace sm100;
  using Vec = SpVec<kBf16>;
  constexpr int kN = Vec::kN, kStep = 32 * kN;  // logits of a warp step
  extern __shared__ uint4 smem[];
  __shared__ SpShared sh;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank(), ranks = cluster_nctarank();
  const int r = blockIdx.x / ranks;
  const int64_t row = a.rows ? a.rows[r] : r;
  const int V = a.V;
  if (row < 0 || row >= a.num_rows) {  // (the same for the whole cluster)
    if (row != -1 && rank == 0 && tid == 0 && a.status) atomicOr(a.status, TSD_STATUS_BAD_PATH);
    if (kMode == kSample && rank == 0)
      for (int i = tid; i < a.draws; i += kSpThreads) {
        a.tokens[(size_t)r * a.draws + i] = -1;
        a.logprob[(size_t)r * a.draws + i] = 0.f;
      }
    return;
  }
  const int pr = r / a.per_param;
  const float T = a.temperature ? a.temperature[pr] : 1.f;
  const bool greedy = !(T >= 1.1754944e-38f);
  int k = a.top_k ? a.top_k[pr] : 0;
  if (k <= 0 || k > V) k = V;
  if (greedy) k = 1;
  const float top_p = a.top_p ? a.top_p[pr] : 1.f;
  const float min_p = a.min_p ? fminf(a.min_p[pr], 1.f) : 0.f;

  // ---- the run of this warp, -inf past the row's end; a lane reads what it wrote itself ----
  const int id0 = ((int)rank * kSpWarps + warp) * a.per_warp;
  uint4 *mine = smem + (size_t)warp * (a.per_warp / kN) + lane;
  Run<kBf16> run;
  run.at = mine;
  run.steps = a.per_warp / kStep;
  run.id = id0 + lane * kN;
  run.inv_t = greedy ? 1.f : __fdiv_rn(1.f, T);
  run.rank = rank;
  run.ranks = ranks;
  {
    using Raw = typename std::conditional<kBf16, uint16_t, uint32_t>::type;
    const Raw *src = reinterpret_cast<const Raw *>(a.logits) + row * V;
    const bool vec = (reinterpret_cast<uintptr_t>(src) & 15) == 0;
    const uint32_t none = kBf16 ? 0xFF80FF80u : 0xFF800000u;
    for (int s = 0; s < run.steps; ++s) {
      const int id = run.id + s * kStep;
      if (vec && id + kN <= V) {
        cp_async_16(smem_addr(mine + s * 32), src + id);
      } else {
        Raw e[kN];
#pragma unroll
        for (int i = 0; i < kN; ++i) e[i] = id + i < V ? src[id + i] : (Raw)none;
        if constexpr (kBf16)
          mine[s * 32] = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
        else
          mine[s * 32] = make_uint4(e[0], e[1], e[2], e[3]);
      }
    }
    for (int b = tid; b < kBins; b += kSpThreads) sh.hist[b] = 0u;
    if (tid == 0) {
      sh.sum_all = sh.sum_near = sh.sum_above = 0ull;
      sh.count_all = sh.count_above = sh.listed = sh.mine = 0;
      sh.failed = false;
    }
    cp_async_wait_all();
  }
  float m = -INFINITY;
  for (int s = 0; s < run.steps; ++s) {
    Vec x;
    x.read(mine + s * 32);
#pragma unroll
    for (int i = 0; i < kN; i += 2) m = max3_nan(m, x.x[i], x.x[i + 1]);
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
  if (lane == 0) sh.wmax[warp] = m;
  __syncthreads();
  if (tid == 0) {
    for (int w = 0; w < kSpWarps; ++w) m = max_nan(m, sh.wmax[w]);
    sh.max = m;
  }
  cluster_sync();
  m = -INFINITY;
  for (uint32_t p = 0; p < ranks; ++p) m = max_nan(m, __uint_as_float(ld_peer32(&sh.max, p)));
  run.m = m;

  const bool bad = !(m < INFINITY), empty = m == -INFINITY;
  if (bad || empty) {
    if (bad && rank == 0 && tid == 0 && a.status) atomicOr(a.status, TSD_STATUS_NONFINITE);
    if (kMode == kSample) {
      if (rank == 0)
        for (int i = tid; i < a.draws; i += kSpThreads) {
          a.tokens[(size_t)r * a.draws + i] = -1;
          a.logprob[(size_t)r * a.draws + i] = bad ? NAN : -INFINITY;
        }
    } else {
      const float x = bad ? NAN : kMode == kProbs ? 0.f : -INFINITY;
      for (int i = id0 + lane; i < min(V, id0 + a.per_warp); i += 32) a.out[(size_t)r * V + i] = x;
    }
    cluster_sync();  // (no CTA leaves while another reads its shared memory)
    return;
  }

  int turn = 0;
  Border kept;
  long long total = -1;  // weight of what is kept, once known

  // ---- the filters' borders ----
#pragma unroll 1
  for (int stage = 0; stage < 2; ++stage) {
    const bool by_count = stage == 0;
    if (by_count ? k >= V : top_p >= 1.f) continue;
    // top-p: from its border on there is more than (1 - p) of a weight of 1 or more, so no
    // logit at or above it has less than (1 - p) / V; what has only adds to the sum
    const float inv_unit = by_count ? 1.f : 1.f / run.inv_t;
    const float near = by_count ? INFINITY : logf((float)V) - logf(1.f - top_p) + 0.05f;
    Bins bins{0.f, by_count ? kCountScale : kWeightScale};
    Verdict v;
    bool again = false;  // a histogram was made
#pragma unroll 1
    for (int level = 0;;) {
      // histogram of what is kept so far
      const float inv_scale = 1.f / bins.scale;
      Fixed all, over;  // over: weight near the top, and once bins are cut again, above them
      int count = 0, count_over = 0;
      const float from = level ? logit_of(bins, kBins, m, inv_unit) : -INFINITY;
      if (by_count) {
        run.each(from, [&](float x, int) {
          const bool in = x > -INFINITY;
          float rest;
          const int b = bin_of(__fsub_rn(m, x), bins, rest);
          count += in;
          if (in && (unsigned)b < (unsigned)kBins) atomicAdd(&sh.hist[b], 1u);
          count_over += b < 0;
        });
      } else {
        run.each_vec(from, [&](const float (&x)[kN], int first) {
          float w[kN];
#pragma unroll
          for (int i = 0; i < kN; ++i) {
            const float d = run.scaled(x[i]);
            const bool in = stage == 0 || k >= V || kept.has(x[i], first + i);
            w[i] = in ? expf(d) : 0.f;
            if (in && d >= -near) {
              float rest;
              const int b = bin_of(-d, bins, rest);
              if (level == 0 || b < 0) over.add(w[i]);
              if ((unsigned)b < (unsigned)kBins) {
                const float z = rest * inv_scale;  // ln of (the bin's weight / this one)
                const float share = fmaf(z, fmaf(z, 0.5f, -1.f), 1.f) * kShare;
                atomicAdd(&sh.hist[b], __float_as_uint(__fadd_rn(share, kRound)) - 0x4B400000u);
              }
            }
          }
          if (level == 0) {
#pragma unroll
            for (int i = 0; i < kN; i += 2) all.add2(w[i], w[i + 1]);
          }
        });
      }
      const long long sums = block_total(sh, count, all.value());
      const long long overs = warp_sum(over.value());
      count_over = __reduce_add_sync(0xffffffffu, count_over);
      if (lane == 0) {
        if (count_over) add_first32(&sh.count_above, count_over);
        if (overs) add_first64(level ? &sh.sum_above : &sh.sum_near, (unsigned long long)overs);
      }
      if (tid == 0 && !again) {
        add_first32(&sh.count_all, count);
        add_first64(&sh.sum_all, (unsigned long long)sums);
      }
      again = true;
      cluster_sync();
      if (rank == 0) {
        if (by_count && sh.count_all <= k) {
          if (tid == 0) sh.verdict.what = kNone;
        } else {
          if (tid == 0) {
            const double all = (double)(long long)sh.sum_all, want = max((double)top_p * all, 1.0);
            sh.need = by_count ? (float)(k - sh.count_above) : (float)((want - (double)(long long)sh.sum_above) * (double)kUnit);
            sh.room = (float)((all - want) * (double)kUnit);
            sh.skipped = (float)((long long)sh.sum_all - (long long)sh.sum_near) * kUnit;
          }
          __syncthreads();
          find_bins(sh, bins, by_count, sh.need, sh.room, !by_count && level == 0, sh.skipped, ranks, level, V);
        }
        __syncthreads();
        // (before the others put their lists there)
        for (int b = tid; b < kBins; b += kSpThreads) sh.hist[b] = 0u;
        if (tid == 0) {
          sh.sum_above = 0ull;
          sh.count_above = 0;
          if (sh.verdict.what == kNone || sh.verdict.what == kBitwise) {
            sh.sum_all = sh.sum_near = 0ull;
            sh.count_all = 0;
          }
        }
      }
      cluster_sync();
      v.what = (int)ld_peer32(&sh.verdict.what, 0);
      v.lo = (int)ld_peer32(&sh.verdict.lo, 0);
      v.hi = (int)ld_peer32(&sh.verdict.hi, 0);
      if (rank != 0)
        for (int b = tid; b < kBins; b += kSpThreads) sh.hist[b] = 0u;  // (for the next one)
      __syncthreads();
      if (v.what == kWiden) {
        bins.scale = kWideScale;
        continue;
      }
      if (v.what != kZoom) break;
      // the border's bins, a little widened, are cut again
      const float width = (float)(v.hi - v.lo + 1) / bins.scale;
      bins.from += ((float)v.lo - 0.5f) / bins.scale - 0.01f * width;
      bins.scale = (float)(kBins - 1) / (1.02f * width);
      ++level;
    }
    if (v.what == kNone) continue;
    if (v.what != kBitwise) {
      // ---- what lies in the border's bins (kGather: and above them) goes to the first CTA ----
      const int lo = v.what == kGather ? -1 : v.lo;
      Fixed over;
      int count = 0;
      run.each(logit_of(bins, v.hi, m, inv_unit), [&](float x, int id) {
        if (!kept.has(x, id)) return;
        const float d = by_count ? __fsub_rn(x, m) : run.scaled(x);
        float rest;
        const int b = bin_of(-d, bins, rest);
        if (b > v.hi) return;
        if (b < lo) {
          ++count;
          if (!by_count) over.add(expf(d));
          return;
        }
        const int at = atomicAdd(rank == 0 ? &sh.listed : &sh.mine, 1);
        if (at < kList) sh.list[at] = ((unsigned long long)ordered(x) << 32) | (uint32_t)~id;
      });
      if (v.what == kCollect) {
        const long long sums = block_total(sh, count, over.value());
        if (tid == 0) {
          add_first32(&sh.count_above, count);
          add_first64(&sh.sum_above, (unsigned long long)sums);
        }
      }
      __syncthreads();
      if (rank != 0) {
        const int n = sh.mine;
        if (tid == 0) sh.wcount[0] = (int)take_first32(&sh.listed, n);
        __syncthreads();
        const int at = sh.wcount[0];
        for (int i = tid; i < min(n, kList); i += kSpThreads)
          if (at + i < kList) st_first64(&sh.list[at + i], sh.list[i]);
        __syncthreads();
        if (tid == 0) sh.mine = 0;
      }
      cluster_sync();
      if (rank == 0) {
        const int n = sh.listed;
        const long long base = (long long)sh.sum_above, everything = (long long)sh.sum_all;
        const int more = sh.count_above;
        __syncthreads();
        if (tid == 0) {
          sh.failed = n > kList;
          sh.border_x = kept.x;
          sh.border_id = kept.id;
          sh.total = 0;
        }
        constexpr int kMine = kList / kSpThreads;
        unsigned long long c[kMine];
        float w[kMine];
        long long before[kMine], fw[kMine];
        int place[kMine];
        const bool weigh = v.what == kGather || !by_count;
#pragma unroll
        for (int e = 0; e < kMine; ++e) {
          const int i = tid + e * kSpThreads;
          c[e] = i < min(n, kList) ? sh.list[i] : 0ull;
          w[e] = 0.f;
          if (c[e] && weigh) {
            w[e] = expf(run.scaled(unordered((uint32_t)(c[e] >> 32))));
            sh.weight[i] = (unsigned long long)fixed(w[e]);
          }
          fw[e] = fixed(w[e]);
          before[e] = 0;
          place[e] = 0;
        }
        __syncthreads();
        if (n <= kList) {
          // rank, and the weight of what ranks higher
          for (int j = 0; j < n; ++j) {
            const unsigned long long o = sh.list[j];
            const long long ow = weigh ? (long long)sh.weight[j] : 0;
#pragma unroll
            for (int e = 0; e < kMine; ++e)
              if (o > c[e]) {
                ++place[e];
                before[e] += ow;
              }
          }
          bool in[kMine];
          if (v.what == kGather) {
            // all that may be kept is here: top-k, then top-p of what that left, then min-p
            long long s = 0;
            int unused = 0;
#pragma unroll
            for (int e = 0; e < kMine; ++e) {
              in[e] = c[e] != 0ull && (stage == 1 || place[e] < k);
              if (in[e]) s += fw[e];
            }
            if (top_p < 1.f) {
              s = block_total(sh, unused, s);
              const long long want = (long long)ceil((double)top_p * (double)(stage == 0 ? s : everything));
#pragma unroll
              for (int e = 0; e < kMine; ++e) in[e] = in[e] && (place[e] == 0 || before[e] < want);
            }
          } else {
            // one filter's border
            const long long want = by_count ? 0 : (long long)ceil((double)top_p * (double)everything);
            if (!by_count && base >= want) sh.failed = true;  // (it lies above the list)
#pragma unroll
            for (int e = 0; e < kMine; ++e)
              in[e] = c[e] != 0ull && (by_count ? more + place[e] < k : base + before[e] < want);
          }
          // the border is the lowest that is kept
          int kept_here = 0;
          long long s = 0;
#pragma unroll
          for (int e = 0; e < kMine; ++e) kept_here += in[e];
          block_total(sh, kept_here, 0);
#pragma unroll
          for (int e = 0; e < kMine; ++e) {
            if (in[e] && place[e] == kept_here - 1) {
              sh.border_x = unordered((uint32_t)(c[e] >> 32));
              sh.border_id = (int)~(uint32_t)c[e];
            }
            if (v.what == kGather) in[e] = in[e] && !(w[e] < min_p);
            if (in[e]) s += fw[e];
          }
          if (kept_here == 0) sh.failed = true;
          int unused = 0;
          s = block_total(sh, unused, s);
          if (tid == 0) sh.total = v.what == kGather ? s : by_count || min_p > 0.f ? -1 : base + s;
          if constexpr (kMode == kSample) {
            if (v.what == kGather) {
              // the draws: the weight of what is kept and has a lower id
#pragma unroll
              for (int e = 0; e < kMine; ++e) {
                if (c[e]) sh.weight[tid + e * kSpThreads] = in[e] ? (unsigned long long)fw[e] : 0ull;
                before[e] = 0;
              }
              if (tid < a.draws) {
                const float u = a.u[(size_t)r * a.draws + tid];
                sh.at[tid] = min(u > 0.f ? (long long)floor((double)u * (double)s) : 0, s - 1);
              }
              __syncthreads();
              for (int j = 0; j < n; ++j) {
                const uint32_t o = (uint32_t)sh.list[j];
                const long long ow = (long long)sh.weight[j];
#pragma unroll
                for (int e = 0; e < kMine; ++e)
                  if (o > (uint32_t)c[e]) before[e] += ow;
              }
              const float log_total = logf((float)s * kUnit);
              for (int q = 0; q < a.draws; ++q) {
                const long long at = sh.at[q];
#pragma unroll
                for (int e = 0; e < kMine; ++e)
                  if (in[e] && at >= before[e] && at < before[e] + fw[e]) {
                    a.tokens[(size_t)r * a.draws + q] = (int32_t)~(uint32_t)c[e];
                    a.logprob[(size_t)r * a.draws + q] = run.scaled(unordered((uint32_t)(c[e] >> 32))) - log_total;
                  }
              }
            }
          }
        }
        __syncthreads();
        for (int b = tid; b < kBins; b += kSpThreads) sh.hist[b] = 0u;  // (it lies over the list)
        if (tid == 0) {
          sh.listed = sh.count_all = sh.count_above = 0;
          sh.sum_all = sh.sum_near = sh.sum_above = 0ull;
        }
      } else {
        for (int b = tid; b < kBins; b += kSpThreads) sh.hist[b] = 0u;
      }
      if (kMode == kSample && v.what == kGather) return;  // (nothing of this CTA is read any more)
      cluster_sync();
      if (ld_peer32(&sh.failed, 0) & 0xFFu) v.what = kBitwise;
      kept.x = __uint_as_float(ld_peer32(&sh.border_x, 0));
      kept.id = (int)ld_peer32(&sh.border_id, 0);
      total = (long long)ld_peer64(&sh.total, 0);
    }
    if (v.what == kBitwise) {
      kept = bitwise_border(sh, run, turn, kept, by_count ? k : 0, top_p);
      total = -1;
    }
    if (v.what == kGather) break;
  }

  // ---- what is kept ----
  auto weight = [&](float x, int id) -> float {  // 0: not kept
    if (!kept.has(x, id)) return 0.f;
    const float w = expf(run.scaled(x));
    return w < min_p ? 0.f : w;
  };
  if (kMode == kSample || (kMode == kProbs && total < 0)) {
    Fixed f;
    run.each(kept.x, [&](float x, int id) { f.add(weight(x, id)); });
    int unused = 0;
    total = cluster_total(sh, turn, ranks, unused, f.value());
  }
  if constexpr (kMode == kSample) {
    long long before = 0;  // of this warp's run
    for (uint32_t p = 0; p < rank; ++p) before += (long long)ld_peer64(&sh.sum[turn ^ 1], p);
    for (int w = 0; w < warp; ++w) before += sh.wsum[w];
    const long long here = sh.wsum[warp];
    const float log_total = logf((float)total * kUnit);
    if (tid < a.draws) {
      const float u = a.u[(size_t)r * a.draws + tid];
      sh.at[tid] = min(u > 0.f ? (long long)floor((double)u * (double)total) : 0, total - 1);
    }
    __syncthreads();
    for (int q = 0; q < a.draws; ++q) {
      long long at = sh.at[q] - before;
      if (at < 0 || at >= here) continue;
      for (int s = 0; s < run.steps; ++s) {
        Vec x;
        x.read(run.at + s * 32);
        float w[kN];
        long long sum = 0;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          w[i] = weight(x.x[i], run.id + s * kStep + i);
          sum += fixed(w[i]);
        }
        long long upto = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const long long o = __shfl_up_sync(0xffffffffu, upto, off);
          if (lane >= off) upto += o;
        }
        const long long all = __shfl_sync(0xffffffffu, upto, 31);
        if (at < all) {
          long long left = at - (upto - sum);
          if (left >= 0 && left < sum) {
            int i = 0;
            float d = 0.f;
#pragma unroll
            for (int j = 0; j < kN; ++j) {
              const long long one = fixed(w[j]);
              if (i == j) {
                d = run.scaled(x.x[j]);
                if (left >= one && j + 1 < kN) {
                  left -= one;
                  ++i;
                }
              }
            }
            a.tokens[(size_t)r * a.draws + q] = run.id + s * kStep + i;
            a.logprob[(size_t)r * a.draws + q] = d - log_total;
          }
          break;
        }
        at -= all;
      }
    }
  } else {
    const float inv = 1.f / ((float)total * kUnit);
    float *dst = a.out + (size_t)r * V;
    const bool vec = (reinterpret_cast<uintptr_t>(dst) & 15) == 0;
    for (int s = 0; s < run.steps; ++s) {
      Vec x;
      x.read(run.at + s * 32);
      const int id = run.id + s * kStep;
      float y[kN];
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const float d = run.scaled(x.x[i]);
        bool in = kept.has(x.x[i], id + i);
        float w = 0.f;
        if (in && (kMode == kProbs || min_p > 0.f)) {
          w = expf(d);
          in = !(w < min_p);
        }
        y[i] = kMode == kProbs ? (in ? w * inv : 0.f) : in ? d : -INFINITY;
      }
      if (vec && id + kN <= V) {
#pragma unroll
        for (int i = 0; i < kN; i += 4)
          __stcs(reinterpret_cast<float4 *>(dst + id + i), make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]));
      } else {
#pragma unroll
        for (int i = 0; i < kN; ++i)
          if (id + i < V) dst[id + i] = y[i];
      }
    }
  }
  cluster_sync();
}

template <bool kBf16, int kMode>
cudaError_t sp_launch(SpArgs &a, cudaStream_t s) {
  constexpr int kN = kBf16 ? 8 : 4, kStep = 32 * kN;
  int c = 1;
  while (c < kMaxCluster && (int64_t)c * kSpWarps * kStep < a.V) c *= 2;
  a.per_warp = ((a.V + c * kSpWarps - 1) / (c * kSpWarps) + kStep - 1) / kStep * kStep;
  const size_t smem = (size_t)a.per_warp * kSpWarps * (kBf16 ? 2 : 4);
  if (!set_smem((const void *)sampling_kernel<kBf16, kMode>, kMaxVocab / kMaxCluster * (kBf16 ? 2 : 4)))
    return cudaErrorUnknown;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.R * c);
  cfg.blockDim = dim3(kSpThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = c;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, sampling_kernel<kBf16, kMode>, a);
}

int sp_check(const SpArgs &a) {
  if (a.R < 0 || a.V < 1 || a.num_rows < 0 || a.per_param < 1) return TSD_ERR_ARG;
  if (a.V > kMaxVocab || a.R > (1 << 24)) return TSD_ERR_LIMIT;
  return TSD_OK;
}

}  // namespace
}  // namespace tsd

TSD_API int tsd_token_sample(const void *logits, int bf16, const int32_t *rows, int R, int64_t num_rows,
                             int V, const float *u, int draws, const float *temperature,
                             const int32_t *top_k, const float *top_p, const float *min_p, int per_param,
                             int32_t *tokens, float *logprob, int32_t *status, tsd_stream_t stream) {
  using namespace tsd;
  SpArgs a{logits, rows, u, temperature, top_p, min_p, top_k, num_rows, R, V, draws, per_param, 0, tokens,
           logprob, nullptr, status};
  const int rc = sp_check(a);
  if (rc != TSD_OK) return rc;
  if (draws < 1) return TSD_ERR_ARG;
  if (draws > kMaxDraws) return TSD_ERR_LIMIT;
  if (R == 0) return TSD_OK;
  if (!logits || !u || !tokens || !logprob) return TSD_ERR_ARG;
  if (!rows && R > num_rows) return TSD_ERR_ARG;
  if (!aligned(logits, bf16 ? 2 : 4)) return TSD_ERR_ARG;
  const cudaError_t e = bf16 ? sp_launch<true, kSample>(a, as_cuda(stream)) : sp_launch<false, kSample>(a, as_cuda(stream));
  return e == cudaSuccess ? TSD_OK : TSD_ERR_CUDA;
}

TSD_API int tsd_logits_filter(const void *logits, int bf16, int R, int V, int probs,
                              const float *temperature, const int32_t *top_k, const float *top_p,
                              const float *min_p, int per_param, float *out, int32_t *status,
                              tsd_stream_t stream) {
  using namespace tsd;
  SpArgs a{logits, nullptr, nullptr, temperature, top_p, min_p, top_k, R, R, V, 0, per_param, 0, nullptr,
           nullptr, out, status};
  const int rc = sp_check(a);
  if (rc != TSD_OK || R == 0) return rc;
  if (!logits || !out) return TSD_ERR_ARG;
  if (!aligned(logits, bf16 ? 2 : 4) || !aligned(out, 4)) return TSD_ERR_ARG;
  const cudaStream_t s = as_cuda(stream);
  const cudaError_t e = bf16 ? (probs ? sp_launch<true, kProbs>(a, s) : sp_launch<true, kLogits>(a, s))
                             : (probs ? sp_launch<false, kProbs>(a, s) : sp_launch<false, kLogits>(a, s));
  return e == cudaSuccess ? TSD_OK : TSD_ERR_CUDA;
}
