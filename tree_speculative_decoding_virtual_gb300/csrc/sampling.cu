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
// A cluster of up to 8 CTAs takes row after row; a row is read once and stays in shared
// memory, each warp with a run of consecutive ids, and the next row's copies start as soon
// as a lane is through with this one's.  A filter's border is found by
//   histogram  2048 bins: for top-k counts of m - x, 32 bins a unit; for top-p weights of
//              (m - x) / T, 64 a unit, relative to the bin's (13 bits a weight: good to
//              1e-4) besides the exact sum of all; the first CTA adds up the cluster's by
//              groups of 32 bins, then the bins of two groups, and finds the bin, or the few
//              bins, that must hold the border
//   list       what lies in them (a handful to 512) goes to the first CTA, with the exact
//              weight above them, and is ranked there (up to 32 by one warp)
// When what lies in those bins and above fits the list (ordinary settings of top-k and
// top-p), the first CTA has all that can be kept, and finishes alone: both filters, min-p
// and the draws.  Bins that hold more than the list are cut into 2048 again; where that does
// not part them either (hundreds of equal logits), the border is found bit by bit.
//
// What bounds it is not the one read of the row (the floor of 508 rows of 128256 fp32 logits
// is 38 us) but some 25 instructions a logit for the histogram (10k cycles of a row's 42k
// with 8 CTAs) and the chain of exchanges in the cluster (three barriers of 3k cycles, bins
// 5k, list 5k, the first CTA's end 5k).  CTAs exchange by loads of what each left in its own
// shared memory: adds from eight CTAs to one place took 6k to 14k cycles.  Measured with a cold
// L2, 128256 logits: one fp32 row with top-k 50 and top-p 0.95 24 us (18 in a graph, 8 CTAs),
// 63 such rows filtered 57; 64 bf16 rows of mixed settings 63 to 72 (6 CTAs); 508 fp32 rows
// with top-p 0.9 and four draws 250 to 350 by the rows' shape, to probabilities 310 to 460
// (8 CTAs).  Rows that do not begin on 16 bytes are copied value by value, not under the end of
// the row before, and take up to 30% longer: 508 fp32 rows with top-p 0.9 and four draws 127 us
// for 50256 logits, 158 for 50257; 64 bf16 rows with top-k 50 31 and 33.
#include <cuda_bf16.h>

#include <cmath>
#include <mutex>
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
constexpr int kMaxRowBytes = kMaxVocab / kMaxCluster * 4;  // of a CTA's share
constexpr int kBins = 2048;
constexpr int kGroup = 32, kGroups = kBins / kGroup;  // bins are looked for by groups of 32 first
constexpr int kList = 512, kCounted = 128, kSmallList = 32;
constexpr float kCountScale = 32.f, kWideScale = 0.5f, kWeightScale = 64.f;  // bins a unit at first
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
constexpr float kRound = 12582912.f;  // 1.5 * 2^23: a sum with it is rounded to a whole number
struct Bins {
  float from, scale, shift;  // shift: kRound - from * scale
  __device__ __forceinline__ void set(float f, float s) {
    from = f;
    scale = s;
    shift = fmaf(-f, s, kRound);
  }
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
  long long wsum[kSpWarps], wabove[kSpWarps];
  int wcount_above[kSpWarps];
  float scan[kSpWarps];
  float max;
  // this CTA's parts of what the first CTA adds up
  struct {
    long long all, above;
    float skipped;
    int count, count_above;
  } part;
  // the first CTA's sums
  long long sum_all, sum_above;
  float skipped;
  int count_all, count_above, listed;
  float u[kMaxDraws];
  alignas(16) float2 groups[kGroups];  // weight, and number of logits
  // exchanged by the bitwise search and the draws (two places, by turn)
  int count[2];
  long long sum[2];
  // the first CTA's findings
  Verdict verdict;
  float border_x;
  int border_id;
  long long total;
  unsigned long long extra[kMaxCluster * kSpWarps];  // kept weight of the list, by warp run
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
  // The sum over the warp's lanes.
  __device__ __forceinline__ long long warp() const {
    constexpr unsigned all = 0xffffffffu;
    const long long h = ((long long)__reduce_add_sync(all, hi >> 8) << 8) + __reduce_add_sync(all, hi & 255u);
    return (h << 23) + ((long long)__reduce_add_sync(all, lo >> 8) << 8) + __reduce_add_sync(all, lo & 255);
  }
};
constexpr float kUnit = 0x1p-43f;

// ln of a sum that holds the largest weight, 1: to the last places where it is near 0 too.
__device__ __forceinline__ float log_sum(long long total) { return log1pf((float)(total - (1ll << 43)) * kUnit); }

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

__device__ __forceinline__ float warp_sum(float x) {
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
  // Calls f(logits, id of the first, the largest) for every vector of this lane that holds a logit of
  // `from` or more.
  template <class F>
  __device__ __forceinline__ void each_vec(float from, F f) const {
    constexpr int kAhead = 4;  // vectors read before the first is looked at
#pragma unroll 1
    for (int s0 = 0; s0 < steps; s0 += kAhead) {
      uint4 raw[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) raw[j] = at[min(s0 + j, steps - 1) * 32];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (s0 + j >= steps) break;
        SpVec<kBf16> v;
        v.read(&raw[j]);
        float most = fmaxf(v.x[0], v.x[1]);
#pragma unroll
        for (int i = 2; i < kN; i += 2) most = sm100::fmax3(most, v.x[i], v.x[i + 1]);
        if (most >= from) f(v.x, id + (s0 + j) * (32 * kN), most);
      }
    }
  }
  // Calls f(logit, id) for every logit of `from` or more (and some others).
  template <class F>
  __device__ __forceinline__ void each(float from, F f) const {
    each_vec(from, [&](const float (&x)[kN], int first, float) {
#pragma unroll
      for (int i = 0; i < kN; ++i) f(x[i], first + i);
    });
  }
};

// The bin of a distance: -1 above the bins, kBins below them; `y` is kRound + the bin.  The
// same rounding for every logit, so that a larger logit is never in a later bin.
__device__ __forceinline__ int bin_of(float distance, const Bins &b, float &y) {
  y = fminf(fmaxf(fmaf(distance, b.scale, b.shift), kRound - 1.f), kRound + kBins);
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

// This CTA's sums for the first CTA.
__device__ __forceinline__ void block_parts(SpShared &sh, const Fixed &f_all, const Fixed &f_above, float skipped,
                                            int count, int count_above) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long all = f_all.warp(), above = f_above.warp();
  skipped = warp_sum(skipped);
  count = __reduce_add_sync(0xffffffffu, count);
  count_above = __reduce_add_sync(0xffffffffu, count_above);
  if (lane == 0) {
    sh.wsum[warp] = all;
    sh.wabove[warp] = above;
    sh.scan[warp] = skipped;
    sh.wcount[warp] = count;
    sh.wcount_above[warp] = count_above;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    all = above = 0;
    skipped = 0.f;
    count = count_above = 0;
#pragma unroll
    for (int w = 0; w < kSpWarps; ++w) {
      all += sh.wsum[w];
      above += sh.wabove[w];
      skipped += sh.scan[w];
      count += sh.wcount[w];
      count_above += sh.wcount_above[w];
    }
    sh.part.all = all;
    sh.part.above = above;
    sh.part.skipped = skipped;
    sh.part.count = count;
    sh.part.count_above = count_above;
  }
}

// First CTA, first warp: the cluster's sums (what is added up once stays, the others are
// new).  In two halves, so that the loads' latency passes while others are under way.
struct Parts {
  long long all, above;
  float skipped;
  int count, count_above;
  __device__ __forceinline__ void load(SpShared &sh, uint32_t ranks) {
    const int lane = threadIdx.x & 31;
    const bool on = lane < (int)ranks;
    all = on ? (long long)ld_peer64(&sh.part.all, lane) : 0;
    above = on ? (long long)ld_peer64(&sh.part.above, lane) : 0;
    skipped = on ? __uint_as_float(ld_peer32(&sh.part.skipped, lane)) : 0.f;
    count = on ? (int)ld_peer32(&sh.part.count, lane) : 0;
    count_above = on ? (int)ld_peer32(&sh.part.count_above, lane) : 0;
  }
  __device__ __forceinline__ void sum(SpShared &sh) {
    all = warp_sum(all);
    above = warp_sum(above);
    skipped = warp_sum(skipped);
    count = __reduce_add_sync(0xffffffffu, count);
    count_above = __reduce_add_sync(0xffffffffu, count_above);
    if ((threadIdx.x & 31) == 0) {
      sh.sum_all += all;
      sh.sum_above = above;
      sh.skipped = skipped;
      sh.count_all += count;
      sh.count_above = count_above;
    }
  }
};

// Sum over the threads before this one.
__device__ __forceinline__ long long block_scan(SpShared &sh, long long mine) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long upto = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, upto, off);
    if (lane >= off) upto += o;
  }
  __syncthreads();
  if (lane == 31) sh.wsum[warp] = upto;
  __syncthreads();
  long long before = upto - mine;
  for (int w = 0; w < warp; ++w) before += sh.wsum[w];
  return before;
}

// Sorts a[0, size), size a power of two of at most twice the block's threads, in place (a
// bitonic network; steps within 64 elements stay in a warp).  Starts and ends with a
// barrier.
template <bool kDown, class T>
__device__ __forceinline__ void sort(T *a, int size) {
  const int t = threadIdx.x;
  __syncthreads();
  for (int span = 2; span <= size; span *= 2)
    for (int stride = span / 2; stride; stride /= 2) {
      if (2 * t < size) {
        const int i = 2 * t - (t & (stride - 1)), j = i + stride;
        const T x = a[i], y = a[j];
        const bool down = ((i & span) == 0) == kDown;
        if (down ? x < y : y < x) {
          a[i] = y;
          a[j] = x;
        }
      }
      // (after a span of 64 the next step crosses warps)
      if (stride > 32 || (stride == 1 && span >= 64)) __syncthreads();
      else __syncwarp();
    }
  __syncthreads();
}

// Where a draw falls: the first weight whose sum exceeds this is drawn.  The product of u
// (24 bits) and the sum is exact in 64 bits and a shift.
__device__ __forceinline__ long long place_of(float u, long long total) {
  if (!(u > 0.f)) return 0;
  if (u >= 1.f) return total - 1;
  const uint32_t bits = __float_as_uint(u);
  const int e = (int)(bits >> 23);  // u = f 2^(e - 150), f < 2^24
  const unsigned long long f = e ? (bits & 0x7FFFFFu) | 0x800000u : bits & 0x7FFFFFu;
  const int shift = 150 - (e ? e : 1);
  const unsigned long long hi = __umul64hi(f, (unsigned long long)total), lo = f * (unsigned long long)total;
  const unsigned long long at = shift >= 128 ? 0ull : shift >= 64 ? hi >> (shift - 64) : (hi << (64 - shift)) | (lo >> shift);
  return min((long long)at, total - 1);
}

// block_total over the cluster; `turn` is which of the two places is used.
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

// What each group of this CTA's bins holds; after a barrier behind the histogram.
__device__ __forceinline__ void sum_groups(SpShared &sh, const Bins &bins, bool by_count) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float width = 1.f / bins.scale;
  const float own = by_count ? 1.f : expf(-(bins.from + (float)lane * width)) * (1.f / kShare);
  static_assert(kGroups / kSpWarps == 8, "");
  float n[8], w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t h = sh.hist[(warp * 8 + i) * kGroup + lane];
    n[i] = (float)__reduce_add_sync(0xffffffffu, h);
    w[i] = (float)h * own;
  }
  // eight sums over the lanes at once: lane l ends with that of group l / 4
#pragma unroll
  for (int off = 16, left = 4; left; off /= 2, left /= 2)
#pragma unroll
    for (int i = 0; i < left; ++i) {
      const bool up = lane & off;
      const float mine = up ? w[i + left] : w[i], theirs = up ? w[i] : w[i + left];
      w[i] = mine + __shfl_xor_sync(0xffffffffu, theirs, off);
    }
  w[0] += __shfl_xor_sync(0xffffffffu, w[0], 2);
  w[0] += __shfl_xor_sync(0xffffffffu, w[0], 1);
  float mine = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i == lane / 4) mine = n[i];
  const int g = warp * 8 + lane / 4;
  // (from shares at most 2% too many)
  if (lane % 4 == 0)
    sh.groups[g] = by_count ? make_float2(mine, mine) : make_float2(w[0] * expf(-(float)(g * kGroup) * width), mine * (1.02f / kShare));
}

// First CTA, first warp: the bins that hold the border, from the cluster's histograms:
// the groups that must, then the bins of two groups.  Counts are added up from the bins'
// top until there are as many as wanted; so are weights, but at first from their end, until
// there is more than may be left behind the border (the exact sum less the share wanted:
// what is left is small, and known better by itself than as a difference).
__device__ __forceinline__ void find_bins(SpShared &sh, const Bins bins, bool by_count, int k, float top_p,
                                          uint32_t ranks, int level) {
  const int lane = threadIdx.x;
  const bool from_end = !by_count && level == 0;
  static_assert(kGroups == 64, "two a lane");
  Parts parts;
  parts.load(sh, ranks);
  // (loads before their uses: one takes some 700 cycles)
  uint4 x[kMaxCluster];
#pragma unroll
  for (uint32_t p = 0; p < kMaxCluster; ++p)
    x[p] = p < ranks ? ld_peer128(&sh.groups[2 * lane], p) : make_uint4(0u, 0u, 0u, 0u);
  float w[2] = {0.f, 0.f}, n[2] = {0.f, 0.f};
#pragma unroll
  for (uint32_t p = 0; p < kMaxCluster; ++p) {
    w[0] += __uint_as_float(x[p].x);
    n[0] += __uint_as_float(x[p].y);
    w[1] += __uint_as_float(x[p].z);
    n[1] += __uint_as_float(x[p].w);
  }
  parts.sum(sh);
  __syncwarp();
  const double all = (double)sh.sum_all, want = max((double)top_p * all, 1.0);
  const float need = by_count ? (float)(k - sh.count_above) : (float)((want - (double)sh.sum_above) * (double)kUnit);
  const float room = (float)((all - want) * (double)kUnit), skipped = sh.skipped;
  const float e = by_count ? 0.f : kShareError;
  // whether the border may, and must, lie at or before a bin (or group), by the sum up to it
  // or, from the end, of what lies behind it
  auto may = [&](float sum) { return from_end ? sum * (1.f - e) <= room : sum * (1.f + e) >= need; };
  auto must = [&](float sum) { return from_end ? sum * (1.f + e) <= room : sum * (1.f - e) >= need; };
  // sums over the lanes before this one, or after it
  auto scan = [&](float v) -> float {
    float upto = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const float y = from_end ? __shfl_down_sync(0xffffffffu, upto, off) : __shfl_up_sync(0xffffffffu, upto, off);
      if (from_end ? lane + off < 32 : lane >= off) upto += y;
    }
    return upto - v;
  };
  auto first = [&](bool a, bool b) -> int {  // place 2 lane (+ 1) of the first true
    return (int)__reduce_min_sync(0xffffffffu, (unsigned)(a ? 2 * lane : b ? 2 * lane + 1 : 64));
  };
  const float out = scan(w[0] + w[1]) + (from_end ? skipped : 0.f);
  const float s0 = from_end ? out + w[1] : out + w[0], s1 = from_end ? out : out + w[0] + w[1];
  const int glo = first(may(s0), may(s1)), ghi = min(first(must(s0), must(s1)), kGroups - 1);
  int lo = kBins, hi = kBins - 1;
  float in_border = 0.f, up_to = 0.f;
  if (glo < kGroups) {
    const int g0 = min(glo, kGroups - 2);  // the two groups that are looked at
    uint32_t h[2] = {0u, 0u};
    unsigned long long y[kMaxCluster];
#pragma unroll
    for (uint32_t p = 0; p < kMaxCluster; ++p)
      y[p] = p < ranks ? ld_peer64(&sh.hist[g0 * kGroup + 2 * lane], p) : 0ull;
#pragma unroll
    for (uint32_t p = 0; p < kMaxCluster; ++p) {
      h[0] += (uint32_t)y[p];
      h[1] += (uint32_t)(y[p] >> 32);
    }
    const float width = 1.f / bins.scale, at = bins.from + (float)(g0 * kGroup + 2 * lane) * width;
    const float own = by_count ? 1.f : expf(-at) * (1.f / kShare);
    const float f0 = (float)h[0] * own, f1 = (float)h[1] * (by_count ? 1.f : own * expf(-width));
    // what lies outside the two groups, on the side that is added up from
    const float outside = warp_sum((from_end ? 2 * lane > g0 + 1 : 2 * lane < g0) ? w[0] : 0.f) +
                          warp_sum((from_end ? 2 * lane + 1 > g0 + 1 : 2 * lane + 1 < g0) ? w[1] : 0.f) +
                          (from_end ? skipped : 0.f);
    const float in = scan(f0 + f1) + outside;
    const float t0 = from_end ? in + f1 : in + f0, t1 = from_end ? in : in + f0 + f1;
    const int flo = first(may(t0), may(t1)), fhi = first(must(t0), must(t1));
    lo = g0 * kGroup + min(flo, 63);
    const float share = by_count ? 1.f : 1.02f / kShare;
    const float before = warp_sum((2 * lane < g0 ? n[0] : 0.f) + (2 * lane + 1 < g0 ? n[1] : 0.f));
    if (fhi < 64) {
      hi = g0 * kGroup + fhi;
      in_border = warp_sum((2 * lane >= flo && 2 * lane <= fhi ? (float)h[0] : 0.f) +
                           (2 * lane + 1 >= flo && 2 * lane + 1 <= fhi ? (float)h[1] : 0.f)) * share;
      up_to = before + warp_sum((2 * lane <= fhi ? (float)h[0] : 0.f) + (2 * lane + 1 <= fhi ? (float)h[1] : 0.f)) * share;
    } else {
      hi = (ghi + 1) * kGroup - 1;
      up_to = warp_sum((2 * lane <= ghi ? n[0] : 0.f) + (2 * lane + 1 <= ghi ? n[1] : 0.f));
      in_border = up_to - before;
    }
  }
  if (lane == 0) {
    const int what = by_count && sh.count_all <= k            ? kNone
                     : lo == kBins                            ? (by_count && bins.scale == kCountScale ? kWiden : kBitwise)
                     : level == 0 && up_to <= (float)kList    ? kGather
                     : in_border <= (float)kList              ? kCollect
                     : level < kLevels                        ? kZoom
                                                              : kBitwise;
    sh.verdict = Verdict{what, lo, hi};
    if (what == kNone || what == kBitwise) {
      sh.sum_all = 0;
      sh.count_all = 0;
    }
  }
}

// What the first CTA knows when it has the list.
struct Found {
  bool gathered;  // all that may be kept is in the list
  bool by_count;
  int k;
  float top_p, min_p;
  int n, more;                 // logits in the list, above it
  long long base, everything;  // weight above the list, of all that was binned
};

// Over a list of at most kCounted entries, for this thread's: how many are ranked before
// it, and their weight (kById: how much weight those of a smaller id have).
template <bool kById>
__device__ __forceinline__ void list_scan(const SpShared &sh, int n, unsigned long long mine, int &place, long long &before) {
  auto less = [&](unsigned long long other) {
    return kById ? (uint32_t)other > (uint32_t)mine : other > mine;  // (the low word is ~id)
  };
  place = 0;
  before = 0;
  if ((int)(threadIdx.x & ~31u) >= n) return;
#pragma unroll 4
  for (int j = 0; j < n; j += 2) {  // (an odd list ends with a zero)
    const ulonglong2 o = *reinterpret_cast<const ulonglong2 *>(&sh.list[j]);
    const ulonglong2 w = *reinterpret_cast<const ulonglong2 *>(&sh.weight[j]);
    if (less(o.x)) {
      ++place;
      before += (long long)w.x;
    }
    if (less(o.y)) {
      ++place;
      before += (long long)w.y;
    }
  }
}

// The first CTA's end of it: ranks the list, finds the border, and where everything
// is in the list the sum of what is kept and the draws.  By the whole block: a short list's
// entries are compared with all, a long one is sorted (with all lists of more than
// kSmallList sorted one row takes 29 us instead of 24, 63 filtered rows 61 instead of 57, 508
// rows as long; comparing all took 508 rows with top-p 0.9 7% longer when it was tried).
template <bool kBf16, int kMode>
__device__ __forceinline__ void settle(SpShared &sh, const Run<kBf16> &run, const Found &f, const SpArgs &a, int r) {
  const int tid = threadIdx.x, n = f.n;
  const bool weigh = f.gathered || !f.by_count;
  const bool counted = n <= kCounted;
  unsigned long long c[2];
  float x[2], w[2] = {0.f, 0.f};
  int id[2], place[2];
  long long fw[2], before[2];
  bool in[2];
  if (!counted) {
    int size = 2;
    while (size < n) size *= 2;
    for (int i = n + tid; i < size; i += kSpThreads) sh.list[i] = 0ull;
    sort<true>(sh.list, size);
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {  // sorted: the ranks 2 tid and 2 tid + 1
    const int i = counted ? tid + e * kSpThreads : 2 * tid + e;
    in[e] = i < n;
    c[e] = in[e] ? sh.list[i] : 0ull;
    x[e] = unordered((uint32_t)(c[e] >> 32));
    id[e] = (int)~(uint32_t)c[e];
    if (in[e] && weigh) w[e] = expf(run.scaled(x[e]));
    fw[e] = fixed(w[e]);
    place[e] = i;
  }
  if (counted) {
    if (tid < kCounted) sh.weight[tid] = (unsigned long long)fw[0];
    if (tid == n) sh.list[n] = 0ull;
    __syncthreads();
    list_scan<false>(sh, n, c[0], place[0], before[0]);
    before[1] = 0;
  } else {
    before[0] = block_scan(sh, fw[0] + fw[1]);
    before[1] = before[0] + fw[0];
  }
  int here = 0;
  if (f.gathered) {
    // top-k, then top-p of what that left
#pragma unroll
    for (int e = 0; e < 2; ++e) in[e] = in[e] && place[e] < f.k;
    if (f.top_p < 1.f) {
      const long long left = f.by_count ? block_total(sh, here, (in[0] ? fw[0] : 0) + (in[1] ? fw[1] : 0)) : f.everything;
      const long long want = (long long)ceil((double)f.top_p * (double)left);
#pragma unroll
      for (int e = 0; e < 2; ++e) in[e] = in[e] && (place[e] == 0 || before[e] < want);
    }
  } else {
    // one filter's border
    const long long want = f.by_count ? 0 : (long long)ceil((double)f.top_p * (double)f.everything);
    if (!f.by_count && f.base >= want) sh.failed = true;  // (it lies above the list)
#pragma unroll
    for (int e = 0; e < 2; ++e) in[e] = in[e] && (f.by_count ? f.more + place[e] < f.k : f.base + before[e] < want);
  }
  // the border is the last that is kept; then min-p, which the weight alone decides
  here = in[0] + in[1];
  block_total(sh, here, 0);
  if (here == 0) sh.failed = true;
  int left = 0;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    if (in[e] && place[e] == here - 1) {
      sh.border_x = x[e];
      sh.border_id = id[e];
    }
    if (f.gathered) in[e] = in[e] && !(w[e] < f.min_p);
  }
  const long long s = block_total(sh, left, (in[0] ? fw[0] : 0) + (in[1] ? fw[1] : 0));
  if (tid == 0) sh.total = f.gathered ? s : f.by_count || f.min_p > 0.f ? -1 : f.base + s;
  if constexpr (kMode == kSample) {
    if (!f.gathered) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (in[e] && fw[e]) atomicAdd(&sh.extra[id[e] / a.per_warp], (unsigned long long)fw[e]);
      return;
    }
    // the draws: the same by id
    if (counted) {
      if (!in[0]) fw[0] = 0;
      if (tid < kCounted) sh.weight[tid] = (unsigned long long)fw[0];
      __syncthreads();
      list_scan<true>(sh, n, c[0], place[0], before[0]);
    } else {
      static_assert(kMaxVocab * kList <= (1 << 27), "id and rank in a word");
      uint32_t *by_id = reinterpret_cast<uint32_t *>(sh.list);
      float *logit = reinterpret_cast<float *>(by_id + kList);
      __syncthreads();  // (the list was read)
      int size = 2;
      while (size < n) size *= 2;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = 2 * tid + e;
        if (i < size) by_id[i] = in[e] ? (uint32_t)id[e] * kList + i : 0xFFFFFFFFu;
        logit[i] = x[e];
        sh.weight[i] = (unsigned long long)fw[e];
      }
      sort<false>(by_id, size);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t one = 2 * tid + e < size ? by_id[2 * tid + e] : 0xFFFFFFFFu;
        const bool any = one != 0xFFFFFFFFu;
        id[e] = (int)(one / kList);
        fw[e] = any ? (long long)sh.weight[one % kList] : 0;
        x[e] = any ? logit[one % kList] : 0.f;
      }
      before[0] = block_scan(sh, fw[0] + fw[1]);
      before[1] = before[0] + fw[0];
    }
    const float log_total = log_sum(s);
    for (int q = 0; q < a.draws; ++q) {
      const long long at = place_of(sh.u[q], s);
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (at >= before[e] && at < before[e] + fw[e]) {
          a.tokens[(size_t)r * a.draws + q] = id[e];
          a.logprob[(size_t)r * a.draws + q] = run.scaled(x[e]) - log_total;
        }
    }
  }
}

// The same for at most 32 logits, by the first warp: a lane each, all compared with all.
template <bool kBf16, int kMode>
__device__ __forceinline__ void settle_few(SpShared &sh, const Run<kBf16> &run, const Found &f, const SpArgs &a, int r) {
  const int lane = threadIdx.x, n = f.n;
  const unsigned long long c = lane < n ? sh.list[lane] : 0ull;
  const float x = unordered((uint32_t)(c >> 32));
  const int id = (int)~(uint32_t)c;
  const float w = lane < n ? expf(run.scaled(x)) : 0.f;
  const long long fw = fixed(w);
  auto shuffle = [](unsigned long long v, int from) { return __shfl_sync(0xffffffffu, v, from); };
  int place = 0;
  long long before = 0;
  for (int j = 0; j < n; ++j) {
    const unsigned long long o = shuffle(c, j);
    const long long ow = (long long)shuffle((unsigned long long)fw, j);
    if (o > c) {
      ++place;
      before += ow;
    }
  }
  bool in = lane < n;
  if (f.gathered) {
    in = in && place < f.k;
    if (f.top_p < 1.f) {
      const long long left = f.by_count ? warp_sum(in ? fw : 0ll) : f.everything;
      in = in && (place == 0 || before < (long long)ceil((double)f.top_p * (double)left));
    }
  } else {
    const long long want = f.by_count ? 0 : (long long)ceil((double)f.top_p * (double)f.everything);
    if (!f.by_count && f.base >= want) sh.failed = true;
    in = in && (f.by_count ? f.more + place < f.k : f.base + before < want);
  }
  const int here = __popc(__ballot_sync(0xffffffffu, in));
  if (here == 0) sh.failed = true;
  if (in && place == here - 1) {
    sh.border_x = x;
    sh.border_id = id;
  }
  if (f.gathered) in = in && !(w < f.min_p);
  const long long s = warp_sum(in ? fw : 0ll);
  if (lane == 0) sh.total = f.gathered ? s : f.by_count || f.min_p > 0.f ? -1 : f.base + s;
  if constexpr (kMode == kSample) {
    if (!f.gathered) {
      if (in && fw && !f.by_count) atomicAdd(&sh.extra[id / a.per_warp], (unsigned long long)fw);
      return;
    }
    before = 0;
    for (int j = 0; j < n; ++j) {
      const int o = __shfl_sync(0xffffffffu, in ? id : kMaxVocab, j);
      const long long ow = (long long)shuffle((unsigned long long)fw, j);
      if (o < id) before += ow;
    }
    const float log_total = log_sum(s);
    for (int q = 0; q < a.draws; ++q) {
      const long long at = place_of(sh.u[q], s);
      if (in && at >= before && at < before + fw) {
        a.tokens[(size_t)r * a.draws + q] = id;
        a.logprob[(size_t)r * a.draws + q] = run.scaled(x) - log_total;
      }
    }
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
  const int V = a.V, clusters = gridDim.x / ranks;
  // The run of this warp, -inf past the row's end.  A lane reads nothing but what it copied
  // itself, so the next row's copies start as soon as a lane is through with this one's.
  const int id0 = ((int)rank * kSpWarps + warp) * a.per_warp;
  uint4 *mine = smem + (size_t)warp * (a.per_warp / kN) + lane;
  Run<kBf16> run;
  run.at = mine;
  run.steps = a.per_warp / kStep;
  run.id = id0 + lane * kN;
  run.rank = rank;
  run.ranks = ranks;
  auto fetch = [&](int r) {
    const int64_t row = r >= a.R ? -1 : a.rows ? a.rows[r] : r;
    if (row < 0 || row >= a.num_rows) return;
    using Raw = typename std::conditional<kBf16, uint16_t, uint32_t>::type;
    const Raw *src = reinterpret_cast<const Raw *>(a.logits) + row * V;
    const bool vec = (reinterpret_cast<uintptr_t>(src) & 15) == 0;
    const uint32_t none = kBf16 ? 0xFF80FF80u : 0xFF800000u;
    for (int s = 0; s < run.steps; ++s) {
      const int id = run.id + s * kStep;
      // (a row that does not begin on 16 bytes is waited for here: slower, see the top)
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
  };
  const int first_row = blockIdx.x / ranks;
  fetch(first_row);
  for (int b = tid; b < kBins; b += kSpThreads) sh.hist[b] = 0u;
#pragma unroll 1
  for (int r = first_row; r < a.R; r += clusters) {
  const int64_t row = a.rows ? a.rows[r] : r;
  if (row < 0 || row >= a.num_rows) {  // (the same for the whole cluster)
    if (row != -1 && rank == 0 && tid == 0 && a.status) atomicOr(a.status, TSD_STATUS_BAD_PATH);
    if (kMode == kSample && rank == 0)
      for (int i = tid; i < a.draws; i += kSpThreads) {
        a.tokens[(size_t)r * a.draws + i] = -1;
        a.logprob[(size_t)r * a.draws + i] = 0.f;
      }
    fetch(r + clusters);
    continue;
  }
  const int pr = r / a.per_param;
  // (a T that is not finite is the largest: 0 times the -inf of a masked logit would be NaN)
  const float T = a.temperature ? fminf(a.temperature[pr], 3.4028235e38f) : 1.f;
  const bool greedy = !(T >= 1.1754944e-38f);
  int k = a.top_k ? a.top_k[pr] : 0;
  if (k <= 0 || k > V) k = V;
  if (greedy) k = 1;
  // (below zero is zero: rank 0 alone, and `near` below stays positive; NaN: off)
  const float top_p = !a.top_p ? 1.f : a.top_p[pr] < 0.f ? 0.f : a.top_p[pr];
  const float min_p = a.min_p && a.min_p[pr] > 0.f ? fminf(a.min_p[pr], 1.f) : 0.f;  // (NaN: off)
  run.inv_t = greedy ? 1.f : __fdiv_rn(1.f, T);
  __syncthreads();  // (the row before is done with)
  if (kMode == kSample && tid < a.draws) sh.u[tid] = a.u[(size_t)r * a.draws + tid];
  if (tid == 0) {
    sh.sum_all = 0;
    sh.count_all = sh.listed = sh.mine = 0;
    sh.failed = false;
  }
  cp_async_wait_all();
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
  m = lane < (int)ranks ? __uint_as_float(ld_peer32(&sh.max, lane)) : -INFINITY;
#pragma unroll
  for (int off = kMaxCluster / 2; off; off >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
  m = __shfl_sync(0xffffffffu, m, 0);
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
    fetch(r + clusters);
    cluster_sync();  // (no CTA goes on while another reads its shared memory)
    continue;
  }

  int turn = 0;
  Border kept;
  long long total = -1;  // weight of what is kept, once known
  bool through = false;  // the first CTA has all it needs for the draws

  // ---- the filters' borders ----
#pragma unroll 1
  for (int stage = 0; stage < 2; ++stage) {
    const bool by_count = stage == 0;
    if (by_count ? k >= V : !(top_p < 1.f)) continue;
    // top-p: from its border on there is more than (1 - p) of a weight of 1 or more, so no
    // logit at or above it has less than (1 - p) / V (up to the sums' last place, 2^-43 a
    // logit); what has only adds to the sum, and is neither binned nor listed.  The 0.05 are
    // three bins: what lies behind the bin in front of `near`'s weighs less than 0.97 of
    // (1 - p), so the border is found there or before, and a list's length is what was binned.
    // (near is in (0, 29.2]; the first bins end at 32)
    const float inv_unit = by_count ? 1.f : 1.f / run.inv_t;
    const float near = by_count ? INFINITY : logf((float)V) - logf(1.f - top_p) + 0.05f;
    Bins bins;
    bins.set(0.f, by_count ? kCountScale : kWeightScale);
    Verdict v;
    bool again = false;  // a histogram was made
#pragma unroll 1
    for (int level = 0;;) {
      // histogram of what is kept so far
      const float inv_scale = 1.f / bins.scale;
      // a logit's share of its bin, e^z with z = -rest / scale, to second order
      const float share2 = 0.5f * kShare * inv_scale * inv_scale, share1 = -kShare * inv_scale;
      Fixed all, over;    // over: weight above the bins, once they are cut again
      float skipped = 0.f;  // weight too small to be binned
      int count = 0, count_over = 0;
      const float from = level ? logit_of(bins, kBins, m, inv_unit) : -INFINITY;
      if (by_count) {
        run.each(from, [&](float x, int) {
          const bool in = x > -INFINITY;
          float y;
          const int b = bin_of(__fsub_rn(m, x), bins, y);
          count += in;
          if (in && (unsigned)b < (unsigned)kBins) atomicAdd(&sh.hist[b], 1u);
          count_over += b < 0;
        });
      } else {
        const bool all_kept = k >= V;
        auto bin = [&](float d, float w) {
          float y;
          const int b = bin_of(-d, bins, y);
          if (level && b < 0) over.add(w);
          if (!level || (unsigned)b < (unsigned)kBins) {
            const float rest = fmaf(-d, bins.scale, __fsub_rn(bins.shift, y));
            const float share = fmaf(rest, fmaf(rest, share2, share1), kShare + kRound);
            atomicAdd(&sh.hist[b], __float_as_uint(share) - 0x4B400000u);
          }
        };
        if (level) {
          run.each(from, [&](float x, int id) {
            const float d = run.scaled(x);
            if ((all_kept || kept.has(x, id)) && d >= -near) bin(d, expf(d));
          });
        } else {
          const float near_x = m - near * inv_unit * 1.00001f - fabsf(m) * 0x1p-21f;  // (or a little lower)
          run.each_vec(-INFINITY, [&](const float (&x)[kN], int first, float most) {
            float d[kN], w[kN];
#pragma unroll
            for (int i = 0; i < kN; ++i) {
              d[i] = run.scaled(x[i]);
              w[i] = expf(d[i]);
              if (!all_kept && !kept.has(x[i], first + i)) {
                d[i] = -INFINITY;
                w[i] = 0.f;
              }
            }
#pragma unroll
            for (int i = 0; i < kN; i += 2) all.add2(w[i], w[i + 1]);
            if (most < near_x) {
#pragma unroll
              for (int i = 0; i < kN; i += 4) skipped += (w[i] + w[i + 1]) + (w[i + 2] + w[i + 3]);
            } else {
#pragma unroll
              for (int i = 0; i < kN; ++i) {
                if (d[i] >= -near) bin(d[i], w[i]);
                else skipped += w[i];
              }
            }
          });
        }
      }
      if (again) {
        all = Fixed();
        count = 0;
      }
      block_parts(sh, all, over, skipped, count, count_over);
      again = true;
      sum_groups(sh, bins, by_count);
      cluster_sync();
      if (rank == 0) {
        if (warp == 0) find_bins(sh, bins, by_count, k, top_p, ranks, level);
        __syncthreads();
        // (before the others put their lists there)
        for (int b = tid; b < kBins; b += kSpThreads) sh.hist[b] = 0u;
      }
      cluster_sync();
      v.what = (int)ld_peer32(&sh.verdict.what, 0);
      v.lo = (int)ld_peer32(&sh.verdict.lo, 0);
      v.hi = (int)ld_peer32(&sh.verdict.hi, 0);
      if (rank != 0)
        for (int b = tid; b < kBins; b += kSpThreads) sh.hist[b] = 0u;  // (for the next one)
      __syncthreads();
      if (v.what == kWiden) {
        bins.set(0.f, kWideScale);
        continue;
      }
      if (v.what != kZoom) break;
      // the border's bins, a little widened, are cut again
      const float width = (float)(v.hi - v.lo + 1) / bins.scale;
      bins.set(bins.from + ((float)v.lo - 0.5f) / bins.scale - 0.01f * width, (float)(kBins - 1) / (1.02f * width));
      ++level;
    }
    if (v.what == kNone) continue;
    if (v.what != kBitwise) {
      // ---- what lies in the border's bins (kGather: and above them) goes to the first CTA ----
      const int lo = v.what == kGather ? -1 : v.lo;
      Fixed over;
      int count = 0;
      auto list = [&](float x, int id) {
        const int at = atomicAdd(rank == 0 ? &sh.listed : &sh.mine, 1);
        if (at < kList) sh.list[at] = ((unsigned long long)ordered(x) << 32) | (uint32_t)~id;
      };
      run.each_vec(logit_of(bins, v.hi, m, inv_unit), [&](const float (&x)[kN], int first, float) {
        float w[kN];
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          const bool in = kept.has(x[i], first + i);
          const float d = by_count ? __fsub_rn(x[i], m) : run.scaled(x[i]);
          float y;
          const int b = bin_of(-d, bins, y);
          w[i] = by_count ? 0.f : expf(d);
          w[i] = in && b < lo ? w[i] : 0.f;
          count += in && b < lo;
          // (the last bins may reach beyond what was binned)
          if (in && d >= -near && (unsigned)(b - lo) <= (unsigned)(v.hi - lo)) list(x[i], first + i);
        }
        if (!by_count && v.what == kCollect) {
#pragma unroll
          for (int i = 0; i < kN; i += 2) over.add2(w[i], w[i + 1]);
        }
      });
      through = kMode == kSample && v.what == kGather;
      if (through) fetch(r + clusters);
      block_parts(sh, Fixed(), over, 0.f, 0, count);
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
        // (not with kGather: there is nothing above, and the other CTAs of a draw may be gone)
        if (v.what == kCollect && warp == 0) {
          Parts parts;
          parts.load(sh, ranks);
          parts.sum(sh);
        }
        // (in front of the barrier: from here on single warps set these and add to them)
        if (tid == 0) {
          sh.failed = sh.listed > kList;
          sh.border_x = kept.x;
          sh.border_id = kept.id;
          sh.total = 0;
        }
        if (tid < kMaxCluster * kSpWarps) sh.extra[tid] = 0ull;
        __syncthreads();
        const int n = sh.listed;
        const long long base = sh.sum_above, everything = sh.sum_all;
        const int more = sh.count_above;
        const Found found{v.what == kGather, by_count, stage == 0 ? k : kMaxVocab, top_p, min_p, n, more, base, everything};
        if (n <= kSmallList) {
          if (warp == 0) settle_few<kBf16, kMode>(sh, run, found, a, r);
        } else if (n <= kList) {
          settle<kBf16, kMode>(sh, run, found, a, r);
        }
        __syncthreads();
        for (int b = tid; b < kBins; b += kSpThreads) sh.hist[b] = 0u;  // (it lies over the list)
        if (tid == 0) {
          sh.listed = sh.count_all = 0;
          sh.sum_all = 0;
        }
      } else {
        for (int b = tid; b < kBins; b += kSpThreads) sh.hist[b] = 0u;
      }
      if (through) break;  // (nothing of this CTA is read any more)
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
  if (through) continue;

  // ---- what is kept ----
  auto weight = [&](float x, int id) -> float {  // 0: not kept
    if (!kept.has(x, id)) return 0.f;
    const float w = expf(run.scaled(x));
    return w < min_p ? 0.f : w;
  };
  const bool summed = total >= 0;  // (and then, for draws, the runs' sums are known too)
  if ((kMode == kSample || kMode == kProbs) && !summed) {
    Fixed f;
    run.each(kept.x, [&](float x, int id) { f.add(weight(x, id)); });
    int unused = 0;
    total = cluster_total(sh, turn, ranks, unused, f.value());
  }
  if constexpr (kMode == kSample) {
    // the kept weight of the runs before this warp's, and of its own
    long long before = 0, here;
    if (summed) {
      long long v[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int one = 2 * lane + e;
        v[e] = one < (int)ranks * kSpWarps
                   ? (long long)ld_peer64(&sh.wabove[one % kSpWarps], one / kSpWarps) + (long long)ld_peer64(&sh.extra[one], 0)
                   : 0;
      }
      const int own = (int)rank * kSpWarps + warp;
      before = warp_sum((2 * lane < own ? v[0] : 0) + (2 * lane + 1 < own ? v[1] : 0));
      here = __shfl_sync(0xffffffffu, own & 1 ? v[1] : v[0], own / 2);
    } else {
      for (uint32_t p = 0; p < rank; ++p) before += (long long)ld_peer64(&sh.sum[turn ^ 1], p);
      for (int w = 0; w < warp; ++w) before += sh.wsum[w];
      here = sh.wsum[warp];
    }
    const float log_total = log_sum(total);
    // one pass over the run, as long as a draw falls into what is left of it; lane q holds
    // where draws q and q + 32 fall
    static_assert(kMaxDraws == 64, "two draws a lane");
    long long at[2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
      at[e] = lane + 32 * e < a.draws ? place_of(sh.u[lane + 32 * e], total) - before : -1;
    constexpr int kAhead = 16 / kN;
    for (int s0 = 0; s0 < run.steps; s0 += kAhead) {
      if (!__any_sync(0xffffffffu, (at[0] >= 0 && at[0] < here) || (at[1] >= 0 && at[1] < here))) break;
      float x[kAhead][kN], w[kAhead][kN];
      Fixed f[kAhead];
      long long all[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        Vec v;
        v.read(run.at + min(s0 + j, run.steps - 1) * 32);
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          x[j][i] = v.x[i];
          const float one = expf(run.scaled(v.x[i]));
          w[j][i] = kept.has(v.x[i], run.id + (s0 + j) * kStep + i) && !(one < min_p) && s0 + j < run.steps ? one : 0.f;
        }
#pragma unroll
        for (int i = 0; i < kN; i += 2) f[j].add2(w[j][i], w[j][i + 1]);
      }
      Fixed together;
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        together.hi += f[j].hi;
        together.lo += f[j].lo;
      }
      const long long most = together.warp();
      if (!__any_sync(0xffffffffu, (at[0] >= 0 && at[0] < most) || (at[1] >= 0 && at[1] < most))) {
        at[0] -= most;
        at[1] -= most;
        here -= most;
        continue;
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) all[j] = f[j].warp();
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
          for (unsigned hits = __ballot_sync(0xffffffffu, at[e] >= 0 && at[e] < all[j]); hits; hits &= hits - 1) {
            const int q = __ffs(hits) - 1;
            const long long sum = f[j].value();
            long long upto = sum;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
              const long long o = __shfl_up_sync(0xffffffffu, upto, off);
              if (lane >= off) upto += o;
            }
            long long left = __shfl_sync(0xffffffffu, at[e], q) - (upto - sum);
            if (left >= 0 && left < sum) {
              int i = 0;
              float d = 0.f;
#pragma unroll
              for (int c = 0; c < kN; ++c) {
                const long long one = fixed(w[j][c]);
                if (i == c) {
                  d = run.scaled(x[j][c]);
                  if (left >= one && c + 1 < kN) {
                    left -= one;
                    ++i;
                  }
                }
              }
              a.tokens[(size_t)r * a.draws + q + 32 * e] = run.id + (s0 + j) * kStep + i;
              a.logprob[(size_t)r * a.draws + q + 32 * e] = d - log_total;
            }
          }
        at[0] -= all[j];
        at[1] -= all[j];
        here -= all[j];
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
  fetch(r + clusters);
  cluster_sync();
  }
}

// A row's logits on c CTAs: of a warp, and the bytes of a CTA.
template <bool kBf16>
void sp_share(int V, int c, int &per_warp, size_t &smem) {
  constexpr int kStep = 32 * SpVec<kBf16>::kN;
  per_warp = ((V + c * kSpWarps - 1) / (c * kSpWarps) + kStep - 1) / kStep * kStep;
  smem = (size_t)per_warp * kSpWarps * (kBf16 ? 2 : 4);
}

// How many clusters of c CTAs run at once, by c (asked once for each kernel, device and
// vocabulary; 0: too much shared memory).
struct Fits {
  const void *fn;
  int dev, V;
  int n[kMaxCluster + 1];
};
template <bool kBf16>
Fits clusters_at_once(const void *kernel, int V, cudaLaunchConfig_t cfg) {
  static std::mutex mu;
  static Fits known[32];
  static unsigned used = 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) dev = -1;
  std::lock_guard<std::mutex> lock(mu);
  for (const Fits &k : known)
    if (k.fn == kernel && k.dev == dev && k.V == V) return k;
  Fits f = {kernel, dev, V, {}};
  for (int c = 1; c <= kMaxCluster; ++c) {
    int per_warp;
    sp_share<kBf16>(V, c, per_warp, cfg.dynamicSmemBytes);
    if (cfg.dynamicSmemBytes > kMaxRowBytes) continue;
    cfg.attrs[0].val.clusterDim.x = c;
    cfg.gridDim = dim3((unsigned)c);
    if (cudaOccupancyMaxActiveClusters(&f.n[c], kernel, &cfg) != cudaSuccess || f.n[c] < 1) f.n[c] = sm_count() / c + 1;
  }
  return known[used++ % 32] = f;
}

template <bool kBf16, int kMode>
cudaError_t sp_launch(SpArgs &a, cudaStream_t s) {
  if (!set_smem((const void *)sampling_kernel<kBf16, kMode>, kMaxRowBytes)) return cudaErrorUnknown;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kSpThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const Fits fits = clusters_at_once<kBf16>((const void *)sampling_kernel<kBf16, kMode>, a.V, cfg);
  // As many clusters as run at once, each taking row after row.  A row costs some 20 us and
  // 1.4 us for each 1000 logits of a CTA (fitted to clusters of 1 to 8 CTAs over 8000 to
  // 262144 logits, 1 to 2000 rows; the choice is the fastest measured or within 2 us, the
  // timer's step, of it): few rows are spread over as many CTAs as can be, of many rows those
  // CTAs stay together that let the SMs fill up.  With top-p 0.9 and a cold L2: 64 rows of
  // 128256 bf16 logits 8 CTAs a row 102 us, 6 74 us; 508 such rows 8 CTAs 436 us, 4 328 us;
  // 508 rows of 8000 fp32 8 CTAs 217 us, 1 68 us.
  int most = 1;
  while (most < kMaxCluster && most * kSpWarps * 32 * SpVec<kBf16>::kN < a.V) ++most;
  int best = 0;
  int64_t least = 0;
  for (int c = most; c >= 1; --c) {
    if (fits.n[c] < 1) continue;
    const int64_t cost = (int64_t)((a.R + fits.n[c] - 1) / fits.n[c]) * (a.V / c + 14000);
    if (best == 0 || cost < least) {
      best = c;
      least = cost;
    }
  }
  if (best == 0) return cudaErrorUnknown;  // (kMaxCluster CTAs hold kMaxVocab logits)
  sp_share<kBf16>(a.V, best, a.per_warp, cfg.dynamicSmemBytes);
  attr[0].val.clusterDim.x = best;
  cfg.gridDim = dim3((unsigned)(a.R < fits.n[best] ? a.R : fits.n[best]) * best);
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
