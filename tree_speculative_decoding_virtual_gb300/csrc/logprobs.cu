// Log probabilities of given tokens, with the row's entropy and its k most
// probable tokens.
//
// For a row x of V logits and a token t, with m = max x, d = x - m and
// S = sum e^d:
//   logprob = d_t - log S,   entropy = log S - (sum e^d d) / S,
// and the k best tokens by (logit descending, id ascending), each with its
// log probability.  Written for what a verify step emits ("Speculative
// Decoding Hierárquico: Medusa, EAGLE-2 e Multi-Token Prediction": the target
// scores every node of the tree in one pass): the rows of the accepted path,
// read through path / accept_len / bonus without a round trip to the host, or
// any rows.
//
// One pass over the logits, so the kernel is bound by HBM (4 or 2 bytes a
// logit).  A cluster of up to 8 CTAs takes a row (one CTA where the rows alone
// fill the GPU); a CTA walks its slice in chunks of 4096 logits, 16 a thread.  With
// alternatives they come through a ring in shared memory, three chunks ahead: it keeps
// the stream going while the CTA settles its first chunk, and what passes the
// threshold is looked up there.  Without, and where rows are not aligned to 16
// bytes, the next 16 are on the way to registers.  (Rows of 128256 fp32, ring /
// registers: 1216 rows, 20 best 106 / 114 us, none 102 / 95; 508 rows, 1 best 51 / 49.)
//   reference  the maximum of the CTA's first chunk is the m of its sums; a warp
//              that meets a value more than 40 above its m moves it (e^40 leaves
//              fp32 sums far from overflow), whether it is among the k best or
//              not: with a masked first chunk m is the mask's value, and the
//              threshold, which all warps raise, says nothing about a warp's own m
//   threshold  the k-th largest of the 256 threads' maxima over the first chunk:
//              at least k values reach it, so only what does can be among the k
//              best.  For independent logits hardly more than k of 4096 do.
//   a chunk    S and T by thread, and what passes the threshold into a list in
//              shared memory; no barrier
//   settling   after chunks 4, 16, 64, ... and at the end the list is cut down to
//              its k best (ranks counted) and the k-th becomes the threshold:
//              later ids lose its ties, so from then on only more passes
// Values that equal the first threshold are listed apart: where there are more
// of them than that list holds (masked vocabularies), the first ones in id order
// are looked up.  Where more pass than the list holds, the slice is taken again
// at the end, chunk by chunk, each chunk's k-th largest value found bit by bit
// (508 rows of 128256 with the first 4096 logits masked and a tenth of the others
// not: 0.9 ms; with a tenth of all, as long as without a mask).
// The CTAs' results meet through distributed shared memory; nothing is written
// but the outputs.

#include <cuda_bf16.h>

#include "sm100_ptx.cuh"
#include "tsd_common.cuh"

namespace tsd {
namespace {

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kPerThread = 16;
constexpr int kChunk = kLpThreads * kPerThread;  // logits held at a time
constexpr int kMaxTop = 32;
constexpr int kLpRing = 3 * kChunk * 4;  // bytes of a CTA's copies in flight
constexpr int kCap = 512;      // candidates the list holds (kMaxTop more for ties)
constexpr int kTies = 64;      // values equal to the threshold that are listed
constexpr float kMove = 40.f;  // the reference follows a value so far above it
constexpr float kLog2e = 1.4426950408889634f;

struct LpArgs {
  const void *logits;
  const int32_t *tokens;
  // explicit rows: rows [R] or null (row r); path mode: the rest
  const int32_t *rows;
  const int32_t *path, *accept_len, *bonus, *err;
  int N_max, D_max;
  int64_t num_rows;
  int V, k, per;  // per: logits of one CTA of the cluster, a multiple of 8
  int32_t *emitted;
  float *logprob, *entropy;
  int32_t *top_ids;
  float *top_lp;
  int32_t *status;
};

struct LpShared {
  uint32_t sorted[kLpWarps][32];  // the threads' first maxima, descending by warp
  float sum[kLpWarps], dsum[kLpWarps], ref[kLpWarps];
  alignas(16) unsigned long long cand[kCap + kTies];
  int tie[kTies];
  int found[kLpWarps][kMaxTop], n_found[kLpWarps];
  int n_cand, n_tie, lost;  // lost: more passed than the list holds
  uint32_t thr;
  int reduce[kLpWarps];
  alignas(16) float m;
  float S, T, xt;  // the CTA's reference, sum e^d, sum e^d d, and the token's logit
};

// Integers that order as the floats do; both zeros alike, NaN above all.
__device__ __forceinline__ uint32_t ordered(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
  if (o == 0xFFFFFFFFu) return __uint_as_float(0x7FC00000u);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
__device__ __forceinline__ unsigned long long lp_key(uint32_t ord, int id) {
  return ((unsigned long long)ord << 32) | (uint32_t)~id;
}

__device__ __forceinline__ unsigned long long f2_mul(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// NaN where an operand is one
__device__ __forceinline__ float fmax3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}
__device__ __forceinline__ int block_sum(int x, int *buf) {
  x = __reduce_add_sync(0xffffffffu, x);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
  __syncthreads();
  int s = 0;
#pragma unroll
  for (int w = 0; w < kLpWarps; ++w) s += buf[w];
  return s;
}
__device__ __forceinline__ int block_min(int x, int *buf) {
  x = __reduce_min_sync(0xffffffffu, x);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
  __syncthreads();
  int s = buf[0];
#pragma unroll
  for (int w = 1; w < kLpWarps; ++w) s = min(s, buf[w]);
  return s;
}

// Where a thread's e-th logit of a chunk lies.
template <bool kBf16, bool kVec>
__device__ __forceinline__ int chunk_pos(int e, int tid) {
  constexpr int kW = kVec ? (kBf16 ? 8 : 4) : 1;
  return ((e / kW) * kLpThreads + tid) * kW + e % kW;
}

// The thread's part of [c0, end) as loaded: 16 fp32 words, or 8 of bf16 pairs
// (one word a logit without vector loads); -inf past the end.
template <bool kBf16, bool kVec>
struct LpRaw {
  static constexpr int kWords = kBf16 && kVec ? kPerThread / 2 : kPerThread;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const void *row, int c0, int end, int tid) {
    if constexpr (!kVec) {
#pragma unroll
      for (int e = 0; e < kPerThread; ++e) {
        const int i = c0 + chunk_pos<kBf16, kVec>(e, tid);
        if (kBf16)
          w[e] = i < end ? (uint32_t)__ldcs(reinterpret_cast<const uint16_t *>(row) + i) << 16 : 0xFF800000u;
        else
          w[e] = i < end ? __ldcs(reinterpret_cast<const uint32_t *>(row) + i) : 0xFF800000u;
      }
    } else {
      constexpr int kW = kBf16 ? 8 : 4;
      constexpr uint32_t none = kBf16 ? 0xFF80FF80u : 0xFF800000u;
#pragma unroll
      for (int g = 0; g < kPerThread / kW; ++g) {
        const int i = c0 + chunk_pos<kBf16, kVec>(g * kW, tid);
        const uint4 v = i < end ? __ldcs(reinterpret_cast<const uint4 *>(row) + i / kW)
                                : make_uint4(none, none, none, none);
        w[4 * g] = v.x;
        w[4 * g + 1] = v.y;
        w[4 * g + 2] = v.z;
        w[4 * g + 3] = v.w;
      }
    }
  }
  // The same part by way of shared memory: every thread copies, and later reads,
  // its own 16 bytes of each group, so that no barrier is needed.
  static constexpr int kGroups = kWords / 4;
  static constexpr int kStage = kLpThreads * kGroups * 16;
  static constexpr int kStages = kLpRing / kStage;
  static __device__ __forceinline__ void fetch(uint32_t stage, const void *row, int c0, int end, int tid) {
    constexpr int kW = kBf16 ? 8 : 4;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const int i = c0 + chunk_pos<kBf16, kVec>(g * kW, tid);
      if (i < end) sm100::cp_async_16(stage + (g * kLpThreads + tid) * 16, reinterpret_cast<const uint4 *>(row) + i / kW);
    }
    asm volatile("cp.async.commit_group;\n" ::: "memory");
  }
  __device__ __forceinline__ void read(const uint8_t *stage, int c0, int end, int tid) {
    constexpr int kW = kBf16 ? 8 : 4;
    constexpr uint32_t none = kBf16 ? 0xFF80FF80u : 0xFF800000u;
    asm volatile("cp.async.wait_group %0;\n" ::"n"(kStages - 1) : "memory");
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const int i = c0 + chunk_pos<kBf16, kVec>(g * kW, tid);
      uint4 v = *reinterpret_cast<const uint4 *>(stage + (g * kLpThreads + tid) * 16);
      if (i >= end) v = make_uint4(none, none, none, none);
      w[4 * g] = v.x;
      w[4 * g + 1] = v.y;
      w[4 * g + 2] = v.z;
      w[4 * g + 3] = v.w;
    }
  }
  static __device__ __forceinline__ float one(const uint8_t *stage, int e, int tid) {
    constexpr int kW = kBf16 ? 8 : 4;
    const uint8_t *p = stage + (e / kW * kLpThreads + tid) * 16;
    if constexpr (kBf16)
      return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(p)[e % kW] << 16);
    else
      return reinterpret_cast<const float *>(p)[e % kW];
  }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (kBf16 && kVec)
      return __uint_as_float((e & 1) ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16);
    else
      return __uint_as_float(w[e]);
  }
};

template <bool kBf16>
__device__ __forceinline__ float one_logit(const void *row, int i) {
  if constexpr (kBf16)
    return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(row)[i] << 16);
  else
    return reinterpret_cast<const float *>(row)[i];
}

// Keeps the k best of sh.cand[0, n), descending, in place; returns how many
// there are.  Called by the whole block with the buffer complete; leaves it
// complete.
__device__ __forceinline__ int keep_best(LpShared &sh, int n, int k) {
  __syncthreads();
  constexpr int kMine = (kCap + kTies + kLpThreads - 1) / kLpThreads;
  unsigned long long mine[kMine];
  int rank[kMine];
#pragma unroll
  for (int q = 0; q < kMine; ++q) {
    const int c = threadIdx.x + q * kLpThreads;
    mine[q] = c < n ? sh.cand[c] : 0ull;
    rank[q] = kCap;
    if (c < n) {
      int r = 0, o = 0;
#pragma unroll 4
      for (; o + 1 < n; o += 2) {  // two at a time
        const ulonglong2 two = *reinterpret_cast<const ulonglong2 *>(sh.cand + o);
        r += (two.x > mine[q] ? 1 : 0) + (two.y > mine[q] ? 1 : 0);
      }
      if (o < n) r += sh.cand[o] > mine[q] ? 1 : 0;
      rank[q] = r;
    }
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kMine; ++q)
    if (rank[q] < k) sh.cand[rank[q]] = mine[q];
  const int left = min(n, k);
  if (threadIdx.x == 0) sh.n_cand = left;
  __syncthreads();
  return left;
}

// The k best of a slice in which more values pass the threshold than the list
// holds: chunk by chunk, the k-th largest value T of the chunk bit by bit (the
// largest T that k values reach), then T's ties in id order.  Out of line: it is
// rare, and its registers are not the main path's.
template <bool kBf16, bool kVec>
__device__ __noinline__ void select_exact(LpShared &sh, const void *row, int first, int last, int k) {
  const int tid = threadIdx.x;
  int held = 0;
  for (int c0 = first; c0 < last; c0 += kChunk) {
    const int end = min(last, c0 + kChunk);
    LpRaw<kBf16, kVec> x;
    x.load(row, c0, end, tid);
    uint32_t T = 0;
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t t = T | (1u << bit);
      int mine = 0;
#pragma unroll
      for (int e = 0; e < kPerThread; ++e)
        mine += (c0 + chunk_pos<kBf16, kVec>(e, tid) < end && ordered(x.get(e)) >= t) ? 1 : 0;
      if (block_sum(mine, sh.reduce) >= k) T = t;
    }
    __syncthreads();
    if (tid == 0) sh.n_cand = held;
    __syncthreads();
    int above = 0;
#pragma unroll
    for (int e = 0; e < kPerThread; ++e) {
      const int id = c0 + chunk_pos<kBf16, kVec>(e, tid);
      const uint32_t o = ordered(x.get(e));
      if (id < end && o > T) {  // fewer than k of them
        sh.cand[atomicAdd(&sh.n_cand, 1)] = lp_key(o, id);
        ++above;
      }
    }
    int left = k - block_sum(above, sh.reduce);
    int after = -1;  // the last tie taken
    for (; left > 0; --left) {
      int id = 0x7FFFFFFF;
#pragma unroll
      for (int e = 0; e < kPerThread; ++e) {
        const int i = c0 + chunk_pos<kBf16, kVec>(e, tid);
        if (i < end && i > after && ordered(x.get(e)) == T) id = min(id, i);
      }
      id = block_min(id, sh.reduce);
      if (id == 0x7FFFFFFF) break;
      if (tid == 0) sh.cand[sh.n_cand++] = lp_key(T, id);
      after = id;
    }
    __syncthreads();
    held = keep_best(sh, sh.n_cand, k);
  }
}

// The first `need` (at most 32) ids of [first, last) whose logit equals the
// threshold, appended to the list: every warp looks through its share from the
// front, then the shares' finds are taken in order.
template <bool kBf16>
__device__ __noinline__ void find_ties(LpShared &sh, const void *row, int first, int last, int need) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t thr = sh.thr;
  const int share = (last - first + kLpWarps - 1) / kLpWarps;
  const int a = first + warp * share, z = min(last, a + share);
  int got = 0;
  for (int i0 = a; i0 < z && got < need; i0 += 32) {
    const int i = i0 + lane;
    const bool hit = i < z && ordered(one_logit<kBf16>(row, i)) == thr;
    const unsigned hits = __ballot_sync(0xffffffffu, hit);
    const int at = got + __popc(hits & ((1u << lane) - 1u));
    if (hit && at < need) sh.found[warp][at] = i;
    got += __popc(hits);
  }
  if (lane == 0) sh.n_found[warp] = min(got, need);
  __syncthreads();
  if (threadIdx.x == 0) {
    int n = sh.n_cand;
    for (int w = 0; w < kLpWarps && need > 0; ++w)
      for (int f = 0; f < sh.n_found[w] && need > 0; ++f, --need) sh.cand[n++] = lp_key(thr, sh.found[w][f]);
    sh.n_cand = n;
  }
  __syncthreads();
}

// Cuts the list down to the k best of [first, end), the part of the slice seen so
// far, and makes the k-th the threshold when there are k.  `settled`: the
// threshold is such a one, and its ties are not wanted.  Returns whether it is
// now.  Called by the whole block.
template <bool kBf16>
__device__ __forceinline__ bool settle(LpShared &sh, const void *row, int first, int end, int k, bool settled) {
  __syncthreads();
  int n = sh.n_cand;
  const int ties = sh.n_tie;
  __syncthreads();
  if (n > kCap) {  // (stays lost; the list goes on from nothing)
    if (threadIdx.x == 0) {
      sh.lost = 1;
      sh.n_cand = 0;
    }
    __syncthreads();
    return settled;
  }
  if (!settled && n < k) {
    if (ties > kTies) {
      find_ties<kBf16>(sh, row, first, end, k - n);
    } else {
      if (threadIdx.x < ties) sh.cand[n + threadIdx.x] = lp_key(sh.thr, sh.tie[threadIdx.x]);
      if (threadIdx.x == 0) sh.n_cand = n + ties;
      __syncthreads();
    }
    n = sh.n_cand;
  }
  n = keep_best(sh, n, k);
  if (n < k) return settled;
  if (threadIdx.x == 0) sh.thr = (uint32_t)(sh.cand[k - 1] >> 32);
  __syncthreads();
  return true;
}

// Output row r: its row of logits and its token; false where there is none
// (the outputs are then the defaults).
__device__ __forceinline__ bool lp_resolve(const LpArgs &a, int r, int64_t &row, int &token,
                                           bool &bad) {
  bad = false;
  if (!a.path) {
    row = a.rows ? (int64_t)a.rows[r] : (int64_t)r;
    token = a.tokens[r];
    if (row == -1) return false;
    bad = row < 0 || row >= a.num_rows;
    return !bad;
  }
  const int cols = a.D_max + 1;
  const int b = r / cols, s = r % cols;
  if (a.err && a.err[b] != 0) return false;
  const int A = a.accept_len[b];
  if (A < 0 || A > a.D_max) {
    bad = s == 0;
    return false;
  }
  if (s > A) return false;
  const int node = a.path[r] - 1;
  const int next = s < A ? a.path[r + 1] - 1 : 0;
  if (node < 0 || node >= a.N_max || next < 0 || next >= a.N_max) {
    bad = true;
    return false;
  }
  row = (int64_t)b * a.N_max + node;
  token = s < A ? a.tokens[(int64_t)b * a.N_max + next] : a.bonus[b];
  return true;
}

template <bool kBf16, bool kVec, bool kRing>
__global__ void __launch_bounds__(kLpThreads, 4) logprobs_kernel(const LpArgs a) {
  using namespace sm100;
  __shared__ LpShared sh;
  extern __shared__ __align__(16) uint8_t ring[];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = cluster_ctarank(), ctas = cluster_nctarank();
  const int r = blockIdx.x / ctas;
  const int k = a.k;
  int64_t row = 0;
  int token = -1;
  bool bad;
  if (!lp_resolve(a, r, row, token, bad)) {  // the whole cluster leaves
    if (rank == 0) {
      if (tid == 0) {
        a.logprob[r] = 0.f;
        if (a.entropy) a.entropy[r] = 0.f;
        if (a.emitted) a.emitted[r] = -1;
        if (bad && a.status) atomicOr(a.status, TSD_STATUS_BAD_PATH);
      }
      if (tid < k) {
        a.top_ids[(size_t)r * k + tid] = -1;
        a.top_lp[(size_t)r * k + tid] = -INFINITY;
      }
    }
    return;
  }
  const void *src = reinterpret_cast<const char *>(a.logits) + (size_t)row * a.V * (kBf16 ? 2 : 4);
  if (tid == 0) {
    sh.n_cand = 0;
    sh.n_tie = 0;
    sh.lost = 0;
    sh.xt = -INFINITY;
  }
  const int first = rank * a.per, last = min(a.V, first + a.per);
  if (first < last) {
    // the logit asked for, read apart from the stream (its line is in flight
    // anyway)
    if (tid == 0 && token >= first && token < last) sh.xt = one_logit<kBf16>(src, token);
    using Raw = LpRaw<kBf16, kVec>;
    Raw x, next;
    const uint32_t ring_at = smem_addr(ring);
    if constexpr (kRing) {
#pragma unroll
      for (int i = 0; i < Raw::kStages; ++i)  // one group a stage, an empty one past the end
        Raw::fetch(ring_at + i * Raw::kStage, src, first + i * kChunk, last, tid);
      x.read(ring, first, last, tid);
    } else {
      x.load(src, first, min(last, first + kChunk), tid);
    }
    // (fmaxf drops a NaN: a threshold may be too low, not too high, and the sums
    // keep the NaN)
    float top = -INFINITY;
#pragma unroll
    for (int e = 0; e < kPerThread; ++e) top = fmaxf(top, x.get(e));
    uint32_t o = ordered(top);
    if (k > 0) {  // descending over the warp's lanes
#pragma unroll
      for (int size = 2; size <= 32; size <<= 1) {
#pragma unroll
        for (int step = size >> 1; step; step >>= 1) {
          const uint32_t other = __shfl_xor_sync(0xffffffffu, o, step);
          const bool high = ((lane & step) == 0) == ((lane & size) == 0 || size == 32);
          o = high ? max(o, other) : min(o, other);
        }
      }
    } else {
      o = __reduce_max_sync(0xffffffffu, o);
    }
    sh.sorted[warp][lane] = o;
    __syncthreads();
    float m = unordered(__reduce_max_sync(0xffffffffu, sh.sorted[lane & (kLpWarps - 1)][0]));
    if (lane < k) {
      // rank of this thread's maximum among all 256 (equal ones by warp)
      int above = lane;
      for (int w = 0; w < kLpWarps; ++w) {
        if (w == warp) continue;
        int lo = 0, hi = 32;
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          const uint32_t v = sh.sorted[w][mid];
          if (v > o || (v == o && w < warp)) lo = mid + 1; else hi = mid;
        }
        above += lo;
      }
      if (above == k - 1) sh.thr = o;
    }
    __syncthreads();
    // What reaches `gate` is looked at: it may be listed (it reaches the threshold; a
    // settled one it has to pass), or it moves the reference (it is above m + 40, as
    // rounded: for a mask of -1e30 above m, for one of -inf anything else).  Both
    // bounds can be beyond the largest number; then +inf itself is looked at.
    uint32_t thr_ord = k > 0 ? sh.thr : 0xFFFFFFFFu;
    bool settled = false;
    auto gate_of = [&] {
      const float moves = unordered(ordered(m + kMove) + 1u);
      const float lists = unordered(settled && thr_ord != 0xFFFFFFFFu ? thr_ord + 1u : thr_ord);
      return fminf(fminf(lists, moves), INFINITY);  // (of a NaN and a number the number)
    };
    float gate = gate_of();
    int next_settle = first + 4 * kChunk;

    unsigned long long S2 = 0ull, T2 = 0ull;  // two sums each
    int stage = 0;  // x's
    for (int c0 = first; c0 < last; c0 += kChunk) {
      const int end = min(last, c0 + kChunk);
      if constexpr (!kRing) {
        if (end < last) next.load(src, end, min(last, end + kChunk), tid);
      }
      float most = x.get(0);
#pragma unroll
      for (int e = 1; e + 1 < kPerThread; e += 2) most = fmax3_nan(most, x.get(e), x.get(e + 1));
      const bool below = fmax3_nan(most, most, x.get(kPerThread - 1)) < gate;  // (false for a NaN)
      if (!below) {
        uint32_t mine = 0u;
#pragma unroll
        for (int e = 0; e < kPerThread; ++e) mine |= (x.get(e) < gate ? 0u : 1u) << e;
        top = -INFINITY;
        // (the few that pass are read again: indexing the registers would spill them)
        for (; mine; mine &= mine - 1) {
          const int e = __ffs(mine) - 1, id = c0 + chunk_pos<kBf16, kVec>(e, tid);
          if (id >= end) continue;
          const float v = kRing ? Raw::one(ring + stage * Raw::kStage, e, tid) : one_logit<kBf16>(src, id);
          const uint32_t vo = ordered(v);
          top = fmaxf(top, v);
          if (k == 0) continue;
          if (vo > thr_ord) {
            const int at = atomicAdd(&sh.n_cand, 1);
            if (at < kCap) sh.cand[at] = lp_key(vo, id);
          } else if (vo == thr_ord && !settled && sh.n_tie <= kTies) {
            const int at = atomicAdd(&sh.n_tie, 1);
            if (at < kTies) sh.tie[at] = id;
          }
        }
      }
      // (x and what was read again are used: the stage can be refilled)
      if constexpr (kRing)
        Raw::fetch(ring_at + stage * Raw::kStage, src, c0 + Raw::kStages * kChunk, last, tid);
      __syncwarp();
      if (__any_sync(0xffffffffu, !below && top > m + kMove)) {  // the warp's reference follows
        const float up = unordered(__reduce_max_sync(0xffffffffu, ordered(below ? -INFINITY : top)));
        const float f = m == -INFINITY ? 0.f : ex2_approx((m - up) * kLog2e);
        const float2 s = f2_unpack(S2), t = f2_unpack(T2);
        T2 = f == 0.f ? 0ull : f2_pack(f * (t.x + s.x * (m - up)), f * (t.y + s.y * (m - up)));
        S2 = f2_pack(f * s.x, f * s.y);
        m = up;
        gate = gate_of();
      }
      // d = -200 stands for every d that e^d rounds to zero for, -inf included; a
      // NaN reaches S and T through e^d, and so does +inf (m = +inf: inf - inf)
      const float base = m == -INFINITY ? 0.f : -m;
      const unsigned long long base2 = f2_pack(base, base), log2e = f2_pack(kLog2e, kLog2e);
#pragma unroll
      for (int e = 0; e < kPerThread; e += 2) {
        const unsigned long long d2 = f2_add(f2_pack(x.get(e), x.get(e + 1)), base2);
        const float2 d = f2_unpack(d2), t = f2_unpack(f2_mul(d2, log2e));
        const unsigned long long p = f2_pack(ex2_approx(t.x), ex2_approx(t.y));
        S2 = f2_add(S2, p);
        T2 = f2_fma(p, f2_pack(fmaxf(d.x, -200.f), fmaxf(d.y, -200.f)), T2);
      }
      if (k > 0 && (end == next_settle || end == last)) {
        settled = settle<kBf16>(sh, src, first, end, k, settled);
        if (settled) {
          thr_ord = sh.thr;
          gate = gate_of();
        }
        next_settle = first + 4 * (next_settle - first);
      }
      if constexpr (kRing) {
        if (++stage == Raw::kStages) stage = 0;
        if (end < last) x.read(ring + stage * Raw::kStage, end, last, tid);
      } else {
        x = next;
      }
    }
    if constexpr (kRing) cp_async_wait_all();
    float S = warp_sum(f2_unpack(S2).x + f2_unpack(S2).y);
    float T = warp_sum(f2_unpack(T2).x + f2_unpack(T2).y);
    if (lane == 0) {
      sh.sum[warp] = S;
      sh.dsum[warp] = T;
      sh.ref[warp] = m;
    }
    __syncthreads();
    if (tid == 0) {
      float M = -INFINITY;
      for (int w = 0; w < kLpWarps; ++w) M = fmaxf(M, sh.ref[w]);
      S = 0.f;
      T = 0.f;
      for (int w = 0; w < kLpWarps; ++w) {
        const float r = sh.ref[w];
        // (a reference of -inf: nothing but -inf, or NaN, since all else moves it)
        const float f = r == M || r == -INFINITY ? 1.f : ex2_approx((r - M) * kLog2e);
        const float by = r == M || r == -INFINITY ? 0.f : r - M;
        S += f * sh.sum[w];
        T += f == 0.f ? 0.f : f * (sh.dsum[w] + sh.sum[w] * by);
      }
      sh.m = M;
      sh.S = S;
      sh.T = T;
    }
    if (sh.lost) {  // (the barriers above made it visible)
      __syncthreads();
      select_exact<kBf16, kVec>(sh, src, first, last, k);
    }
  } else if (tid == 0) {
    sh.m = -INFINITY;
    sh.S = 0.f;
    sh.T = 0.f;
  }
  __syncthreads();
  if (ctas > 1) {
    cluster_arrive();
    cluster_wait();
  }
  if (rank == 0) {
    // the whole row's statistics (each thread the same), from every CTA's
    float M = -INFINITY, xt = -INFINITY;
    bool nan = false;
    float cm[8], cS[8], cT[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      if (c >= ctas) break;
      const float4 v = ld_dsmem_f4(smem_addr(&sh.m), c);
      cm[c] = v.x;
      cS[c] = v.y;
      cT[c] = v.z;
      nan = nan || v.y != v.y;
      M = fmaxf(M, v.x);
      if (token >= c * a.per && token < (c + 1) * a.per) xt = v.w;
    }
    float S = 0.f, T = 0.f;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      if (c >= ctas) break;
      if (cm[c] == -INFINITY) continue;
      const float f = ex2_approx((cm[c] - M) * kLog2e);
      S += f * cS[c];
      T += f == 0.f ? 0.f : f * (cT[c] + cS[c] * (cm[c] - M));
    }
    if (nan) S = T = __uint_as_float(0x7FC00000u);
    const float logS = logf(S);
    const bool empty = M == -INFINITY && !nan;  // every logit is -inf
    if (tid == 0) {
      a.logprob[r] = empty || token < 0 || token >= a.V ? -INFINITY : (xt - M) - logS;
      if (a.entropy) a.entropy[r] = empty ? 0.f : logS - T / S;
      if (a.emitted) a.emitted[r] = token;
    }
    // the CTAs' sorted lists: a candidate's rank is the number of larger keys
    for (int c = warp; c < ctas; c += kLpWarps) {
      // lane l reads entries 2 (l % 16) and 2 (l % 16) + 1 of the list of CTA c
      if (lane < kMaxTop / 2) {
        const float4 v = ld_dsmem_f4(smem_addr(&sh.cand[lane * 2]), c);
        const unsigned long long k0 =
            (unsigned long long)__float_as_uint(v.x) | ((unsigned long long)__float_as_uint(v.y) << 32);
        const unsigned long long k1 =
            (unsigned long long)__float_as_uint(v.z) | ((unsigned long long)__float_as_uint(v.w) << 32);
        sh.cand[c * kMaxTop + lane * 2] = k0;
        sh.cand[c * kMaxTop + lane * 2 + 1] = k1;
      }
    }
    __syncthreads();
    for (int x = tid; x < ctas * k; x += kLpThreads) {
      const int c = x / k, i = x % k;
      const int mine_n = min(k, max(0, min(a.V, (c + 1) * a.per) - c * a.per));
      if (i >= mine_n) continue;
      const unsigned long long key = sh.cand[c * kMaxTop + i];
      int rk = i;
      for (int o = 0; o < ctas; ++o) {
        if (o == c) continue;
        int lo = 0, hi = min(k, max(0, min(a.V, (o + 1) * a.per) - o * a.per));
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (sh.cand[o * kMaxTop + mid] > key) lo = mid + 1; else hi = mid;
        }
        rk += lo;
      }
      if (rk < k) {
        const float xv = unordered((uint32_t)(key >> 32));
        a.top_ids[(size_t)r * k + rk] = (int)~(uint32_t)key;
        a.top_lp[(size_t)r * k + rk] = empty ? -INFINITY : (xv - M) - logS;
      }
    }
  }
  if (ctas > 1) {  // no CTA leaves while rank 0 may still read its shared memory
    cluster_arrive();
    cluster_wait();
  }
}

template <bool kBf16, bool kVec, bool kRing>
cudaError_t lp_launch(const LpArgs &a, int R, int ctas, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas * (unsigned)R);
  cfg.blockDim = dim3(kLpThreads);
  if (kRing) {
    if (!set_smem((const void *)logprobs_kernel<kBf16, kVec, kRing>, kLpRing)) return cudaErrorUnknown;
    cfg.dynamicSmemBytes = kLpRing;
  }
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, logprobs_kernel<kBf16, kVec, kRing>, a);
}

int lp_run(LpArgs &a, int R, int bf16, tsd_stream_t stream) {
  // CTAs of a row: as many (a power of two, up to 8, at most one a chunk) as leave
  // no SM with two; a slice's first chunk and its end cost more than sharing saves.
  // Measured (128256 fp32 logits, 20 best; 1, 2, 4, 8 CTAs): 8 rows 22.6, 17.5, 14.4,
  // 13.4 us; 38 rows 24.1, 18.3, 16.8, 19.7; 76 rows 24.1, 19.3, 23.6, 29.7; 152 rows
  // 25.6, 24.4, 34.6; 304 rows 33.3, 37.7.
  int ctas = 1;
  while (ctas < 8 && (int64_t)ctas * kChunk < a.V && 2ll * ctas * R <= sm_count()) ctas *= 2;
  a.per = ((a.V + ctas - 1) / ctas + 7) / 8 * 8;
  const bool vec = aligned(a.logits, 16) && a.V % (bf16 ? 8 : 4) == 0;
  const cudaStream_t s = as_cuda(stream);
  const bool ring = vec && a.k > 0;
  const cudaError_t e = bf16 ? (ring  ? lp_launch<true, true, true>(a, R, ctas, s)
                                : vec ? lp_launch<true, true, false>(a, R, ctas, s)
                                      : lp_launch<true, false, false>(a, R, ctas, s))
                             : (ring  ? lp_launch<false, true, true>(a, R, ctas, s)
                                : vec ? lp_launch<false, true, false>(a, R, ctas, s)
                                      : lp_launch<false, false, false>(a, R, ctas, s));
  return e == cudaSuccess ? TSD_OK : TSD_ERR_CUDA;
}

int lp_check(int64_t num_rows, int R, int V, int k) {
  if (num_rows < 0 || R < 0 || V < 1 || k < 0) return TSD_ERR_ARG;
  if (R > (1 << 27) || V > (1 << 24) || k > kMaxTop || k > V) return TSD_ERR_LIMIT;
  return TSD_OK;
}

}  // namespace
}  // namespace tsd

TSD_API int tsd_token_logprobs(const void *logits, int bf16, const int32_t *tokens,
                               const int32_t *rows, int R, int64_t num_rows, int V, int k,
                               float *logprob, float *entropy, int32_t *top_ids,
                               float *top_logprobs, int32_t *status, tsd_stream_t stream) {
  using namespace tsd;
  const int rc = lp_check(num_rows, R, V, k);
  if (rc != TSD_OK || R == 0) return rc;
  if (!logits || !tokens || !logprob || (k > 0 && (!top_ids || !top_logprobs))) return TSD_ERR_ARG;
  if (!rows && R > num_rows) return TSD_ERR_ARG;
  if (!aligned(logits, bf16 ? 2 : 4)) return TSD_ERR_ARG;
  LpArgs a = {};
  a.logits = logits;
  a.tokens = tokens;
  a.rows = rows;
  a.num_rows = num_rows;
  a.V = V;
  a.k = k;
  a.logprob = logprob;
  a.entropy = entropy;
  a.top_ids = top_ids;
  a.top_lp = top_logprobs;
  a.status = status;
  return lp_run(a, R, bf16, stream);
}

TSD_API int tsd_tree_path_logprobs(const void *logits, int bf16, const int32_t *tokens,
                                   const int32_t *path, const int32_t *accept_len,
                                   const int32_t *bonus, const int32_t *err, int B, int N_max, int V,
                                   int D_max, int k, int32_t *emitted, float *logprob, float *entropy,
                                   int32_t *top_ids, float *top_logprobs, int32_t *status,
                                   tsd_stream_t stream) {
  using namespace tsd;
  if (B < 0) return TSD_ERR_ARG;
  if (N_max < 1 || N_max > kMaxNodes || D_max < 0 || D_max > kMaxDepth || B > 65535) return TSD_ERR_LIMIT;
  if ((int64_t)B * (D_max + 1) > 65535) return TSD_ERR_LIMIT;
  const int rc = lp_check((int64_t)B * N_max, B * (D_max + 1), V, k);
  if (rc != TSD_OK || B == 0) return rc;
  if (!logits || !tokens || !path || !accept_len || !bonus || !emitted || !logprob ||
      (k > 0 && (!top_ids || !top_logprobs)))
    return TSD_ERR_ARG;
  if (!aligned(logits, bf16 ? 2 : 4)) return TSD_ERR_ARG;
  LpArgs a = {};
  a.logits = logits;
  a.tokens = tokens;
  a.path = path;
  a.accept_len = accept_len;
  a.bonus = bonus;
  a.err = err;
  a.N_max = N_max;
  a.D_max = D_max;
  a.num_rows = (int64_t)B * N_max;
  a.V = V;
  a.k = k;
  a.emitted = emitted;
  a.logprob = logprob;
  a.entropy = entropy;
  a.top_ids = top_ids;
  a.top_lp = top_logprobs;
  a.status = status;
  return lp_run(a, B * (D_max + 1), bf16, stream);
}
