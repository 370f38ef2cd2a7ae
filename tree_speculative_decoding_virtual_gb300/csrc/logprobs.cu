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
// logit).  A cluster of up to 8 CTAs takes a row; a CTA holds kChunk logits at
// a time in registers (32 a thread), which serve the maximum, the sums and the
// selection without a second read.  Selection: the minimum of the maxima of 32
// disjoint groups of the chunk is at most its 32nd largest value, so only
// values at or above it can be among the k <= 32 best; for independent logits
// about 110 of 8192 remain, and their ranks are counted in shared memory.
// Rows with long ties (masked vocabularies) can leave more than the buffer
// holds: then the k-th largest value is found bit by bit and its ties are
// taken in id order.  The CTAs' results meet through distributed shared
// memory; nothing is written but the outputs.

#include <cuda_bf16.h>

#include "sm100_ptx.cuh"
#include "tsd_common.cuh"

namespace tsd {
namespace {

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kPerThread = 32;
constexpr int kChunk = kLpThreads * kPerThread;  // logits held at a time
constexpr int kMaxTop = 32;
constexpr int kGroups = 32;  // groups of 8 threads
constexpr int kCap = 512;    // candidates the shared buffer holds
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
  uint32_t group_max[kGroups];
  float sum[kLpWarps], dsum[kLpWarps];
  unsigned long long cand[kCap];
  alignas(16) unsigned long long best[kMaxTop];  // this CTA's best so far, descending
  int n_cand, n_best;
  int reduce[kLpWarps];
  alignas(16) float m;
  float S, T, xt;  // running: maximum, sum e^d, sum e^d d, the token's logit
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

// The thread's logits of [c0, end); -inf past it.
template <bool kBf16, bool kVec>
__device__ __forceinline__ void load_chunk(const void *row, int c0, int end, int tid,
                                           float (&x)[kPerThread]) {
  constexpr int kW = kVec ? (kBf16 ? 8 : 4) : 1;
  if constexpr (!kVec) {
#pragma unroll
    for (int e = 0; e < kPerThread; ++e) {
      const int i = c0 + chunk_pos<kBf16, kVec>(e, tid);
      if (kBf16) {
        const uint16_t *p = reinterpret_cast<const uint16_t *>(row);
        x[e] = i < end ? __uint_as_float((uint32_t)__ldcs(p + i) << 16) : -INFINITY;
      } else {
        const float *p = reinterpret_cast<const float *>(row);
        x[e] = i < end ? __ldcs(p + i) : -INFINITY;
      }
    }
  } else {
    uint4 w[kPerThread / kW];
#pragma unroll
    for (int g = 0; g < kPerThread / kW; ++g) {
      const int i = c0 + chunk_pos<kBf16, kVec>(g * kW, tid);
      const uint32_t none = kBf16 ? 0xFF80FF80u : 0xFF800000u;
      w[g] = i < end ? __ldcs(reinterpret_cast<const uint4 *>(row) + i / kW)
                     : make_uint4(none, none, none, none);
    }
#pragma unroll
    for (int g = 0; g < kPerThread / kW; ++g) {
      const uint32_t u[4] = {w[g].x, w[g].y, w[g].z, w[g].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (kBf16) {
          x[g * kW + 2 * j] = __uint_as_float(u[j] << 16);
          x[g * kW + (2 * j + 1) % kW] = __uint_as_float(u[j] & 0xFFFF0000u);
        } else {
          x[g * kW + j] = __uint_as_float(u[j]);
        }
      }
    }
  }
}

// Merges the chunk's candidates with the best so far (all of them in
// sh.cand[0, n)) into sh.best.
__device__ __forceinline__ void rank_candidates(LpShared &sh, int n, int k) {
  __syncthreads();
  for (int c = threadIdx.x; c < n; c += kLpThreads) {
    const unsigned long long mine = sh.cand[c];
    int rank = 0;
    for (int o = 0; o < n; ++o) rank += sh.cand[o] > mine ? 1 : 0;
    if (rank < k) sh.best[rank] = mine;
  }
  if (threadIdx.x == 0) sh.n_best = min(n, k);
  __syncthreads();
}

// The chunk's part in the k best (see the head of the file).  floor_ord: the
// minimum of the groups' maxima.
template <bool kBf16, bool kVec>
__device__ __forceinline__ void select_chunk(LpShared &sh, const float (&x)[kPerThread], int c0,
                                             int end, int k, uint32_t floor_ord) {
  const int tid = threadIdx.x;
  const int nb = sh.n_best;
  if (nb == k) floor_ord = max(floor_ord, (uint32_t)(sh.best[k - 1] >> 32));
  if (tid < nb) sh.cand[tid] = sh.best[tid];
  if (tid == 0) sh.n_cand = nb;
  __syncthreads();
  const float lowest = unordered(floor_ord);
#pragma unroll
  for (int e = 0; e < kPerThread; ++e) {
    // (a NaN floor leaves only NaN, a NaN logit passes any floor)
    if (!(x[e] < lowest)) {
      const int id = c0 + chunk_pos<kBf16, kVec>(e, tid);
      const uint32_t o = ordered(x[e]);
      if (id < end && o >= floor_ord) {
        const int at = atomicAdd(&sh.n_cand, 1);
        if (at < kCap) sh.cand[at] = lp_key(o, id);
      }
    }
  }
  __syncthreads();
  const int n = sh.n_cand;
  if (n <= kCap) {
    rank_candidates(sh, n, k);
    return;
  }
  // Too many: the k-th largest value of the chunk, bit by bit (the largest T
  // with at least k values >= T), then its ties in id order.
  uint32_t T = 0;
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t t = T | (1u << bit);
    int mine = 0;
#pragma unroll
    for (int e = 0; e < kPerThread; ++e)
      mine += (c0 + chunk_pos<kBf16, kVec>(e, tid) < end && ordered(x[e]) >= t) ? 1 : 0;
    if (block_sum(mine, sh.reduce) >= k) T = t;
  }
  __syncthreads();
  if (tid == 0) sh.n_cand = nb;
  __syncthreads();
  int above = 0;
#pragma unroll
  for (int e = 0; e < kPerThread; ++e) {
    const int id = c0 + chunk_pos<kBf16, kVec>(e, tid);
    const uint32_t o = ordered(x[e]);
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
      if (i < end && i > after && ordered(x[e]) == T) id = min(id, i);
    }
    id = block_min(id, sh.reduce);
    if (id == 0x7FFFFFFF) break;
    if (tid == 0) sh.cand[sh.n_cand++] = lp_key(T, id);
    after = id;
  }
  __syncthreads();
  rank_candidates(sh, sh.n_cand, k);
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

template <bool kBf16, bool kVec>
__global__ void __launch_bounds__(kLpThreads, 3) logprobs_kernel(const LpArgs a) {
  using namespace sm100;
  __shared__ LpShared sh;
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
    sh.n_best = 0;
    sh.m = -INFINITY;
    sh.S = 0.f;
    sh.T = 0.f;
    sh.xt = -INFINITY;
  }
  const int first = rank * a.per, last = min(a.V, first + a.per);
  for (int c0 = first; c0 < last; c0 += kChunk) {
    const int end = min(last, c0 + kChunk);
    float x[kPerThread];
    load_chunk<kBf16, kVec>(src, c0, end, tid, x);
    float top = -INFINITY;  // fmaxf drops a NaN, so those are looked for apart
    bool nan = false;
#pragma unroll
    for (int e = 0; e < kPerThread; ++e) {
      top = fmaxf(top, x[e]);
      nan = nan || x[e] != x[e];
    }
    uint32_t best = nan ? 0xFFFFFFFFu : ordered(top);
#pragma unroll
    for (int off = 1; off < 8; off <<= 1)
      best = max(best, __shfl_xor_sync(0xffffffffu, best, off));
    __syncthreads();  // the previous chunk's shared state is read
    if ((lane & 7) == 0) sh.group_max[tid >> 3] = best;
    __syncthreads();
    const uint32_t gm = sh.group_max[lane];
    const float m = unordered(__reduce_max_sync(0xffffffffu, gm));
    const uint32_t floor_ord = __reduce_min_sync(0xffffffffu, gm);
    // d = -200 stands for every d that e^d rounds to zero for (-inf included);
    // a maximum that is NaN or +inf makes the row's sums NaN below
    float S = 0.f, T = 0.f;
#pragma unroll
    for (int e = 0; e < kPerThread; ++e) {
      const float d = fmaxf(x[e] - m, -200.f);
      const float p = ex2_approx(d * kLog2e);
      S += p;
      T = fmaf(p, d, T);
    }
    if (token >= c0 && token < end && kVec) {
      const int o = token - c0;
      constexpr int kW = kBf16 ? 8 : 4;
      if ((o / kW) % kLpThreads == tid) {
#pragma unroll
        for (int e = 0; e < kPerThread; ++e)
          if (chunk_pos<kBf16, kVec>(e, tid) == o) sh.xt = x[e];
      }
    } else if (token >= c0 && token < end) {
#pragma unroll
      for (int e = 0; e < kPerThread; ++e)
        if (chunk_pos<kBf16, kVec>(e, tid) == token - c0) sh.xt = x[e];
    }
    S = warp_sum(S);
    T = warp_sum(T);
    if (lane == 0) {
      sh.sum[warp] = S;
      sh.dsum[warp] = T;
    }
    __syncthreads();
    if (tid == 0) {
      S = 0.f;
      T = 0.f;
#pragma unroll
      for (int w = 0; w < kLpWarps; ++w) {
        S += sh.sum[w];
        T += sh.dsum[w];
      }
      if (m == -INFINITY) S = T = 0.f;
      if (!(m < INFINITY)) S = T = __uint_as_float(0x7FC00000u);
      // join with the chunks before it
      const float m0 = sh.m;
      const float M = (m0 != m0 || m != m) ? __uint_as_float(0x7FC00000u) : fmaxf(m0, m);
      float S1 = 0.f, T1 = 0.f;
      if (m0 != -INFINITY) {
        const float f = ex2_approx((m0 - M) * kLog2e);
        S1 = f * sh.S;
        T1 = f == 0.f ? 0.f : f * (sh.T + sh.S * (m0 - M));
      }
      if (m != -INFINITY) {
        const float f = ex2_approx((m - M) * kLog2e);
        S1 += f * S;
        T1 += f == 0.f ? 0.f : f * (T + S * (m - M));
      }
      sh.m = M;
      sh.S = S1;
      sh.T = T1;
    }
    if (k > 0) select_chunk<kBf16, kVec>(sh, x, c0, end, k, floor_ord);
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
      nan = nan || v.x != v.x;
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
        const float4 v = ld_dsmem_f4(smem_addr(&sh.best[lane * 2]), c);
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

template <bool kBf16, bool kVec>
cudaError_t lp_launch(const LpArgs &a, int R, int ctas, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas * (unsigned)R);
  cfg.blockDim = dim3(kLpThreads);
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
  return cudaLaunchKernelEx(&cfg, logprobs_kernel<kBf16, kVec>, a);
}

int lp_run(LpArgs &a, int R, int bf16, tsd_stream_t stream) {
  // a CTA for every chunk of a row, up to 8 (a power of two)
  int ctas = 1;
  while (ctas < 8 && (int64_t)ctas * kChunk < a.V) ctas *= 2;
  a.per = ((a.V + ctas - 1) / ctas + 7) / 8 * 8;
  const bool vec = aligned(a.logits, 16) && a.V % (bf16 ? 8 : 4) == 0;
  const cudaStream_t s = as_cuda(stream);
  const cudaError_t e = bf16 ? (vec ? lp_launch<true, true>(a, R, ctas, s) : lp_launch<true, false>(a, R, ctas, s))
                             : (vec ? lp_launch<false, true>(a, R, ctas, s) : lp_launch<false, false>(a, R, ctas, s));
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
