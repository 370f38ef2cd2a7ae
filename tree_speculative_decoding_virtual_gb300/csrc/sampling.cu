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
// One cluster of up to 8 CTAs a row; the row stays in shared memory, each warp with a
// run of consecutive ids.
#include <cuda_bf16.h>

#include <cmath>

#include "sm100_ptx.cuh"
#include "tsd_common.cuh"

namespace tsd {
namespace {

constexpr int kSpThreads = 512;
constexpr int kSpWarps = kSpThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxVocab = 262144;
constexpr int kMaxDraws = 64;
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

struct SpShared {
  float max[2];
  int count[2];
  long long sum[2];
  float wmax[kSpWarps];
  int wcount[kSpWarps];
  long long wsum[kSpWarps];
};

__device__ __forceinline__ uint32_t ordered(float x) {  // no NaN; both zeros alike
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
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
__device__ __forceinline__ void cluster_sync() {
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
  __device__ __forceinline__ long long value() const { return ((long long)hi << 23) + lo; }
};
constexpr float kUnit = 0x1p-43f;

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

// What is kept: everything from (hi, lo) on, in (ordered logit, kMaxVocab - 1 - id).
struct Border {
  uint32_t hi = 0u, lo = 0u;
  __device__ __forceinline__ bool has(uint32_t key, int id) const {
    return key > hi || (key == hi && (uint32_t)(kMaxVocab - 1 - id) >= lo);
  }
};

template <bool kBf16, int kMode>
__global__ void __launch_bounds__(kSpThreads) sampling_kernel(const SpArgs a) {
  using namespace sm100;
  using Vec = SpVec<kBf16>;
  constexpr int kStep = 32 * Vec::kN;  // logits of a warp step
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
  const float inv_t = greedy ? 1.f : __fdiv_rn(1.f, T);
  int k = a.top_k ? a.top_k[pr] : 0;
  if (k <= 0 || k > V) k = V;
  if (greedy) k = 1;
  const float top_p = a.top_p ? a.top_p[pr] : 1.f;
  const float min_p = a.min_p ? fminf(a.min_p[pr], 1.f) : 0.f;

  // ---- the run [id0, id0 + per_warp) of this warp, -inf past the row's end ----
  const int id0 = ((int)rank * kSpWarps + warp) * a.per_warp;
  const int steps = a.per_warp / kStep;
  uint4 *run = smem + (size_t)warp * (a.per_warp / Vec::kN);
  float m = -INFINITY;
  {
    using Raw = typename std::conditional<kBf16, uint16_t, uint32_t>::type;
    const Raw *src = reinterpret_cast<const Raw *>(a.logits) + row * V;
    const bool vec = (reinterpret_cast<uintptr_t>(src) & 15) == 0;
    const uint32_t none = kBf16 ? 0xFF80FF80u : 0xFF800000u;
    for (int s = 0; s < steps; ++s) {
      const int id = id0 + s * kStep + lane * Vec::kN;
      uint4 v = make_uint4(none, none, none, none);
      if (vec && id + Vec::kN <= V) {
        v = __ldcs(reinterpret_cast<const uint4 *>(src + id));
      } else {
        Raw e[Vec::kN];
#pragma unroll
        for (int i = 0; i < Vec::kN; ++i) e[i] = id + i < V ? src[id + i] : (Raw)none;
        if constexpr (kBf16)
          v = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
        else
          v = make_uint4(e[0], e[1], e[2], e[3]);
      }
      run[s * 32 + lane] = v;
      Vec x;
      x.read(&v);
#pragma unroll
      for (int i = 0; i < Vec::kN; ++i) m = max_nan(m, x.x[i]);
    }
  }
  // (a lane reads what it wrote itself until the draws)

  int turn = 0;  // which of the exchanged values' two places
  auto cluster_total = [&](int &count, Fixed f) -> long long {
    const long long sum = warp_sum(f.value());
    count = __reduce_add_sync(0xffffffffu, count);
    __syncthreads();
    if (lane == 0) {
      sh.wsum[warp] = sum;
      sh.wcount[warp] = count;
    }
    __syncthreads();
    if (tid == 0) {
      long long t = 0;
      int c = 0;
      for (int w = 0; w < kSpWarps; ++w) {
        t += sh.wsum[w];
        c += sh.wcount[w];
      }
      sh.sum[turn] = t;
      sh.count[turn] = c;
    }
    cluster_sync();
    long long t = 0;
    count = 0;
    for (uint32_t p = 0; p < ranks; ++p) {
      t += (long long)ld_peer64(&sh.sum[turn], p);
      count += (int)ld_peer32(&sh.count[turn], p);
    }
    turn ^= 1;
    return t;
  };

#pragma unroll
  for (int off = 16; off; off >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
  if (lane == 0) sh.wmax[warp] = m;
  __syncthreads();
  if (tid == 0) {
    for (int w = 0; w < kSpWarps; ++w) m = max_nan(m, sh.wmax[w]);
    sh.max[0] = m;
  }
  cluster_sync();
  m = -INFINITY;
  for (uint32_t p = 0; p < ranks; ++p) m = max_nan(m, __uint_as_float(ld_peer32(&sh.max[0], p)));

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

  auto scaled = [&](float x) { return __fmul_rn(__fsub_rn(x, m), inv_t); };
  // number and weight of what lies above a border
  auto above = [&](const Border &b, int &count) -> long long {
    Fixed f;
    count = 0;
    for (int s = 0; s < steps; ++s) {
      Vec x;
      x.read(run + s * 32 + lane);
#pragma unroll
      for (int i = 0; i < Vec::kN; ++i) {
        const bool in = x.x[i] > -INFINITY && b.has(ordered(x.x[i]), id0 + s * kStep + lane * Vec::kN + i);
        count += in;
        if (in) f.add(expf(scaled(x.x[i])));
      }
    }
    return cluster_total(count, f);
  };
  // the highest border that enough lies above
  auto settle = [&](auto enough) -> Border {
    Border b;
    for (int bit = 31; bit >= 0; --bit) {
      Border t{b.hi | 1u << bit, 0u};
      int n;
      const long long sum = above(t, n);
      if (enough(n, sum)) b = t;
    }
    for (int bit = 17; bit >= 0; --bit) {
      Border t{b.hi, b.lo | 1u << bit};
      int n;
      const long long sum = above(t, n);
      if (enough(n, sum)) b = t;
    }
    return b;
  };
  Border kept;
  if (k < V) {
    int n;
    above(kept, n);
    if (n > k) kept = settle([&](int c, long long) { return c >= k; });
  }
  if (top_p < 1.f) {
    int n;
    const double want = (double)top_p * (double)above(kept, n);
    const long long least = want > 1.0 ? (long long)ceil(want) : 1;
    const Border b = settle([&](int, long long s) { return s >= least; });
    if (b.hi > kept.hi || (b.hi == kept.hi && b.lo > kept.lo)) kept = b;
  }

  // ---- what is kept, by warp ----
  auto weight = [&](float x, int id) -> float {  // 0: not kept
    if (!(x > -INFINITY) || !kept.has(ordered(x), id)) return 0.f;
    const float w = expf(scaled(x));
    return w < min_p ? 0.f : w;
  };
  Fixed f;
  for (int s = 0; s < steps; ++s) {
    Vec x;
    x.read(run + s * 32 + lane);
#pragma unroll
    for (int i = 0; i < Vec::kN; ++i) f.add(weight(x.x[i], id0 + s * kStep + lane * Vec::kN + i));
  }
  int unused = 0;
  const long long total = cluster_total(unused, f);
  if constexpr (kMode == kSample) {
    long long before = 0;  // of this warp's run
    for (uint32_t p = 0; p < rank; ++p) before += (long long)ld_peer64(&sh.sum[turn ^ 1], p);
    for (int w = 0; w < warp; ++w) before += sh.wsum[w];
    const long long mine = sh.wsum[warp];
    const float log_total = logf((float)total * kUnit);
    for (int q = 0; q < a.draws; ++q) {
      const float u = a.u[(size_t)r * a.draws + q];
      long long at = u > 0.f ? (long long)floor((double)u * (double)total) : 0;
      at = min(at, total - 1) - before;
      if (at < 0 || at >= mine) continue;
      for (int s = 0; s < steps; ++s) {
        Vec x;
        x.read(run + s * 32 + lane);
        float w[Vec::kN];
        long long sum = 0;
#pragma unroll
        for (int i = 0; i < Vec::kN; ++i) {
          w[i] = weight(x.x[i], id0 + s * kStep + lane * Vec::kN + i);
          Fixed one;
          one.add(w[i]);
          sum += one.value();
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
#pragma unroll
            for (int j = 0; j < Vec::kN - 1; ++j) {
              Fixed one;
              one.add(w[j]);
              if (i == j && left >= one.value()) {
                left -= one.value();
                ++i;
              }
            }
            float d = 0.f;
#pragma unroll
            for (int j = 0; j < Vec::kN; ++j)
              if (j == i) d = scaled(x.x[j]);
            a.tokens[(size_t)r * a.draws + q] = id0 + s * kStep + lane * Vec::kN + i;
            a.logprob[(size_t)r * a.draws + q] = d - log_total;
          }
          break;
        }
        at -= all;
      }
    }
  } else {
    const float inv = 1.f / ((float)total * kUnit);
    for (int s = 0; s < steps; ++s) {
      Vec x;
      x.read(run + s * 32 + lane);
#pragma unroll
      for (int i = 0; i < Vec::kN; ++i) {
        const int id = id0 + s * kStep + lane * Vec::kN + i;
        if (id >= V) continue;
        const bool in = x.x[i] > -INFINITY && kept.has(ordered(x.x[i]), id) &&
                        !(min_p > 0.f && expf(scaled(x.x[i])) < min_p);
        a.out[(size_t)r * V + id] =
            kMode == kProbs ? (in ? expf(scaled(x.x[i])) * inv : 0.f) : in ? scaled(x.x[i]) : -INFINITY;
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
