// The 4-bit paged cache: its writer, its reader and the commit of an accepted
// path (format: q4.cuh).
//
// All three move a few bytes per value.  For a step's tree they are bound by launch
// latency.  For prompts the reader and the commit are bound by HBM; the writer by the
// pipe of the integer and conversion instructions (32768 tokens, 8 heads of 128: 35
// us for 172 MB, that pipe 70% busy; the reader of the same 30 us), which is why its
// two lanes of a group share the scales' computation (one K's, one V's), quotients
// are rounded by packed fp32 sums, and item positions are counted, not divided for:
// 47 us without these.

#include <cuda_bf16.h>

#include "commit_core.cuh"
#include "q4.cuh"
#include "q4_encode.cuh"
#include "sm100_ptx.cuh"
#include "tsd_common.cuh"

namespace tsd {
namespace {

// Writer and reader: a lane holds 8 consecutive values (16 bytes of bf16, 4 code
// bytes), so a warp's loads and stores are contiguous on both sides; two lanes
// share a group and its scale.
constexpr int kRowThreads = 256;
constexpr int kLaneValues = 8;
constexpr int kBlockItems = 4 * kRowThreads;  // lanes' worth of work of a block

struct RowArgs {
  const int32_t *slots;
  int64_t T;
  int num_blocks, Hkv, tokens;  // tokens: of one block
  int32_t *status;
};

// Slot of token t; -1 when there is none (the one lane that `report`s tells).
__device__ __forceinline__ int row_slot(const RowArgs &a, int64_t t, bool report) {
  const int slot = a.slots[t];
  if (slot >= 0 && (int64_t)slot < (int64_t)a.num_blocks * kPage) return slot;
  if (slot != -1 && report && a.status) atomicOr(a.status, TSD_STATUS_BAD_PAGE);
  return -1;
}

// A block takes a.tokens tokens, K and V.
template <int D>
__global__ void __launch_bounds__(kRowThreads)
kv_write_q4_kernel(const RowArgs a, const uint16_t *__restrict__ k, int64_t k_stride,
                   const uint16_t *__restrict__ v, int64_t v_stride, uint8_t *__restrict__ kc,
                   uint8_t *__restrict__ vc) {
  using L = Q4Page<D>;
  constexpr int kLanes = D / kLaneValues;  // of one head's row
  pdl_wait();
  const int per = a.Hkv * kLanes;
  const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
  const int items = (int)min((int64_t)a.tokens, a.T - t0) * per;
  const int step_t = kRowThreads / per, step_c = kRowThreads % per;
  int tl = threadIdx.x / per, c = threadIdx.x % per;  // of item x: token, lane of its row
  const bool second = threadIdx.x & 1;  // of the two lanes of a group
  // (whole warps: a lane past the end encodes zeros for its partner's sake)
#pragma unroll 2
  for (int x = threadIdx.x; x < (items + 31) / 32 * 32; x += kRowThreads) {
    const int64_t t = t0 + tl;
    const int slot = x < items ? row_slot(a, t, c == 0) : -1;
    uint4 kin = make_uint4(0u, 0u, 0u, 0u), vin = kin;
    if (slot >= 0) {
      kin = __ldcs(reinterpret_cast<const uint4 *>(k + t * k_stride + c * kLaneValues));
      vin = __ldcs(reinterpret_cast<const uint4 *>(v + t * v_stride + c * kLaneValues));
    }
    bool odd = false;
    const uint32_t k_most = q4_amax(kin, odd), v_most = q4_amax(vin, odd);
    // the group's first lane finds K's scale, the second V's
    const uint32_t theirs = __shfl_xor_sync(0xffffffffu, second ? k_most : v_most, 1);
    float recip;
    const uint32_t byte = q4_group_scale(__uint_as_float(max(second ? v_most : k_most, theirs)), recip);
    const float other = __shfl_xor_sync(0xffffffffu, recip, 1);
    const uint32_t ck = q4_codes(kin, second ? other : recip), cv = q4_codes(vin, second ? recip : other);
    if (slot >= 0) {
      const int h = c / kLanes, i = c % kLanes;
      const size_t page = ((size_t)(slot / kPage) * a.Hkv + h) * L::kBytes;
      const int row = slot % kPage;
      *reinterpret_cast<uint32_t *>(kc + page + row * L::kRow + i * 4) = ck;
      *reinterpret_cast<uint32_t *>(vc + page + row * L::kRow + i * 4) = cv;
      (second ? vc : kc)[page + L::kScales + row * L::kScaleRow + i / 2] = (uint8_t)byte;
      if (odd && a.status) atomicOr(a.status, TSD_STATUS_NONFINITE);
    }
    tl += step_t;
    c += step_c;
    if (c >= per) {
      c -= per;
      ++tl;
    }
  }
}

// Two fp16 values of a page (exact in bf16) as a bf16 pair.
__device__ __forceinline__ uint32_t half2_to_bf16x2(uint32_t h) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
  const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t *>(&b);
}

__device__ __forceinline__ uint4 q4_values(uint32_t code, uint32_t scale_byte) {
  const uint32_t s = q4_scale2(scale_byte);
  uint32_t a[4];
  q4_decode8(code, a);
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = half2_to_bf16x2(q4_mul2(a[i], s));
  return make_uint4(a[0], a[1], a[2], a[3]);
}

template <int D>
__global__ void __launch_bounds__(kRowThreads)
kv_read_q4_kernel(const RowArgs a, const uint8_t *__restrict__ kc, const uint8_t *__restrict__ vc,
                  uint16_t *__restrict__ k, uint16_t *__restrict__ v) {
  using L = Q4Page<D>;
  constexpr int kLanes = D / kLaneValues;
  pdl_wait();
  const int per = a.Hkv * kLanes;
  const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
  const int items = (int)min((int64_t)a.tokens, a.T - t0) * per;
  const int step_t = kRowThreads / per, step_c = kRowThreads % per;
  int tl = threadIdx.x / per, c = threadIdx.x % per;  // of item x: token, lane of its row
#pragma unroll 4
  for (int x = threadIdx.x; x < items; x += kRowThreads) {
    const int64_t t = t0 + tl;
    const int slot = row_slot(a, t, c == 0);
    uint32_t ck = 0, cv = 0, sk = 0, sv = 0;
    if (slot >= 0) {
      const int h = c / kLanes, i = c % kLanes;
      const size_t page = ((size_t)(slot / kPage) * a.Hkv + h) * L::kBytes;
      const int row = slot % kPage;
      ck = *reinterpret_cast<const uint32_t *>(kc + page + row * L::kRow + i * 4);
      cv = *reinterpret_cast<const uint32_t *>(vc + page + row * L::kRow + i * 4);
      sk = kc[page + L::kScales + row * L::kScaleRow + i / 2];
      sv = vc[page + L::kScales + row * L::kScaleRow + i / 2];
    }
    const size_t at = (size_t)t * per + c;
    __stcs(reinterpret_cast<uint4 *>(k) + at, q4_values(ck, sk));
    __stcs(reinterpret_cast<uint4 *>(v) + at, q4_values(cv, sv));
    tl += step_t;
    c += step_c;
    if (c >= per) {
      c -= per;
      ++tl;
    }
  }
}

constexpr int kCommitThreads = 128;

// One block per (kv head, sequence, layer), as the bf16 commit: warp 0 plans
// the sequence's moves, then every source row (codes and scales, 4-byte words)
// is staged before any destination is written, because a destination can be
// the source of a later path element.
template <int D>
__global__ void __launch_bounds__(kCommitThreads)
commit_q4_kernel(const CommitArgs a, uint8_t *kc, uint8_t *vc, const int32_t *__restrict__ n_nodes,
                 const int32_t *__restrict__ accept_len, const int32_t *__restrict__ path,
                 const int32_t *__restrict__ err, int N_max, int D_max) {
  using L = Q4Page<D>;
  constexpr int kCodeWords = L::kRow / 4, kWords = kCodeWords + L::kScaleRow / 4;
  __shared__ CommitMoves mv;
  __shared__ uint32_t stage[2][kMaxMoves * kWords];
  pdl_wait();
  const int h = blockIdx.x, b = blockIdx.y, layer = blockIdx.z;
  if (threadIdx.x < 32)
    commit_plan_warp(a, b, N_max, D_max, n_nodes, err, accept_len, path, h == 0 && layer == 0, mv,
                     threadIdx.x);
  __syncthreads();
  uint32_t *kp = reinterpret_cast<uint32_t *>(kc + (size_t)layer * (size_t)a.layer_stride);
  uint32_t *vp = reinterpret_cast<uint32_t *>(vc + (size_t)layer * (size_t)a.layer_stride);
  auto at = [&](int page, int slot, int w) -> size_t {
    const size_t p = ((size_t)page * a.Hkv + h) * (L::kBytes / 4);
    return p + (w < kCodeWords ? slot * kCodeWords + w
                               : L::kScales / 4 + slot * (L::kScaleRow / 4) + (w - kCodeWords));
  };
  const int items = mv.n * kWords;
  for (int x = threadIdx.x; x < items; x += kCommitThreads) {
    const int m = x / kWords;
    const size_t s = at(mv.src_page[m], mv.src_slot[m], x % kWords);
    stage[0][x] = kp[s];
    stage[1][x] = vp[s];
  }
  __syncthreads();
  for (int x = threadIdx.x; x < items; x += kCommitThreads) {
    const int m = x / kWords;
    const size_t d = at(mv.dst_page[m], mv.dst_slot[m], x % kWords);
    kp[d] = stage[0][x];
    vp[d] = stage[1][x];
  }
}

// Checks shared by the writer and the reader; TSD_OK with T == 0 means an
// empty call.
int rows_check(int64_t T, int num_blocks, int Hkv, int D) {
  if (T < 0 || num_blocks < 1 || Hkv < 1) return TSD_ERR_ARG;
  if (D != 64 && D != 128) return TSD_ERR_LIMIT;
  if (Hkv > 65535 || (int64_t)num_blocks * kPage > 0x7FFFFFFFll || T > 0x7FFFFFFFll) return TSD_ERR_LIMIT;
  return TSD_OK;
}

RowArgs row_args(const int32_t *slots, int64_t T, int num_blocks, int Hkv, int D, int32_t *status) {
  // a block's work: kBlockItems lanes, or fewer so that a step's tree still
  // reaches every SM
  const int per = Hkv * (D / kLaneValues);
  const int64_t fill = (T * per + 2 * sm_count() - 1) / (2 * sm_count());
  const int64_t lanes = fill < kBlockItems ? fill : kBlockItems;
  const int tokens = (int)(lanes / per);
  return RowArgs{slots, T, num_blocks, Hkv, tokens > 0 ? tokens : 1, status};
}

}  // namespace
}  // namespace tsd

TSD_API int tsd_kv_write_q4(const uint16_t *k, int64_t k_stride, const uint16_t *v, int64_t v_stride,
                            const int32_t *slots, int64_t T, int num_blocks, int Hkv, int D,
                            uint8_t *k_cache, uint8_t *v_cache, int32_t *status, tsd_stream_t stream) {
  using namespace tsd;
  const int rc = rows_check(T, num_blocks, Hkv, D);
  if (rc != TSD_OK || T == 0) return rc;
  if (!k || !v || !slots || !k_cache || !v_cache) return TSD_ERR_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16))
    return TSD_ERR_ARG;
  const int64_t row = (int64_t)Hkv * D;
  if (T > 1 && (k_stride < row || v_stride < row)) return TSD_ERR_ARG;
  if (k_stride % 8 != 0 || v_stride % 8 != 0) return TSD_ERR_ARG;
  const RowArgs a = row_args(slots, T, num_blocks, Hkv, D, status);
  const dim3 grid((unsigned)((T + a.tokens - 1) / a.tokens));
  const cudaError_t e =
      D == 128 ? launch(kv_write_q4_kernel<128>, grid, dim3(kRowThreads), 0, as_cuda(stream), a, k,
                        k_stride, v, v_stride, k_cache, v_cache)
               : launch(kv_write_q4_kernel<64>, grid, dim3(kRowThreads), 0, as_cuda(stream), a, k,
                        k_stride, v, v_stride, k_cache, v_cache);
  return e == cudaSuccess ? TSD_OK : TSD_ERR_CUDA;
}

TSD_API int tsd_kv_read_q4(const uint8_t *k_cache, const uint8_t *v_cache, const int32_t *slots,
                           int64_t T, int num_blocks, int Hkv, int D, uint16_t *k, uint16_t *v,
                           int32_t *status, tsd_stream_t stream) {
  using namespace tsd;
  const int rc = rows_check(T, num_blocks, Hkv, D);
  if (rc != TSD_OK || T == 0) return rc;
  if (!k || !v || !slots || !k_cache || !v_cache) return TSD_ERR_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16))
    return TSD_ERR_ARG;
  const RowArgs a = row_args(slots, T, num_blocks, Hkv, D, status);
  const dim3 grid((unsigned)((T + a.tokens - 1) / a.tokens));
  const cudaError_t e =
      D == 128 ? launch(kv_read_q4_kernel<128>, grid, dim3(kRowThreads), 0, as_cuda(stream), a, k_cache,
                        v_cache, k, v)
               : launch(kv_read_q4_kernel<64>, grid, dim3(kRowThreads), 0, as_cuda(stream), a, k_cache,
                        v_cache, k, v);
  return e == cudaSuccess ? TSD_OK : TSD_ERR_CUDA;
}

TSD_API int tsd_kv_commit_path_q4(uint8_t *k_cache, uint8_t *v_cache, int num_layers,
                                  int64_t layer_stride, const int32_t *block_table, int max_blocks,
                                  int num_blocks, const int32_t *prefix_len, const int32_t *n_nodes,
                                  const int32_t *accept_len, const int32_t *path, const int32_t *err,
                                  const int32_t *tail_base, int B, int N_max, int Hkv, int D, int D_max,
                                  int32_t *new_len, int32_t *moved, int32_t *status,
                                  tsd_stream_t stream) {
  using namespace tsd;
  if (B < 0 || num_layers < 0 || Hkv < 1 || max_blocks < 1 || num_blocks < 1) return TSD_ERR_ARG;
  if (D != 64 && D != 128) return TSD_ERR_LIMIT;
  if (N_max < 1 || N_max > kMaxNodes || D_max < 0 || D_max > kMaxDepth || B > 65535 ||
      Hkv > 65535 || num_layers > 65535)
    return TSD_ERR_LIMIT;
  if (B == 0 || num_layers == 0) return TSD_OK;
  if (!k_cache || !v_cache || !block_table || !prefix_len || !accept_len || !path || !new_len)
    return TSD_ERR_ARG;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16)) return TSD_ERR_ARG;
  const int64_t pool = (int64_t)num_blocks * Hkv * 9 * D;
  if (num_layers > 1 && (layer_stride < pool || layer_stride % 16 != 0)) return TSD_ERR_ARG;
  const dim3 grid(Hkv, B, num_layers);
  const CommitArgs a{nullptr, nullptr, num_layers, layer_stride, block_table, max_blocks, num_blocks,
                     prefix_len, tail_base, Hkv, new_len, moved, status};
  const cudaError_t e =
      D == 128 ? launch(commit_q4_kernel<128>, grid, dim3(kCommitThreads), 0, as_cuda(stream), a,
                        k_cache, v_cache, n_nodes, accept_len, path, err, N_max, D_max)
               : launch(commit_q4_kernel<64>, grid, dim3(kCommitThreads), 0, as_cuda(stream), a,
                        k_cache, v_cache, n_nodes, accept_len, path, err, N_max, D_max);
  return e == cudaSuccess ? TSD_OK : TSD_ERR_CUDA;
}
