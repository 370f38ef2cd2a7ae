// The 4-bit paged cache: its writer, its reader and the commit of an accepted
// path (format: q4.cuh).
//
// All three move a few bytes per value and compute next to nothing, so they
// are bound by HBM for prompts and by launch latency for a step's tree.

#include <cuda_bf16.h>

#include "commit_core.cuh"
#include "q4.cuh"
#include "tsd_common.cuh"

namespace tsd {
namespace {

constexpr int kRowThreads = 256;

// One group of 16 bf16 values -> eight code bytes and a scale byte.
//   scale = nearest (ties to even) to amax / 6, at most 10240;
//   code  = nearest (ties to even) to x / scale.
// amax and x have 8 significant bits and every rounding boundary (times 6, or
// times the scale) at most 7, so a quotient that is not a tie differs from
// the boundary by 2^-9 relative or more: deciding on the correctly rounded
// fp32 quotient gives the decision of exact arithmetic.  NaN counts as 0 and
// an infinity as the largest value; both are reported.
__device__ __forceinline__ uint2 q4_encode(const uint4 (&in)[2], uint32_t &scale_byte, bool &odd) {
  float x[16];
  const uint32_t w[8] = {in[0].x, in[0].y, in[0].z, in[0].w, in[1].x, in[1].y, in[1].z, in[1].w};
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  bool finite = true;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if (!isfinite(x[i])) {
      finite = false;
      if (isnan(x[i])) x[i] = 0.f;
    }
    amax = fmaxf(amax, fabsf(x[i]));
  }
  odd = odd || !finite;
  const float r = fminf(__fdiv_rn(amax, 6.f), 10240.f);
  uint32_t byte;
  if (r < 6.103515625e-05f) {  // below 2^-14: steps of 2^-17
    byte = (uint32_t)rintf(r * 131072.f);
  } else {
    uint32_t u = __float_as_uint(r);
    u += 0x7FFFFu + ((u >> 20) & 1u);
    byte = (u >> 20) - (112u << 3);
  }
  scale_byte = byte;
  const float scale =
      byte < 8 ? (float)byte * 7.62939453125e-06f : __uint_as_float((byte + (112u << 3)) << 20);
  uint32_t code[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = byte ? __fdiv_rn(x[2 * i], scale) : copysignf(0.f, x[2 * i]);
    const float b = byte ? __fdiv_rn(x[2 * i + 1], scale) : copysignf(0.f, x[2 * i + 1]);
    uint16_t two;  // the first source of the conversion goes to the high nibble
    asm("{\n .reg .b8 t;\n cvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n cvt.u16.u8 %0, t;\n}\n"
        : "=h"(two)
        : "f"(b), "f"(a));
    code[i / 4] |= (uint32_t)two << (8 * (i % 4));
  }
  return make_uint2(code[0], code[1]);
}

// One thread per (token, kv head, group): reads 32 bytes of K and of V, writes
// 8 code bytes and a scale byte of each.
template <int D>
__global__ void __launch_bounds__(kRowThreads)
kv_write_q4_kernel(const uint16_t *__restrict__ k, int64_t k_stride, const uint16_t *__restrict__ v,
                   int64_t v_stride, const int32_t *__restrict__ slots, int64_t items, int num_blocks,
                   int Hkv, uint8_t *__restrict__ kc, uint8_t *__restrict__ vc, int32_t *status) {
  using L = Q4Page<D>;
  constexpr int kGroups = D / kQ4Group;
  pdl_wait();
  const int64_t x = (int64_t)blockIdx.x * kRowThreads + threadIdx.x;
  if (x >= items) return;
  const int per = Hkv * kGroups;  // groups of one token
  const int64_t t = x / per;
  const int hg = (int)(x - t * per);
  const int h = hg / kGroups, gi = hg % kGroups;
  const int slot = slots[t];
  if (slot < 0 || (int64_t)slot >= (int64_t)num_blocks * kPage) {
    if (slot != -1 && hg == 0 && status) atomicOr(status, TSD_STATUS_BAD_PAGE);
    return;
  }
  const uint4 *ks = reinterpret_cast<const uint4 *>(k + t * k_stride + hg * kQ4Group);
  const uint4 *vs = reinterpret_cast<const uint4 *>(v + t * v_stride + hg * kQ4Group);
  const uint4 kin[2] = {ks[0], ks[1]}, vin[2] = {vs[0], vs[1]};
  const size_t page = ((size_t)(slot / kPage) * Hkv + h) * L::kBytes;
  const int row = slot % kPage;
  bool odd = false;
  uint32_t sk, sv;
  const uint2 ck = q4_encode(kin, sk, odd), cv = q4_encode(vin, sv, odd);
  *reinterpret_cast<uint2 *>(kc + page + row * L::kRow + gi * 8) = ck;
  kc[page + L::kScales + row * L::kScaleRow + gi] = (uint8_t)sk;
  *reinterpret_cast<uint2 *>(vc + page + row * L::kRow + gi * 8) = cv;
  vc[page + L::kScales + row * L::kScaleRow + gi] = (uint8_t)sv;
  if (odd && status) atomicOr(status, TSD_STATUS_NONFINITE);
}

// Two fp16 values of a page (exact in bf16) as a bf16 pair.
__device__ __forceinline__ uint32_t half2_to_bf16x2(uint32_t h) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
  const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t *>(&b);
}

__device__ __forceinline__ void q4_row_out(uint2 code, uint32_t scale_byte, uint16_t *dst) {
  const uint32_t s = q4_scale2(scale_byte);
  uint32_t a[4], b[4];
  q4_decode8(code.x, a);
  q4_decode8(code.y, b);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] = half2_to_bf16x2(q4_mul2(a[i], s));
    b[i] = half2_to_bf16x2(q4_mul2(b[i], s));
  }
  uint4 *d = reinterpret_cast<uint4 *>(dst);
  d[0] = make_uint4(a[0], a[1], a[2], a[3]);
  d[1] = make_uint4(b[0], b[1], b[2], b[3]);
}

// One thread per (token, kv head, group), K and V: 9 bytes in, 32 out.
template <int D>
__global__ void __launch_bounds__(kRowThreads)
kv_read_q4_kernel(const uint8_t *__restrict__ kc, const uint8_t *__restrict__ vc,
                  const int32_t *__restrict__ slots, int64_t items, int num_blocks, int Hkv,
                  uint16_t *__restrict__ k, uint16_t *__restrict__ v, int32_t *status) {
  using L = Q4Page<D>;
  constexpr int kGroups = D / kQ4Group;
  pdl_wait();
  const int64_t x = (int64_t)blockIdx.x * kRowThreads + threadIdx.x;
  if (x >= items) return;
  const int per = Hkv * kGroups;
  const int64_t t = x / per;
  const int hg = (int)(x - t * per);
  const int h = hg / kGroups, gi = hg % kGroups;
  const int slot = slots[t];
  uint2 ck = make_uint2(0u, 0u), cv = ck;
  uint32_t sk = 0, sv = 0;
  if (slot >= 0 && (int64_t)slot < (int64_t)num_blocks * kPage) {
    const size_t page = ((size_t)(slot / kPage) * Hkv + h) * L::kBytes;
    const int row = slot % kPage;
    ck = *reinterpret_cast<const uint2 *>(kc + page + row * L::kRow + gi * 8);
    cv = *reinterpret_cast<const uint2 *>(vc + page + row * L::kRow + gi * 8);
    sk = kc[page + L::kScales + row * L::kScaleRow + gi];
    sv = vc[page + L::kScales + row * L::kScaleRow + gi];
  } else if (slot != -1 && hg == 0 && status) {
    atomicOr(status, TSD_STATUS_BAD_PAGE);
  }
  q4_row_out(ck, sk, k + x * kQ4Group);
  q4_row_out(cv, sv, v + x * kQ4Group);
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
  if ((T * Hkv * (D / kQ4Group) + kRowThreads - 1) / kRowThreads > 0x7FFFFFFFll) return TSD_ERR_LIMIT;
  return TSD_OK;
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
  const int64_t items = T * Hkv * (D / kQ4Group);
  const dim3 grid((unsigned)((items + kRowThreads - 1) / kRowThreads));
  const cudaError_t e =
      D == 128 ? launch(kv_write_q4_kernel<128>, grid, dim3(kRowThreads), 0, as_cuda(stream), k,
                        k_stride, v, v_stride, slots, items, num_blocks, Hkv, k_cache, v_cache, status)
               : launch(kv_write_q4_kernel<64>, grid, dim3(kRowThreads), 0, as_cuda(stream), k,
                        k_stride, v, v_stride, slots, items, num_blocks, Hkv, k_cache, v_cache, status);
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
  const int64_t items = T * Hkv * (D / kQ4Group);
  const dim3 grid((unsigned)((items + kRowThreads - 1) / kRowThreads));
  const cudaError_t e =
      D == 128 ? launch(kv_read_q4_kernel<128>, grid, dim3(kRowThreads), 0, as_cuda(stream), k_cache,
                        v_cache, slots, items, num_blocks, Hkv, k, v, status)
               : launch(kv_read_q4_kernel<64>, grid, dim3(kRowThreads), 0, as_cuda(stream), k_cache,
                        v_cache, slots, items, num_blocks, Hkv, k, v, status);
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
