// Keys and values into the paged cache, with the norms and the rotation of
// queries and keys on the way ("EAGLE-Pangu: Accelerator-Safe Tree Speculative
// Decoding on Ascend NPUs", technical summary 2.1: the speculative branch's
// entries are written behind the committed prefix; a tree's node stands at
// position P_b + depth).
//
// For a head's row x of a token at position p (per axis):
//   y = x rsqrt(mean x^2 + eps) w                 (where a weight is given)
//   pairs (y_i, y_j) of frequency f turn by the angle p_axis(f) inv_freq_f
// in fp32, rounded to bf16 once.  Queries go to q_out, keys and values to their
// slots; a 4-bit cache takes the rounded keys as tsd_kv_write_q4 would.
//
// Angles: an fp32 product loses the angle of a far position (at 2^18 it is off by
// 2^-7), so a frequency is held as 64-bit fixed-point turns and multiplied by the
// position modulo one turn.  The 64 bits come from a whole-number product of the
// frequency's mantissa and 128 bits of 1 / (2 pi) and are off by less than two of their last
// places (frequencies below 2^64), the angle at position 2^31 by less than 2^-32 of a turn;
// the rest is a fraction of a turn in [-1/2, 1/2).
//
// Each byte is read and written once, so memory bounds many tokens and the launch few.  A
// block takes a few tokens: their cosines and sines are computed once, into shared memory,
// and used by all heads; a lane then holds two 16-byte chunks of a row that turn into each
// other (chunks l and l + R/16, or with neighbouring pairs 2l and 2l + 1), and the
// arithmetic goes two columns to an instruction.  What holds the loads in flight is the
// number of warps: 8 blocks of 128 threads and 4 tokens.  Measured at 32768 tokens of 64 +
// 2 x 8 heads of 128 (1.34 GB moved): 249 us, 5.4 TB/s; blocks of 256 threads with 16 tokens
// 261 us, with the loads of two steps on the way (and half the warps) 355 us, warps that
// keep a token's cosines in registers 282 us.  The same into 4 bits (1.25 GB): 231 us, 5.4
// TB/s.  One token of 32 + 2 x 8 heads: 2.5 us in a graph, 8 cold; 496 tokens of 32 + 2 x 8
// heads 10 us cold, into 16 bits and into 4: the launch, and one wave of blocks whose loads,
// angles and stores follow one another.
#include <cuda_bf16.h>

#include "q4.cuh"
#include "q4_encode.cuh"
#include "sm100_ptx.cuh"
#include "tsd_common.cuh"

namespace tsd {
namespace {

constexpr int kApThreads = 128;
constexpr int kApWarps = kApThreads / 32;
constexpr int kApTokens = 4;  // tokens of a block at most
constexpr int kMaxAxes = 4;

struct AppendArgs {
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride, q_out_stride;
  uint16_t *q_out;
  const int32_t *slots;
  int64_t T;
  int Hq, Hkv, R, axes, interleaved;
  const float *inv_freq;
  const int32_t *freq_axis, *pos, *base;
  int64_t per_base;
  const uint16_t *q_weight, *k_weight;
  float eps, rot_scale;
  int num_blocks;
  uint8_t *kc, *vc;
  int tokens, steps;  // of a block: tokens, warp steps of a token
  int32_t *status;
};

// inv_freq / (2 pi) as a 64-bit fraction of a turn, whole turns dropped.
__device__ __forceinline__ uint64_t turns(float inv_freq) {
  constexpr uint64_t kHi = 0x28BE60DB9391054Aull, kLo = 0x7F09D5F47D4D3770ull;  // 2^128 / (2 pi)
  const uint32_t bits = __float_as_uint(inv_freq), e = bits >> 23 & 255u;
  if (e == 255u) return 0ull;  // infinity, NaN
  const uint64_t m = bits & 0x7FFFFFu | (e ? 0x800000u : 0u);  // |inv_freq| = m 2^(max(e, 1) - 150)
  const int shift = 214 - (int)max(e, 1u);  // of the product, down to multiples of 2^-64: -40 .. 213
  const uint64_t w0 = m * kLo, w1 = m * kHi + __umul64hi(m, kLo);
  const uint64_t w2 = __umul64hi(m, kHi) + (w1 < m * kHi);
  const int word = shift >> 6, bit = shift & 63;
  const uint64_t x = word == 0 ? w0 : word == 1 ? w1 : word == 2 ? w2 : 0ull;
  const uint64_t y = word == -1 ? w0 : word == 0 ? w1 : word == 1 ? w2 : 0ull;
  const uint64_t t = bit ? x >> bit | y << (64 - bit) : x;
  return bits >> 31 ? 0ull - t : t;
}

// Two neighbouring columns in one 64-bit register, as the two-wide fp32 instructions take
// them.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  return sm100::f2_pack(lo, hi);
}
__device__ __forceinline__ float lo_of(uint64_t x) { return __uint_as_float((uint32_t)x); }
__device__ __forceinline__ float hi_of(uint64_t x) { return __uint_as_float((uint32_t)(x >> 32)); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ void unpack8(uint4 x, uint64_t (&f)[4]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = (uint64_t)(w[i] & 0xFFFF0000u) << 32 | w[i] << 16;
}
__device__ __forceinline__ uint4 pack8(const uint64_t (&f)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo_of(f[i]), hi_of(f[i]));
    w[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Block (x, y): tokens [x * tokens, ...), warp steps [y * steps, ...) of each.  A
// step is 32 / (D / 16) heads of the token's row q heads, k heads, v heads.
template <int D, bool kQ4>
__global__ void __launch_bounds__(kApThreads, 8) kv_append_kernel(const AppendArgs a) {
  constexpr int kLanes = D / 16;       // of one head's row
  constexpr int kHeads = 32 / kLanes;  // of one warp step
  // of frequencies 8 l + 2 i and the next, at [i][l]: both cosines, then both sines
  __shared__ float4 cs[kApTokens][4][kLanes];
  __shared__ uint4 weight[2][D / 8];
  __shared__ int slot_of[kApTokens];
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
  const int nt = (int)min((int64_t)a.tokens, a.T - t0);
  const int heads = a.Hq + 2 * a.Hkv;
  const int s0 = blockIdx.y * a.steps;
  const int per = min(a.steps, (heads + kHeads - 1) / kHeads - s0);  // steps of a token here
  const int l = lane % kLanes, hl = lane / kLanes;

  // The block's steps go round its warps, a token's after the other's.
  // a warp's next step: its lane's source, or null, and the two chunks there
  struct Item {
    const uint16_t *src;
    uint4 x, y;
    int tok, h;  // h: head of the row q | k | v
  };
  const int step_t = kApWarps / per, step_s = kApWarps % per;
  int tok = warp / per, s = warp % per;
  // A rotated lane's two chunks, and those of a lane that only copies.
  const int half = a.interleaved ? 0 : a.R / 16;  // lanes whose chunks are half a rotation apart
  auto chunks = [&](int h, int &c0, int &c1) {
    const bool apart = h < a.Hq + a.Hkv && l < half;
    c0 = apart ? l : 2 * l;
    c1 = apart ? l + half : 2 * l + 1;
    return apart;
  };
  auto fetch = [&](Item &it) {
    it.tok = tok;
    it.h = (s0 + s) * kHeads + hl;
    it.src = nullptr;
    it.x = it.y = make_uint4(0u, 0u, 0u, 0u);
    if (tok < nt && it.h < heads) {
      const int64_t t = t0 + tok;
      it.src = it.h < a.Hq           ? a.q + t * a.q_stride + (int64_t)it.h * D
               : it.h < a.Hq + a.Hkv ? a.k + t * a.k_stride + (int64_t)(it.h - a.Hq) * D
                                     : a.v + t * a.v_stride + (int64_t)(it.h - a.Hq - a.Hkv) * D;
      int c0, c1;
      chunks(it.h, c0, c1);
      it.x = __ldcs(reinterpret_cast<const uint4 *>(it.src) + c0);
      it.y = __ldcs(reinterpret_cast<const uint4 *>(it.src) + c1);
    }
    tok += step_t;
    s += step_s;
    if (s >= per) {
      s -= per;
      ++tok;
    }
  };
  Item it;  // on the way while the angles are computed, and while the step before is worked on
  fetch(it);

  {
    int lanes = 1;  // threads of one token's angles: a power of two
    while (lanes < a.R / 2) lanes *= 2;
    const int j = tid & (lanes - 1);
    if (j < a.R / 2) {
      const uint64_t freq = turns(a.inv_freq[j]);
      const int ax = a.freq_axis ? a.freq_axis[j] : 0;
      const int64_t off = ax > 0 && ax < a.axes ? ax * a.T : 0;
      for (int i = tid / lanes; i < nt; i += kApThreads / lanes) {
        const int64_t t = t0 + i;
        int64_t p = a.pos ? a.pos[off + t] : t % a.per_base;
        if (a.base) p += a.base[t / a.per_base];
        const uint64_t frac = freq * (uint64_t)p;
        const float z = (float)(int32_t)((frac + 0x80000000ull) >> 32) * 0x1p-31f;
        float sn, cn;
        sincospif(z, &sn, &cn);
        float *at = reinterpret_cast<float *>(&cs[i][(j & 7) >> 1][j >> 3]) + (j & 1);
        at[0] = cn * a.rot_scale;
        at[2] = sn * a.rot_scale;
      }
    }
    if (tid < D / 8 && a.q_weight) weight[0][tid] = reinterpret_cast<const uint4 *>(a.q_weight)[tid];
    if (tid < D / 8 && a.k_weight) weight[1][tid] = reinterpret_cast<const uint4 *>(a.k_weight)[tid];
    if (tid < nt) {
      int slot = a.slots[t0 + tid];
      if (slot < 0 || (int64_t)slot >= (int64_t)a.num_blocks * kPage) {
        if (slot != -1 && blockIdx.y == 0 && a.status) atomicOr(a.status, TSD_STATUS_BAD_PAGE);
        slot = -1;
      }
      slot_of[tid] = slot;
    }
  }
  __syncthreads();

  while (it.tok < nt) {  // (the same for the whole warp)
    const Item now = it;
    fetch(it);
    uint4 cx = now.x, cy = now.y;
    const bool is_q = now.h < a.Hq, is_v = now.h >= a.Hq + a.Hkv;
    int c0, c1;
    const bool apart = chunks(now.h, c0, c1);
    const uint16_t *w = is_q ? a.q_weight : a.k_weight;
    const bool normed = w && !is_v, turned = !is_v && l < a.R / 16;
    if (__any_sync(0xffffffffu, normed || turned)) {
      uint64_t f[4], g[4];
      unpack8(cx, f);
      unpack8(cy, g);
      if (__any_sync(0xffffffffu, normed)) {
        uint64_t sum = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) sum = sm100::f2_fma(g[i], g[i], sm100::f2_fma(f[i], f[i], sum));
        float ss = lo_of(sum) + hi_of(sum);
#pragma unroll
        for (int off = kLanes / 2; off; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
        if (normed) {
          const float r = rsqrtf(ss * (1.f / D) + a.eps);
          const uint64_t r2 = pair(r, r);
          uint64_t wf[4], wg[4];
          unpack8(weight[is_q ? 0 : 1][c0], wf);
          unpack8(weight[is_q ? 0 : 1][c1], wg);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            f[i] = mul2(f[i], mul2(r2, wf[i]));
            g[i] = mul2(g[i], mul2(r2, wg[i]));
          }
        }
      }
      if (turned) {
        if (apart) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 r = cs[now.tok][i][l];
            const uint64_t c = pair(r.x, r.y), sn = pair(r.z, r.w), x = f[i];
            f[i] = sm100::f2_fma(x, c, mul2(g[i], sn ^ 0x8000000080000000ull));
            g[i] = sm100::f2_fma(g[i], c, mul2(x, sn));
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {  // frequency 8 l + i turns one pair
            uint64_t &e = i < 4 ? f[i & 3] : g[i & 3];
            const float4 r = cs[now.tok][i / 2][l];
            const float c = i & 1 ? r.y : r.x, sn = i & 1 ? r.w : r.z;
            const float e0 = lo_of(e), e1 = hi_of(e);
            e = pair(e0 * c - e1 * sn, e1 * c + e0 * sn);
          }
        }
      }
      if (normed || turned) {
        cx = pack8(f);
        cy = pack8(g);
      }
    }
    const int slot = slot_of[now.tok];
    const bool cached = now.src && !is_q && slot >= 0;
    const int h = is_v ? now.h - a.Hq - a.Hkv : now.h - a.Hq;
    if (now.src && is_q) {
      uint4 *dst = reinterpret_cast<uint4 *>(a.q_out + (t0 + now.tok) * a.q_out_stride + (int64_t)now.h * D);
      __stcs(dst + c0, cx);
      __stcs(dst + c1, cy);
    }
    if constexpr (!kQ4) {
      if (cached) {
        uint4 *dst = reinterpret_cast<uint4 *>(is_v ? a.vc : a.kc) +
                     (((size_t)(slot / kPage) * a.Hkv + h) * kPage + slot % kPage) * (D / 8);
        dst[c0] = cx;
        dst[c1] = cy;
      }
    } else if (__any_sync(0xffffffffu, cached)) {
      // Groups of 16 columns: both chunks of a lane, or, where its chunks lie apart,
      // each with the neighbour's.
      using L = Q4Page<D>;
      bool odd = false;
      uint32_t m0 = q4_amax(cx, odd), m1 = q4_amax(cy, odd);
      const uint32_t n0 = __shfl_xor_sync(0xffffffffu, m0, 1), n1 = __shfl_xor_sync(0xffffffffu, m1, 1);
      m0 = max(m0, apart ? n0 : m1);
      m1 = apart ? max(m1, n1) : m0;
      float r0, r1;
      const uint32_t b0 = q4_group_scale(__uint_as_float(m0), r0), b1 = q4_group_scale(__uint_as_float(m1), r1);
      const uint32_t e0 = q4_codes(cx, r0), e1 = q4_codes(cy, r1);
      if (cached) {
        uint8_t *page = (is_v ? a.vc : a.kc) + ((size_t)(slot / kPage) * a.Hkv + h) * L::kBytes;
        const int row = slot % kPage;
        *reinterpret_cast<uint32_t *>(page + row * L::kRow + c0 * 4) = e0;
        *reinterpret_cast<uint32_t *>(page + row * L::kRow + c1 * 4) = e1;
        uint8_t *scale = page + L::kScales + row * L::kScaleRow;
        if (!apart || (l & 1) == 0) scale[c0 / 2] = (uint8_t)b0;
        if (apart && (l & 1)) scale[c1 / 2] = (uint8_t)b1;
        if (odd && a.status) atomicOr(a.status, TSD_STATUS_NONFINITE);
      }
    }
  }
}

template <int D, bool kQ4>
cudaError_t append_launch(AppendArgs &a, cudaStream_t s) {
  constexpr int kHeads = 32 / (D / 16);
  const int steps = (a.Hq + 2 * a.Hkv + kHeads - 1) / kHeads;
  // Enough blocks for every SM: few tokens are shared out by heads, many go up to
  // kApTokens a block.
  const int64_t want = 8ll * sm_count();
  const int64_t tokens = a.T / want;
  a.tokens = (int)(tokens < 1 ? 1 : tokens > kApTokens ? kApTokens : tokens);
  const int64_t blocks = (a.T + a.tokens - 1) / a.tokens;
  const int64_t parts = want / blocks, most = (steps + kApWarps - 1) / kApWarps;
  const int ny = (int)(parts < 1 ? 1 : parts > most ? most : parts);
  a.steps = (steps + ny - 1) / ny;
  const dim3 grid((unsigned)blocks, (unsigned)((steps + a.steps - 1) / a.steps));
  return launch(kv_append_kernel<D, kQ4>, grid, dim3(kApThreads), 0, s, a);
}

int append(AppendArgs &a, bool q4, int D, tsd_stream_t stream) {
  if (a.T < 0 || a.Hq < 0 || a.Hkv < 1 || a.num_blocks < 1 || a.R < 0 || a.axes < 1) return TSD_ERR_ARG;
  if (D != 64 && D != 128) return TSD_ERR_LIMIT;
  if (a.R > D || a.R % 32 != 0 || a.axes > kMaxAxes || a.Hq > 65535 || a.Hkv > 65535 || a.T > 0x7FFFFFFFll ||
      (int64_t)a.num_blocks * kPage > 0x7FFFFFFFll)
    return TSD_ERR_LIMIT;
  if (a.T == 0) return TSD_OK;
  if (!a.k || !a.v || !a.slots || !a.kc || !a.vc || (a.Hq > 0 && (!a.q || !a.q_out))) return TSD_ERR_ARG;
  if (a.R > 0 && !a.inv_freq) return TSD_ERR_ARG;
  if (a.per_base < 1 || !(a.eps >= 0.f)) return TSD_ERR_ARG;
  if (!aligned(a.q, 16) || !aligned(a.k, 16) || !aligned(a.v, 16) || !aligned(a.q_out, 16) ||
      !aligned(a.kc, 16) || !aligned(a.vc, 16) || !aligned(a.q_weight, 16) || !aligned(a.k_weight, 16))
    return TSD_ERR_ARG;
  if (a.q_stride % 8 || a.k_stride % 8 || a.v_stride % 8 || a.q_out_stride % 8) return TSD_ERR_ARG;
  const int64_t qrow = (int64_t)a.Hq * D, row = (int64_t)a.Hkv * D;
  if (a.T > 1 && (a.q_stride < qrow || a.q_out_stride < qrow || a.k_stride < row || a.v_stride < row))
    return TSD_ERR_ARG;
  const cudaStream_t s = as_cuda(stream);
  const cudaError_t e = q4 ? (D == 128 ? append_launch<128, true>(a, s) : append_launch<64, true>(a, s))
                           : (D == 128 ? append_launch<128, false>(a, s) : append_launch<64, false>(a, s));
  return e == cudaSuccess ? TSD_OK : TSD_ERR_CUDA;
}

}  // namespace
}  // namespace tsd

TSD_API int tsd_kv_append_rope(const uint16_t *q, int64_t q_stride, const uint16_t *k, int64_t k_stride,
                               const uint16_t *v, int64_t v_stride, const int32_t *slots, int64_t T,
                               int Hq, int Hkv, int D, const float *inv_freq, int R,
                               const int32_t *freq_axis, int axes, int interleaved, float rot_scale,
                               const int32_t *pos, const int32_t *base, int64_t per_base,
                               const uint16_t *q_weight, const uint16_t *k_weight, float eps,
                               int num_blocks, uint16_t *k_cache, uint16_t *v_cache, uint16_t *q_out,
                               int64_t q_out_stride, int32_t *status, tsd_stream_t stream) {
  tsd::AppendArgs a{q, k, v, q_stride, k_stride, v_stride, q_out_stride, q_out, slots, T, Hq, Hkv, R, axes,
                    interleaved, inv_freq, freq_axis, pos, base, per_base, q_weight, k_weight, eps,
                    rot_scale, num_blocks, reinterpret_cast<uint8_t *>(k_cache),
                    reinterpret_cast<uint8_t *>(v_cache), 0, 0, status};
  return tsd::append(a, false, D, stream);
}

TSD_API int tsd_kv_append_rope_q4(const uint16_t *q, int64_t q_stride, const uint16_t *k,
                                  int64_t k_stride, const uint16_t *v, int64_t v_stride,
                                  const int32_t *slots, int64_t T, int Hq, int Hkv, int D,
                                  const float *inv_freq, int R, const int32_t *freq_axis, int axes,
                                  int interleaved, float rot_scale, const int32_t *pos,
                                  const int32_t *base, int64_t per_base, const uint16_t *q_weight,
                                  const uint16_t *k_weight, float eps, int num_blocks, uint8_t *k_cache,
                                  uint8_t *v_cache, uint16_t *q_out, int64_t q_out_stride,
                                  int32_t *status, tsd_stream_t stream) {
  tsd::AppendArgs a{q, k, v, q_stride, k_stride, v_stride, q_out_stride, q_out, slots, T, Hq, Hkv, R, axes,
                    interleaved, inv_freq, freq_axis, pos, base, per_base, q_weight, k_weight, eps,
                    rot_scale, num_blocks, k_cache, v_cache, 0, 0, status};
  return tsd::append(a, true, D, stream);
}
