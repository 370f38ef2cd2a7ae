// Tree-masked attention over the 4-bit paged cache (format: q4.cuh), for one
// query token per sequence as well as for draft trees.
//
// "EAGLE-Pangu: Accelerator-Safe Tree Speculative Decoding on Ascend NPUs",
// technical summary 2.3: every node of the tree attends, in one pass, to the
// committed prefix and to its own ancestor path; the rows of a kv head are
// node-major (row = node * g + head-in-group), so a GQA group shares K and V.
//
// Few rows (tree_attn_q4_rows): the kernel is bound by the cache's bytes (9 D
// a page, a quarter of bf16), so K and V go from the page to the tensor
// core's operand registers without a second pass through shared memory.  A
// warp owns whole pages: its lanes copy a page's K and V asynchronously, 16 bytes
// each, into the warp's ring (bulk copies of a page's 9 D bytes took 80 ns each,
// whatever the ring's depth), and it computes, for 8 rows at a time,
//   S^T (16 keys x 8 rows) = K Q^T      A = K, decoded in registers
//   P^T = exp2(S^T * c - m)             fp32, packed to fp16, transposed in
//                                       registers by movmatrix
//   O^T (D x 8 rows) += V^T P^T         A = V^T, decoded in registers
// with fp16 operands and fp32 accumulation (m16n8k16).  Decoded values are
// exact in fp16.  q (bf16) is scaled per row by a power of two that brings
// its largest magnitude to [2^13, 2^14) and then converted: exact for every
// element within 2^-27 of that magnitude, below which the rounding (2^-25
// absolute) is lost in the fp32 accumulation anyway; the power goes into the
// softmax's factor.  P lies in (0, 2^15] (the reference m is 8 below the row's
// first maximum and follows when a score passes that maximum by 7), so fp16
// keeps 11 bits of every probability down to 2^-22 of the largest, 3 bits more
// than bf16 would; the row sum uses the unrounded fp32 values.
//
// Operand layout.  The contraction index of an MMA may be permuted freely, so
// lane (i, t) = (lane / 4, lane % 4) takes, as A rows i and i + 8 of K, D/4
// consecutive columns of two keys (one 16-byte read for D = 128), and of V
// the D/8 consecutive columns from i D/8 on of four keys.  The order of a
// page's keys over the A rows (i ^ (i >> 1 & 1)) makes the K reads free of
// bank conflicts and the V reads two-way.
//
// Cutting up the key ranges: one cluster a range, equal parts of all ranges end to
// end (attention_q4.cuh), or, for batches beyond a plan, uniform pieces; partial rows are
// joined in fp32, in shared memory or by a second kernel.
//
// Measured (device time): one token behind 4096 keys, 32 query and 8 kv heads of 128: 9 us; 32
// tokens behind 512 to 16384 keys, 64 / 8 heads: 70 us for 312 MB (66% of the copy
// bandwidth); behind 16384 each, 32 / 8 heads: 111 us for 604 MB (80%).  Batches of 128 and
// 256 tokens behind 512 to 16384 keys, 64 / 8 heads, in uniform pieces: 252 and 455 us (73
// and 81%), with a bound of 131072 keys 262 and 455; 65 tokens 139, with that bound 170 (64
// tokens, planned: 125 with any bound).  A warp takes two
// pages at a time (with up to 8 rows; more would not leave the registers): one at a
// time, with some 350 instructions a page, the three took 9, 75 and 125 us, the copies
// of the second alone 56 and its arithmetic alone 66; and of that kernel ten
// warps a block (96 registers) took 80 us, three blocks an SM (80 registers) 125, the
// next page's scores ahead of this page's products 77, a ring of five pages 76.

#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "attention_q4.cuh"
#include "sm100_ptx.cuh"

namespace tsd {
namespace {

constexpr int kRowsThreads = 256;
constexpr int kRowsWarps = kRowsThreads / 32;
constexpr float kOffset = 8.f;  // P of the reference score is 2^8
constexpr float kSlack = 7.f;   // P stays at or below 2^15
constexpr float kRowsLn2 = 0.6931471805599453f;

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9},"
      " {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}
template <int N>
__device__ __forceinline__ void lds_words(const uint8_t *p, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    const uint4 x = *reinterpret_cast<const uint4 *>(p);
    w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
  } else if constexpr (N == 2) {
    const uint2 x = *reinterpret_cast<const uint2 *>(p);
    w[0] = x.x; w[1] = x.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t *>(p);
  }
}

template <int D, int NT>
struct RowsLayout {
  static constexpr int kPageBytes = Q4Page<D>::kBytes;
  // Pages that a warp takes at a time, and the stages of its ring of such items
  static constexpr int kItem = NT == 1 ? 2 : 1, kStages = 4 / kItem;
  static constexpr int kPair = 2 * kPageBytes;  // a page's K and V
  static constexpr int kStage = kItem * kPair;
  static constexpr int kChunks = kPair / 16;  // 16-byte copies of a K and a V page
  static constexpr int kRing = kRowsWarps * kStages * kStage;
  static constexpr int kMerge = kRowsWarps * 8 * NT * D * 4;  // O of every warp
  static constexpr int kBlock = 8 * NT * D * 4;               // O of the block
  static constexpr int kBytes = kRing > kMerge + kBlock ? kRing : kMerge + kBlock;
  static_assert(kPageBytes % 16 == 0, "copies start on 16 bytes");
};

// Four columns of a finished row: O / sum in bf16, and the row's lse.
__device__ __forceinline__ void rows_out(const Q4Attn &p, size_t orow, int D, int c, float4 a, float M,
                                         float sum, bool skip) {
  const bool empty = skip || sum == 0.f;
  const float inv = empty ? 0.f : 1.f / sum;
  *reinterpret_cast<uint2 *>(p.out + orow * D + 4 * c) =
      empty ? make_uint2(0u, 0u)
            : make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
  if (c == 0 && p.lse) p.lse[orow] = empty ? -INFINITY : (M + log2f(sum)) * kRowsLn2;
}

struct RowsShared {
  float2 ml[kRowsWarps][16];  // (reference, sum) of each warp's rows
  float4 block_ml[16];        // and of the block's (sum -1: bad page)
  int bad;
  Q4Plan plan;
};

// Grid (splits * row blocks * Hkv, B).  A block owns 8 NT rows of one kv head
// and one piece of the key range; its warps take the piece's pages in turn.
// With p.cluster the pieces of a range are one thread-block cluster: each
// sequence is cut into equal parts of its own length, and the parts meet
// through distributed shared memory, without a workspace or a second kernel.
template <int D, int NT>
__global__ void __launch_bounds__(kRowsThreads, 2) tree_attn_q4_rows_kernel(const Q4Attn p) {
  using namespace sm100;
  using L = RowsLayout<D, NT>;
  using Page = Q4Page<D>;
  constexpr int kSteps = D / 16;      // contraction steps of S
  constexpr int kWordsK = D / 32;     // code words of a lane's part of a key
  constexpr int kWordsV = D / 64;     // code words of a lane's part of a V row
  constexpr int kTiles = D / 16;      // M tiles of O^T
  constexpr int kItem = L::kItem, kStages = L::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ RowsShared sh;
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int qi = lane >> 2, qt = lane & 3;  // (i, t)
  pdl_wait();
  if (p.planned && warp == 0) q4_plan(p, sh.plan);
  __syncthreads();
  Q4Seg seg;
  int g = p.planned ? blockIdx.x * sh.plan.part : 0;
  while (q4_next(p, sh.plan, g, seg)) {
    __syncthreads();  // the last segment's shared memory is read
    if (tid == 0) sh.bad = 0;
    __syncthreads();
    const int b = seg.b, h = seg.h, P = seg.P, nb = seg.nb, first = seg.first, last = seg.last;
    const int row0 = seg.rb * 8 * NT;
    const int rows_valid = nb * p.g;
    const bool work = row0 < rows_valid && first < last;
    if (!work && !seg.direct && !p.cluster) continue;

    float o[NT][kTiles][4];
    float l[NT][2], trig[NT][2], ref[NT][2], mul[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int j = 0; j < kTiles; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][j][e] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[n][e] = 0.f;
        trig[n][e] = -INFINITY;  // the score that moves the reference
        ref[n][e] = 0.f;
        mul[n][e] = 0.f;
      }
    }

    if (work) {
      // ---- the page stream: each item is one group of the lanes' copies ----
      const int32_t *trow = p.table + (size_t)b * p.max_blocks;
      const int items = (last - first + kItem - 1) / kItem;
      const int mine = items > warp ? (items - warp + kRowsWarps - 1) / kRowsWarps : 0;
      const uint32_t ring = smem_addr(smem) + warp * kStages * L::kStage;
      const uint8_t *ring_p = smem + warp * kStages * L::kStage;
      auto page_of = [&](int it, int h) { return first + (warp + it * kRowsWarps) * kItem + h; };
      int ids = 0;  // lane i: the id of this warp's page 32 * batch + i
      bool stop = false;
      constexpr int kBatch = 32 / kItem;  // items whose ids are read together
      auto fetch_ids = [&](int it) {
        const int j = it + lane / kItem, page = page_of(j, lane % kItem);
        const int id = j < mine && page < last ? trow[page] : 0;
        const bool bad = id < 0 || id >= p.num_blocks;
        if (__any_sync(0xffffffffu, bad)) {
          stop = true;
          if (lane == 0) sh.bad = 1;
        }
        ids = id;
      };
      // The lane's c-th copy is chunk 32 c + lane of K's page followed by V's; only
      // round kMixed (chunks of both) depends on the lane.
      constexpr int kHalfChunks = L::kChunks / 2, kMixed = kHalfChunks / 32;
      const uint8_t *k_lane = p.k + 16 * lane, *v_lane = p.v - 16 * kHalfChunks + 16 * lane;
      const uint8_t *mixed = kMixed * 32 + lane < kHalfChunks ? k_lane : v_lane;
      auto issue = [&](int it) {
        const uint32_t dst0 = ring + (it % kStages) * L::kStage + 16 * lane;
#pragma unroll
        for (int hp = 0; hp < kItem; ++hp) {
          if (hp > 0 && page_of(it, hp) >= last) break;  // (an odd end; its scores are masked)
          const int id = __shfl_sync(0xffffffffu, ids, (it % kBatch) * kItem + hp);
          const size_t off = ((size_t)id * p.Hkv + h) * L::kPageBytes;
          const uint32_t dst = dst0 + hp * L::kPair;
#pragma unroll
          for (int c = 0; c < (L::kChunks + 31) / 32; ++c) {
            const uint8_t *src = (c < kMixed ? k_lane : c == kMixed ? mixed : v_lane) + off + 512 * c;
            if ((c + 1) * 32 <= L::kChunks || c * 32 + lane < L::kChunks) cp_async_16(dst + 512 * c, src);
          }
        }
      };
      auto commit = [] { asm volatile("cp.async.commit_group;\n" ::: "memory"); };
      if (mine > 0) fetch_ids(0);
      int issued = 0;
      for (int i = 0; i < kStages; ++i) {  // one group a stage, an empty one past the end
        if (!stop && issued < mine) issue(issued++);
        commit();
      }

      // ---- Q^T as B operands: row i of each 8-row tile ----
      uint32_t qf[NT][kSteps][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int r = row0 + 8 * n + qi;
        uint32_t raw[D / 8];  // D/4 bf16 columns from qt * D/4 on
        if (r < rows_valid) {
          const uint4 *src = reinterpret_cast<const uint4 *>(p.q + q4_out_row(p, b, h, r) * D + qt * (D / 4));
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            const uint4 x = src[c];
            raw[4 * c] = x.x; raw[4 * c + 1] = x.y; raw[4 * c + 2] = x.z; raw[4 * c + 3] = x.w;
          }
        } else {
#pragma unroll
          for (int c = 0; c < D / 8; ++c) raw[c] = 0u;
        }
        float amax = 0.f;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          amax = fmaxf(amax, fabsf(__uint_as_float(raw[c] << 16)));
          amax = fmaxf(amax, fabsf(__uint_as_float(raw[c] & 0xFFFF0000u)));
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const int e = q4_exponent(amax);
        const float up1 = q4_pow2(e / 2), up2 = q4_pow2(e - e / 2);
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const float lo = __uint_as_float(raw[c] << 16) * up1 * up2;
          const float hi = __uint_as_float(raw[c] & 0xFFFF0000u) * up1 * up2;
          // columns 4 s + {0, 1} feed b0 of step s, 4 s + {2, 3} its b1
          qf[n][c / 2][c & 1] = pack_half2(lo, hi);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {  // this lane's score columns are rows 2 t and 2 t + 1
          const int er = __shfl_sync(0xffffffffu, e, (2 * qt + s) * 4);
          mul[n][s] = p.scale_log2 * q4_pow2(-(er / 2)) * q4_pow2(-(er - er / 2));
        }
      }

      const int key_a = qi ^ ((qi >> 1) & 1);  // A row i; row i + 8 is key_a + 8
      // V's contraction indices 2t, 2t+1, 2t+8, 2t+9 are A rows 2t, 2t+1, ...
      const int kv0 = (2 * qt) ^ (qt & 1), kv1 = (2 * qt + 1) ^ (qt & 1);

      for (int it = 0; it < mine && !stop; ++it) {
        asm volatile("cp.async.wait_group %0;\n" ::"n"(kStages - 1) : "memory");
        __syncwarp();
        const uint8_t *item = ring_p + (it % kStages) * L::kStage;
        const int t0 = page_of(it, 0) * kPage;  // first key slot

        // S^T
        float s[kItem][NT][4];
#pragma unroll
        for (int hp = 0; hp < kItem; ++hp) {
          const uint8_t *kp = item + hp * L::kPair;
#pragma unroll
          for (int n = 0; n < NT; ++n) s[hp][n][0] = s[hp][n][1] = s[hp][n][2] = s[hp][n][3] = 0.f;
          uint32_t wa[kWordsK], wb[kWordsK];
          lds_words(kp + key_a * Page::kRow + qt * (D / 8), wa);
          lds_words(kp + (key_a + 8) * Page::kRow + qt * (D / 8), wb);
          uint32_t sa[2], sb[2];  // scales of the lane's (one or two) groups of 16 columns
          if constexpr (D == 128) {
            const uint32_t xa = *reinterpret_cast<const uint16_t *>(kp + Page::kScales + key_a * 8 + 2 * qt);
            const uint32_t xb =
                *reinterpret_cast<const uint16_t *>(kp + Page::kScales + (key_a + 8) * 8 + 2 * qt);
            sa[0] = (xa & 0xFFu) * 0x00800080u;
            sa[1] = (xa >> 8) * 0x00800080u;
            sb[0] = (xb & 0xFFu) * 0x00800080u;
            sb[1] = (xb >> 8) * 0x00800080u;
          } else {
            sa[0] = sa[1] = kp[Page::kScales + key_a * 4 + qt] * 0x00800080u;
            sb[0] = sb[1] = kp[Page::kScales + (key_a + 8) * 4 + qt] * 0x00800080u;
          }
#pragma unroll
          for (int w = 0; w < kWordsK; ++w) {
            uint32_t ra[4], rb4[4];
            q4_decode8(wa[w], ra);
            q4_decode8(wb[w], rb4);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              ra[e] = q4_mul2(ra[e], sa[w / 2]);
              rb4[e] = q4_mul2(rb4[e], sb[w / 2]);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma_f16(s[hp][n], ra[0], rb4[0], ra[1], rb4[1], qf[n][2 * w][0], qf[n][2 * w][1]);
              mma_f16(s[hp][n], ra[2], rb4[2], ra[3], rb4[3], qf[n][2 * w + 1][0], qf[n][2 * w + 1][1]);
            }
          }
        }

        // V's codes and scales; slots past the sequence read as zero
        uint32_t wv[kItem][4][kWordsV], sv[kItem][4];
        const int kk[4] = {kv0, kv1, kv0 + 8, kv1 + 8};
#pragma unroll
        for (int hp = 0; hp < kItem; ++hp) {
          const uint8_t *vp = item + hp * L::kPair + L::kPageBytes;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            lds_words(vp + kk[e] * Page::kRow + qi * (D / 16), wv[hp][e]);
            sv[hp][e] = vp[Page::kScales + kk[e] * Page::kScaleRow + qi * (D / 8) / kQ4Group];
          }
        }
        // the item is in registers: its stage can be refilled
        __syncwarp();
        if (issued < mine) {
          if (issued % kBatch == 0) fetch_ids(issued);
          if (!stop) issue(issued++);
        }
        commit();

        // softmax: t = s * mul, and what the row may not see is -inf
#pragma unroll
        for (int hp = 0; hp < kItem; ++hp)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            s[hp][n][0] *= mul[n][0];
            s[hp][n][1] *= mul[n][1];
            s[hp][n][2] *= mul[n][0];
            s[hp][n][3] *= mul[n][1];
          }
        if (t0 + kItem * kPage > P) {
#pragma unroll
          for (int hp = 0; hp < kItem; ++hp) {
            const int at = t0 + hp * kPage;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int r = row0 + 8 * n + 2 * qt + e;
                const uint32_t vis = r < rows_valid ? q4_visible(p, b, r / p.g, at - P, nb) : 0u;
                if (!((vis >> key_a) & 1u)) s[hp][n][e] = -INFINITY;
                if (!((vis >> (key_a + 8)) & 1u)) s[hp][n][2 + e] = -INFINITY;
              }
            }
            // V's slots past the sequence read as zero.  Scale bytes that no writer makes
            // can only be met here, in slots of the tree that were not written: they read
            // as the largest scale, so that P = 0 really leaves them out.
#pragma unroll
            for (int e = 0; e < 4; ++e) sv[hp][e] = at + kk[e] >= P + nb ? 0u : min(sv[hp][e], kQ4MaxScale);
          }
        }
        float most[NT][2];  // the lane's largest scores
        bool over = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            most[n][e] = fmaxf(s[0][n][e], s[0][n][2 + e]);
            if constexpr (kItem == 2) most[n][e] = fmax3(most[n][e], s[1][n][e], s[1][n][2 + e]);
            over = over || most[n][e] > trig[n][e];
          }
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
          for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float m = most[n][e];
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
              if (m > trig[n][e]) {  // the same decision in the eight lanes of the row
                // (for scores whose ulp is coarser than these steps: at the maximum)
                const float to = m - (m - kOffset) <= kOffset ? m - kOffset : m;
                const float f = trig[n][e] == -INFINITY ? 0.f : ex2_approx(ref[n][e] - to);
                trig[n][e] = (m + kSlack) - m <= kSlack ? m + kSlack : m;
                ref[n][e] = to;
                l[n][e] *= f;
#pragma unroll
                for (int j = 0; j < kTiles; ++j) {
                  o[n][j][e] *= f;
                  o[n][j][2 + e] *= f;
                }
              }
            }
          }
        }
#pragma unroll
        for (int hp = 0; hp < kItem; ++hp) {
          uint32_t pb[NT][2];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const float p0 = ex2_approx(s[hp][n][0] - ref[n][0]), p1 = ex2_approx(s[hp][n][1] - ref[n][1]);
            const float p2 = ex2_approx(s[hp][n][2] - ref[n][0]), p3 = ex2_approx(s[hp][n][3] - ref[n][1]);
            l[n][0] += p0 + p2;
            l[n][1] += p1 + p3;
            pb[n][0] = transpose8x8(pack_half2(p0, p1));
            pb[n][1] = transpose8x8(pack_half2(p2, p3));
          }

          // O^T: M tile j holds columns i D/8 + 2 j (row i) and the next (row i + 8).  An
          // operand register holds one column of two keys, so the codes of two keys are
          // interleaved before they are decoded (three operations for eight registers;
          // after, it takes a byte permutation each, on the pipe that also converts).
          const uint32_t s01 = sv[hp][0] * 0x80u + sv[hp][1] * 0x00800000u;
          const uint32_t s23 = sv[hp][2] * 0x80u + sv[hp][3] * 0x00800000u;
#pragma unroll
          for (int w = 0; w < kWordsV; ++w) {
            const uint32_t v0 = wv[hp][0][w], v1 = wv[hp][1][w], v2 = wv[hp][2][w], v3 = wv[hp][3][w];
            uint32_t a0[4], a1[4], a2[4], a3[4];
            q4_decode8((v0 & 0x0F0F0F0Fu) | (v1 * 16u & 0xF0F0F0F0u), a0);
            q4_decode8(((v0 >> 4) & 0x0F0F0F0Fu) | (v1 & 0xF0F0F0F0u), a1);
            q4_decode8((v2 & 0x0F0F0F0Fu) | (v3 * 16u & 0xF0F0F0F0u), a2);
            q4_decode8(((v2 >> 4) & 0x0F0F0F0Fu) | (v3 & 0xF0F0F0F0u), a3);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              a0[j] = q4_mul2(a0[j], s01);
              a1[j] = q4_mul2(a1[j], s01);
              a2[j] = q4_mul2(a2[j], s23);
              a3[j] = q4_mul2(a3[j], s23);
#pragma unroll
              for (int n = 0; n < NT; ++n)
                mma_f16(o[n][4 * w + j], a0[j], a1[j], a2[j], a3[j], pb[n][0], pb[n][1]);
            }
          }
        }
      }
      cp_async_wait_all();  // before the ring's memory is used again
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 4);
          l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 8);
          l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 16);
        }
    }

    // ---- join the warps: every ring is drained, its memory holds their O ----
    __syncthreads();
    float *merge = reinterpret_cast<float *>(smem);
    float *block_o = reinterpret_cast<float *>(smem + L::kMerge);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * n + 2 * qt + e;
        if (qi == 0)
          sh.ml[warp][r] = make_float2(trig[n][e] == -INFINITY && l[n][e] == 0.f ? -INFINITY : ref[n][e], l[n][e]);
        float *dst = merge + ((size_t)warp * 8 * NT + r) * D + qi * (D / 8);
#pragma unroll
        for (int j = 0; j < kTiles; j += 2)
          *reinterpret_cast<float4 *>(dst + 2 * j) =
              make_float4(o[n][j][e], o[n][j][2 + e], o[n][j + 1][e], o[n][j + 1][2 + e]);
      }
    }
    __syncthreads();
    const bool bad = sh.bad != 0;
    if (tid == 0 && bad && p.status) atomicOr(p.status, TSD_STATUS_BAD_PAGE);
    constexpr int kVec = D / 4;  // float4 of a row
    for (int x = tid; x < 8 * NT * kVec; x += kRowsThreads) {
      const int rl = x / kVec, c = x % kVec, r = row0 + rl;
      if (r >= p.rows) break;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kRowsWarps; ++w) M = fmaxf(M, sh.ml[w][rl].x);
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
      float sum = 0.f;
      if (M > -INFINITY) {
#pragma unroll
        for (int w = 0; w < kRowsWarps; ++w) {
          const float2 ml = sh.ml[w][rl];
          const float f = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - M);
          const float4 v = *reinterpret_cast<const float4 *>(merge + ((size_t)w * 8 * NT + rl) * D + 4 * c);
          a.x += f * v.x;
          a.y += f * v.y;
          a.z += f * v.z;
          a.w += f * v.w;
          sum += f * ml.y;
        }
      }
      if (p.cluster) {
        *reinterpret_cast<float4 *>(block_o + rl * D + 4 * c) = a;
        if (c == 0) sh.block_ml[rl] = make_float4(M, bad ? -1.f : sum, 0.f, 0.f);
      } else if (!seg.direct) {
        if (r >= rows_valid) continue;
        const size_t pr = seg.part + rl;
        *reinterpret_cast<float4 *>(p.part_o + pr * D + 4 * (c ^ (rl & 7))) = a;  // (see the join)
        if (c == 0) p.part_ml[pr] = make_float2(M, bad ? -1.f : sum);
      } else if (!p.planned || r < rows_valid) {  // (planned: the join writes the others)
        rows_out(p, q4_out_row(p, b, h, r), D, c, a, M, sum, r >= rows_valid || bad);
      }
    }
    if (!p.cluster) continue;
    // every block of the cluster takes a share of the rows' columns
    const int split = cluster_ctarank();
    cluster_arrive();
    cluster_wait();
    for (int x = split * kRowsThreads + tid; x < 8 * NT * kVec; x += p.splits * kRowsThreads) {
      const int rl = x / kVec, c = x % kVec, r = row0 + rl;
      if (r >= p.rows) break;
      float M = -INFINITY;
      bool skip = r >= rows_valid;
      for (int s = 0; s < p.splits; ++s) {
        const float4 ml = ld_dsmem_f4(smem_addr(&sh.block_ml[rl]), s);
        M = fmaxf(M, ml.x);
        skip = skip || ml.y == -1.f;
      }
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
      float sum = 0.f;
      if (M > -INFINITY) {
        for (int s = 0; s < p.splits; ++s) {
          const float4 ml = ld_dsmem_f4(smem_addr(&sh.block_ml[rl]), s);
          const float4 v = ld_dsmem_f4(smem_addr(block_o + rl * D + 4 * c), s);
          const float f = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - M);
          a.x += f * v.x;
          a.y += f * v.y;
          a.z += f * v.z;
          a.w += f * v.w;
          sum += f * ml.y;
        }
      }
      rows_out(p, q4_out_row(p, b, h, r), D, c, a, M, sum, skip);
    }
    cluster_arrive();  // no block leaves while another reads its shared memory
    cluster_wait();
  }
}

// One warp per output row: joins the pieces of its key range (fp32), rounds
// once to bf16.  Rows of skipped sequences and padding nodes become 0 / -inf.
template <int D>
__global__ void __launch_bounds__(256) tree_attn_q4_join_kernel(const Q4Attn p) {
  using namespace sm100;
  constexpr int kPer = D / 32;  // columns of a lane
  pdl_trigger();
  pdl_wait();
  const int64_t x = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (x >= (int64_t)p.B * p.Hkv * p.rows) return;
  const int r = (int)(x % p.rows);
  const int64_t bh = x / p.rows;
  const int h = (int)(bh % p.Hkv), b = (int)(bh / p.Hkv);
  int P, nb;
  bool bad_len;
  const bool ok = q4_seq(p, b, P, nb, bad_len) && r < nb * p.g;
  const int rb = r / p.rows_per_block;
  const int rl = r % p.rows_per_block;
  int pieces = 0, k0 = 0;  // planned: the block of the range's first unit
  if (ok && p.planned) {
    const int4 plan = p.plan[b];
    const int t = plan.y, rbs = plan.z >> 2, last_w = plan.z & 3, part = plan.w;
    const int full = p.range_cost + t * p.row_tiles;
    const int first = plan.x + h * (rbs * full - t * (p.row_tiles - last_w)) + rb * full + p.range_cost;
    k0 = first / part;
    pieces = (first + (t - 1) * (rb == rbs - 1 ? last_w : p.row_tiles)) / part - k0 + 1;
    if (pieces == 1) return;  // its block has written it
  } else if (ok) {
    pieces = ((P + nb + kPage - 1) / kPage + p.chunk - 1) / p.chunk;
  }
  const size_t base = p.planned ? 0 : q4_part_row(p, b, h, rb, 0);
  auto part_row = [&](int s) -> size_t {
    if (!p.planned) return base + (size_t)s * p.rows_per_block + rl;
    return ((size_t)(k0 + s) * 2 + (s == 0 ? 1 : 0)) * p.rows_per_block + rl;
  };
  // lane l holds the (reference, sum) of pieces l, l + 32, ...: at most 64
  float2 ml[2] = {make_float2(-INFINITY, 0.f), make_float2(-INFINITY, 0.f)};
#pragma unroll
  for (int e = 0; e < 2; ++e)
    if (lane + 32 * e < pieces) ml[e] = p.part_ml[part_row(lane + 32 * e)];
  const bool bad = __any_sync(0xffffffffu, ml[0].y == -1.f || ml[1].y == -1.f);
  float M = fmaxf(ml[0].x, ml[1].x);
#pragma unroll
  for (int off = 16; off; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  float f[2], sum = 0.f;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    f[e] = ml[e].x == -INFINITY ? 0.f : ex2_approx(ml[e].x - M);
    sum += f[e] * ml[e].y;
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  const bool empty = !ok || bad || sum == 0.f;
  float a[kPer];
#pragma unroll
  for (int c = 0; c < kPer; ++c) a[c] = 0.f;
  for (int s = 0; s < pieces; ++s) {
    const float fs = __shfl_sync(0xffffffffu, s < 32 ? f[0] : f[1], s & 31);
    // (a partial row's 16-byte chunks are swizzled by its place in the block, which
    // spreads the many-row kernel's stores over the banks)
    const float *src = p.part_o + part_row(s) * D + ((lane * kPer / 4) ^ (rl & 7)) * 4 + lane * kPer % 4;
    if constexpr (kPer == 4) {
      const float4 v = *reinterpret_cast<const float4 *>(src);
      a[0] += fs * v.x;
      a[1] += fs * v.y;
      a[2] += fs * v.z;
      a[3] += fs * v.w;
    } else {
      const float2 v = *reinterpret_cast<const float2 *>(src);
      a[0] += fs * v.x;
      a[1] += fs * v.y;
    }
  }
  const float inv = empty ? 0.f : 1.f / sum;
  const size_t orow = q4_out_row(p, b, h, r);
  uint32_t w[kPer / 2];
#pragma unroll
  for (int c = 0; c < kPer / 2; ++c) w[c] = empty ? 0u : pack_bf16x2(a[2 * c] * inv, a[2 * c + 1] * inv);
  uint16_t *dst = p.out + orow * D + lane * kPer;
  if constexpr (kPer == 4)
    *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
  else
    *reinterpret_cast<uint32_t *>(dst) = w[0];
  if (lane == 0 && p.lse) p.lse[orow] = empty ? -INFINITY : (M + log2f(sum)) * kRowsLn2;
}

// Key ranges of up to this many pages are the work of one cluster where all clusters
// run at once: no workspace, and no second launch.  Alone, a cluster is faster up
// to 16384 keys or so (one token, 8 kv heads, clusters / planned parts: 1024 keys 7.0 /
// 12.2 us, 4096 9.0 / 13.0, 8192 11.8 / 16.1, 16384 17.9 / 19.1, 32768 28 / 24).  In a
// batch every cluster has the same number of blocks, and the longest range is what
// counts: 16 sequences of 4096 keys 22.8 / 25.9 us, of 64 to 8192 keys 41 / 29.
constexpr int kClusterPages = 1024, kClusterPagesBatch = 288;

struct Q4Shape {
  bool tc;       // the many-row kernel
  bool cluster;  // pieces joined inside a cluster
  bool planned;  // equal parts of all ranges end to end
  int nt, rows_per_block, row_blocks, splits, chunk, blocks;
  size_t plan_bytes, ml_bytes, bytes;  // workspace: the plan, (reference, sum) of the partial rows, the rows
};


// Fixed cost of a key range, in units of 128 keys of one row tile.  Measured (with
// kernels a little slower than these), 16 trees of up to 31 nodes over 512 to 8192 slots,
// many-row kernel: 0: 110 us, 4: 79, 6: 74, 8: 71, 10: 71, 16: 78; 32 tokens over 512
// to 16384 slots, few-row kernel: 0: 94 us, 2: 83, 5: 73, 7: 70, 10: 70.  64 trees
// take 216 us with 7, 208 with 8, 203 with 9 and 10.  Equal long ranges take the same
// time with any.
constexpr int kTcRangeCost = 9, kRowsRangeCost = 7;

// The many-row kernel needs some 15 us more to get going, and then takes 128 or 256 rows
// through a decoded tile where the few-row kernel takes 16: it runs from this much
// work on, in units of 128 keys of 16 rows and with a range's fixed cost.  Measured, few
// / many rows (8 kv heads; rows of one, sequences, keys): 32, 1, 2048: 14 / 27 us; 252,
// 1, 2048: 23 / 30; 32, 8, 1024: 17 / 28; 64, 1, 8192: 27 / 29; 64, 8, 512: 27 / 24;
// 64, 8, 1024: 32 / 28; 64, 1, 16384: 39 / 31; 32, 32, 8192: 212 / 163.
constexpr int64_t kTcMinWork = 3080;

// Host: how a call is cut up.
Q4Shape q4_shape(int B, int N_max, int Hq, int Hkv, int D, int max_slots) {
  Q4Shape pl = {};
  const int rows = N_max * (Hq / Hkv);
  const int pages = (max_slots + kPage - 1) / kPage, units = (pages + kUnitPages - 1) / kUnitPages;
  pl.tc = rows > 16 && (int64_t)B * Hkv * ((rows + 15) / 16) * (units + kRowsRangeCost) > kTcMinWork;
  pl.nt = rows > 8 ? 2 : 1;
  pl.rows_per_block = pl.tc ? (rows > 128 ? 256 : 128) : 8 * pl.nt;
  pl.row_blocks = (rows + pl.rows_per_block - 1) / pl.rows_per_block;
  const int64_t base = (int64_t)B * Hkv * pl.row_blocks;
  const int slots = (pl.tc ? 1 : 2) * sm_count();
  pl.splits = 1;
  pl.chunk = pages;
  // one piece a range: short ranges, or so many that they fill the GPU many times
  if (units <= 2 || base >= 64ll * slots) return pl;
  if (!pl.tc && pages <= (B == 1 ? kClusterPages : kClusterPagesBatch) && 2 * base <= slots) {
    // Short ranges of few blocks: a cluster of 2, 4 or 8, as long as all run at once.
    int c = 2;
    while (c < 8 && 2 * c * base <= slots && c < units) c *= 2;
    pl.cluster = true;
    pl.splits = c;
    return pl;
  }
  size_t pieces;
  if (B <= kPlanSeqs && base * (2 * units + 64) < (1ll << 30)) {
    pl.planned = true;
    // as many parts as blocks run at a time; parts are longer where that would cut
    // a range into more than kPlanPieces
    pl.blocks = slots;
    pieces = 2 * (size_t)pl.blocks;
  } else {
    // Batches too large to plan: enough pieces of the longest range for four
    // blocks a slot.
    const int64_t want = std::min<int64_t>((4ll * slots + base - 1) / base, std::min(units, 32));
    pl.chunk = (int)((units + want - 1) / want) * kUnitPages;
    pl.splits = (pages + pl.chunk - 1) / pl.chunk;
    if (pl.splits == 1) return pl;
    pieces = (size_t)base * pl.splits;
  }
  const size_t part_rows = pieces * pl.rows_per_block;
  pl.plan_bytes = align_up(kPlanSeqs * sizeof(int4), 256);
  pl.ml_bytes = align_up(part_rows * sizeof(float2), 256);
  pl.bytes = pl.plan_bytes + pl.ml_bytes + part_rows * D * sizeof(float);
  return pl;
}

template <int D, int NT>
cudaError_t rows_launch(const Q4Attn &p, int blocks, cudaStream_t s) {
  const int smem = RowsLayout<D, NT>::kBytes;
  if (!set_smem((const void *)tree_attn_q4_rows_kernel<D, NT>, smem)) return cudaErrorUnknown;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = p.planned ? dim3(blocks) : dim3((unsigned)p.splits * p.Hkv * p.row_blocks, p.B);
  cfg.blockDim = dim3(kRowsThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.cluster ? p.splits : 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, tree_attn_q4_rows_kernel<D, NT>, p);
}

int q4_check(int B, int N_max, int Hq, int Hkv, int D, int max_slots) {
  if (B < 0 || N_max < 1 || Hq < 1 || Hkv < 1 || max_slots < 1) return TSD_ERR_ARG;
  if (D != 64 && D != 128) return TSD_ERR_LIMIT;
  if (N_max > kMaxNodes || Hq % Hkv != 0 || Hq / Hkv > 16 || B > 65535 || Hkv > 65535 ||
      max_slots > 262144)
    return TSD_ERR_LIMIT;
  return TSD_OK;
}

}  // namespace
}  // namespace tsd

TSD_API size_t tsd_tree_attn_q4_workspace_bytes(int B, int N_max, int Hq, int Hkv, int D,
                                                int max_slots) {
  using namespace tsd;
  if (B == 0 || q4_check(B, N_max, Hq, Hkv, D, max_slots) != TSD_OK) return 0;
  return q4_shape(B, N_max, Hq, Hkv, D, max_slots).bytes;
}

TSD_API int tsd_tree_attn_fwd_q4(const uint16_t *q, const uint8_t *k_cache, const uint8_t *v_cache,
                                 const int32_t *block_table, int max_blocks, int num_blocks,
                                 const int32_t *prefix_len, const int32_t *n_nodes,
                                 const uint32_t *mask, const int32_t *err, int B, int N_max, int Hq,
                                 int Hkv, int D, int max_slots, float scale, uint16_t *out, float *lse,
                                 void *workspace, size_t ws_bytes, int32_t *status,
                                 tsd_stream_t stream) {
  using namespace tsd;
  const int rc = q4_check(B, N_max, Hq, Hkv, D, max_slots);
  if (rc != TSD_OK) return rc;
  if (max_blocks < 1 || num_blocks < 1 || !std::isfinite(scale)) return TSD_ERR_ARG;
  if (B == 0) return TSD_OK;
  if (!q || !k_cache || !v_cache || !block_table || !prefix_len || !out) return TSD_ERR_ARG;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16))
    return TSD_ERR_ARG;
  const Q4Shape pl = q4_shape(B, N_max, Hq, Hkv, D, max_slots);
  if (pl.bytes > 0 && (!workspace || ws_bytes < pl.bytes)) return TSD_ERR_WORKSPACE;
  if (pl.bytes > 0 && !aligned(workspace, 16)) return TSD_ERR_ARG;
  Q4Attn p = {};
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
  p.B = B;
  p.N_max = N_max;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.g = Hq / Hkv;
  p.W = (N_max + 31) / 32;
  p.max_slots = max_slots;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.rows = N_max * p.g;
  p.rows_per_block = pl.rows_per_block;
  p.row_blocks = pl.row_blocks;
  p.splits = pl.splits;
  p.chunk = pl.chunk;
  p.cluster = pl.cluster ? pl.splits : 0;
  p.planned = pl.planned;
  p.slots = pl.blocks;
  p.row_tiles = pl.tc ? pl.rows_per_block / 128 : 1;
  p.range_cost = pl.tc ? kTcRangeCost : kRowsRangeCost;
  p.min_part = p.range_cost + 2 * p.row_tiles;  // a shorter part would be mostly set-up
  if (pl.bytes) {
    char *ws = reinterpret_cast<char *>(workspace);
    p.plan = reinterpret_cast<int4 *>(ws);
    p.part_ml = reinterpret_cast<float2 *>(ws + pl.plan_bytes);
    p.part_o = reinterpret_cast<float *>(ws + pl.plan_bytes + pl.ml_bytes);
  }
  p.out = out;
  p.lse = lse;
  p.status = status;
  p.wait_limit_ns = (uint64_t)option(TSD_OPT_WAIT_LIMIT_NS);
  p.test_stall = (int)option(TSD_OPT_TEST_STALL);
  const cudaStream_t s = as_cuda(stream);
  cudaError_t e;
  if (pl.tc)
    e = q4_tc_launch(p, D, pl.blocks, s);
  else if (D == 128)
    e = pl.nt == 2 ? rows_launch<128, 2>(p, pl.blocks, s) : rows_launch<128, 1>(p, pl.blocks, s);
  else
    e = pl.nt == 2 ? rows_launch<64, 2>(p, pl.blocks, s) : rows_launch<64, 1>(p, pl.blocks, s);
  if (e != cudaSuccess) return TSD_ERR_CUDA;
  if (pl.bytes) {
    const int64_t rows = (int64_t)B * Hkv * p.rows;
    const dim3 grid((unsigned)((rows + 7) / 8));
    e = D == 128 ? launch(tree_attn_q4_join_kernel<128>, grid, dim3(256), 0, s, p)
                 : launch(tree_attn_q4_join_kernel<64>, grid, dim3(256), 0, s, p);
    if (e != cudaSuccess) return TSD_ERR_CUDA;
  }
  return TSD_OK;
}
