// Parameters and helpers shared by the 4-bit tree attention's kernels.
#pragma once

#include "q4.cuh"
#include "tsd_common.cuh"

namespace tsd {

struct Q4Attn {
  const uint16_t *q;
  const uint8_t *k, *v;
  const int32_t *table;
  int max_blocks, num_blocks;
  const int32_t *prefix_len, *n_nodes;
  const uint32_t *mask;  // null: node i sees nodes 0..i
  const int32_t *err;
  int B, N_max, Hq, Hkv, g, W, max_slots;
  float scale_log2;
  int rows;        // N_max * g, query rows of one kv head
  int row_blocks;  // blocks over them
  int splits;      // pieces of the longest key range
  int chunk;       // pages (of 16 keys) in one piece
  int cluster;     // few-row kernel: the pieces of a range are a thread-block cluster
  float *part_o;   // [B * Hkv][splits][rows][D]: unnormalised fp32 outputs
  float2 *part_ml;  // [B * Hkv][splits][rows]: (reference in log2 units, sum), sum -1: bad page
  uint16_t *out;
  float *lse;
  int32_t *status;
  uint64_t wait_limit_ns;
};

// Lengths of sequence b; false when it is skipped (and then `bad` says whether
// its lengths are why).
__device__ __forceinline__ bool q4_seq(const Q4Attn &p, int b, int &P, int &nb, bool &bad) {
  bad = false;
  P = p.prefix_len[b];
  nb = p.n_nodes ? p.n_nodes[b] : p.N_max;
  if (p.err && p.err[b] != 0) return false;
  bad = nb < 1 || nb > p.N_max || P < 0 || (int64_t)P + nb > (int64_t)p.max_slots ||
        (int64_t)P + nb > (int64_t)p.max_blocks * kPage;
  return !bad;
}

// Visibility of the 16 slots of a page that starts at tail index j0 (slot -
// P; negative: prefix) for node i: bit s set when slot s is seen.
__device__ __forceinline__ uint32_t q4_visible(const Q4Attn &p, int b, int i, int j0, int nb) {
  if (j0 <= -kPage) return 0xFFFFu;
  uint32_t tail;  // bits of tail nodes from max(j0, 0) on
  const int first = max(j0, 0);
  if (p.mask) {
    const uint32_t *m = p.mask + ((size_t)b * p.N_max + i) * p.W;
    const int w = first >> 5;
    const uint32_t lo = w < p.W ? m[w] : 0u, hi = w + 1 < p.W ? m[w + 1] : 0u;
    tail = __funnelshift_r(lo, hi, first & 31);
  } else {
    const int n = i + 1 - first;  // nodes first..i
    tail = n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u;
  }
  const int left = nb - first;  // nodes of the tree from there on
  if (left < 32) tail &= left <= 0 ? 0u : (1u << left) - 1u;
  if (j0 < 0) tail = (tail << -j0) | ((1u << -j0) - 1u);
  return tail & 0xFFFFu;
}

// The exponent e for which 2^e brings amax to [2^13, 2^14); 0 for zero, inf or
// NaN.  It reaches 140, so 2^e is applied as two factors.
__device__ __forceinline__ int q4_exponent(float amax) {
  if (!(amax > 0.f) || !isfinite(amax)) return 0;
  return 13 - (((int)(__float_as_uint(amax) >> 23) & 0xFF) - 127);
}
// 2^e, |e| <= 126.
__device__ __forceinline__ float q4_pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// Output row of row r of kv head h of sequence b.
__device__ __forceinline__ size_t q4_out_row(const Q4Attn &p, int b, int h, int r) {
  return ((size_t)b * p.N_max + r / p.g) * p.Hq + h * p.g + r % p.g;
}

// The many-row kernel (attention_q4_tc.cu).
cudaError_t q4_tc_launch(const Q4Attn &p, int D, int rows_per_block, cudaStream_t s);

}  // namespace tsd
