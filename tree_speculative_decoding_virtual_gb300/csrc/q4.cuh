// The 4-bit paged cache's format, shared by its writer, reader, commit and
// attention.
//
// A page holds 16 token slots of one kv head: 16 rows of D/2 code bytes (even
// column in the low nibble), then 16 rows of D/16 scale bytes, 9 D bytes in
// all.  Sixteen consecutive columns of a row share one scale.
//   code   E2M1: sign, two exponent bits, one fraction bit; the magnitudes
//          are 0, 0.5, 1, 1.5, 2, 3, 4, 6.
//   scale  five exponent and three fraction bits, no sign (a scale is never
//          negative): the half-precision number whose bits are byte << 7.
//          No writer makes a byte above kQ4MaxScale (10240).  Where a page may
//          hold slots that were not written, its bytes are read as at most that,
//          so that a value is finite whatever the page holds.
// A value is code * scale: at most six significant bits and between 2^-18
// and 61440 in magnitude, so it is exact in fp16 (and bf16), which is what
// lets the attention decode straight to fp16 MMA operands without rounding.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "tsd_common.cuh"

namespace tsd {

constexpr int kQ4Group = 16;
constexpr uint32_t kQ4MaxScale = 0xE2;

template <int D>
struct Q4Page {
  static constexpr int kRow = D / 2;            // code bytes of one slot
  static constexpr int kScaleRow = D / kQ4Group;  // scale bytes of one slot
  static constexpr int kScales = kPage * kRow;  // offset of the scale rows
  static constexpr int kBytes = kPage * (kRow + kScaleRow);
};
static_assert(Q4Page<128>::kBytes == 9 * 128 && Q4Page<64>::kBytes == 9 * 64, "9 D bytes a page");

// Eight codes (one word) as four fp16 pairs, lowest column first.
__device__ __forceinline__ void q4_decode8(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}
// The scale of `byte` as an fp16 pair (the same value twice).
__device__ __forceinline__ uint32_t q4_scale2(uint32_t byte) {
  return min(byte, kQ4MaxScale) * 0x00800080u;
}
__device__ __forceinline__ uint32_t q4_mul2(uint32_t a, uint32_t s) {
  const __half2 r = __hmul2(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&s));
  return *reinterpret_cast<const uint32_t *>(&r);
}

}  // namespace tsd
