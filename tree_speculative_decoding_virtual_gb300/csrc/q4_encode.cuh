// Quantisation to the 4-bit cache's format (q4.cuh), shared by its writers.
#pragma once

#include "q4.cuh"
#include "sm100_ptx.cuh"

namespace tsd {

// Quantisation of a group of 16 values:
//   scale = nearest (ties to even) to amax / 6, at most 10240;
//   code  = nearest (ties to even) to x / scale.
// amax and x have 8 significant bits and every rounding boundary (times 6, or times
// the scale) at most 7, so a quotient that is not a tie differs from the boundary by
// 2^-9 relative or more: a quotient that is off by 2^-20 and then rounded to 16 bits,
// or to multiples of 2^-14 where the boundaries are multiples of 1/4, gives the
// decision of exact arithmetic.  NaN counts as 0 and an infinity as the largest
// value; both are reported.

// The largest magnitude of eight bf16 values, as the bits of a float; NaN becomes 0.
__device__ __forceinline__ uint32_t q4_amax(uint4 &in, bool &odd) {
  uint32_t w[4] = {in.x, in.y, in.z, in.w};
  // bf16 magnitudes order as integers, infinity and then NaN above the others
  auto largest = [&]() {
    const uint32_t m = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu),
                                __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
    return max(m << 16, m & 0xFFFF0000u);
  };
  uint32_t most = largest();
  if (most >= 0x7F800000u) {
    odd = true;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if ((w[i] & 0x7FFFu) > 0x7F80u) w[i] &= 0xFFFF0000u;
      if ((w[i] & 0x7FFF0000u) > 0x7F800000u) w[i] &= 0xFFFFu;
    }
    most = largest();
    in = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return most;
}

// The scale byte of a group, and the reciprocal of its scale to 2^-23.  (1 for the
// scale 0: the group's values are below 2^-15 then, which makes every code 0.)
__device__ __forceinline__ uint32_t q4_group_scale(float amax, float &recip) {
  // amax / 6 to 16 bits
  const float y = fminf(amax, 61440.f) * 0x1.555556p-3f;
  const float r = __uint_as_float((__float_as_uint(y) + 0x80u) & 0xFFFFFF00u);
  uint32_t byte;
  if (r < 6.103515625e-05f) {  // below 2^-14: steps of 2^-17
    byte = (uint32_t)rintf(r * 131072.f);
  } else {
    uint32_t u = __float_as_uint(r);
    u += 0x7FFFFu + ((u >> 20) & 1u);
    byte = (u >> 20) - (112u << 3);
  }
  const float scale =
      byte < 8 ? (float)byte * 7.62939453125e-06f : __uint_as_float((byte + (112u << 3)) << 20);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(recip) : "f"(scale));
  if (byte == 0u) recip = 1.f;
  return byte;
}

// Rounds down: a - a is -0.
__device__ __forceinline__ unsigned long long f2_add_down(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.rm.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Eight values -> four code bytes.
__device__ __forceinline__ uint32_t q4_codes(uint4 in, float recip) {
  using namespace sm100;
  const uint32_t w[4] = {in.x, in.y, in.z, in.w};
  // x / scale to a multiple of 2^-14, the sum's last place; then 2^-30 of the quotient,
  // which is lost unless that was 0 and then keeps the sign of x.  (The difference is
  // exact; a zero of it is -0, so that -0 x stays -0.)
  constexpr float kGrid = 768.f;  // 1.5 * 2^9
  const unsigned long long recip2 = f2_pack(recip, recip), up = f2_pack(kGrid, kGrid),
                           down = f2_pack(-kGrid, -kGrid),
                           trace = f2_pack(recip * 0x1p-30f, recip * 0x1p-30f);
  float z[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const unsigned long long x = f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    const float2 y = f2_unpack(f2_fma(x, trace, f2_add_down(f2_fma(x, recip2, up), down)));
    z[2 * i] = y.x;
    z[2 * i + 1] = y.y;
  }
  uint32_t code;  // (a conversion's first source goes to the high nibble)
  asm("{\n .reg .b8 a, b, c, d;\n cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
      " cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(code)
      : "f"(z[0]), "f"(z[1]), "f"(z[2]), "f"(z[3]), "f"(z[4]), "f"(z[5]), "f"(z[6]), "f"(z[7]));
  return code;
}

}  // namespace tsd
