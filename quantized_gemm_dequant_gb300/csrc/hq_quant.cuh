// Steps that the kernels which make 8- and 4-bit activations share: bf16 loads to fp32, e4m3 conversions, exact
// division by a scale and the largest magnitude of bf16 values.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace hq {

__device__ __forceinline__ void bf16x8_to_f32(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// two floats -> bf16x2, round to nearest even (lo = a)
__device__ __forceinline__ uint32_t bf16x2_of(float a, float b) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
  return d;
}
__device__ __forceinline__ uint4 bf16x8_of(const float (&f)[8]) {
  return make_uint4(bf16x2_of(f[0], f[1]), bf16x2_of(f[2], f[3]), bf16x2_of(f[4], f[5]), bf16x2_of(f[6], f[7]));
}

// two floats -> two e4m3 bytes (lo = a), round to nearest even, saturating
__device__ __forceinline__ uint32_t cvt_e4m3x2(float a, float b) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(b), "f"(a));
  return d;
}

// x / y rounded to nearest even (IEEE binary32) from yi = RN(1 / y): q = RN(x * yi) is faithful, the residual
// x - q * y is exact with one FMA, and RN(q + residual * yi) is the correctly rounded quotient (P. Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor", IBM J. Res. Dev. 34(1), 1990).  Valid
// while the residual stays a normal number: the callers use it only when the scale is at least 2^-100 (every quotient
// that can round to a nonzero code then has |x| >= 2^-110), and take the plain division otherwise.
__device__ __forceinline__ float div_by(float x, float y, float yi) {
  const float q = __fmul_rn(x, yi);
  const float r = __fmaf_rn(-q, y, x);
  return __fmaf_rn(r, yi, q);
}
constexpr float kDivMinScale = 7.8886091e-31f;  // 2^-100

// largest bf16 magnitude of 8 values (4 words), as the 16-bit pattern: finite non-negative bf16 values order like
// their bit patterns, so a SIMD unsigned max of the sign-cleared halves suffices
__device__ __forceinline__ uint32_t bf16x8_absmax_bits(const uint4& v, uint32_t m) {
  m = __vmaxu2(m, v.x & 0x7FFF7FFFu);
  m = __vmaxu2(m, v.y & 0x7FFF7FFFu);
  m = __vmaxu2(m, v.z & 0x7FFF7FFFu);
  m = __vmaxu2(m, v.w & 0x7FFF7FFFu);
  return m;
}
__device__ __forceinline__ float absmax_bits_to_f32(uint32_t m) {
  const uint32_t h = (m & 0xFFFFu) > (m >> 16) ? (m & 0xFFFFu) : (m >> 16);
  return __uint_as_float(h << 16);
}

// The e4m3 scale of values whose largest magnitude has the bits `amax`: s = amax / 448, and what division by it needs.
// Magnitudes are compared as unsigned bit patterns, which order like the numbers and put infinity and NaN on top, so a
// NaN is not lost: it becomes the scale.
struct E4m3Scale {
  float s, inv;
  bool on, fast;
  __device__ __forceinline__ explicit E4m3Scale(uint32_t amax) {
    s = __fdiv_rn(__uint_as_float(amax), 448.0f);
    inv = __frcp_rn(s);
    on = s > 0.0f;          // a scale of zero (or NaN) has zero codes
    fast = s >= 0x1p-60f;  // div_by's residual is exact: the quotients that matter are above 2^-10
  }
  // e4m3 codes of eight values
  __device__ __forceinline__ uint2 codes(const float (&f)[8]) const {
    if (!on) return make_uint2(0u, 0u);
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      b[i] = fast ? cvt_e4m3x2(div_by(f[2 * i], s, inv), div_by(f[2 * i + 1], s, inv))
                  : cvt_e4m3x2(__fdiv_rn(f[2 * i], s), __fdiv_rn(f[2 * i + 1], s));
    return make_uint2(b[0] | (b[1] << 16), b[2] | (b[3] << 16));
  }
};

// largest magnitude of eight values, as its bits
__device__ __forceinline__ uint32_t absmax_bits(const float (&f)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
  return m;
}

}  // namespace hq
