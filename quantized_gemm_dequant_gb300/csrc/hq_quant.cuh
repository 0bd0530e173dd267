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

// ---- eight values as four pairs (two fp32 operations an instruction)
__device__ __forceinline__ void bf16x8_to_f32x2(const uint4& v, float2 (&f)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
__device__ __forceinline__ uint4 bf16x8_of(const float2 (&f)[4]) {
  return make_uint4(bf16x2_of(f[0].x, f[0].y), bf16x2_of(f[1].x, f[1].y), bf16x2_of(f[2].x, f[2].y),
                    bf16x2_of(f[3].x, f[3].y));
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// the larger of three magnitudes; a NaN among them wins
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(fabsf(b)), "f"(fabsf(c)));
  return d;
}
// largest magnitude of `m` (not negative) and eight values, as its bits: unsigned bit patterns order like the numbers
// and put infinity and NaN on top, so that further maxima keep a NaN
__device__ __forceinline__ uint32_t absmax_bits(const float2 (&f)[4], float m = 0.0f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max3_nan(m, f[i].x, f[i].y);
  return __float_as_uint(m) & 0x7FFFFFFFu;
}

// The e4m3 scale of values whose largest magnitude has the bits `amax`: s = amax / 448, and the codes of values divided
// by it.  Quotients are those of IEEE division: div_by's two steps after a multiplication by the reciprocal (of the
// scale: approximated, with one Newton step), in the range where its residuals are exact (what matters is above 2^-10,
// so that they stay above 2^-93 from a scale of 2^-60 on), plain division outside.
struct E4m3Scale {
  float s, inv;
  bool fast;
  __device__ __forceinline__ explicit E4m3Scale(uint32_t amax) {
    const float m = __uint_as_float(amax);
    fast = m >= 0x1p-50f && m <= 0x1p126f;
    s = fast ? div_by(m, 448.0f, 1.0f / 448.0f) : __fdiv_rn(m, 448.0f);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
    inv = fmaf(inv, fmaf(-s, inv, 1.0f), inv);
  }
  // (every lane of the warp calls it: one plain scale among them takes the warp the plain way)
  __device__ __forceinline__ uint2 codes(const float2 (&f)[4]) const {
    uint32_t b[4];
    if (__all_sync(0xffffffffu, fast)) {
      const float2 y = both(inv), ns = both(-s);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 q = __fmul2_rn(f[i], y);
        const float2 r = __ffma2_rn(q, ns, f[i]);
        const float2 z = __ffma2_rn(r, y, q);
        b[i] = cvt_e4m3x2(z.x, z.y);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)  // a scale of zero, or one that is no number, has zero codes
        b[i] = s > 0.0f ? cvt_e4m3x2(__fdiv_rn(f[i].x, s), __fdiv_rn(f[i].y, s)) : 0u;
    }
    return make_uint2(b[0] | (b[1] << 16), b[2] | (b[3] << 16));
  }
};

}  // namespace hq
