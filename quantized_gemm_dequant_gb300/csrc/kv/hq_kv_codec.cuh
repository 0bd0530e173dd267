// Conversions between fp32 / bf16 values and the cache's codes.
#pragma once
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../../include/hq.h"

namespace hq {

// The first device-found error of a call stays in the workspace's status word.
__device__ __forceinline__ void kv_report(int* status) { atomicCAS(status, HQ_OK, HQ_ERR_INVALID_ARG); }

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {  // round to nearest even
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint4 pack_bf16x8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// two floats -> two e4m3 bytes (low byte = a), nearest even, saturating
__device__ __forceinline__ uint32_t pack_e4m3x2(float a, float b) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(b), "f"(a));
  return d;
}
// two e4m3 bytes -> f16x2, exact
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t b) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)b));
  return h;
}
__device__ __forceinline__ float2 f16x2_to_f32x2(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// eight floats -> eight e2m1 codes (code i in nibble i), nearest even, saturating; a zero code loses its sign: a
// nibble's magnitude m + 7 sets bit 3 exactly when m != 0 and never carries, and that bit keeps or clears the sign
__device__ __forceinline__ uint32_t pack_e2m1x8(const float (&v)[8]) {
  uint32_t d;
  asm("{\n\t.reg .b8 t0, t1, t2, t3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t3, %8, %7;\n\t"
      "mov.b32 %0, {t0, t1, t2, t3};\n\t}"
      : "=r"(d)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  const uint32_t s = (d & 0x77777777u) + 0x77777777u;
  return d & (s | 0x77777777u);
}

// eight e2m1 codes -> fp32.  The code's e and m bits, put at an f16's lowest exponent bit and highest fraction bit,
// are the value times 2^-14 (subnormals too), sign on top; the multiplication back is exact.
__device__ __forceinline__ void unpack_e2m1x8(uint32_t w, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // nibbles i and i + 4 sit in the two halves
    const uint32_t x = w << (12 - 4 * i);
    const uint32_t h = (x & 0x80008000u) | ((x >> 3) & 0x0E000E00u);
    const float2 v = f16x2_to_f32x2(h);
    f[i] = v.x * 16384.0f;
    f[i + 4] = v.y * 16384.0f;
  }
}

}  // namespace hq
