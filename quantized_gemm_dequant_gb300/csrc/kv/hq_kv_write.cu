// Norm, rotation and quantised append: the fused projection's rows -> queries in bf16, keys and values in the cache.
//
//   y = x * rsqrt(mean(x^2) + eps) * w,   (a, b) -> (a cos - b sin, b cos + a sin),   then one rounding:
//   bf16; e4m3 of y / s with s = absmax / 448; or e2m1 of y / d with d = e4m3(absmax_16 / (6 g)) * g.
// All steps are fp32; the divisions that decide a code are IEEE divisions.
//
// Memory-bound: every element is read once and written once.  D / 8 lanes hold a head's row, 8 dims each (one 16-byte
// load), so a head's sum of squares and largest magnitude are shuffles inside the group, and the rotation's partner
// dims are a lane's own or another lane's of the group.  A warp takes one token and NS steps of 256 / D heads: all its
// rows are loaded before the first is worked on, and the angles' cosines and sines (as many bytes as two heads' rows)
// are loaded once for all of them.  Few tokens take one step a warp instead, which spreads them over the SMs.
#include <cuda_runtime.h>
#include <stdint.h>

#include "../hq_launch.h"
#include "../hq_ptx.cuh"
#include "hq_kv.h"
#include "hq_kv_codec.cuh"

namespace hq {

namespace {

constexpr int KW_THREADS = 128;

// x / y rounded to nearest even from yi = RN(1 / y): RN(x yi) is faithful, its residual is exact with one FMA, and one
// more FMA gives the correctly rounded quotient (P. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", IBM J. Res. Dev. 34(1), 1990).  Valid while the residual stays a normal number; callers take
// it for y >= 2^-100 and divide otherwise.
__device__ __forceinline__ float quotient(float x, float y, float yi, bool fast) {
  if (!fast) return __fdiv_rn(x, y);
  const float q = __fmul_rn(x, yi);
  return __fmaf_rn(__fmaf_rn(-q, y, x), yi, q);
}
constexpr float KW_FAST = 7.8886091e-31f;  // 2^-100

template <int KIND, int D, int NS>
__global__ void __launch_bounds__(KW_THREADS) kv_write_kernel(const KvWriteArgs a, int parts) {
  constexpr int LPH = D / 8;      // lanes of a head's row
  constexpr int HPW = 32 / LPH;   // heads of one step
  constexpr int RB = kv_row_bytes(KIND, D);
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, l = lane % LPH, sub = lane / LPH;
  const int64_t task = (int64_t)blockIdx.x * (KW_THREADS / 32) + (threadIdx.x >> 5);
  const int64_t t = task / parts;
  if (t >= a.T) return;
  const int part = (int)(task - t * parts);
  const int H = a.kv.heads, Hq = a.q_heads, all = Hq + 2 * H;
  const int h0 = part * NS * HPW + sub, d0 = 8 * l;

  uint4 raw[NS];
  const uint16_t* src = a.qkv + t * a.row_stride + (int64_t)h0 * D + d0;
#pragma unroll
  for (int s = 0; s < NS; ++s)
    raw[s] = h0 + s * HPW < all ? __ldcs(reinterpret_cast<const uint4*>(src + s * HPW * D)) : make_uint4(0, 0, 0, 0);

  // the row's place, and its angles
  const int64_t slot = a.slots[t];
  const bool cached = slot >= 0 && slot < a.kv.num_pages * a.kv.page_size;
  if (slot >= 0 && !cached && part == 0 && lane == 0) kv_report(a.status);
  const int64_t page = cached ? slot / a.kv.page_size : 0;
  const int off = cached ? (int)(slot - page * a.kv.page_size) : 0;
  const int half = a.rotary >> 1;
  const bool turn = d0 < a.rotary;
  float cs[8], sn[8];  // the rotation is x cs + partner sn
  int partner = lane;
  if (a.rotary) {
    const int64_t pos = a.positions[t];
    if (pos < 0 || pos >= a.num_positions) {
      if (part == 0 && lane == 0) kv_report(a.status);
      return;
    }
    const float* row = a.cos_sin + pos * a.rotary;
    if (turn) {
      if (a.interleaved) {  // pairs (2i, 2i + 1): four angles, each for two dims
        const float4 c = *reinterpret_cast<const float4*>(row + d0 / 2);
        const float4 s = *reinterpret_cast<const float4*>(row + half + d0 / 2);
        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) cs[i] = cc[i / 2], sn[i] = (i & 1) ? ss[i / 2] : -ss[i / 2];
      } else {  // dim i pairs with i + half: eight angles
        const int i0 = d0 < half ? d0 : d0 - half;
        partner = d0 < half ? lane + half / 8 : lane - half / 8;
        const float sign = d0 < half ? -1.0f : 1.0f;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float4 c = *reinterpret_cast<const float4*>(row + i0 + 4 * q);
          const float4 s = *reinterpret_cast<const float4*>(row + half + i0 + 4 * q);
          cs[4 * q] = c.x, cs[4 * q + 1] = c.y, cs[4 * q + 2] = c.z, cs[4 * q + 3] = c.w;
          sn[4 * q] = sign * s.x, sn[4 * q + 1] = sign * s.y;
          sn[4 * q + 2] = sign * s.z, sn[4 * q + 3] = sign * s.w;
        }
      }
    }
  }
  const uint4 wq = a.q_norm ? *reinterpret_cast<const uint4*>(a.q_norm + d0) : make_uint4(0, 0, 0, 0);
  const uint4 wk = a.k_norm ? *reinterpret_cast<const uint4*>(a.k_norm + d0) : make_uint4(0, 0, 0, 0);
  const bool any_norm = a.q_norm != nullptr || a.k_norm != nullptr;

#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const int h = h0 + s * HPW, first = h - sub;  // the lane's head, the warp's first one
    if (first >= all) break;
    const bool live = h < all, is_q = h < Hq, is_k = !is_q && h < Hq + H;
    float x[8];
    unpack_bf16x8(raw[s], x);
    if (first < Hq + H) {  // the warp's query and key heads (its shuffles are whole)
      if (any_norm) {
        float sq = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sq = fmaf(x[i], x[i], sq);
#pragma unroll
        for (int o = LPH / 2; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
        if (is_q ? a.q_norm != nullptr : (is_k && a.k_norm != nullptr)) {
          const float r = rsqrtf(sq * (1.0f / D) + a.eps);
          float w[8];
          unpack_bf16x8(is_q ? wq : wk, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
        }
      }
      if (a.rotary) {
        float y[8];
        if (a.interleaved) {
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = x[i ^ 1];
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], partner);
        }
        if (turn && (is_q || is_k)) {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = fmaf(x[i], cs[i], y[i] * sn[i]);
        }
      }
    }
    if (is_q) *reinterpret_cast<uint4*>(a.q_out + (t * Hq + h) * D + d0) = pack_bf16x8(x);
    if (first + HPW <= Hq) continue;  // query heads only
    // keys and values into the cache
    const bool put = live && !is_q && cached;
    const int64_t row = (page * H + (is_k ? h - Hq : h - Hq - H)) * a.kv.page_size + off;
    uint8_t* dst = (is_k ? a.kv.k : a.kv.v) + row * RB;
    if constexpr (KIND == HQ_KV_BF16) {
      if (put) *reinterpret_cast<uint4*>(dst + 16 * l) = pack_bf16x8(x);
    } else {
      float m = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
      if constexpr (KIND == HQ_KV_E4M3) {
#pragma unroll
        for (int o = LPH / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float sc = __fdiv_rn(m, 448.0f), inv = __frcp_rn(sc);
        const bool fast = sc >= KW_FAST;
        uint32_t c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          c[i] = sc > 0.0f ? pack_e4m3x2(quotient(x[2 * i], sc, inv, fast), quotient(x[2 * i + 1], sc, inv, fast)) : 0u;
        if (put) {
          *reinterpret_cast<uint2*>(dst + 8 * l) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
          if (l == 0) reinterpret_cast<float*>(is_k ? a.kv.k_scale : a.kv.v_scale)[row] = sc;
        }
      } else {
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));  // a block of 16 dims is two lanes
        const float g = put ? *(is_k ? a.kv.k_global : a.kv.v_global) : 1.0f;
        const uint32_t sb = g > 0.0f ? pack_e4m3x2(__fdiv_rn(m, __fmul_rn(6.0f, g)), 0.0f) & 0xFFu : 0u;
        const float d = __fmul_rn(f16x2_to_f32x2(e4m3x2_to_f16x2(sb)).x, g), inv = __frcp_rn(d);
        const bool fast = d >= KW_FAST;
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = d > 0.0f ? quotient(x[i], d, inv, fast) : 0.0f;
        if (put) {
          *reinterpret_cast<uint32_t*>(dst + 4 * l) = pack_e2m1x8(y);
          if (!(l & 1)) (is_k ? a.kv.k_scale : a.kv.v_scale)[row * (D / 16) + l / 2] = (uint8_t)sb;
        }
      }
    }
  }
}

template <int KIND, int D, int NS>
cudaError_t launch_ns(const KvWriteArgs& a, int steps, cudaStream_t stream) {
  const int parts = (steps + NS - 1) / NS;  // warps of one token
  const int64_t ctas = (a.T * parts + KW_THREADS / 32 - 1) / (KW_THREADS / 32);
  if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  return launch_kernel(kv_write_kernel<KIND, D, NS>, dim3((unsigned)ctas), dim3(KW_THREADS), 0, stream, a, parts);
}

template <int KIND, int D>
cudaError_t launch(const KvWriteArgs& a, cudaStream_t stream) {
  constexpr int HPW = 256 / D;
  const int steps = (a.q_heads + 2 * a.kv.heads + HPW - 1) / HPW;
  // four steps a warp once that leaves every SM 16 warps
  return a.T * steps >= 4 * 16 * 152 ? launch_ns<KIND, D, 4>(a, steps, stream) : launch_ns<KIND, D, 1>(a, steps, stream);
}

template <int KIND>
cudaError_t by_dim(int dim, const KvWriteArgs& a, cudaStream_t stream) {
  return dim == 64 ? launch<KIND, 64>(a, stream) : (dim == 128 ? launch<KIND, 128>(a, stream)
                                                               : launch<KIND, 256>(a, stream));
}

}  // namespace

cudaError_t launch_kv_write(int kind, int dim, const KvWriteArgs& a, cudaStream_t stream) {
  return kind == HQ_KV_BF16 ? by_dim<HQ_KV_BF16>(dim, a, stream)
                            : (kind == HQ_KV_E4M3 ? by_dim<HQ_KV_E4M3>(dim, a, stream)
                                                  : by_dim<HQ_KV_NVFP4>(dim, a, stream));
}

}  // namespace hq
