// Norm, rotation and quantised append: the fused projection's rows -> queries in bf16, keys and values in the cache.
//
//   y = x * rsqrt(mean(x^2) + eps) * w,   (a, b) -> (a cos - b sin, b cos + a sin),   then one rounding:
//   bf16; e4m3 of y / s with s = absmax / 448; or e2m1 of y / d with d = e4m3(absmax_16 / (6 g)) * g.
// All steps are fp32; the divisions that decide a code are IEEE divisions.
//
// Memory-bound: every element is read once and written once, and the instructions per element decide whether that is
// reached.  A CTA takes one token; its four warps take every fourth step of 256 / D heads of one kind (query, key or
// value), four query steps and the first key and value step in flight at once.  D / 8 lanes hold a head's row.  For a
// rotation by halves a lane holds four dims of the first half and their four partners, so that the rotation needs no
// exchange between lanes and a lane's four angles serve both; otherwise it holds eight neighbouring dims.  Sums of
// squares and largest magnitudes are shuffles inside the head's lanes.
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

// A head's row in its lanes: dims lo .. lo + 3 and hi .. hi + 3 of each lane.
struct Row {
  uint2 lo, hi;
};
__device__ __forceinline__ Row load_row(const uint16_t* p, int lo, int hi, bool live) {
  Row r;
  r.lo = live ? __ldcs(reinterpret_cast<const uint2*>(p + lo)) : make_uint2(0, 0);
  r.hi = live ? __ldcs(reinterpret_cast<const uint2*>(p + hi)) : make_uint2(0, 0);
  return r;
}
__device__ __forceinline__ void unpack_row(const Row& r, float (&x)[8]) {
  x[0] = bf16_lo(r.lo.x), x[1] = bf16_hi(r.lo.x), x[2] = bf16_lo(r.lo.y), x[3] = bf16_hi(r.lo.y);
  x[4] = bf16_lo(r.hi.x), x[5] = bf16_hi(r.hi.x), x[6] = bf16_lo(r.hi.y), x[7] = bf16_hi(r.hi.y);
}
__device__ __forceinline__ void store_row(uint16_t* p, int lo, int hi, const float (&x)[8]) {
  *reinterpret_cast<uint2*>(p + lo) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
  *reinterpret_cast<uint2*>(p + hi) = make_uint2(pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

template <int LPH>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = LPH / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int LPH>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int o = LPH / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float largest(const float (&x)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
  return m;
}

// Norm (w: the lane's weights; on: whether there is one) and rotation of a row.  The rotated pairs are (x[i], x[i + 4])
// for a rotation by halves, (x[2 i], x[2 i + 1]) for an interleaved one; cs, sn are their four angles'.
template <int LPH>
__device__ __forceinline__ void norm_rotate(float (&x)[8], bool on, const float (&w)[8], float eps, bool turn,
                                            bool interleaved, const float (&cs)[4], const float (&sn)[4]) {
  if (on) {
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sq = fmaf(x[i], x[i], sq);
    const float r = rsqrtf(lanes_sum<LPH>(sq) * (1.0f / (8 * LPH)) + eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
  }
  if (!turn) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (interleaved) {
      const float p = x[2 * i], q = x[2 * i + 1];
      x[2 * i] = fmaf(p, cs[i], -q * sn[i]);
      x[2 * i + 1] = fmaf(q, cs[i], p * sn[i]);
    } else {
      const float p = x[i], q = x[i + 4];
      x[i] = fmaf(p, cs[i], -q * sn[i]);
      x[i + 4] = fmaf(q, cs[i], p * sn[i]);
    }
  }
}

// A row (dims lo .. and hi .. of each lane; NVFP4: eight neighbouring dims) into the pool.  The shuffles are the whole
// warp's; only lanes that `put` store.
template <int KIND, int D>
__device__ __forceinline__ void store_held(uint8_t* codes, uint8_t* scales, const float* global, int64_t row, int l,
                                           int lo, int hi, const float (&x)[8], bool put) {
  uint8_t* dst = codes + row * kv_row_bytes(KIND, D);
  if constexpr (KIND == HQ_KV_BF16) {
    if (put) store_row(reinterpret_cast<uint16_t*>(dst), lo, hi, x);
  } else if constexpr (KIND == HQ_KV_E4M3) {
    const float s = __fdiv_rn(lanes_max<D / 8>(largest(x)), 448.0f), inv = __frcp_rn(s);
    const bool fast = s >= KW_FAST;
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c[i] = s > 0.0f ? pack_e4m3x2(quotient(x[2 * i], s, inv, fast), quotient(x[2 * i + 1], s, inv, fast)) : 0u;
    if (put) {
      *reinterpret_cast<uint32_t*>(dst + lo) = c[0] | (c[1] << 16);
      *reinterpret_cast<uint32_t*>(dst + hi) = c[2] | (c[3] << 16);
      if (l == 0) reinterpret_cast<float*>(scales)[row] = s;
    }
  } else {
    const float m = lanes_max<2>(largest(x)), g = *global;  // a block of 16 dims is two lanes
    const uint32_t sb = g > 0.0f ? pack_e4m3x2(__fdiv_rn(m, __fmul_rn(6.0f, g)), 0.0f) & 0xFFu : 0u;
    const float d = __fmul_rn(f16x2_to_f32x2(e4m3x2_to_f16x2(sb)).x, g), inv = __frcp_rn(d);
    const bool fast = d >= KW_FAST;
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = d > 0.0f ? quotient(x[i], d, inv, fast) : 0.0f;
    if (put) {
      *reinterpret_cast<uint32_t*>(dst + 4 * l) = pack_e2m1x8(y);
      if (!(l & 1)) scales[row * (D / 16) + l / 2] = (uint8_t)sb;
    }
  }
}

template <int KIND, int D>
__global__ void __launch_bounds__(KW_THREADS) kv_write_kernel(const KvWriteArgs a) {
  constexpr int LPH = D / 8;     // lanes of a head's row
  constexpr int HPW = 32 / LPH;  // heads of one step
  constexpr int WARPS = KW_THREADS / 32, NS = 4;
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % LPH, sub = lane / LPH;
  const int64_t t = blockIdx.x;
  const int H = a.kv.heads, Hq = a.q_heads, R = a.rotary;
  const bool halves = R > 0 && !a.interleaved, turn = 8 * l < R;
  // the lane's dims: by halves of the rotated part and of the rest, or eight neighbours
  int lo = 8 * l, hi = 8 * l + 4;
  if (halves && turn) lo = 4 * l, hi = R / 2 + 4 * l;
  const uint16_t* qs = a.qkv + t * a.row_stride;
  const uint16_t* ks = qs + (int64_t)Hq * D;
  const uint16_t* vs = ks + (int64_t)H * D;
  const bool neighbours = KIND == HQ_KV_NVFP4 && halves;  // key rows by neighbours all the same: blocks of 16 dims
  const int klo = neighbours ? 8 * l : lo, khi = neighbours ? 8 * l + 4 : hi;
  const int kv0 = warp * HPW + sub;
  Row kr = load_row(ks + (int64_t)kv0 * D, klo, khi, kv0 < H);
  Row vr = load_row(vs + (int64_t)kv0 * D, 8 * l, 8 * l + 4, kv0 < H);

  const int64_t slot = a.slots[t];
  const bool cached = slot >= 0 && slot < a.kv.num_pages * a.kv.page_size;
  if (slot >= 0 && !cached && threadIdx.x == 0) kv_report(a.status);
  float cs[4] = {1.0f, 1.0f, 1.0f, 1.0f}, sn[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  const float* angles = nullptr;
  if (R > 0) {
    const int64_t pos = a.positions[t];
    if (pos < 0 || pos >= a.num_positions) {
      if (threadIdx.x == 0) kv_report(a.status);
      return;
    }
    angles = a.cos_sin + pos * R;
    if (turn) {
      const float4 c = *reinterpret_cast<const float4*>(angles + 4 * l);
      const float4 s = *reinterpret_cast<const float4*>(angles + R / 2 + 4 * l);
      cs[0] = c.x, cs[1] = c.y, cs[2] = c.z, cs[3] = c.w;
      sn[0] = s.x, sn[1] = s.y, sn[2] = s.z, sn[3] = s.w;
    }
  }

  // ---- query heads
  float w[8];
  if (a.q_norm) unpack_row(load_row(a.q_norm, lo, hi, true), w);
  for (int h0 = warp * HPW; h0 < Hq; h0 += NS * WARPS * HPW) {
    Row r[NS];
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int h = h0 + s * WARPS * HPW + sub;
      r[s] = load_row(qs + (int64_t)h * D, lo, hi, h < Hq);
    }
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int h = h0 + s * WARPS * HPW + sub;
      if (h - sub >= Hq) break;
      float x[8];
      unpack_row(r[s], x);
      norm_rotate<LPH>(x, a.q_norm != nullptr, w, a.eps, turn, a.interleaved, cs, sn);
      if (h < Hq) store_row(a.q_out + (t * Hq + h) * D, lo, hi, x);
    }
  }

  // ---- key and value heads
  if (!cached) return;  // (the whole CTA's token)
  const uint32_t ps = (uint32_t)a.kv.page_size;
  const int64_t page = slot >> 32 ? slot / ps : (uint32_t)slot / ps;
  const int64_t row0 = page * H * ps + (slot - page * ps);
  if (a.k_norm) unpack_row(load_row(a.k_norm, klo, khi, true), w);
  for (int h = kv0; h - sub < H; h += WARPS * HPW) {
    if (h != kv0) {
      kr = load_row(ks + (int64_t)h * D, klo, khi, h < H);
      vr = load_row(vs + (int64_t)h * D, 8 * l, 8 * l + 4, h < H);
    }
    float x[8];
    unpack_row(kr, x);
    if (!neighbours) {
      norm_rotate<LPH>(x, a.k_norm != nullptr, w, a.eps, turn, a.interleaved, cs, sn);
    } else {  // eight neighbouring dims pair with those of another lane
      norm_rotate<LPH>(x, a.k_norm != nullptr, w, a.eps, false, false, cs, sn);
      const int half = R / 2, i0 = 8 * l < half ? 8 * l : 8 * l - half;
      const int partner = turn ? (8 * l < half ? lane + half / 8 : lane - half / 8) : lane;
      const float sign = 8 * l < half ? -1.0f : 1.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float y = __shfl_sync(0xffffffffu, x[i], partner);
        if (turn) x[i] = fmaf(x[i], angles[i0 + i], sign * y * angles[half + i0 + i]);
      }
    }
    store_held<KIND, D>(a.kv.k, a.kv.k_scale, a.kv.k_global, row0 + (int64_t)h * ps, l, klo, khi, x, h < H);
    unpack_row(vr, x);
    store_held<KIND, D>(a.kv.v, a.kv.v_scale, a.kv.v_global, row0 + (int64_t)h * ps, l, 8 * l, 8 * l + 4, x, h < H);
  }
}

template <int KIND, int D>
cudaError_t launch(const KvWriteArgs& a, cudaStream_t stream) {
  return launch_kernel(kv_write_kernel<KIND, D>, dim3((unsigned)a.T), dim3(KW_THREADS), 0, stream, a);
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
