// Norm, rotation and quantised append: the fused projection's rows -> queries in bf16, keys and values in the cache.
//
//   y = x * rsqrt(mean(x^2) + eps) * w,   (a, b) -> (a cos - b sin, b cos + a sin),   then one rounding:
//   bf16; e4m3 of y / s with s = absmax / 448; or e2m1 of y / d with d = e4m3(absmax_16 / (6 g)) * g.
// All steps are fp32; the divisions that decide a code give what IEEE divisions give, overflow included: most are
// products with a reciprocal and their correction.
//
// Memory-bound: every element is read once and written once, and the instructions per element decide whether that is
// reached.  A CTA takes one token; its four warps take every fourth step of 256 / D heads of one kind (query, key or
// value), up to four query steps and the first key and value step in flight at once.  Where the heads do not fill the
// warps' steps, the warps take their places in turn from token to token, since a CTA holds its room on the SM until its
// slowest warp is done (8 / 1 heads of 128 dims, 20000 tokens e4m3: 78 us without, 63 so).  D / 8 lanes hold a head's
// row.  For a rotation by halves a lane holds four dims of the first half and their four partners, so that the rotation
// needs no exchange between lanes and a lane's four angles serve both; otherwise it holds eight neighbouring dims.  Sums
// of squares and largest magnitudes are shuffles inside the head's lanes.
// Measured on a GB300, 8192 tokens of 32 query and 8 key-value heads of 128 dims into e4m3: 38.4 us, 73% of the measured
// copy bandwidth (a warp per token and two heads: 160; without the next token on its way: 47); bf16 36.7, 83%; NVFP4 41,
// 66%.  Fewer heads leave it further off: 16 / 4 of 128 dims, 9029 tokens NVFP4 29.2 us, 51%; 14 / 2 of 64, 20000 tokens
// bf16 33, 44%; 8 / 1 of 128, 20000 tokens e4m3 41, 39%.  The four CTAs of an SM have one more token each on its way:
// 48, 24, 9 and 10 KB for 32 / 8, 16 / 4, 14 / 2 and 8 / 1 heads, where 44 GB/s an SM over about 1 us of latency take 44.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "../hq_launch.h"
#include "../hq_ptx.cuh"
#include "hq_kv.h"
#include "hq_kv_codec.cuh"

namespace hq {

namespace {

constexpr int KW_THREADS = 128;

// x / y rounded to nearest even from yi = RN(1 / y): RN(x yi) is faithful, its residual is exact with one FMA, and one
// more FMA gives the correctly rounded quotient (P. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", IBM J. Res. Dev. 34(1), 1990).  quick() says for which y callers take it, and they divide
// otherwise: 1 / y is a normal number there, and the residual, a multiple of ulp(quotient) * ulp(y), is one of 2^-149
// for every quotient from 2^-10 on; smaller ones become zero codes however they are rounded.  (A row's largest magnitude
// over 448, kept in all its bits, has a residual of multiples of 2^-140.)  The quotient must be finite: of an infinite
// one the residual would make a NaN, where a division's saturates.
__device__ __forceinline__ float quotient(float x, float y, float yi) {
  const float q = __fmul_rn(x, yi);
  return __fmaf_rn(__fmaf_rn(-q, y, x), yi, q);
}
constexpr float KW_LEAST = 1.0097420e-28f, KW_MOST = 4.2535296e+37f;  // 2^-93, 2^125
__device__ __forceinline__ bool quick(float y) { return y == 0.0f || (y >= KW_LEAST && y <= KW_MOST); }

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
// the larger of two; KEEP: a NaN if either is one
template <bool KEEP>
__device__ __forceinline__ float larger(float a, float b) {
  if constexpr (!KEEP) return fmaxf(a, b);
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}
template <int LPH, bool KEEP>
__device__ __forceinline__ float lanes_largest(const float (&x)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = larger<KEEP>(m, fabsf(x[i]));
#pragma unroll
  for (int o = LPH / 2; o > 0; o >>= 1) m = larger<KEEP>(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

enum { NO_TURN = 0, BY_HALVES = 1, INTERLEAVED = 2 };

// Norm (w: the lane's weights, ones where there is none) and rotation of a row, without branches, so that several rows'
// shuffles and chains overlap.  The rotated pairs are (x[i], x[i + 4]) for a rotation by halves, (x[2 i], x[2 i + 1])
// for an interleaved one; cs, sn are their four angles'.
template <int LPH, int MODE>
__device__ __forceinline__ void norm_rotate(float (&x)[8], bool on, const float (&w)[8], float eps, bool turn,
                                            const float (&cs)[4], const float (&sn)[4]) {
  float sq = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) sq = fmaf(x[i], x[i], sq);
  const float r = on ? rsqrtf(lanes_sum<LPH>(sq) * (1.0f / (8 * LPH)) + eps) : 1.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
  if constexpr (MODE != NO_TURN) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float& p = x[MODE == INTERLEAVED ? 2 * i : i];
      float& q = x[MODE == INTERLEAVED ? 2 * i + 1 : i + 4];
      const float p0 = p, q0 = q, p1 = fmaf(p0, cs[i], -q0 * sn[i]), q1 = fmaf(q0, cs[i], p0 * sn[i]);
      p = turn ? p1 : p0;
      q = turn ? q1 : q0;
    }
  }
}

// NVFP4's global scale of one side and what block scales are divided by
struct Global {
  float g, six, inverse;  // g, 6 g, 1 / (6 g)
  float most;             // largest magnitudes below it are taken by quotient(): 1024 * 6 g, far into saturation; 0: none is
  __device__ __forceinline__ explicit Global(float x) : g(x) {
    six = __fmul_rn(6.0f, x);
    inverse = __frcp_rn(six);
    most = six >= KW_LEAST && six <= KW_MOST ? six * 1024.0f : 0.0f;
  }
};

// The scale that a lane's eight dims are divided by: e4m3's of the row, NVFP4's of the block of 16 dims (two lanes) with
// its byte.  0 where all codes are zero.  A NaN is a code of its own in e4m3 and does not count for the scale; e2m1 has
// none, so it makes its block's scale NaN.  fits: no dim's quotient by the scale passes fp32's range (e4m3: it is 449 at
// most, or quick() refuses the scale; NVFP4: a scale is 2^-9 g at least, so it is below 2^22).
template <int KIND, int D>
__device__ __forceinline__ float scale_of(const float (&x)[8], const Global& g, uint32_t& byte, bool& fits) {
  if constexpr (KIND == HQ_KV_E4M3) {
    const float m = lanes_largest<D / 8, false>(x);
    fits = true;
    return m >= KW_LEAST && m < INFINITY ? quotient(m, 448.0f, 1.0f / 448.0f) : __fdiv_rn(m, 448.0f);
  } else {
    const float m = lanes_largest<2, true>(x);
    fits = m < g.most;
    const float y = fits ? quotient(m, g.six, g.inverse) : __fdiv_rn(m, g.six);
    byte = g.g > 0.0f ? pack_e4m3x2(y, 0.0f) & 0xFFu : 0u;
    return __fmul_rn(f16x2_to_f32x2(e4m3x2_to_f16x2(byte)).x, g.g);
  }
}

// What a lane's dims are divided by: the scale, or one for e4m3's zero scale, whose dims are zeros (or so small that
// they become zeros) and NaN.
template <int KIND>
__device__ __forceinline__ float divisor(float s) {
  return KIND == HQ_KV_E4M3 && s == 0.0f ? 1.0f : s;
}

// A quantised row into the pool; x holds the quotients.
template <int KIND, int D>
__device__ __forceinline__ void store_codes(uint8_t* codes, uint8_t* scales, int64_t row, int l, int lo, int hi,
                                            const float (&x)[8], float s, uint32_t byte) {
  uint8_t* dst = codes + row * kv_row_bytes(KIND, D);
  if constexpr (KIND == HQ_KV_E4M3) {
    const uint32_t c0 = pack_e4m3x2(x[0], x[1]) | (pack_e4m3x2(x[2], x[3]) << 16);
    const uint32_t c1 = pack_e4m3x2(x[4], x[5]) | (pack_e4m3x2(x[6], x[7]) << 16);
    const uint32_t keep = s > 0.0f ? ~0u : 0x7F7F7F7Fu;  // of a zero scale no sign, but a NaN
    *reinterpret_cast<uint32_t*>(dst + lo) = c0 & keep;
    *reinterpret_cast<uint32_t*>(dst + hi) = c1 & keep;
    if (l == 0) reinterpret_cast<float*>(scales)[row] = s;
  } else {
    const uint32_t c = pack_e2m1x8(x);
    *reinterpret_cast<uint32_t*>(dst + 4 * l) = s > 0.0f ? c : 0u;
    if (!(l & 1)) scales[row * (D / 16) + l / 2] = (uint8_t)byte;
  }
}

// What a warp reads of one token.
template <int STEPS>
struct Token {
  Row q[STEPS], k, v;
  float4 cs, sn;  // the lane's four angles
  int64_t slot;
  int64_t pos;
};

constexpr int KW_STEPS = 4;  // query steps of a warp that are kept in registers, at most

// STEPS: query steps of a warp that are kept in registers, 1, 2 or KW_STEPS.  A step without heads costs its instructions
// all the same (with KW_STEPS alone: 16 / 4 heads of 128 dims, 9029 tokens NVFP4 35.1 us, where this was 27.5; 8 / 1 heads,
// 20000 tokens e4m3 63 and 41).  Five CTAs per SM where one step leaves the registers are no faster.
// MORE: a warp has at least two query steps beyond those that its registers hold; they are loaded as many at a time (56
// heads of 256 dims: 243 us one by one, 194 so).  With one beyond them it is loaded on its own: the batch's registers
// cost 32 heads of 128 dims 38.4 us -> 40.2.
template <int KIND, int D, int MODE, int STEPS, bool MORE>
__global__ void __launch_bounds__(KW_THREADS, 4) kv_write_kernel(const KvWriteArgs a) {
  constexpr int LPH = D / 8;     // lanes of a head's row
  constexpr int HPW = 32 / LPH;  // heads of one step
  constexpr int NEXT = KW_THREADS / 32 * HPW;
  constexpr bool halves = MODE == BY_HALVES;
  constexpr bool neighbours = KIND == HQ_KV_NVFP4 && halves;  // key rows by neighbours all the same: blocks of 16 dims
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % LPH, sub = lane / LPH;
  const int H = a.kv.heads, Hq = a.q_heads, R = a.rotary;
  const bool turn = 8 * l < R;
  // the lane's dims: by halves of the rotated part and of the rest, or eight neighbours
  int lo = 8 * l, hi = 8 * l + 4;
  if (halves && turn) lo = 4 * l, hi = R / 2 + 4 * l;
  const int klo = neighbours ? 8 * l : lo, khi = neighbours ? 8 * l + 4 : hi;
  int h0 = warp * HPW + sub;  // the lane's first head of the token; the warps take the places in turn
  const int ktok = Hq * D, vtok = ktok + H * D;

  auto read_place = [&](int64_t t, Token<STEPS>& x) {
    const bool live = t < a.T;
    x.slot = live ? a.slots[t] : -1;
    x.pos = MODE != NO_TURN && live ? a.positions[t] : 0;
  };
  const int by = H % NEXT || Hq % NEXT ? HPW : 0;
  auto next_h0 = [&](int h) { return h + by < NEXT ? h + by : h + by - NEXT; };
  auto read_rows = [&](int64_t t, int h0, Token<STEPS>& x) {  // its position is known
    const bool live = t < a.T;
    const uint16_t* row = a.qkv + t * a.row_stride + h0 * D;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) x.q[s] = load_row(row + s * NEXT * D, lo, hi, live && h0 + s * NEXT < Hq);
    x.k = load_row(row + ktok, klo, khi, live && h0 < H);
    x.v = load_row(row + vtok, 8 * l, 8 * l + 4, live && h0 < H);
    if constexpr (MODE != NO_TURN) {
      const float* angles = a.cos_sin + (x.pos >= 0 && x.pos < a.num_positions ? x.pos : 0) * R;
      x.cs = *reinterpret_cast<const float4*>(angles + (turn ? 4 * l : 0));
      x.sn = *reinterpret_cast<const float4*>(angles + R / 2 + (turn ? 4 * l : 0));
    }
  };

  float w[8];
  Row kw = {make_uint2(0x3F803F80u, 0x3F803F80u), make_uint2(0x3F803F80u, 0x3F803F80u)};  // ones
  unpack_row(a.q_norm ? load_row(a.q_norm, lo, hi, true) : kw, w);
  if (a.k_norm) kw = load_row(a.k_norm, klo, khi, true);
  const bool q_on = a.q_norm != nullptr, k_on = a.k_norm != nullptr;
  const Global kg(KIND == HQ_KV_NVFP4 ? *a.kv.k_global : 1.0f), vg(KIND == HQ_KV_NVFP4 ? *a.kv.v_global : 1.0f);
  const uint32_t ps = (uint32_t)a.kv.page_size;
  const int64_t G = gridDim.x, slots = a.kv.num_pages * ps;
  Token<STEPS> x, y, z;
  read_place(blockIdx.x, x);
  read_place(blockIdx.x + G, y);
  read_rows(blockIdx.x, h0, x);
  for (int64_t t = blockIdx.x; t < a.T; t += G, x = y, y.slot = z.slot, y.pos = z.pos, h0 = next_h0(h0)) {
    read_rows(t + G, next_h0(h0), y);
    read_place(t + 2 * G, z);
    const bool cached = x.slot >= 0 && x.slot < slots;
    const bool placed = MODE == NO_TURN || (x.pos >= 0 && x.pos < a.num_positions);
    if (threadIdx.x == 0 && ((x.slot >= 0 && !cached) || !placed)) kv_report(a.status);
    if (!placed) continue;
    const float cs[4] = {x.cs.x, x.cs.y, x.cs.z, x.cs.w}, sn[4] = {x.sn.x, x.sn.y, x.sn.z, x.sn.w};

    // ---- query heads
    uint16_t* out = a.q_out + (t * Hq + h0) * D;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      float f[8];
      unpack_row(x.q[s], f);
      norm_rotate<LPH, MODE>(f, q_on, w, a.eps, turn, cs, sn);
      if (h0 + s * NEXT < Hq) store_row(out + s * NEXT * D, lo, hi, f);
    }
    for (int h = h0 + STEPS * NEXT; MORE && h - sub < Hq; h += STEPS * NEXT) {
      const uint16_t* row = a.qkv + t * a.row_stride + (int64_t)h * D;
#pragma unroll
      for (int s = 0; s < STEPS; ++s) x.q[s] = load_row(row + s * NEXT * D, lo, hi, h + s * NEXT < Hq);
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        float f[8];
        unpack_row(x.q[s], f);
        norm_rotate<LPH, MODE>(f, q_on, w, a.eps, turn, cs, sn);
        if (h + s * NEXT < Hq) store_row(out + (int64_t)(h - h0 + s * NEXT) * D, lo, hi, f);
      }
    }

    for (int h = h0 + STEPS * NEXT; !MORE && h - sub < Hq; h += NEXT) {
      float f[8];
      unpack_row(load_row(a.qkv + t * a.row_stride + (int64_t)h * D, lo, hi, h < Hq), f);
      norm_rotate<LPH, MODE>(f, q_on, w, a.eps, turn, cs, sn);
      if (h < Hq) store_row(out + (int64_t)(h - h0) * D, lo, hi, f);
    }

    // ---- key and value heads
    if (!cached) continue;
    const int64_t page = x.slot >> 32 ? x.slot / ps : (uint32_t)x.slot / ps;
    const int64_t row0 = page * H * ps + (x.slot - page * ps);
    for (int h = h0; h - sub < H; h += NEXT) {
      if (h != h0) {
        const uint16_t* row = a.qkv + t * a.row_stride + (int64_t)h * D;
        x.k = load_row(row + ktok, klo, khi, h < H);
        x.v = load_row(row + vtok, 8 * l, 8 * l + 4, h < H);
      }
      float f[8], g[8];
      unpack_row(x.k, f);
      unpack_row(kw, g);
      norm_rotate<LPH, neighbours ? NO_TURN : MODE>(f, k_on, g, a.eps, turn, cs, sn);
      if constexpr (neighbours) {  // eight neighbouring dims pair with those of another lane
        const int half = R / 2, i0 = 8 * l < half ? 8 * l : 8 * l - half;
        const int partner = turn ? (8 * l < half ? lane + half / 8 : lane - half / 8) : lane;
        const float sign = 8 * l < half ? -1.0f : 1.0f;
        const float4* angles = reinterpret_cast<const float4*>(a.cos_sin + x.pos * R + (turn ? i0 : 0));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float4 ac = angles[i], as = angles[half / 4 + i];
          const float kc[4] = {ac.x, ac.y, ac.z, ac.w}, kn[4] = {as.x, as.y, as.z, as.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float& y = f[4 * i + j];
            const float p = __shfl_sync(0xffffffffu, y, partner);
            if (turn) y = fmaf(y, kc[j], sign * p * kn[j]);
          }
        }
      }
      unpack_row(x.v, g);
      const int64_t row = row0 + (int64_t)h * ps;
      if constexpr (KIND == HQ_KV_BF16) {
        if (h < H) {
          store_row(reinterpret_cast<uint16_t*>(a.kv.k) + row * D, klo, khi, f);
          store_row(reinterpret_cast<uint16_t*>(a.kv.v) + row * D, 8 * l, 8 * l + 4, g);
        }
      } else {
        uint32_t kb = 0, vb = 0;
        bool kfit, vfit;
        const float ks = scale_of<KIND, D>(f, kg, kb, kfit), vs = scale_of<KIND, D>(g, vg, vb, vfit);
        const float kd = divisor<KIND>(ks), vd = divisor<KIND>(vs);
        if (__all_sync(0xffffffffu, kfit && vfit && quick(kd) && quick(vd))) {
          const float ki = __frcp_rn(kd), vi = __frcp_rn(vd);
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = quotient(f[i], kd, ki), g[i] = quotient(g[i], vd, vi);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = __fdiv_rn(f[i], kd), g[i] = __fdiv_rn(g[i], vd);
        }
        if (h < H) {
          store_codes<KIND, D>(a.kv.k, a.kv.k_scale, row, l, klo, khi, f, ks, kb);
          store_codes<KIND, D>(a.kv.v, a.kv.v_scale, row, l, 8 * l, 8 * l + 4, g, vs, vb);
        }
      }
    }
  }
}

template <int KIND, int D, int MODE, int STEPS, bool MORE>
cudaError_t launch_steps(const KvWriteArgs& a, cudaStream_t stream) {
  static std::atomic<int> resident{0};  // CTAs that the device holds at once
  int n = resident.load(std::memory_order_relaxed);
  if (n == 0) {
    int dev = 0, sms = 0, per = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kv_write_kernel<KIND, D, MODE, STEPS, MORE>, KW_THREADS, 0);
    if (e != cudaSuccess) return e;
    n = (per > 0 ? per : 1) * (sms > 0 ? sms : 1);
    resident.store(n, std::memory_order_relaxed);
  }
  return launch_kernel(kv_write_kernel<KIND, D, MODE, STEPS, MORE>, dim3((unsigned)(a.T < n ? a.T : n)),
                       dim3(KW_THREADS), 0, stream, a);
}

template <int KIND, int D, int MODE>
cudaError_t launch(const KvWriteArgs& a, cudaStream_t stream) {
  constexpr int NEXT = KW_THREADS / 32 * (256 / D);
  if (a.q_heads <= NEXT) return launch_steps<KIND, D, MODE, 1, false>(a, stream);
  if (a.q_heads <= 2 * NEXT) return launch_steps<KIND, D, MODE, 2, false>(a, stream);
  return a.q_heads > (KW_STEPS + 1) * NEXT ? launch_steps<KIND, D, MODE, KW_STEPS, true>(a, stream)
                                           : launch_steps<KIND, D, MODE, KW_STEPS, false>(a, stream);
}

template <int KIND, int D>
cudaError_t by_mode(const KvWriteArgs& a, cudaStream_t stream) {
  if (a.rotary == 0) return launch<KIND, D, NO_TURN>(a, stream);
  return a.interleaved ? launch<KIND, D, INTERLEAVED>(a, stream) : launch<KIND, D, BY_HALVES>(a, stream);
}

template <int KIND>
cudaError_t by_dim(int dim, const KvWriteArgs& a, cudaStream_t stream) {
  return dim == 64 ? by_mode<KIND, 64>(a, stream)
                   : (dim == 128 ? by_mode<KIND, 128>(a, stream) : by_mode<KIND, 256>(a, stream));
}

}  // namespace

cudaError_t launch_kv_write(int kind, int dim, const KvWriteArgs& a, cudaStream_t stream) {
  return kind == HQ_KV_BF16 ? by_dim<HQ_KV_BF16>(dim, a, stream)
                            : (kind == HQ_KV_E4M3 ? by_dim<HQ_KV_E4M3>(dim, a, stream)
                                                  : by_dim<HQ_KV_NVFP4>(dim, a, stream));
}

}  // namespace hq
