// A layer's rows made into the activations of its next product, in one pass over memory:
//   add_rms_norm   r = x + residual, residual_out = bf16(r), y = r / sqrt(mean(r^2) + eps) * w
//   swiglu         y = silu(gate) * up of the rows [gate | up]
//   (rows as they are, for hq_quantize_act's block scales)
// with y out as bf16, as e4m3 with one fp32 scale per row, or as e4m3 with one per 128 elements (scale = absmax / 448).
// y is never rounded on the way: fp32 until its code.
//
// All of them are bound by memory: a row is read once and stays in registers between its statistics and its codes.
// Measured, inputs past L2: norm of 8192 x 7168 with a residual 62.2 us with a scale per row (6610 GB/s, 97% of copy
// bandwidth), 66.2 us with one per 128 (6240 GB/s), 74.8 us to bf16 (6280 GB/s); rows as they are 28.0 us (6360 GB/s).
// SwiGLU of 8192 x 7168 with a scale per 128 50.4 us (5860 GB/s) and of 32768 x 768 with one per row 24.6 us (5120 GB/s):
// issue slots are two thirds full there (190 instructions for 8 outputs a lane, 18 of them powers and reciprocals).
#include <cuda_runtime.h>
#include <float.h>
#include <stdint.h>

#include <atomic>

#include "../hq_launch.h"
#include "../hq_ptx.cuh"
#include "../hq_quant.cuh"
#include "hq_row_ops.h"

namespace hq {

namespace {

enum RowSrc { SRC_NORM = 0, SRC_ADD_NORM = 1, SRC_SWIGLU = 2 };

// silu(g) * u = g * u / (1 + exp(-g)) of eight values (every lane of the warp calls it).  exp(-g) = 2^t with
// t = -g log2(e) in two parts: the product's fp32 rounding error, found by an FMA, together with the part of log2(e)
// below fp32, corrects the power to first order (2^(t + d) = 2^t (1 + d ln 2)), which without it would be off by up to
// |t| 2^-24.  The reciprocal gets one Newton step.  Two values go through each instruction but the power's and the
// reciprocal's.  Where a power over- or underflows (and where a gate is infinite) the quotient is taken as 0 or 1; true is
// returned to all lanes, and silu_far has the values behind the zeros.
__device__ __forceinline__ bool silu_mul(float2 (&g)[4], const float2 (&u)[4]) {
  constexpr float kHi = -1.44269504f, kLo = -1.925963033e-8f, kLn2 = 0.693147181f;
  float2 t[4], r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    t[i] = __fmul2_rn(g[i], both(kHi));
    const float2 d = __ffma2_rn(g[i], both(kLo), __ffma2_rn(g[i], both(kHi), make_float2(-t[i].x, -t[i].y)));
    float2 p;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p.x) : "f"(t[i].x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p.y) : "f"(t[i].y));
    const float2 q = __fadd2_rn(__ffma2_rn(p, __fmul2_rn(d, both(kLn2)), p), both(1.0f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r[i].x) : "f"(q.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r[i].y) : "f"(q.y));
    r[i] = __ffma2_rn(r[i], __ffma2_rn(make_float2(-q.x, -q.y), r[i], both(1.0f)), r[i]);
  }
  const bool ends = __any_sync(0xffffffffu, !(__uint_as_float(absmax_bits(t)) <= 126.0f));
  if (ends) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (fabsf(t[i].x) > 126.0f) r[i].x = t[i].x > 0.0f ? 0.0f : 1.0f;
      if (fabsf(t[i].y) > 126.0f) r[i].y = t[i].y > 0.0f ? 0.0f : 1.0f;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) g[i] = __fmul2_rn(__fmul2_rn(g[i], r[i]), u[i]);
  return ends;
}

// silu(g) * u where t = -g log2(e) is above 126: there 1 / (1 + exp(-g)) is exp(g) to fp32's precision and leaves its
// normal range, but g exp(g) u need not.  exp(g) = 2^-t is therefore taken 2^192 times larger (t - 192 is exact), with
// the correction of silu_mul's power, and the factor divided out in halves, u's first: what that loses of a small u is
// below fp32's smallest number in the result.  Past t = 290 the largest u leaves less than half of that number.
// Gate and up are read again, so that a path which ordinary activations never take costs the others no registers (with
// the values at hand 8192 x 7168 took 55 us for 53, 2048 x 32768 80 for 70).
__device__ __forceinline__ void silu_far(float2 (&y)[4], const uint4* gate, const uint4* up) {
  const auto far = [](uint32_t gbits, uint32_t ubits, float y) {
    constexpr float kHi = -1.44269504f, kLo = -1.925963033e-8f, kLn2 = 0.693147181f;
    const float g = __uint_as_float(gbits), u = __uint_as_float(ubits), t = __fmul_rn(g, kHi);
    if (!(t > 126.0f && t <= 290.0f)) return y;
    const float d = fmaf(g, kLo, fmaf(g, kHi, -t));
    float p;
    asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(p) : "f"(192.0f - t));
    p = fmaf(p, -kLn2 * d, p);
    return __fmul_rn(__fmul_rn(__fmul_rn(g, p), __fmul_rn(u, 0x1p-96f)), 0x1p-96f);
  };
  const uint4 vg = *gate, vu = *up;
  const uint32_t g[4] = {vg.x, vg.y, vg.z, vg.w}, u[4] = {vu.x, vu.y, vu.z, vu.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[i].x = far(g[i] << 16, u[i] << 16, y[i].x);
    y[i].y = far(g[i] & 0xFFFF0000u, u[i] & 0xFFFF0000u, y[i].y);
  }
}

// Reductions over a row's threads: a warp, or the CTA (every thread calls them; `turn` alternates between the two
// buffers, so that one barrier per reduction is enough).
template <bool WARP, typename T, typename F>
__device__ __forceinline__ T row_reduce(T v, T zero, T (*red)[32], int& turn, F&& f) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
  if (WARP) return v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) red[turn][warp] = v;
  __syncthreads();
  v = lane < (int)(blockDim.x >> 5) ? red[turn][lane] : zero;
  turn ^= 1;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// SwiGLU rows with gates far below zero (silu_far), done again with a scale per row after the row kernel's own loop: a
// function of its own, whose registers ordinary rows do not pay for.
template <bool WARP>
__device__ __noinline__ void swiglu_rows_again(const uint16_t* rows_in, int64_t rows, int width, void* out, float* scale,
                                               uint32_t (*red)[32]) {
  const int t = WARP ? (threadIdx.x & 31) : threadIdx.x, n = WARP ? 32 : blockDim.x, chunks = width >> 3;
  const auto most = [](uint32_t p, uint32_t q) { return max(p, q); };
  int turn = 0;
  if (!WARP) __syncthreads();
  for (int64_t row = (int64_t)blockIdx.x * (WARP ? 4 : 1) + (WARP ? (threadIdx.x >> 5) : 0); row < rows;
       row += (int64_t)gridDim.x * (WARP ? 4 : 1)) {
    const uint4* x = reinterpret_cast<const uint4*>(rows_in) + row * 2 * chunks;
    const auto chunk = [&](int c, float2 (&f)[4]) {  // (the whole warp's: zeros behind the row)
      const uint4 none = make_uint4(0u, 0u, 0u, 0u);
      float2 u[4];
      bf16x8_to_f32x2(c < chunks ? x[c] : none, f);
      bf16x8_to_f32x2(c < chunks ? x[chunks + c] : none, u);
      const bool ends = silu_mul(f, u);
      if (ends && c < chunks) silu_far(f, x + c, x + chunks + c);
      return ends;
    };
    float2 f[4];
    uint32_t m = 0;
    bool ends = false;
#pragma unroll 1
    for (int c0 = 0; c0 < chunks; c0 += n) {
      ends |= chunk(t + c0, f);
      m = max(m, absmax_bits(f));
    }
    if (!row_reduce<WARP>((uint32_t)ends, 0u, red, turn, most)) continue;
    m = row_reduce<WARP>(m, 0u, red, turn, most);
    const E4m3Scale s(m);
    if (t == 0) scale[row] = s.s;
#pragma unroll 1
    for (int c0 = 0; c0 < chunks; c0 += n) {
      chunk(t + c0, f);
      const uint2 q = s.codes(f);
      if (t + c0 < chunks) static_cast<uint2*>(out)[row * chunks + t + c0] = q;
    }
  }
}

// One row per CTA, or per warp (WARP, four rows a CTA), CH chunks of 8 elements per thread; the next row of the same
// threads is loaded while the current one is reduced and written.  LONG: rows past 2048 chunks on 1024 threads, whose
// registers leave no room for that, nor for the norm's weights, which every row reads again (from L2): 2048 x 32768 with a
// residual 81.4 us with a scale per row (5770 GB/s), 85.9 with one per 128, 86.1 to bf16 (6240 GB/s); SwiGLU 67.8 us
// (4950 GB/s).  Four of the seven instances spill 4 to 36 bytes.
template <int SRC, int OUT, int CH, bool WARP, bool LONG>
__global__ void __launch_bounds__(WARP || (SRC == SRC_SWIGLU && CH == 2) ? 128 : (CH == 1 || LONG ? 1024 : 512),
                                  SRC == SRC_SWIGLU && CH == 2 ? 9 : 0) row_kernel(const RowArgs a) {
  __shared__ float red_f[2][32];
  __shared__ uint32_t red_u[2][32];
  constexpr bool NORM = SRC != SRC_SWIGLU;
  constexpr bool TWO = SRC != SRC_NORM;  // two operands a chunk: x and residual, or gate and up
  int turn_f = 0, turn_u = 0;
  const int t = WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int n = WARP ? 32 : blockDim.x;
  const int chunks = a.width >> 3;
  const int64_t step = (int64_t)gridDim.x * (WARP ? 4 : 1);
  int64_t row = (int64_t)blockIdx.x * (WARP ? 4 : 1) + (WARP ? (threadIdx.x >> 5) : 0);
  pdl_trigger();
  pdl_wait();
  const uint4 none = make_uint4(0u, 0u, 0u, 0u);
  uint4 w[LONG ? 1 : CH], va[LONG ? 1 : CH], vb[LONG ? 1 : CH];
  auto first = [&](int64_t r) { return reinterpret_cast<const uint4*>(a.x + r * a.x_stride); };
  auto second = [&](int64_t r) {
    return SRC == SRC_SWIGLU ? first(r) + chunks : reinterpret_cast<const uint4*>(a.residual + r * a.residual_stride);
  };
  auto weight = [&](int c) { return c < chunks ? reinterpret_cast<const uint4*>(a.weight)[c] : none; };
  auto load = [&](int64_t r) {
    const uint4 *pa = first(r), *pb = TWO ? second(r) : pa;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = t + j * n;
      va[j] = c < chunks ? pa[c] : none;
      if (TWO) vb[j] = c < chunks ? pb[c] : none;
    }
  };
  const float width = (float)a.width, inv_width = __frcp_rn(width);
  if (!LONG) {
    if (row < a.rows) load(row);
    if (NORM) {
#pragma unroll
      for (int j = 0; j < CH; ++j) w[j] = weight(t + j * n);
    }
  }
  bool ends = false;
  for (; row < a.rows; row += step) {
    float2 f[CH][4];
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = t + j * n;
      const uint4 x = LONG ? (c < chunks ? first(row)[c] : none) : va[LONG ? 0 : j];
      bf16x8_to_f32x2(x, f[j]);
      if (TWO) {
        float2 g[4];
        bf16x8_to_f32x2(LONG ? (c < chunks ? second(row)[c] : none) : vb[LONG ? 0 : j], g);
        if (SRC == SRC_SWIGLU) {
          if (!WARP || j * n < chunks) ends |= silu_mul(f[j], g);  // (a warp's short row leaves its last chunks out)
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) f[j][i] = __fadd2_rn(f[j][i], g[i]);
        }
      }
    }
    if (!LONG && row + step < a.rows) load(row + step);
    if (SRC == SRC_ADD_NORM) {
      uint4* ro = reinterpret_cast<uint4*>(a.residual_out + row * a.residual_out_stride);
#pragma unroll
      for (int j = 0; j < CH; ++j)
        if (t + j * n < chunks) ro[t + j * n] = bf16x8_of(f[j]);
    }
    if (NORM) {
      auto add = [](float p, float q) { return p + q; };
      auto squares = [&] {
        float2 s[2] = {both(0.0f), both(0.0f)};
#pragma unroll
        for (int j = 0; j < CH; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[i & 1] = __ffma2_rn(f[j][i], f[j][i], s[i & 1]);
        return row_reduce<WARP>((s[0].x + s[1].x) + (s[0].y + s[1].y), 0.0f, red_f, turn_f, add);
      };
      const float ss = squares();
      // 1 / sqrt(mean + eps): the approximation and one Newton step
      const float v = div_by(ss, width, inv_width) + a.eps;
      float rstd;
      asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(rstd) : "f"(v));
      rstd = fmaf(rstd, fmaf(-0.5f * v * rstd, rstd, 0.5f), rstd);
      // A sum that overflowed (of squares, or of their mean and eps), or one that lost small squares where eps does not
      // cover them, is taken again with the row divided by a power of two near its largest magnitude.  (A row of zeros
      // too: the approximation above takes an eps below 2^-126 as zero.)
      if (!(v <= FLT_MAX) || (ss < 0x1p-80f && a.eps < 0x1p-60f)) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < CH; ++j) m = max(m, absmax_bits(f[j]));
        m = row_reduce<WARP>(m, 0u, red_u, turn_u, [](uint32_t p, uint32_t q) { return max(p, q); });
        if (m < 0x7F800000u) {
          const int e = m > 0u ? ilogbf(__uint_as_float(m)) : 0;
#pragma unroll
          for (int j = 0; j < CH; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) f[j][i] = make_float2(ldexpf(f[j][i].x, -e), ldexpf(f[j][i].y, -e));
          const double ms = (double)squares() / a.width + ldexp((double)a.eps, -2 * e);
          rstd = (float)(1.0 / sqrt(ms));
        }
      }
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        float2 g[4];
        bf16x8_to_f32x2(LONG ? weight(t + j * n) : w[LONG ? 0 : j], g);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[j][i] = __fmul2_rn(__fmul2_rn(f[j][i], both(rstd)), g[i]);
      }
    }
    if (OUT == ROW_BF16) {
      uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + row * a.width);
#pragma unroll
      for (int j = 0; j < CH; ++j)
        if (t + j * n < chunks) o[t + j * n] = bf16x8_of(f[j]);
    } else {
      uint2* o = reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.out) + row * a.width);
      if (OUT == ROW_TOKEN) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < CH; ++j) m = max(m, absmax_bits(f[j]));
        m = row_reduce<WARP>(m, 0u, red_u, turn_u, [](uint32_t p, uint32_t q) { return max(p, q); });
        const E4m3Scale s(m);
        if (t == 0) a.scale[row] = s.s;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
          const uint2 q = s.codes(f[j]);
          if (t + j * n < chunks) o[t + j * n] = q;
        }
      } else {
        // the 16 chunks of a block are 16 neighbouring lanes (the row's threads are a multiple of 32)
#pragma unroll
        for (int j = 0; j < CH; ++j) {
          uint32_t m = absmax_bits(f[j]);
#pragma unroll
          for (int k = 8; k > 0; k >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, k));
          const E4m3Scale s(m);
          const int c = t + j * n;
          const uint2 q = s.codes(f[j]);
          if (c < chunks) o[c] = q;
          if (c < chunks && (t & 15) == 0) a.scale[row * (a.width >> 7) + (c >> 4)] = s.s;
        }
      }
    }
  }
  if (SRC == SRC_SWIGLU && (WARP ? (int)ends : __syncthreads_or(ends))) 
    swiglu_rows_again<WARP>(a.x, a.rows, a.width, a.out, a.scale, red_u);
}

// A scale per 128 outputs needs no statistics of the row: every thread takes U chunks of 8 outputs, all loads first; 16
// neighbouring lanes hold a block.
constexpr int BQ_THREADS = 256;
// i / d for 0 <= i < n.  Up to n = 2^31 by a multiplication: with m = floor(2^(31 + s) / d) + 1 and 2^s >= d the error
// of i m / 2^(31 + s) is below i / 2^(31 + s) < 1 / d.  (Division is a software routine.)
struct RowDivide {
  uint32_t d, m, shift;  // m = 0: plain division
  RowDivide(int64_t n, uint32_t d_) : d(d_), m(0), shift(0) {
    if (n > ((int64_t)1 << 31)) return;
    while ((1u << (shift + 1)) < d) ++shift;  // 2^(shift + 1) >= d, and m below 2^32 as d > 2^shift
    m = (uint32_t)(((uint64_t)1 << (32 + shift)) / d) + 1u;
  }
  __device__ __forceinline__ int64_t of(int64_t i) const {
    return m ? (int64_t)(__umulhi((uint32_t)i, m) >> shift) : i / d;
  }
};
template <bool SWIGLU, int U>
__global__ void __launch_bounds__(BQ_THREADS)
    block_quant_kernel(const uint4* x, int64_t n8, RowDivide per_row, uint2* __restrict__ q,
                       float* __restrict__ s_out) {
  pdl_trigger();
  pdl_wait();
  uint4 va[U], vb[U];
  const int64_t base = (int64_t)blockIdx.x * (BQ_THREADS * U) + threadIdx.x;
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int64_t i = base + j * BQ_THREADS;
    va[j] = vb[j] = make_uint4(0u, 0u, 0u, 0u);
    if (i < n8) {
      if (SWIGLU) {  // [gate | up] rows
        const uint4* p = x + i + per_row.of(i) * per_row.d;
        va[j] = *p;
        vb[j] = p[per_row.d];
      } else {
        va[j] = x[i];
      }
    }
  }
  const auto out = [&](int64_t i, const float2 (&f)[4]) {
    uint32_t m = absmax_bits(f);
#pragma unroll
    for (int k = 8; k > 0; k >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, k));
    const E4m3Scale s(m);
    const uint2 c = s.codes(f);
    if (i < n8) q[i] = c;
    if (i < n8 && (threadIdx.x & 15) == 0) s_out[i >> 4] = s.s;
  };
  bool ends = false;
#pragma unroll
  for (int j = 0; j < U; ++j) {
    float2 f[4];
    bf16x8_to_f32x2(va[j], f);
    if (SWIGLU) {
      float2 u[4];
      bf16x8_to_f32x2(vb[j], u);
      ends |= silu_mul(f, u);
    }
    out(base + j * BQ_THREADS, f);
  }
  if (SWIGLU && ends) {  // a warp with gates far below zero does its chunks again
    for (int j = 0; j < U; ++j) {
      const int64_t i = base + j * BQ_THREADS;
      const uint4 *pg = x, *pu = x;
      float2 f[4], u[4] = {};
      for (int k = 0; k < 4; ++k) f[k] = both(0.0f);
      if (i < n8) {
        pg = x + i + per_row.of(i) * per_row.d;
        pu = pg + per_row.d;
        bf16x8_to_f32x2(*pg, f);
        bf16x8_to_f32x2(*pu, u);
      }
      silu_mul(f, u);
      if (i < n8) silu_far(f, pg, pu);
      out(i, f);
    }
  }
}

int sms() {
  static const int n = [] {
    int dev = 0, v = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return 1;
    return v < 1 ? 1 : v;
  }();
  return n;
}

template <int SRC, int OUT, int CH, bool WARP, bool LONG = false>
cudaError_t launch_row(const RowArgs& a, int threads, cudaStream_t stream) {
  void (*k)(RowArgs) = row_kernel<SRC, OUT, CH, WARP, LONG>;
  const int64_t need = WARP ? (a.rows + 3) / 4 : a.rows;
  int64_t room = sms();
  if (need > room) {  // CTAs an SM holds, asked once for each CTA size
    static std::atomic<int> known[33];
    int per_sm = known[threads / 32].load(std::memory_order_relaxed);
    if (per_sm == 0) {
      if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k, threads, 0) != cudaSuccess || per_sm < 1) per_sm = 1;
      known[threads / 32].store(per_sm, std::memory_order_relaxed);
    }
    room *= per_sm;
  }
  return launch_kernel(k, dim3((unsigned)(need < room ? need : room)), dim3(threads), 0, stream, a);
}

template <int SRC, int OUT>
cudaError_t launch_rows(const RowArgs& a, cudaStream_t stream) {
  const int chunks = a.width / 8;
  const auto threads = [&](int ch) { return ((chunks + ch - 1) / ch + 31) / 32 * 32; };
  // Rows that a warp holds in four chunks a lane, and enough of them to fill the SMs' warps: no barriers (16384 x 1024
  // norms 20.8 -> 19.8 us, 32768 x 768 SwiGLU 32.0 -> 24.9).
  if (chunks <= 128 && a.rows >= 2048) return launch_row<SRC, OUT, 4, true>(a, 128, stream);
  // Few rows: as many threads as the row has chunks, for the shortest chain of work; else four chunks a thread from 2048
  // elements on (8192 x 4096 norms with two: 40.2 -> 42.4 us), two below, and the next row's loads in flight.
  if (a.rows <= 2 * sms() && chunks <= 1024) return launch_row<SRC, OUT, 1, false>(a, threads(1), stream);
  if (chunks <= 256) return launch_row<SRC, OUT, 2, false>(a, threads(2), stream);
  if (chunks <= 2048) return launch_row<SRC, OUT, 4, false>(a, threads(4), stream);
  return launch_row<SRC, OUT, 4, false, true>(a, threads(4), stream);
}

}  // namespace

cudaError_t launch_add_rms_norm(RowOut out, const RowArgs& a, cudaStream_t stream) {
  if (a.residual) {
    if (out == ROW_BF16) return launch_rows<SRC_ADD_NORM, ROW_BF16>(a, stream);
    if (out == ROW_TOKEN) return launch_rows<SRC_ADD_NORM, ROW_TOKEN>(a, stream);
    return launch_rows<SRC_ADD_NORM, ROW_BLOCK>(a, stream);
  }
  if (out == ROW_BF16) return launch_rows<SRC_NORM, ROW_BF16>(a, stream);
  if (out == ROW_TOKEN) return launch_rows<SRC_NORM, ROW_TOKEN>(a, stream);
  return launch_rows<SRC_NORM, ROW_BLOCK>(a, stream);
}

cudaError_t launch_swiglu_token(const RowArgs& a, cudaStream_t stream) {
  return launch_rows<SRC_SWIGLU, ROW_TOKEN>(a, stream);
}

cudaError_t launch_block_quant(bool swiglu, const void* x, int64_t rows, int64_t width, void* data, void* scale,
                               cudaStream_t stream) {
  const int64_t n8 = rows * (width >> 3);
  // One chunk a thread where that leaves no SM more than two CTAs (16 x 7168 SwiGLU: 2.4 -> 2.05 us), else two of the
  // SwiGLU (four: 5.6 -> 6.4 us at 512 x 7168, though 50.5 -> 48.1 at 8192 x 7168) and four of plain rows (two: 28.0 ->
  // 29.5 us at 8192 x 7168).
  const int unroll = n8 <= (int64_t)2 * sms() * BQ_THREADS ? 1 : (swiglu ? 2 : 4);
  const int64_t grid = (n8 + BQ_THREADS * unroll - 1) / (BQ_THREADS * unroll);
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
  void (*k)(const uint4*, int64_t, RowDivide, uint2*, float*) =
      swiglu ? (unroll == 1 ? block_quant_kernel<true, 1> : block_quant_kernel<true, 2>)
             : (unroll == 1 ? block_quant_kernel<false, 1> : block_quant_kernel<false, 4>);
  return launch_kernel(k, dim3((unsigned)grid), dim3(BQ_THREADS), 0, stream, static_cast<const uint4*>(x), n8,
                       RowDivide(n8, (uint32_t)(width >> 3)), static_cast<uint2*>(data), static_cast<float*>(scale));
}

}  // namespace hq
