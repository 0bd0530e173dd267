// Attention of one new token per sequence over a paged cache.
//
// One CTA per (sequence, query head): each warp takes every fourth token with its own running maximum m and sum l, so
// that after token j   m' = max(m, s_j),  l = l exp(m - m') + exp(s_j - m'),  o = o exp(m - m') + exp(s_j - m') v_j;
// the warps' parts are joined the same way.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../hq_launch.h"
#include "../hq_ptx.cuh"
#include "hq_kv.h"
#include "hq_kv_codec.cuh"

namespace hq {

namespace {

constexpr int KA_WARPS = 4;

// value of one dim of a row
template <int KIND, int D>
__device__ __forceinline__ float value(const uint8_t* codes, const uint8_t* scales, float g, int64_t row, int d) {
  if constexpr (KIND == HQ_KV_BF16) {
    return bf16_lo(reinterpret_cast<const uint16_t*>(codes)[row * D + d]);
  } else if constexpr (KIND == HQ_KV_E4M3) {
    return f16x2_to_f32x2(e4m3x2_to_f16x2(codes[row * D + d])).x * reinterpret_cast<const float*>(scales)[row];
  } else {
    const uint32_t c = (codes[row * (D / 2) + d / 2] >> (4 * (d & 1))) & 15u;
    float f[8];
    unpack_e2m1x8(c, f);
    return f[0] * (f16x2_to_f32x2(e4m3x2_to_f16x2(scales[row * (D / 16) + d / 16])).x * g);
  }
}

template <int KIND, int D>
__global__ void __launch_bounds__(KA_WARPS * 32) kv_attention_kernel(const KvAttnArgs a) {
  constexpr int N = D / 32;
  __shared__ float part[KA_WARPS][D + 2];
  pdl_trigger();
  pdl_wait();
  const int H = a.kv.heads, Hq = H * a.group;
  const int64_t b = blockIdx.x / Hq;
  const int hq = (int)(blockIdx.x - b * Hq), h = hq / a.group;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t n = a.lens[b];
  const int64_t most = a.table_stride * a.kv.page_size;
  if (n < 0 || n > most) {
    if (threadIdx.x == 0) kv_report(a.status);
    n = n < 0 ? 0 : most;
  }
  const int64_t j0 = a.window > 0 && n > a.window ? n - a.window : 0;
  float kg = 1.0f, vg = 1.0f;
  if constexpr (KIND == HQ_KV_NVFP4) kg = *a.kv.k_global, vg = *a.kv.v_global;
  float q[N], o[N], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    q[i] = bf16_lo(a.q[(b * Hq + hq) * D + lane + 32 * i]) * a.scale;
    o[i] = 0.0f;
  }
  for (int64_t j = j0 + warp; j < n; j += KA_WARPS) {
    const int64_t page = a.page_table[b * a.table_stride + j / a.kv.page_size];
    if (page < 0 || page >= a.kv.num_pages) {
      if (lane == 0) kv_report(a.status);
      continue;
    }
    const int64_t row = (page * H + h) * a.kv.page_size + j % a.kv.page_size;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) s = fmaf(q[i], value<KIND, D>(a.kv.k, a.kv.k_scale, kg, row, lane + 32 * i), s);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    if (a.softcap > 0.0f) s = a.softcap * tanhf(s / a.softcap);
    const float m1 = fmaxf(m, s), f = m1 == -INFINITY ? 1.0f : expf(m - m1), p = m1 == -INFINITY ? 0.0f : expf(s - m1);
    m = m1;
    l = l * f + p;
#pragma unroll
    for (int i = 0; i < N; ++i)
      o[i] = fmaf(p, value<KIND, D>(a.kv.v, a.kv.v_scale, vg, row, lane + 32 * i), o[i] * f);
  }
  if (lane == 0) part[warp][D] = m, part[warp][D + 1] = l;
#pragma unroll
  for (int i = 0; i < N; ++i) part[warp][lane + 32 * i] = o[i];
  __syncthreads();
  float mm = -INFINITY, ll = 0.0f;
  for (int w = 0; w < KA_WARPS; ++w) mm = fmaxf(mm, part[w][D]);
  for (int w = 0; w < KA_WARPS; ++w) ll += part[w][D] == -INFINITY ? 0.0f : part[w][D + 1] * expf(part[w][D] - mm);
  for (int d = threadIdx.x; d < D; d += KA_WARPS * 32) {
    float y = 0.0f;
    for (int w = 0; w < KA_WARPS; ++w) y += part[w][D] == -INFINITY ? 0.0f : part[w][d] * expf(part[w][D] - mm);
    a.out[(b * Hq + hq) * D + d] = (uint16_t)pack_bf16x2(ll > 0.0f ? y / ll : 0.0f, 0.0f);
  }
  if (threadIdx.x == 0 && a.lse) a.lse[b * Hq + hq] = ll > 0.0f ? mm + logf(ll) : -INFINITY;
}

template <int KIND>
cudaError_t by_dim(int dim, const KvAttnArgs& a, cudaStream_t stream) {
  const dim3 grid((unsigned)(a.B * a.kv.heads * a.group)), block(KA_WARPS * 32);
  return dim == 64 ? launch_kernel(kv_attention_kernel<KIND, 64>, grid, block, 0, stream, a)
                   : (dim == 128 ? launch_kernel(kv_attention_kernel<KIND, 128>, grid, block, 0, stream, a)
                                 : launch_kernel(kv_attention_kernel<KIND, 256>, grid, block, 0, stream, a));
}

}  // namespace

cudaError_t launch_kv_attention(int kind, int dim, const KvAttnArgs& a, cudaStream_t stream) {
  return kind == HQ_KV_BF16 ? by_dim<HQ_KV_BF16>(dim, a, stream)
                            : (kind == HQ_KV_E4M3 ? by_dim<HQ_KV_E4M3>(dim, a, stream)
                                                  : by_dim<HQ_KV_NVFP4>(dim, a, stream));
}

}  // namespace hq
