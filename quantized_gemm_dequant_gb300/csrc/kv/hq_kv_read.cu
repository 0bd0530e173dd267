// Cached tokens back as contiguous bf16 rows.
//
// Memory-bound: a row's codes and scale are read once, its bf16 values are written once.  A CTA takes 16 output rows
// of all heads: the rows are one contiguous stretch of the output, and in the cache each head's rows are contiguous
// as far as the tokens share a page.  16 threads first find their row's sequence (binary search in `starts`) and its
// place in the pools; then every thread converts 8 dims at a time.  Measured on a GB300: e4m3, 9 sequences of up to 16000
// tokens, 8 heads of 128 dims: 78.5 us, 90% of the measured copy bandwidth; NVFP4, one of 50001: 44.5 us, 88%.  With few
// heads a CTA has little to load behind its chain of lookups (one head of 64 dims: 128 pieces for 256 threads): 16 of up
// to 16384 tokens, one head of 64 dims bf16 14.8 us, 75%, e4m3 18.7, 45%, NVFP4 16.3, 43%; one of 128 dims 96%, 69%,
// 63%; two of 128 dims 93%, 80%, 80%.
#include <cuda_runtime.h>
#include <stdint.h>

#include "../hq_launch.h"
#include "../hq_ptx.cuh"
#include "hq_kv.h"
#include "hq_kv_codec.cuh"

namespace hq {

namespace {

constexpr int KR_THREADS = 256;
constexpr int KR_ROWS = 16;

// the 8 values at dim 8 * l of row `row` of one pool, as bf16
template <int KIND, int D>
__device__ __forceinline__ uint4 read8(const uint8_t* codes, const uint8_t* scales, float g, int64_t row, int l) {
  const uint8_t* p = codes + row * kv_row_bytes(KIND, D);
  if constexpr (KIND == HQ_KV_BF16) {
    return __ldcs(reinterpret_cast<const uint4*>(p) + l);
  } else if constexpr (KIND == HQ_KV_E4M3) {
    const uint2 c = __ldcs(reinterpret_cast<const uint2*>(p) + l);
    const float s = reinterpret_cast<const float*>(scales)[row];
    const uint32_t w[2] = {c.x, c.y};
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = f16x2_to_f32x2(e4m3x2_to_f16x2(w[i / 2] >> (16 * (i & 1))));
      f[2 * i] = v.x * s;
      f[2 * i + 1] = v.y * s;
    }
    return pack_bf16x8(f);
  } else {
    const uint32_t c = __ldcs(reinterpret_cast<const uint32_t*>(p) + l);
    const float d = __fmul_rn(f16x2_to_f32x2(e4m3x2_to_f16x2(scales[row * (D / 16) + l / 2])).x, g);
    float f[8];
    unpack_e2m1x8(c, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] *= d;
    return pack_bf16x8(f);
  }
}

template <int KIND, int D>
__global__ void __launch_bounds__(KR_THREADS) kv_read_kernel(const KvReadArgs a) {
  __shared__ int64_t place[KR_ROWS];  // row of head 0 in the pools, -1: not read
  pdl_trigger();
  pdl_wait();
  const int64_t r0 = (int64_t)blockIdx.x * KR_ROWS;
  const int H = a.kv.heads;
  if (threadIdx.x < KR_ROWS) {
    const int64_t r = r0 + threadIdx.x;
    int64_t at = -1;
    if (r < a.total && r >= a.starts[0] && r < a.starts[a.B]) {
      int64_t lo = 0, hi = a.B;  // starts[lo] <= r < starts[hi]
      while (hi - lo > 1) {
        const int64_t mid = (lo + hi) >> 1;
        if (a.starts[mid] <= r) lo = mid;
        else hi = mid;
      }
      const int64_t i = r - a.starts[lo] + (a.first ? a.first[lo] : 0);
      const int64_t col = i >= 0 ? i / a.kv.page_size : -1;
      int64_t page = -1;
      if (col >= 0 && col < a.table_stride) page = a.page_table[lo * a.table_stride + col];
      if (page >= 0 && page < a.kv.num_pages) at = page * H * a.kv.page_size + (i - col * a.kv.page_size);
      else kv_report(a.status);
    }
    if (blockIdx.x == 0 && threadIdx.x == 0 && a.starts[a.B] > a.total) kv_report(a.status);
    place[threadIdx.x] = at;
  }
  float kg = 1.0f, vg = 1.0f;
  if constexpr (KIND == HQ_KV_NVFP4) kg = *a.kv.k_global, vg = *a.kv.v_global;
  __syncthreads();
  constexpr int LPH = D / 8;
  for (int i = threadIdx.x; i < KR_ROWS * H * LPH; i += KR_THREADS) {
    const int l = i % LPH, r = i / LPH % KR_ROWS, h = i / (LPH * KR_ROWS);
    if (place[r] < 0) continue;
    const int64_t row = place[r] + (int64_t)h * a.kv.page_size;
    const int64_t to = ((r0 + r) * H + h) * LPH + l;
    const uint4 k = read8<KIND, D>(a.kv.k, a.kv.k_scale, kg, row, l);
    const uint4 v = read8<KIND, D>(a.kv.v, a.kv.v_scale, vg, row, l);
    __stcs(reinterpret_cast<uint4*>(a.k_out) + to, k);
    __stcs(reinterpret_cast<uint4*>(a.v_out) + to, v);
  }
}

template <int KIND>
cudaError_t by_dim(int dim, const KvReadArgs& a, cudaStream_t stream) {
  const dim3 grid((unsigned)((a.total + KR_ROWS - 1) / KR_ROWS)), block(KR_THREADS);
  return dim == 64 ? launch_kernel(kv_read_kernel<KIND, 64>, grid, block, 0, stream, a)
                   : (dim == 128 ? launch_kernel(kv_read_kernel<KIND, 128>, grid, block, 0, stream, a)
                                 : launch_kernel(kv_read_kernel<KIND, 256>, grid, block, 0, stream, a));
}

}  // namespace

cudaError_t launch_kv_read(int kind, int dim, const KvReadArgs& a, cudaStream_t stream) {
  return kind == HQ_KV_BF16 ? by_dim<HQ_KV_BF16>(dim, a, stream)
                            : (kind == HQ_KV_E4M3 ? by_dim<HQ_KV_E4M3>(dim, a, stream)
                                                  : by_dim<HQ_KV_NVFP4>(dim, a, stream));
}

}  // namespace hq
