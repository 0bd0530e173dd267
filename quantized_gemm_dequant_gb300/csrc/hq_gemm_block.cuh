// e4m3 x e4m3 products with fp32 scales per block of 128 (dense), for sm_103a:
//   C[m, n] = bias[n] + sum_b a_scale[m, b] * w_scale[n / 128, b] * sum_{k in block b} a[m, k] * w[n, k]
//
// The MMA's own block scales are powers of two per 32 elements, so fp32 scales per 128 cannot ride on it: every 128-K
// block is multiplied into an accumulator of its own in tensor memory (four tcgen05.mma kind::f8f6f4 steps of 32 K),
// and warps add it, times its scale, to fp32 sums in registers ("promotion") while the MMA fills the next slot.
#pragma once
#include "hq_gemm_kernel.cuh"

namespace hq {

// Instruction descriptor for kind::f8f6f4 (e4m3 x e4m3 -> fp32, both operands K-major).
__host__ __device__ constexpr uint32_t idesc_e4m3(uint32_t M, uint32_t N) {
  return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
// D[tmem] (+)= A[smem desc] * B[smem desc]^T, K = 32 per instruction
__device__ __forceinline__ void umma_e4m3_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// ------------------------------------------------------------------ clusters
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// shared::cluster address of a shared::cta address in the CTA of cluster rank `rank`
__device__ __forceinline__ uint32_t cluster_addr(uint32_t saddr, uint32_t rank) {
  uint32_t d;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(saddr), "r"(rank));
  return d;
}
__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// ------------------------------------------------------------------ few tokens
// Weights are the MMA's A operand (128 output features, one per tensor-memory lane) and BT tokens its B operand, so
// that a step of one token still fills the MMA's rows.  A tile is 128 features by BT tokens; its K blocks are split
// over the CTAs of a cluster (up to 8), which read each other's fp32 sums from shared memory and add them in rank
// order: one kernel, no workspace, and the result does not depend on timing.
//
// Bound by the weights' bytes: every CTA keeps a ring of 16 KB weight blocks in flight.
template <int BT>
struct BlkCfg {
  static constexpr int STAGE = 16384 + BT * 128;  // weight block, token rows x 128 bytes
  static constexpr int PER_SM = BT <= 64 ? 2 : 1;
  static constexpr int STAGES = BT == 16 ? 6 : (BT == 32 ? 5 : (BT == 64 ? 4 : 6));
  static constexpr int SLOTS = 4;                 // accumulators in tensor memory
  static constexpr int COLS = SLOTS * BT;         // 64 .. 512: two CTAs of up to 64 tokens share an SM's 512 columns
  static constexpr int KC = 8;                    // K blocks per chunk of scales
  static constexpr int RING = STAGES * STAGE;
  static constexpr int SCALES = 2 * KC * BT * 4;
  static constexpr int SMEM = RING + SCALES + 1024 /*align*/ + 512 /*barriers*/;
  static_assert(RING >= BT * TILE_N * 4, "the sums overlay the ring");
  // at most PER_SM CTAs on an SM, so that their tensor memory always fits and no CTA of a cluster waits for columns
  // that another cluster's CTA holds
  static_assert((PER_SM + 1) * (SMEM + 1024) > 228 * 1024 && PER_SM * (SMEM + 1024) <= 228 * 1024, "CTAs per SM");
};
constexpr int BLK_THREADS = 320;
constexpr int BLK_LOAD_WARP = 8, BLK_MMA_WARP = 9;

template <int BT>
struct BlkSmem {
  using C = BlkCfg<BT>;
  uint64_t full[C::STAGES], empty[C::STAGES], dfull[C::SLOTS], dempty[C::SLOTS], drain;
  uint32_t tmem_base;
  int abort_flag;
};

template <int BT>
__global__ void __launch_bounds__(BLK_THREADS, BlkCfg<BT>::PER_SM)
    gemm_block_kernel(const __grid_constant__ GemmArgs args) {
  using C = BlkCfg<BT>;
  static_assert(sizeof(BlkSmem<BT>) <= 512, "shared state");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* scales = reinterpret_cast<float*>(smem + C::RING);  // [2][KC][BT]
  BlkSmem<BT>& sh = *reinterpret_cast<BlkSmem<BT>*>(smem + C::RING + C::SCALES);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int split = args.sk;
  const int rank = (int)(blockIdx.x % (unsigned)split), tile = (int)(blockIdx.x / (unsigned)split);
  const int nt = tile / args.m_tiles, m0 = (tile - nt * args.m_tiles) * BT;  // neighbours share a weight tile
  const int g0 = (int)((int64_t)rank * args.kst / split), nblk = (int)((int64_t)(rank + 1) * args.kst / split) - g0;
  const uint8_t* wblk = args.w + ((int64_t)nt * args.kst + g0) * 16384;
  volatile int* abort_flag = &sh.abort_flag;

  if (warp == 0) {
    tmem_alloc(&sh.tmem_base, C::COLS);
    tmem_relinquish();
  }
  auto load_w = [&](int s, int i) {
    mbar_arrive_expect_tx(&sh.full[s], C::STAGE);
    if (args.w_evict_first)
      bulk_g2s_hint(smem + s * C::STAGE, wblk + (int64_t)i * 16384, 16384, &sh.full[s], l2_evict_first_policy());
    else
      bulk_g2s(smem + s * C::STAGE, wblk + (int64_t)i * 16384, 16384, &sh.full[s]);
  };
  const int npre = nblk < C::STAGES ? nblk : C::STAGES;
  if (tid == BLK_LOAD_WARP * 32) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], 1);
    }
    for (int d = 0; d < C::SLOTS; ++d) {
      mbar_init(&sh.dfull[d], 1);
      mbar_init(&sh.dempty[d], 8);
    }
    mbar_init(&sh.drain, 1);
    sh.abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&args.tmap_a);
    for (int i = 0; i < npre; ++i) load_w(i, i);  // packed weights may be read before the grid dependency wait
  }
  pdl_trigger();
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;
  bool ok = true;
  auto waitf = [&](uint64_t* bar, uint32_t par) {
    if (ok && !mbar_wait(bar, par, abort_flag, args.wait_ns)) {
      *abort_flag = 1;
      atomicCAS(args.status, 0, ERR_TIMEOUT);
      ok = false;
    }
    return ok;
  };

  constexpr int HC = BT / 2;
  float acc[HC];
#pragma unroll
  for (int j = 0; j < HC; ++j) acc[j] = 0.0f;

  if (warp == BLK_LOAD_WARP) {
    if (lane == 0) {
      int s = 0, n = 0;
      uint32_t ph = 0;
      for (; n < nblk; ++n) {
        if (n >= npre) {
          if (!waitf(&sh.empty[s], ph ^ 1)) break;
          load_w(s, n);
        }
        tma_load_2d(smem + s * C::STAGE + 16384, &args.tmap_a, (g0 + n) * 128, m0, &sh.full[s]);
        if (++s == C::STAGES) {
          s = 0;
          ph ^= 1;
        }
      }
      // every copy lands before shared memory is used otherwise or released (the latest fill of each stage)
      int never = 0;
      for (int k = 0; k < C::STAGES; ++k)
        if (n > k) mbar_wait(&sh.full[k], (uint32_t)(((n - 1 - k) / C::STAGES) & 1), &never, DRAIN_WAIT_NS);
    }
  } else if (warp == BLK_MMA_WARP) {
    if (lane == 0) {
      int s = 0, d = 0;
      uint32_t ph = 0, dph = 0;
      for (int i = 0; i < nblk; ++i) {
        if (!waitf(&sh.dempty[d], dph ^ 1) || !waitf(&sh.full[s], ph)) break;
        tc_fence_after();
        const uint32_t w = smem_u32(smem + s * C::STAGE), a = w + 16384;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          umma_e4m3_ss(tmem + d * BT, smem_desc(w + 32 * k, 16, 1024, 2), smem_desc(a + 32 * k, 16, 1024, 2),
                       idesc_e4m3(128, BT), k > 0);
        umma_commit(&sh.empty[s]);
        umma_commit(&sh.dfull[d]);
        if (++s == C::STAGES) {
          s = 0;
          ph ^= 1;
        }
        if (++d == C::SLOTS) {
          d = 0;
          dph ^= 1;
        }
      }
      int never = 0;  // every MMA completes before tensor memory is released
      umma_commit(&sh.drain);
      mbar_wait(&sh.drain, 0, &never, DRAIN_WAIT_NS);
    }
  } else {
    // ------------------------------------------------ promotion: warp -> lane quarter warp % 4, column half warp / 4
    const int h = warp >> 2;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    // a chunk's scales a_scale * w_scale, [KC][BT]: loaded a chunk ahead, in shared memory for the chunk's columns
    constexpr int PER = (C::KC * BT + 255) / 256;
    float next[PER];
    auto load_scales = [&](int i0) {
#pragma unroll
      for (int u = 0; u < PER; ++u) {
        const int idx = tid + 256 * u, i = i0 + (idx & (C::KC - 1)), m = m0 + idx / C::KC;
        next[u] = (idx < C::KC * BT && i < nblk && m < args.M)
                      ? args.a_scale[(int64_t)m * args.kst + g0 + i] * args.w_gscale[(int64_t)nt * args.kst + g0 + i]
                      : 0.0f;
      }
    };
    load_scales(0);
    int d = 0;
    uint32_t dph = 0;
    for (int i0 = 0; i0 < nblk; i0 += C::KC) {
      float* sc = scales + ((i0 / C::KC) & 1) * (C::KC * BT);
#pragma unroll
      for (int u = 0; u < PER; ++u) {
        const int idx = tid + 256 * u;
        if (idx < C::KC * BT) sc[(idx & (C::KC - 1)) * BT + idx / C::KC] = next[u];
      }
      named_bar_sync(1, 256);  // every warp comes here once a chunk, also after a wait has run out
      load_scales(i0 + C::KC);
      const int n = nblk - i0 < C::KC ? nblk - i0 : C::KC;
      for (int i = 0; i < n; ++i) {
        if (waitf(&sh.dfull[d], dph)) {
          tc_fence_after();
          uint32_t v[HC];
#pragma unroll
          for (int j = 0; j < HC; j += 16) {
            if (HC < 16) tmem_ld8(tmem + lane_base + d * BT + h * HC, *reinterpret_cast<uint32_t(*)[8]>(v));
            else tmem_ld16(tmem + lane_base + d * BT + h * HC + j, *reinterpret_cast<uint32_t(*)[16]>(v + j));
          }
          tmem_wait_ld();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.dempty[d]);
          const float* f = sc + i * BT + h * HC;
#pragma unroll
          for (int j = 0; j < HC; j += 4) {
            const float4 s = *reinterpret_cast<const float4*>(f + j);
            acc[j] = fmaf(__uint_as_float(v[j]), s.x, acc[j]);
            acc[j + 1] = fmaf(__uint_as_float(v[j + 1]), s.y, acc[j + 1]);
            acc[j + 2] = fmaf(__uint_as_float(v[j + 2]), s.z, acc[j + 2]);
            acc[j + 3] = fmaf(__uint_as_float(v[j + 3]), s.w, acc[j + 3]);
          }
        }
        if (++d == C::SLOTS) {
          d = 0;
          dph ^= 1;
        }
      }
    }
  }

  // ------------------------------------------------ sums -> shared memory -> output rows
  __syncthreads();  // every copy has landed and every MMA has read its stage
  float* red = reinterpret_cast<float*>(smem);  // [BT][128]
  if (warp < 8) {
    const int r = (warp & 3) * 32 + lane;
#pragma unroll
    for (int j = 0; j < HC; ++j) red[((warp >> 2) * HC + j) * TILE_N + r] = acc[j];
  }
  if (split > 1) cluster_sync();
  else __syncthreads();
  const int nrows = args.M - m0 < BT ? args.M - m0 : BT;
  if (warp < 8) {
    const int n = nt * TILE_N + lane * 4;
    float b[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) b[k] = (args.bias && n + k < args.N) ? bf16_to_f32(args.bias[n + k]) : 0.0f;
    const bool wide = (args.N & 3) == 0 && (reinterpret_cast<uintptr_t>(args.c) & 7) == 0;
    for (int t = warp * split + rank; t < nrows; t += 8 * split) {
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      const uint32_t at = smem_u32(red + t * TILE_N + lane * 4);
      for (int k = 0; k < split; ++k) {
        const float4 p = split > 1 ? ld_cluster_f32x4(cluster_addr(at, (uint32_t)k))
                                   : *reinterpret_cast<const float4*>(red + t * TILE_N + lane * 4);
        v = make_float4(v.x + p.x, v.y + p.y, v.z + p.z, v.w + p.w);
      }
      int row = m0 + t;
#if HQ_DEBUG_BOUNDS
      row = dbg_row(row, args.dbg_c_rows, args.status);
      if (row < 0) continue;
#endif
      uint16_t* o = args.c + (int64_t)row * args.N + n;
      const float y[4] = {v.x + b[0], v.y + b[1], v.z + b[2], v.w + b[3]};
      if (wide && n < args.N) {
        *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (n + k < args.N) o[k] = f32_to_bf16(y[k]);
      }
    }
  }
  if (split > 1) cluster_sync();  // the sums stay until every CTA of the cluster has read them
  else __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, C::COLS);
  }
}

// `cluster` CTAs of consecutive index form a cluster.
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster_kernel(void (*kernel)(KArgs...), int grid, int cluster, int threads, int smem,
                                  cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace hq
