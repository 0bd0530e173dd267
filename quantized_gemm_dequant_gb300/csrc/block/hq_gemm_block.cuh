// e4m3 x e4m3 products with fp32 scales per block of 128 (dense), for sm_103a:
//   C[m, n] = bias[n] + sum_b a_scale[m, b] * w_scale[n / 128, b] * sum_{k in block b} a[m, k] * w[n, k]
//
// The MMA's own block scales are powers of two per 32 elements, so fp32 scales per 128 cannot ride on it: every 128-K
// block is multiplied into an accumulator of its own in tensor memory (four tcgen05.mma kind::f8f6f4 steps of 32 K),
// and warps add it, times its scale, to fp32 sums in registers ("promotion") while the MMA fills the next slot.
#pragma once
#include "../hq_gemm_kernel.cuh"

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

// mbar_wait for waits that are short and on the critical path of every K block: its tests suspend the thread only as
// long as the hardware sees fit.  (With a time hint they become sleeps, whose end comes hundreds of cycles late.)
__device__ __forceinline__ bool mbar_wait_soon(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long c0 = clock64(), lim = 3ll * (long long)limit_ns;  // at least limit_ns at clocks up to 3 GHz
  for (;;) {
    if (clock64() - c0 >= lim || *abort) return false;
    if (mbar_try_wait(bar, parity)) return true;
  }
}
// The same where a limit below a microsecond runs out at a phase that is not complete at once: a kernel needs one such
// wait to end early, the others then see the abort flag.  (In every wait the choice cost 8192 tokens 350 -> 370 us.)
__device__ __forceinline__ bool mbar_wait_strict(uint64_t* bar, uint32_t parity, volatile int* abort,
                                                 uint64_t limit_ns) {
  if (mbar_test_wait(bar, parity)) return true;
  if (limit_ns >= 1000) return mbar_wait_soon(bar, parity, abort, limit_ns);
  const long long c0 = clock64(), lim = 3ll * (long long)limit_ns;
  while (clock64() - c0 < lim && !*abort)
    if (mbar_test_wait(bar, parity)) return true;
  return false;
}

// The whole warp's wait (every lane calls it): each test is put to the vote, so that the lanes stay together.
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const long long c0 = clock64(), lim = 3ll * (long long)limit_ns;
  for (;;) {
    if (__any_sync(0xffffffffu, clock64() - c0 >= lim || *abort)) return false;
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  }
}

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

// ------------------------------------------------------------------ clusters
// The lanes of a warp leave a wait, or a branch of one lane, one by one; barriers and tensor-memory instructions are the
// whole warp's.  Between every such wait or branch and the next of those stands a __syncwarp(), or the wait is one that
// the lanes leave together (mbar_wait_warp's votes): a warp that comes to them in parts is undefined behaviour.
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cta_sync() {
  __syncwarp();
  __syncthreads();
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
// A tile is 128 output features by BT tokens; its K blocks are split over the CTAs of a cluster (up to 8), which read
// each other's fp32 sums from shared memory and add them in rank order: one kernel, no workspace, and the result does
// not depend on timing.
//
// Up to 32 tokens the weights are the MMA's A operand (a feature per tensor-memory lane) and the tokens its B operand,
// so that a step of one token still fills the MMA's rows; a column's scale is then its token's, read from shared memory
// by every warp (128 bytes into the registers for each column).  From 64 tokens on that read takes longer than the rest,
// and the tokens are the A operand: a lane is a token and its scale one register (128 tokens, N = 14336, K = 4096: 19.5
// to 14.8 us).  The A operand of 64 tokens is still 128 rows: the MMA reads what follows them in shared memory, whatever
// it is, into sums that nothing reads.
//
// Bound by the weights' bytes: every CTA keeps a ring of 16 KB weight blocks in flight, and two warps issue the MMAs of
// every second block each (waits and issue take a warp some 500 cycles a block, as long as its bytes take to arrive).
template <int BT>
struct BlkCfg {
  static constexpr bool LANES = BT >= 64;         // tokens on the lanes
  static constexpr int STAGE = 16384 + BT * 128;  // weight block, token rows x 128 bytes
  static constexpr int PER_SM = LANES ? 1 : 2;
  static constexpr int STAGES = BT == 16 ? 6 : (BT == 32 ? 4 : (BT == 64 ? 8 : 6));
  static constexpr int SLOTS = 4;                    // accumulators in tensor memory
  static constexpr int WIDTH = LANES ? TILE_N : BT;  // columns of one
  static constexpr int COLS = SLOTS * WIDTH;         // 64, 128 (two CTAs share an SM's 512 columns), or all 512
  static constexpr int HC = WIDTH / 2;               // columns of a promoting warp
  static constexpr int ACTIVE = LANES ? BT / 16 : 8;  // promoting warps
  static constexpr int KC = 8;                       // K blocks per chunk of scales
  static constexpr int PITCH = LANES ? TILE_N + 4 : TILE_N;  // floats of a token's sums in shared memory
  static constexpr int RING = STAGES * STAGE;
  static constexpr int SCALES = 2 * KC * BT * 4;
  static constexpr int TAIL = SCALES + 512 /*barriers*/;
  // behind the ring there is as much as the MMA reads past the last stage's 64 tokens
  static constexpr int SMEM = RING + (BT == 64 && TAIL < 8192 ? 8192 : TAIL) + 1024 /*align*/;
  static_assert(RING >= BT * PITCH * 4, "the sums overlay the ring");
  // at most PER_SM CTAs on an SM, so that their tensor memory always fits and no CTA of a cluster waits for columns
  // that another cluster's CTA holds
  static_assert((PER_SM + 1) * (SMEM + 1024) > 228 * 1024 && PER_SM * (SMEM + 1024) <= 228 * 1024, "CTAs per SM");
};
constexpr int BLK_THREADS = 352;
constexpr int BLK_LOAD_WARP = 8, BLK_MMA_WARP = 9;  // 9 and 10 issue the MMAs

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
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // the same in all lanes, as the compiler sees it
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
      mbar_init(&sh.dempty[d], C::ACTIVE);
    }
    mbar_init(&sh.drain, 2);
    sh.abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&args.tmap_a);
    for (int i = 0; i < npre; ++i) load_w(i, i);  // packed weights may be read before the grid dependency wait
  }
  pdl_trigger();
  pdl_wait();
  tc_fence_before();
  cta_sync();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;
  bool ok = true;
  auto timed_out = [&] {
    *abort_flag = 1;
    atomicCAS(args.status, 0, ERR_TIMEOUT);
    ok = false;
  };
  auto waitf = [&](uint64_t* bar, uint32_t par) {
    if (ok && !mbar_wait_soon(bar, par, abort_flag, args.wait_ns)) timed_out();
    return ok;
  };

  constexpr int HC = C::HC;
  float2 acc[HC / 2];
#pragma unroll
  for (int j = 0; j < HC / 2; ++j) acc[j] = make_float2(0.0f, 0.0f);

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
  } else if (warp >= BLK_MMA_WARP) {
    // (the whole warp runs the loop, so that descriptors and addresses are uniform registers; one lane issues)
    const bool one = elect_one();
    const uint32_t ring = smem_u32(smem);
    int s = warp - BLK_MMA_WARP, d = warp - BLK_MMA_WARP;
    uint32_t ph = 0, dph = 0;
    // A parity wait tells a barrier's next phase from the one before the last only by what its waiter knows: a warp
    // that took a stage's every second fill could pass on the fill before (copies end out of order).  So the numbers are
    // even, a stage and a slot belong to one warp, which waits for each of their phases in turn.
    static_assert(C::STAGES % 2 == 0 && C::SLOTS % 2 == 0, "a stage and a slot belong to one issuing warp");
    for (int i = warp - BLK_MMA_WARP; i < nblk; i += 2) {
      if (waitf(&sh.dempty[d], dph ^ 1) && !mbar_wait_strict(&sh.full[s], ph, abort_flag, args.wait_ns)) timed_out();
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const uint64_t w = smem_desc(ring + s * C::STAGE, 16, 1024, 2),
                     a = smem_desc(ring + s * C::STAGE + 16384, 16, 1024, 2);
      if (one) {
#pragma unroll
        for (int k = 0; k < 4; ++k)  // 32 bytes further on: the address field counts 16s
          umma_e4m3_ss(tmem + d * C::WIDTH, (C::LANES ? a : w) + 2 * k, (C::LANES ? w : a) + 2 * k,
                       idesc_e4m3(128, C::WIDTH), k > 0);
        umma_commit(&sh.empty[s]);
        umma_commit(&sh.dfull[d]);
      }
      s += 2;
      if (s >= C::STAGES) {
        s -= C::STAGES;
        ph ^= 1;
      }
      d += 2;
      if (d >= C::SLOTS) {
        d -= C::SLOTS;
        dph ^= 1;
      }
    }
    int never = 0;  // every MMA completes before tensor memory is released
    if (one) umma_commit(&sh.drain);
    mbar_wait(&sh.drain, 0, &never, DRAIN_WAIT_NS);
  } else {
    // ------------------------------------------------ promotion: warp -> lane quarter warp % 4, column half warp / 4
    const int h = warp >> 2;
    const bool active = !C::LANES || (warp & 3) * 32 < BT;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    // a chunk's scales a_scale * w_scale, [KC][BT]: loaded a chunk ahead, multiplied on their way to shared memory
    constexpr int PER = (C::KC * BT + 255) / 256;
    const int kb = tid & (C::KC - 1);  // a thread's K block of a chunk
    float na[PER], nw;
    auto load_scales = [&](int i0) {
      const int i = i0 + kb;
      nw = i < nblk ? args.w_gscale[(int64_t)nt * args.kst + g0 + i] : 0.0f;
#pragma unroll
      for (int u = 0; u < PER; ++u) {
        const int idx = tid + 256 * u, m = m0 + idx / C::KC;
        na[u] = (idx < C::KC * BT && i < nblk && m < args.M) ? args.a_scale[(int64_t)m * args.kst + g0 + i] : 0.0f;
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
        if (idx < C::KC * BT) sc[kb * BT + idx / C::KC] = na[u] * nw;
      }
      __syncwarp();
      named_bar_sync(1, 256);  // every warp comes here once a chunk, also after a wait has run out
      load_scales(i0 + C::KC);
      const int n = !active ? 0 : (nblk - i0 < C::KC ? nblk - i0 : C::KC);
      for (int i = 0; i < n; ++i) {
        // (after a wait that has run out the sums are of no use, but nothing is out of place)
        if (ok && !mbar_wait_warp(&sh.dfull[d], dph, abort_flag, args.wait_ns)) timed_out();
        tc_fence_after();
        uint32_t v[HC];
        const uint32_t from = tmem + lane_base + d * C::WIDTH + h * HC;
        if (HC == 8) tmem_ld8(from, *reinterpret_cast<uint32_t(*)[8]>(v));
        if (HC == 16) tmem_ld16(from, *reinterpret_cast<uint32_t(*)[16]>(v));
        if (HC >= 32) tmem_ld32(from, *reinterpret_cast<uint32_t(*)[32]>(v));
        if (HC == 64) tmem_ld32(from + 32, *reinterpret_cast<uint32_t(*)[32]>(v + HC - 32));
        tmem_wait_ld();
        tc_fence_before();
        mbar_arrive_if(&sh.dempty[d], lane == 0);  // (the wait above is the whole warp's)
        const float* f = sc + i * BT + (C::LANES ? (warp & 3) * 32 + lane : h * HC);
        const float own = *f;
#pragma unroll
        for (int j = 0; j < HC; j += 4) {
          const float4 s = C::LANES ? make_float4(own, own, own, own) : *reinterpret_cast<const float4*>(f + j);
          acc[j / 2] = __ffma2_rn(make_float2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), make_float2(s.x, s.y),
                                  acc[j / 2]);
          acc[j / 2 + 1] = __ffma2_rn(make_float2(__uint_as_float(v[j + 2]), __uint_as_float(v[j + 3])),
                                      make_float2(s.z, s.w), acc[j / 2 + 1]);
        }
        if (++d == C::SLOTS) {
          d = 0;
          dph ^= 1;
        }
      }
    }
  }

  // ------------------------------------------------ sums -> shared memory -> output rows
  cta_sync();  // every copy has landed and every MMA has read its stage
  float* red = reinterpret_cast<float*>(smem);  // [BT][PITCH]
  if (warp < 8 && (!C::LANES || (warp & 3) * 32 < BT)) {
    const int r = (warp & 3) * 32 + lane;
    if (C::LANES) {
#pragma unroll
      for (int j = 0; j < HC; j += 4)
        *reinterpret_cast<float4*>(red + r * C::PITCH + (warp >> 2) * HC + j) =
            make_float4(acc[j / 2].x, acc[j / 2].y, acc[j / 2 + 1].x, acc[j / 2 + 1].y);
    } else {
#pragma unroll
      for (int j = 0; j < HC; ++j) red[((warp >> 2) * HC + j) * C::PITCH + r] = j & 1 ? acc[j / 2].y : acc[j / 2].x;
    }
  }
  if (split > 1) cluster_sync();
  else cta_sync();
  const int nrows = args.M - m0 < BT ? args.M - m0 : BT;
  if (warp < 8) {
    const int n = nt * TILE_N + lane * 4;
    float b[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) b[k] = (args.bias && n + k < args.N) ? bf16_to_f32(args.bias[n + k]) : 0.0f;
    const bool wide = (args.N & 3) == 0 && (reinterpret_cast<uintptr_t>(args.c) & 7) == 0;
    for (int t = warp * split + rank; t < nrows; t += 8 * split) {
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      const uint32_t at = smem_u32(red + t * C::PITCH + lane * 4);
      for (int k = 0; k < split; ++k) {
        const float4 p = split > 1 ? ld_cluster_f32x4(cluster_addr(at, (uint32_t)k))
                                   : *reinterpret_cast<const float4*>(red + t * C::PITCH + lane * 4);
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
  else cta_sync();
  if (warp == 0) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::COLS);
  }
}

// ------------------------------------------------------------------ many tokens
// Two CTAs of a cluster share one MMA (cta_group::2): a tile is 256 tokens, the MMA's A operand, by BN features, its B
// operand.  Each CTA loads its own 128 tokens and half of the tile's weight rows, so that both operands are read from
// L2 and written to shared memory once per pair, and holds its tokens' sums: a token is a tensor-memory lane, so a
// thread's sums share one token scale and (128 columns) one weight scale, and a K block costs a thread one scale and
// an FMA per sum.  Two FMAs go in one instruction.
//
// A K block of a 256 x 256 tile keeps the tensor pipe busy for 650 cycles, and the promotion of its 128 x 256 sums per
// CTA by eight warps takes 256 cycles of the FMA pipes and as many of tensor-memory reads, under the next block's MMAs.
// Measured: 8192 tokens, 14336 x 4096, 385 us = 2.5 PFLOP/s (355 to 400 from run to run: a long call draws the card's
// full power); one wave of tiles, 2048 x 2048 x 16384, 55 us = 820 cycles a K block.  With the additions left out that
// takes 45 us, at the MMA's pace; with a quarter of the MMAs and neither reads nor additions 41, which is what copies,
// barriers and hand-overs between the CTAs cost by themselves.  What is left over the MMA is the circle of a slot: filled,
// announced to both CTAs, read, given back.  Tried for it: sixteen promoting warps with 64 columns each (69 us), one MMA
// and slot for 256 columns, which reads a third less shared memory but leaves two slots (59), weights copied and half
// the scales multiplied by two more warps (63), waits by one lane of a warp (70), the next slot tested and read before
// the last additions (56).
// Accumulators are handed over 128 columns at a time (four slots in tensor memory), so that half of the promoting warps
// read one half of a tile while the MMA fills the other.
template <int BN>
struct PairCfg {
  static constexpr int BROWS = BN / 2;  // weight rows a CTA loads
  static constexpr int STAGE = 16384 + BROWS * 128;
  static constexpr int STAGES = BN == 256 ? 6 : 8;
  static constexpr int SN = 128;           // features of an accumulator slot (the MMA's N): one weight tile
  static constexpr int HALVES = BN / SN;  // slots a K block fills
  static constexpr int SLOTS = 512 / SN, DEPTH = SLOTS / HALVES;
  static constexpr int HC = BN / 2;  // columns of a promoting warp
  static constexpr int TILES = BN / 128;           // weight tiles
  static constexpr int SK = 8;                     // K blocks in a group of scales
  static constexpr int SGROUP = SK * TILES * 128;  // [K block][weight tile][token]
  static constexpr int SGROUPS = 2;
  static constexpr int SCALES = SGROUPS * SGROUP * 4;
  static constexpr int OUT_PITCH = 18;  // bf16 values of a row of 16 on their way out
  static constexpr int OUT = 8 * 32 * OUT_PITCH * 2;
  static constexpr int SMEM = STAGES * STAGE + SCALES + OUT + 1024 /*align*/ + 512 /*barriers*/;
  static_assert(SMEM <= 227 * 1024, "shared memory");
};
// warps 0-7 promote, 8 loads, 9 and 10 issue the MMAs (of the cluster's first CTA), 11 multiplies the scales
constexpr int PAIR_THREADS = 384;
// registers: 168 x 384 at launch (the 256-feature kernel spills 24 bytes of them); the promoting warps raise theirs to 216,
// the others go down to 72, and 2 x 216 + 72 = 3 x 168
constexpr int PAIR_TOKENS = 256;
constexpr int PAIR_GROUP = 8;  // token tiles per round of feature tiles: the tiles in flight share operands in L2

template <int BN>
struct PairSmem {
  using C = PairCfg<BN>;
  uint64_t full[C::STAGES], empty[C::STAGES], dfull[C::SLOTS], dempty[C::SLOTS], sfull[C::SGROUPS],
      sempty[C::SGROUPS], drain;
  uint32_t tmem_base;
  int abort_flag;
};

// Token tile and feature tile of a tile index: groups of PAIR_GROUP token tiles, feature tiles inside, token tiles
// innermost.
__host__ __device__ inline void pair_tile(int t, int m_tiles, int n_tiles, int& mt, int& nt) {
  const int per = PAIR_GROUP * n_tiles, g = t / per, in = t - g * per;
  const int left = m_tiles - g * PAIR_GROUP, rows = left < PAIR_GROUP ? left : PAIR_GROUP;
  nt = in / rows;
  mt = g * PAIR_GROUP + in - nt * rows;
}

__device__ __forceinline__ void umma_e4m3_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// arrive on the barrier at this address in both CTAs once every tcgen05 operation issued so far completes
__device__ __forceinline__ void umma_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
// 2-D tensor load into this CTA whose bytes are counted on a barrier of the pair (a shared::cluster address)
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const void* tmap, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, "
      "%3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(tmap), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// Arrival on a barrier of the pair that orders nothing but itself: what it announces, the end of this warp's
// tensor-memory reads, is ordered by their wait and the tcgen05 fence before it.  (A releasing arrival at cluster scope
// waits for the thread's outstanding memory operations, some 1000 cycles a K block: 8192 tokens took 888 us with it.)
__device__ __forceinline__ void mbar_arrive_cluster_if(uint32_t bar, uint32_t on) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n\t}\n" ::"r"(bar),
      "r"(on)
      : "memory");
}
__device__ __forceinline__ void st_global_32b(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

template <int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PAIR_THREADS, 1)
    gemm_block_pair_kernel(const __grid_constant__ GemmArgs args) {
  using C = PairCfg<BN>;
  static_assert(sizeof(PairSmem<BN>) <= 512, "shared state");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* scales = reinterpret_cast<float*>(smem + C::STAGES * C::STAGE);  // [SGROUPS][SK][TILES][128]
  PairSmem<BN>& sh = *reinterpret_cast<PairSmem<BN>*>(smem + C::STAGES * C::STAGE + C::SCALES + C::OUT);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // the same in all lanes, as the compiler sees it
  const int rank = (int)(blockIdx.x & 1), pair = (int)(blockIdx.x >> 1), pairs = (int)(gridDim.x >> 1);
  const int kst = args.kst;
  const int f_tiles = BN == 256 ? (args.n_tiles + 1) / 2 : args.n_tiles;  // tiles of BN features
  const int tiles = args.m_tiles * f_tiles;
  volatile int* abort_flag = &sh.abort_flag;

  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh.tmem_base))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  if (tid == 8 * 32) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], C::HALVES);
    }
    for (int d = 0; d < C::SLOTS; ++d) {
      mbar_init(&sh.dfull[d], 1);
      mbar_init(&sh.dempty[d], 16 / C::HALVES);
    }
    for (int g = 0; g < C::SGROUPS; ++g) {
      mbar_init(&sh.sfull[g], 32);
      mbar_init(&sh.sempty[g], 8);
    }
    mbar_init(&sh.drain, 2);
    sh.abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&args.tmap_a);
    prefetch_tmap(&args.tmap_sf);
  }
  pdl_trigger();
  tc_fence_before();
  cta_sync();
  cluster_sync();  // both CTAs' barriers stand before either is signalled
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;
  bool ok = true;
  auto fail = [&] {
    *abort_flag = 1;
    atomicCAS(args.status, 0, ERR_TIMEOUT);
    ok = false;
  };

  __syncwarp();
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 8 && lane == 0) {
      // ------------------------------------------------ loads: this CTA's tokens and its half of the weight rows
      int s = 0;
      uint32_t ph = 0;
      int64_t n = 0;
      bool waited = false;
      for (int t = pair; t < tiles && ok; t += pairs) {
        int mt, ft;
        pair_tile(t, args.m_tiles, f_tiles, mt, ft);
        const int m0 = mt * PAIR_TOKENS + rank * 128;
        // first rows of this CTA's 64 of each weight tile in the packed buffer, taken as rows of 128 bytes (a weight
        // tile past the last one is loaded from the last: its columns are not stored)
        int w0[C::TILES];
#pragma unroll
        for (int h = 0; h < C::TILES; ++h) {
          const int nt = C::TILES * ft + h;
          w0[h] = (nt < args.n_tiles ? nt : args.n_tiles - 1) * kst * 128 + rank * 64;
        }
        for (int b = 0; b < kst; ++b) {
          if (!mbar_wait_strict(&sh.empty[s], ph ^ 1, abort_flag, args.wait_ns)) {
            fail();
            break;
          }
          const uint32_t bar = cluster_addr(smem_u32(&sh.full[s]), 0);
          uint8_t* dst = smem + s * C::STAGE;
          if (rank == 0) mbar_arrive_expect_tx(&sh.full[s], 2 * C::STAGE);
#pragma unroll
          for (int h = 0; h < C::TILES; ++h)
            tma_load_2d_pair(dst + 16384 + h * 8192, &args.tmap_sf, 0, w0[h] + b * 128, bar);
          if (!waited) {  // packed weights may be read before the grid dependency wait, activations not
            pdl_wait();
            waited = true;
          }
          tma_load_2d_pair(dst, &args.tmap_a, b * 128, m0, bar);
          ++n;
          if (++s == C::STAGES) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      // every copy lands before shared memory is released; the first CTA's barriers count both CTAs' bytes, and the
      // second leaves after the first
      int never = 0;
      if (rank == 0)
        for (int k = 0; k < C::STAGES; ++k)
          if (n > k) mbar_wait(&sh.full[k], (uint32_t)(((n - 1 - k) / C::STAGES) & 1), &never, DRAIN_WAIT_NS);
      if (!ok)
        for (const long long c0 = clock64(); clock64() - c0 < 10000000ll;) {}  // copies that no barrier counts any more
    } else if ((warp == 9 || warp == 10) && rank == 0) {
      // ------------------------------------------------ MMAs of the pair: two warps take a tile's slots in turn (waits
      // and issue take a warp some 250 cycles a slot), each as a whole, so that descriptors and addresses are uniform
      // registers; one lane issues
      const bool one = elect_one();
      const int w = warp - 9;
      uint32_t dph = 0;  // a bit per accumulator slot
      uint32_t base = 0;  // stages of the tiles before
      auto waitf = [&](uint64_t* bar, uint32_t par) {
        if (ok && !mbar_wait_warp(bar, par, abort_flag, args.wait_ns)) fail();
        return ok;
      };
      const uint32_t ring = smem_u32(smem);
      const int h = C::HALVES == 2 ? w : 0;
      constexpr int STEP = C::HALVES == 2 ? 1 : 2;
      const int b1 = C::HALVES == 2 ? 0 : w;  // the first K block of a tile that this warp takes
      if (pair < tiles && b1 < kst &&
          !__all_sync(0xffffffffu, mbar_wait_strict(&sh.full[b1], 0, abort_flag, args.wait_ns)))
        fail();
      for (int t = pair; t < tiles && ok; t += pairs) {
        int s = (int)((base + b1) % C::STAGES);
        uint32_t ph = ((base + b1) / C::STAGES) & 1;
        for (int b = b1; b < kst; b += STEP) {
          const int d = (b & (C::DEPTH - 1)) * C::HALVES + h;  // a tile begins with the first slots
          // The slot first: tiles of 128 features with an odd number of K blocks give a stage to either warp, and that
          // its last fill but one is over, without which a parity wait could pass on it, follows from the slot (block
          // i - 7 or a later one has been promoted, in order, and i - 8 with it).
          if (!waitf(&sh.dempty[d], ~(dph >> d) & 1) || !waitf(&sh.full[s], ph)) break;
          dph ^= 1u << d;
          tc_fence_after();
          const uint64_t x = smem_desc(ring + s * C::STAGE, 16, 1024, 2),
                         y = smem_desc(ring + s * C::STAGE + 16384 + h * 8192, 16, 1024, 2);
          if (one) {
#pragma unroll
            for (int k = 0; k < 4; ++k)  // 32 bytes further on: the address field counts 16s
              umma_e4m3_pair(tmem + d * C::SN, x + 2 * k, y + 2 * k, idesc_e4m3(256, C::SN), k > 0);
            umma_commit_pair(&sh.dfull[d]);
            umma_commit_pair(&sh.empty[s]);
          }
          s += STEP;
          if (s >= C::STAGES) {
            s -= C::STAGES;
            ph ^= 1;
          }
        }
        base += (uint32_t)kst;
      }
      int never = 0;  // every MMA completes before tensor memory is released
      if (one) umma_commit_pair(&sh.drain);
      mbar_wait(&sh.drain, 0, &never, DRAIN_WAIT_NS);
    } else if (warp == 11) {
      // ------------------------------------------------ scales: token scale times weight scale of a group of K blocks,
      // four tokens a thread
      pdl_wait();
      const int r = lane;
      const bool quad = (kst & 3) == 0;
      int g = 0;
      uint32_t ph = 0;
      for (int t = pair; t < tiles && ok; t += pairs) {
        int mt, ft;
        pair_tile(t, args.m_tiles, f_tiles, mt, ft);
        for (int b0 = 0; b0 < kst; b0 += C::SK) {
          if (!mbar_wait_warp(&sh.sempty[g], ph ^ 1, abort_flag, args.wait_ns)) {
            fail();
            break;
          }
          const int end = b0 + C::SK < kst ? b0 + C::SK : kst;
          float* o = scales + g * C::SGROUP + r;
          for (int b = b0; b < end; b += 4) {
            float a[4][4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int m = mt * PAIR_TOKENS + rank * 128 + r + 32 * u;
              const float* p = args.a_scale + (int64_t)m * kst + b;
              if (m < args.M && quad) {
                *reinterpret_cast<float4*>(a[u]) = *reinterpret_cast<const float4*>(p);
              } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) a[u][i] = m < args.M && b + i < kst ? p[i] : 0.0f;
              }
            }
#pragma unroll
            for (int h = 0; h < C::TILES; ++h) {
              const int nt = C::TILES * ft + h < args.n_tiles ? C::TILES * ft + h : args.n_tiles - 1;
              const float* p = args.w_gscale + (int64_t)nt * kst + b;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float w = b + i < kst ? p[i] : 0.0f;
#pragma unroll
                for (int u = 0; u < 4; ++u) o[(i * C::TILES + h) * 128 + 32 * u] = a[u][i] * w;
              }
            }
            o += 4 * C::TILES * 128;
          }
          mbar_arrive(&sh.sfull[g]);
          if (++g == C::SGROUPS) {
            g = 0;
            ph ^= 1;
          }
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    // ------------------------------------------------ promotion: warp -> 32 tokens warp % 4, column half warp / 4
    pdl_wait();
    const int h = warp >> 2;
    // K block b of a tile lies in slot b % DEPTH (of this warp's half, where a slot holds half a tile)
    const uint32_t src = tmem + ((uint32_t)((warp & 3) * 32) << 16) + h * (C::HALVES == 2 ? C::SN : C::HC);
    const uint32_t dempty = cluster_addr(smem_u32(&sh.dempty[C::HALVES == 2 ? h : 0]), 0);
    uint64_t* dfull = &sh.dfull[C::HALVES == 2 ? h : 0];
    constexpr int CHUNKS = C::HC / 32;  // 4 or 2
    constexpr int UNROLL = 8;           // K blocks; divides a group
    uint32_t dph = 0;  // a bit per slot
    const float* sc = scales + (BN == 256 ? h * 128 : 0) + (warp & 3) * 32 + lane;
    int g = 0;
    uint32_t gph = 0;
    // two buffers of 32 columns: a slot is given back when its last columns are read, before they are added
    uint32_t v[2][32];
    // the slot's sums are there: the first of them are on their way
    auto open = [&](int d) {
      if (!mbar_wait_warp(dfull + d * C::HALVES, (dph >> d) & 1, abort_flag, args.wait_ns)) fail();
      dph ^= 1u << d;
      tc_fence_after();
      tmem_ld32(src + d * (C::HALVES * C::SN), v[0]);
      tmem_ld32(src + d * (C::HALVES * C::SN) + 32, v[1]);
    };
    float f, fn = 0.0f;  // this K block's scale and the next one's
    const float* at = sc;
    auto group = [&] {
      if (!mbar_wait_warp(&sh.sfull[g], gph, abort_flag, args.wait_ns)) fail();
      at = sc + g * C::SGROUP;
      fn = *at;
    };
    group();
    for (int t = pair; t < tiles; t += pairs) {
      float2 acc[C::HC / 2];
#pragma unroll
      for (int j = 0; j < C::HC / 2; ++j) acc[j] = make_float2(0.0f, 0.0f);
      auto add = [&](const uint32_t (&x)[32], int c) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
          acc[16 * c + j] = __ffma2_rn(make_float2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])),
                                       make_float2(f, f), acc[16 * c + j]);
      };
      open(0);
      for (int b0 = 0; b0 < kst; b0 += UNROLL) {
#pragma unroll
        for (int i = 0; i < UNROLL; ++i) {
          if (b0 + i >= kst) break;
          const int d = i % C::DEPTH;
          const uint32_t from = src + d * (C::HALVES * C::SN);
          f = fn;
          tmem_wait_ld();
          if (CHUNKS == 4) {
            add(v[0], 0);
            tmem_ld32(from + 64, v[0]);
            add(v[1], 1);
            tmem_ld32(from + 96, v[1]);
            tmem_wait_ld();
          }
          tc_fence_before();
          mbar_arrive_cluster_if(dempty + 8 * C::HALVES * d, lane == 0);
          if (i + 1 < UNROLL) fn = at[(i + 1) * C::TILES * 128];
          add(v[0], CHUNKS - 2);
          add(v[1], CHUNKS - 1);
          if (b0 + i + 1 < kst) open((i + 1) % C::DEPTH);
        }
        const int next = b0 + UNROLL;
        at += UNROLL * C::TILES * 128;
        if (next % C::SK == 0 || next >= kst) {
          mbar_arrive_if(&sh.sempty[g], lane == 0);
          if (++g == C::SGROUPS) {
            g = 0;
            gph ^= 1;
          }
          if (next < kst || t + pairs < tiles) group();
        } else {
          fn = *at;
        }
      }
      if (!__all_sync(0xffffffffu, ok)) break;  // (a warp's lanes stay together: tensor-memory reads are the warp's)
      // ------------------------------------------------ output: a thread's row, HC columns of it
      int mt, ft;
      pair_tile(t, args.m_tiles, f_tiles, mt, ft);
      const int m = mt * PAIR_TOKENS + rank * 128 + (warp & 3) * 32 + lane;
      const int nt = BN == 256 ? 2 * ft + h : ft;
      int row = m < args.M && nt < args.n_tiles ? m : -1;
#if HQ_DEBUG_BOUNDS
      if (row >= 0) row = dbg_row(row, args.dbg_c_rows, args.status);
#endif
      const int n0 = BN == 256 ? nt * 128 : nt * 128 + h * C::HC;
      const bool wide = (args.N & 15) == 0 && (reinterpret_cast<uintptr_t>(args.c) & 31) == 0;
      uint16_t* stage = reinterpret_cast<uint16_t*>(scales + C::SGROUPS * C::SGROUP) + warp * (32 * C::OUT_PITCH);
#pragma unroll
      for (int j = 0; j < C::HC; j += 16) {
        if (n0 + j >= args.N) break;
        float y[16];
#pragma unroll
        for (int k = 0; k < 8; ++k) y[2 * k] = acc[j / 2 + k].x, y[2 * k + 1] = acc[j / 2 + k].y;
        if (args.bias) {
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (n0 + j + k < args.N) y[k] += bf16_to_f32(args.bias[n0 + j + k]);
        }
        uint32_t p[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) p[k] = pack_bf16x2(y[2 * k], y[2 * k + 1]);
        if (wide) {  // a whole 32-byte sector of the thread's row
          if (row >= 0) st_global_32b(args.c + (int64_t)row * args.N + n0 + j, p);
        } else {
          // rows that start anywhere: 16 lanes write 16 neighbouring outputs of a row
#pragma unroll
          for (int k = 0; k < 8; ++k) reinterpret_cast<uint32_t*>(stage + lane * C::OUT_PITCH)[k] = p[k];
          __syncwarp();
          const int c = lane & 15;
#pragma unroll 4
          for (int r = lane >> 4; r < 32; r += 2) {
            const int to = __shfl_sync(0xffffffffu, row, r);
            if (to >= 0 && n0 + j + c < args.N) args.c[(int64_t)to * args.N + n0 + j + c] = stage[r * C::OUT_PITCH + c];
          }
          __syncwarp();
        }
      }
    }
  }

  tc_fence_before();
  cta_sync();
  cluster_sync();  // neither CTA leaves while the other's MMAs, copies or arrivals may still reach it
  if (warp == 0) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
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
