// Instances and launches of the block-scaled e4m3 products (hq_gemm_block.cuh).
#include <atomic>

#include "hq_gemm_block.cuh"

namespace hq {

namespace {

// The shared-memory limit of a kernel, set once per device.
template <typename K>
cudaError_t allow_smem(K kernel, int bytes, std::atomic<int> (&done)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev >= 0 && dev < 64 && done[dev])) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = 1;
  return e;
}

template <int BT>
cudaError_t launch_bt(const GemmArgs& a, int grid, cudaStream_t stream) {
  static std::atomic<int> done[64];
  const cudaError_t e = allow_smem(gemm_block_kernel<BT>, BlkCfg<BT>::SMEM, done);
  if (e != cudaSuccess) return e;
  return launch_cluster_kernel(gemm_block_kernel<BT>, grid, a.sk, BLK_THREADS, BlkCfg<BT>::SMEM, stream, a);
}

// Clusters of n CTAs, one CTA an SM, that the current device holds at once (asked once for each n; 0: no answer).
int clusters_of(int n) {
  static std::atomic<int> known[9];
  int c = known[n].load(std::memory_order_relaxed);
  if (c != 0) return c;
  static std::atomic<int> done[64];
  if (allow_smem(gemm_block_kernel<128>, BlkCfg<128>::SMEM, done) != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)n);
  cfg.blockDim = dim3(BLK_THREADS);
  cfg.dynamicSmemBytes = BlkCfg<128>::SMEM;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)n;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&c, gemm_block_kernel<128>, &cfg) != cudaSuccess || c < 1) {
    cudaGetLastError();
    return 0;
  }
  known[n].store(c, std::memory_order_relaxed);
  return c;
}

template <int BN>
cudaError_t launch_pair(const GemmArgs& a, int grid, cudaStream_t stream) {
  static std::atomic<int> done[64];
  const cudaError_t e = allow_smem(gemm_block_pair_kernel<BN>, PairCfg<BN>::SMEM, done);
  if (e != cudaSuccess) return e;
  return launch_kernel(gemm_block_pair_kernel<BN>, dim3((unsigned)grid), dim3(PAIR_THREADS), PairCfg<BN>::SMEM, stream,
                       a);
}

}  // namespace

// CTAs of the kernel for few tokens that the device holds at once in clusters of sk (0 where there is no device to ask).
// Two of a cluster's CTAs with up to 32 tokens share an SM, which the occupancy query does not see (304 tiles take 3.5
// us, 380 take 5.3): a cluster then takes half as many SMs.
int gemm_block_room(int bt, int sk) {
  if (sk < 1 || sk > 8) return 0;
  return bt > 32 ? clusters_of(sk) * sk : (sk == 1 ? 2 * clusters_of(1) : clusters_of((sk + 1) / 2) * sk);
}

// bn features by 256 tokens a pair of CTAs
cudaError_t launch_gemm_block_pair(const GemmArgs& a, int bn, int grid, cudaStream_t stream) {
  return bn == 256 ? launch_pair<256>(a, grid, stream) : launch_pair<128>(a, grid, stream);
}

// bt tokens a tile, grid = tiles * a.sk CTAs
cudaError_t launch_gemm_block(const GemmArgs& a, int bt, int grid, cudaStream_t stream) {
  switch (bt) {
    case 16: return launch_bt<16>(a, grid, stream);
    case 32: return launch_bt<32>(a, grid, stream);
    case 64: return launch_bt<64>(a, grid, stream);
    case 128: return launch_bt<128>(a, grid, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace hq
