// Instances and launches of the block-scaled e4m3 products (hq_gemm_block.cuh).
#include "hq_gemm_block.cuh"

namespace hq {

namespace {

// The shared-memory limit of a kernel, set once per device.
template <typename K>
cudaError_t allow_smem(K kernel, int bytes, int (&done)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev >= 0 && dev < 64 && done[dev])) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = 1;
  return e;
}

template <int BT>
cudaError_t launch_bt(const GemmArgs& a, int grid, cudaStream_t stream) {
  static int done[64] = {0};
  const cudaError_t e = allow_smem(gemm_block_kernel<BT>, BlkCfg<BT>::SMEM, done);
  if (e != cudaSuccess) return e;
  return launch_cluster_kernel(gemm_block_kernel<BT>, grid, a.sk, BLK_THREADS, BlkCfg<BT>::SMEM, stream, a);
}

template <int BN>
cudaError_t launch_pair(const GemmArgs& a, int grid, cudaStream_t stream) {
  static int done[64] = {0};
  const cudaError_t e = allow_smem(gemm_block_pair_kernel<BN>, PairCfg<BN>::SMEM, done);
  if (e != cudaSuccess) return e;
  return launch_kernel(gemm_block_pair_kernel<BN>, dim3((unsigned)grid), dim3(PAIR_THREADS), PairCfg<BN>::SMEM, stream,
                       a);
}

}  // namespace

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
