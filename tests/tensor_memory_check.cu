// Host-side check that tensor memory never runs out on an SM: whatever mix of this library's tensor-memory kernels fits
// its 228 KB of shared memory together asks for at most 512 columns, so that no allocation ever waits for another CTA.
// (A CTA that waited could wait for one of the next kernel in its stream, launched early, which waits for it.)  Built with
// nvcc and run on the CPU by tests/test_tensor_memory.py; prints "OK" or the first mix that does not fit.
#include <stdio.h>

#include <vector>

#include "../quantized_gemm_dequant_gb300/csrc/block/hq_gemm_block.cuh"

using namespace hq;

struct Kernel {
  const char* name;
  int bt, smem, columns;
};
static std::vector<Kernel> kernels;

template <int PATH, int BT>
static void whole(const char* name) {
  kernels.push_back({name, BT, Cfg<PATH, BT>::SMEM_BYTES, 512});
}
template <int PATH>
static void wholes(const char* name) {
  whole<PATH, 16>(name), whole<PATH, 32>(name), whole<PATH, 64>(name), whole<PATH, 128>(name), whole<PATH, 256>(name);
}
template <int BT>
static void block() {
  kernels.push_back({"e4m3 block", BT, BlkCfg<BT>::SMEM, BlkCfg<BT>::COLS});
}

// mixes of kernels `from`.. added to those that hold `smem` bytes and `columns` already
static int mixes(size_t from, int smem, int columns, std::vector<size_t>& held) {
  if (columns > 512) {
    for (size_t k : held) printf("%s (%d tokens, %d bytes, %d columns)  ", kernels[k].name, kernels[k].bt, kernels[k].smem, kernels[k].columns);
    printf("share an SM\n");
    return 1;
  }
  for (size_t k = from; k < kernels.size(); ++k) {
    if (smem + kernels[k].smem + 1024 > 228 * 1024) continue;
    held.push_back(k);
    if (mixes(k, smem + kernels[k].smem + 1024, columns + kernels[k].columns, held)) return 1;
    held.pop_back();
  }
  return 0;
}

int main() {
  wholes<PATH_INT4>("int4"), wholes<PATH_NVFP4>("nvfp4"), wholes<PATH_MXFP4>("mxfp4");
  wholes<PATH_MXFP4A>("mxfp4 x mxfp8"), wholes<PATH_MXFP4X>("mxfp4 x mxfp4");
  block<16>(), block<32>(), block<64>(), block<128>();
  kernels.push_back({"e4m3 block pair", 128, PairCfg<128>::SMEM, 512});
  kernels.push_back({"e4m3 block pair", 256, PairCfg<256>::SMEM, 512});
  std::vector<size_t> held;
  if (mixes(0, 0, 0, held)) return 1;
  printf("OK\n");
  return 0;
}
