// Paged attention over a nvfp4 cache.
#include "hq_kv_attention.cuh"

namespace hq {

cudaError_t launch_kv_attention_nvfp4(int dim, const KvAttnArgs& a, int sms, int64_t tokens, uint8_t* workspace,
                                    cudaStream_t stream) {
  return launch_ka_dim<HQ_KV_NVFP4>(dim, a, sms, tokens, workspace, stream);
}

}  // namespace hq
