// Paged attention over a bf16 cache.
#include "hq_kv_attention.cuh"

namespace hq {

cudaError_t launch_kv_attention_bf16(int dim, const KvAttnArgs& a, int sms, int64_t tokens, float* slots,
                                    int* counters, cudaStream_t stream) {
  return launch_ka_dim<HQ_KV_BF16>(dim, a, sms, tokens, slots, counters, stream);
}

}  // namespace hq
