// Paged attention over a nvfp4 cache.
#include "hq_kv_attention.cuh"

namespace hq {

cudaError_t launch_kv_attention_nvfp4(int dim, const KvAttnArgs& a, int ctas, float* slots, int* counters,
                                      cudaStream_t stream) {
  return dim == 64 ? launch_ka<HQ_KV_NVFP4, 64>(a, ctas, slots, counters, stream)
                   : (dim == 128 ? launch_ka<HQ_KV_NVFP4, 128>(a, ctas, slots, counters, stream)
                                 : launch_ka<HQ_KV_NVFP4, 256>(a, ctas, slots, counters, stream));
}

}  // namespace hq
