// Paged key-value cache: geometry and kernel arguments shared by the host API and the device code.
//
// Each pool is [num_pages][num_heads][page_size] rows; a row is one (token, head)'s codes.  The 16 tokens of an aligned
// block lie inside one page (page_size is a multiple of 16), so a block's rows of one head are contiguous: 16 * row
// bytes, which is the unit that the attention and the read-back copy.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../../include/hq.h"

namespace hq {

constexpr int KV_BLOCK = 16;            // tokens of a contiguous block of rows
constexpr size_t KV_HEADER_BYTES = 256;  // workspace: device status word, padding

// bytes of one row's codes / scales
__host__ __device__ constexpr int kv_row_bytes(int kind, int dim) {
  return kind == HQ_KV_BF16 ? 2 * dim : (kind == HQ_KV_E4M3 ? dim : dim / 2);
}
__host__ __device__ constexpr int kv_scale_bytes(int kind, int dim) {
  return kind == HQ_KV_BF16 ? 0 : (kind == HQ_KV_E4M3 ? 4 : dim / 16);
}

// The pools as the kernels take them.
struct KvView {
  uint8_t* k;
  uint8_t* v;
  uint8_t* k_scale;
  uint8_t* v_scale;
  const float* k_global;
  const float* v_global;
  int64_t num_pages;
  int page_size;
  int heads;
};

struct KvWriteArgs {
  KvView kv;
  const uint16_t* qkv;
  int64_t row_stride;
  int64_t T;
  int q_heads;
  int rotary;
  int interleaved;
  float eps;
  const uint16_t* q_norm;
  const uint16_t* k_norm;
  const float* cos_sin;
  int64_t num_positions;
  const int32_t* positions;
  const int64_t* slots;
  uint16_t* q_out;
  int* status;
};

struct KvReadArgs {
  KvView kv;
  const int32_t* page_table;
  int64_t table_stride;
  const int64_t* starts;
  const int32_t* first;
  int64_t B;
  int64_t total;
  uint16_t* k_out;
  uint16_t* v_out;
  int* status;
};

struct KvAttnArgs {
  KvView kv;
  const uint16_t* q;
  int group;  // query heads per key-value head
  const int32_t* page_table;
  int64_t table_stride;
  const int32_t* lens;
  int64_t B;
  int64_t most;  // largest length: the table's row, or 2^30
  float scale;
  int64_t window;  // 0: all tokens
  float softcap;   // 0: none
  uint16_t* out;
  float* lse;
  int* status;
};

cudaError_t launch_kv_write(int kind, int dim, const KvWriteArgs& a, cudaStream_t stream);
cudaError_t launch_kv_read(int kind, int dim, const KvReadArgs& a, cudaStream_t stream);
// sms: of the device; tokens: the most that one sequence sees
cudaError_t launch_kv_attention_bf16(int dim, const KvAttnArgs& a, int sms, int64_t tokens, uint8_t* workspace,
                                    cudaStream_t stream);
cudaError_t launch_kv_attention_e4m3(int dim, const KvAttnArgs& a, int sms, int64_t tokens, uint8_t* workspace,
                                    cudaStream_t stream);
cudaError_t launch_kv_attention_nvfp4(int dim, const KvAttnArgs& a, int sms, int64_t tokens, uint8_t* workspace,
                                    cudaStream_t stream);

}  // namespace hq
