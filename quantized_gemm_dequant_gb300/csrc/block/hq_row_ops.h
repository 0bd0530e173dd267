// Launch interface of the kernels that turn a layer's rows into the activations of its next product (hq_row_ops.cu).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace hq {

enum RowOut { ROW_BF16 = 0, ROW_TOKEN = 1, ROW_BLOCK = 2 };  // bf16; e4m3 with a scale per row; e4m3 with one per 128

constexpr int64_t ROW_MAX = 32768;  // longest row whose statistics a CTA takes from registers

struct RowArgs {
  const uint16_t* x;  // norm: the addend; SwiGLU: [gate | up] rows
  int64_t x_stride;
  const uint16_t* residual;  // norm: null = no addition
  int64_t residual_stride;
  const uint16_t* weight;  // norm
  uint16_t* residual_out;
  int64_t residual_out_stride;
  void* out;
  float* scale;
  int64_t rows;
  int width;  // elements of an output row
  float eps;
};

cudaError_t launch_add_rms_norm(RowOut out, const RowArgs& a, cudaStream_t stream);
cudaError_t launch_swiglu_token(const RowArgs& a, cudaStream_t stream);
// rows of `width` outputs, a scale per 128 of them: SwiGLU of [gate | up] rows, or the bf16 rows themselves
cudaError_t launch_block_quant(bool swiglu, const void* x, int64_t rows, int64_t width, void* data, void* scale,
                               cudaStream_t stream);

}  // namespace hq
