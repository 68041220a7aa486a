// grad.h -- host-side declarations of the gradient norm and clipping kernels.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace moe {

constexpr int kGradBatch = 120;       // tensors per launch (the list travels in the kernel's parameters)
// CTAs per SM, measured on 1.5 GB in bf16: reading, 4 take 215 us, 5 225 us and 6
// (not all resident) 268 us; scaling, 4 take 545 us and 6 489 us.
constexpr int kGradNormCtas = 4;
constexpr int kGradScaleCtas = 6;
constexpr int kGradMaxSms = 256;      // the workspace holds partial sums for this many SMs
constexpr int kGradMaxTensors = 1024;

struct GradBatch {
  const void* src[kGradBatch];
  void* dst[kGradBatch];
  int64_t count[kGradBatch];
  uint32_t first[kGradBatch + 1];  // first chunk of each tensor; first[n] = chunks in all
  uint8_t bf16[kGradBatch];
  bool in_place;  // every tensor
  int n;
};
static_assert(sizeof(GradBatch) <= 4000, "kernel parameters hold 4 KB");

// Chunks of a tensor of `count` elements.
int64_t grad_chunks(int64_t count, bool bf16);
int grad_grid(uint32_t chunks, int ctas);
cudaError_t launch_grad_squares(const GradBatch& b, double* part, int grid, cudaStream_t stream);
cudaError_t launch_grad_norm(const double* part, int nparts, float* norm_out, cudaStream_t stream);
cudaError_t launch_grad_scale(const GradBatch& b, const double* part, int nparts, float max_norm, float* norm_out,
                              int grid, cudaStream_t stream);

}  // namespace moe
