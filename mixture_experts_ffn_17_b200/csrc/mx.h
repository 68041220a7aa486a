// mx.h -- host-side declarations of the MXFP4 kernels.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace moe {

constexpr int kMxBlock = 32;  // values that share a scale

// codes, scales of [rows, cols] values (row stride ld elements); up != nullptr:
// of silu(src) * up.
cudaError_t launch_mx_quantise(const void* src, const void* up, bool bf16, int64_t rows, int cols, int64_t ld,
                               uint8_t* codes, uint8_t* scales, int sms, cudaStream_t stream);
// codes [E, N, K / 2], scales [E, N, K / 32] of W [E, K, N].
cudaError_t launch_mx_quantise_weights(const void* W, bool bf16, int E, int K, int N, uint8_t* codes, uint8_t* scales,
                                       cudaStream_t stream);
cudaError_t launch_mx_dequantise(const uint8_t* codes, const uint8_t* scales, int64_t rows, int cols, void* dst,
                                 bool bf16, int sms, cudaStream_t stream);

// Grouped product: Y[r] = A[r] W[e]^T for the rows of each expert.
constexpr int kMxTileTokens = 192;
constexpr int kMxMaxExperts = 1024;

struct MxProduct {
  int64_t rows;  // of A and Y
  int E, K, N;
  const uint8_t* a_scales;   // [rows, K / 32]
  const uint8_t* w_scales;   // [E, N, K / 32]
  const int32_t* offsets;    // [E + 1]
  void* Y;                   // [rows, N]
  uint32_t* status;
  bool withhold;             // tests: no operands are loaded
};

// Tensor maps over the codes as bytes, 128-byte boxes with the 128-byte
// swizzle: W as [E * N, K / 2] in boxes of 128 rows, A as [rows, K / 2] in
// boxes of 16 and of 64.
cudaError_t launch_mx_product(const CUtensorMap& tmW, const CUtensorMap& tmA16, const CUtensorMap& tmA64,
                              const MxProduct& p, bool y_bf16, int sms, cudaStream_t stream);

}  // namespace moe
