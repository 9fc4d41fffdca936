// norm.cuh -- launch of the norm with 8-bit outputs (norm.cu).
#pragma once

#include "kernels.cuh"

namespace w8a8 {

struct NormArgs {
  const uint16_t* x = nullptr;         // [M,K] bf16
  const uint16_t* residual = nullptr;  // [M,K] bf16 or nullptr
  const void* weight = nullptr;        // [K] bf16, or fp32 (weight_f32)
  uint16_t* residual_out = nullptr;    // [M,K] bf16: x + residual (with a residual; may be x or residual)
  uint16_t* y = nullptr;               // [M,K] bf16 or nullptr
  uint8_t* q = nullptr;                // [M,K] int8 or E4M3
  void* scale = nullptr;               // fp32 [M] | fp32 [M, ceil(K / 128)] | E8M0 bytes [M, K / 32]
  int64_t M = 0;
  int K = 0;                           // a multiple of 16 (MXFP8: 32), at most W8A8_MAX_K
  float eps = 0.0f;
  bool weight_f32 = false;
};
// form: 0 int8 with a scale a row, 1 E4M3 with a scale per 128 values, 2 MXFP8.
cudaError_t launch_norm_quant(const NormArgs& a, int form, int num_sms, cudaStream_t stream);

}  // namespace w8a8
