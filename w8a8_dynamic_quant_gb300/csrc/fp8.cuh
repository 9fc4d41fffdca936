// fp8.cuh -- launches of the block-scaled FP8 kernels and of the expert router (declared apart from kernels.cuh: the
// int8 and MXFP8 calls do not depend on this file).
#pragma once

#include "kernels.cuh"

namespace w8a8 {

// Rows to E4M3 codes with a binary32 scale per 128 values (fp8_quant.cu): x [M,K] bf16 -> q [M,K], scale
// [M, ceil(K / 128)]; the same with token row m written to its routed rows dst[m*k + j] (an index < 0 is
// skipped); and of the SwiGLU of y13 [R,2I] (gate half, up half).
cudaError_t launch_fp8_quant(const uint16_t* x, int64_t M, int64_t K, uint8_t* q, float* scale, cudaStream_t stream,
                             int num_sms);
cudaError_t launch_fp8_quant_scatter(const uint16_t* x, int64_t T, int64_t K, const int32_t* dst, int k, uint8_t* q,
                                     float* scale, cudaStream_t stream, int num_sms);
cudaError_t launch_fp8_swiglu_quant(const uint16_t* y13, int64_t R, int64_t I, uint8_t* q, float* scale,
                                    cudaStream_t stream, int num_sms);

// Block-scaled FP8 contraction (fp8_gemm.cu), grouped (group_list) or dense (nullptr: one group of R rows).
struct Fp8GemmArgs {
  const uint8_t* q = nullptr;           // [R,K] E4M3
  const float* x_scale = nullptr;       // [R, ceil(K / 128)]
  const int64_t* group_list = nullptr;  // [E] counts, or nullptr
  int64_t E = 1, R = 0, K = 0, N = 0;
  const uint8_t* w = nullptr;        // [E,N,K] E4M3
  const float* w_scale = nullptr;    // [E, ceil(N / 128), ceil(K / 128)]
  const uint16_t* bias = nullptr;    // [N] bf16 or nullptr (dense only)
  uint16_t* y = nullptr;             // [R,N] bf16
  DeviceStatus* status = nullptr;
};
// Scratch of the contraction (zero-filled once) for R rows, in E groups when grouped.
size_t fp8_gemm_ws_bytes(int64_t E, int64_t R, int64_t N, int64_t K, bool grouped);
cudaError_t launch_fp8_gemm(const Fp8GemmArgs& a, void* ws, cudaStream_t stream);

// Expert router (gate.cu): logits [T,E] fp32 or bf16 -> ids [T,k], weights [T,k].  n_group <= 32, k <= 32.
cudaError_t launch_gate(const void* logits, bool bf16, int64_t T, int E, const float* bias, bool sigmoid, int n_group,
                        int topk_group, bool top2, int k, bool renorm, float scale, int64_t* ids, float* weights,
                        cudaStream_t stream);

}  // namespace w8a8
