// gemm_bf16.cuh -- launch of the bf16 products (gemm_bf16.cu).
#pragma once

#include "kernels.cuh"

namespace w8a8 {

// y = act(x w^T + bias) (+ residual), dense (group_list == nullptr: one group of R rows) or grouped by expert.
struct Bf16GemmArgs {
  const uint16_t* x = nullptr;          // [R,K] bf16
  const int64_t* group_list = nullptr;  // [E] counts, or nullptr
  const uint16_t* w = nullptr;          // [E,N,K] bf16, gated: [E,2N,K], the gate's N rows, then the up projection's
  const uint16_t* bias = nullptr;       // [E, rows of w] bf16 or nullptr
  const uint16_t* residual = nullptr;   // [R,N] bf16 or nullptr
  void* y = nullptr;                    // [R,N] bf16 or fp32
  DeviceStatus* status = nullptr;
  int64_t E = 1, R = 0, K = 0, N = 0;   // N: channels of y
  int act = 0;                          // W8A8_ACT_*
  bool f32 = false;                     // y is fp32
  struct {
    int nt, blocks, per, split, pairs, cut;
  } plan = {};                          // plan_bf16_gemm's
};
// Chooses the tiles and returns the scratch that they need (its counters zero-filled once; grouped products need none).
size_t plan_bf16_gemm(Bf16GemmArgs& a);
constexpr size_t kBf16CounterBytes = 4864;  // at the scratch's start
// The most that a dense product of up to R rows to up to N channels asks for, gated or not, whatever its K.
size_t bf16_gemm_ws_bytes(int64_t R, int64_t N);
cudaError_t launch_bf16_gemm(const Bf16GemmArgs& a, void* ws, cudaStream_t stream);

}  // namespace w8a8
