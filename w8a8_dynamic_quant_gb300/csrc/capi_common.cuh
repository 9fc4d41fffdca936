// capi_common.cuh -- argument checks and per-thread state that the files of the extern "C" boundary share (capi.cu:
// the int8 and MXFP8 calls; capi_fp8.cu: the router and the block-scaled FP8 calls).
#pragma once

#include <mutex>

#include "kernels.cuh"

namespace w8a8 {

inline constexpr int kMaxDevices = 64;
inline constexpr int64_t kMaxE = 1024;

struct DevInfo {
  int sms = 0;
  int supported = -1;  // -1 unknown, 0 no, 1 yes
};
inline DevInfo g_dev[kMaxDevices];
inline std::mutex g_dev_mu;

inline w8a8_status device_info(int& sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return W8A8_ERR_CUDA;
  std::lock_guard<std::mutex> lk(g_dev_mu);
  DevInfo& d = g_dev[dev];
  if (d.supported < 0) {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return W8A8_ERR_CUDA;
    d.supported = (major == 10 && minor == 3) ? 1 : 0;
  }
  if (!d.supported) return W8A8_ERR_UNSUPPORTED;
  sms = d.sms;
  return W8A8_OK;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0u; }
inline w8a8_status cuda_status(cudaError_t e) { return e == cudaSuccess ? W8A8_OK : W8A8_ERR_CUDA; }

inline w8a8_status check_k(int64_t K) {
  if (K <= 0 || K > W8A8_MAX_K) return W8A8_ERR_SHAPE;
  if (K % 16 != 0) return W8A8_ERR_ALIGN;
  return W8A8_OK;
}

// Sizes shared by the routing calls: T tokens with k choices each, R = T*k routed rows.
inline w8a8_status check_route_shape(int64_t T, int64_t k, int64_t E) {
  if (T < 0 || k < 1 || k > INT32_MAX || E < 1 || E > kMaxE) return W8A8_ERR_SHAPE;
  if (T > 0 && k > INT32_MAX / T) return W8A8_ERR_SHAPE;
  return W8A8_OK;
}

// The combine numbers its work items (token, 1024 columns) with 32-bit integers.
inline bool combine_grid_ok(int64_t T, int64_t H) { return T * ((H / 8 + 127) / 128) <= INT32_MAX; }

// The engine of this thread's last contraction (w8a8_last_engine).
inline thread_local int t_last_engine = W8A8_ENGINE_NONE;

}  // namespace w8a8
