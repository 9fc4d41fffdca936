// capi_bf16.cu -- the extern "C" boundary of the norm with 8-bit outputs and of the bf16 products (declared in
// include/w8a8.h): argument validation and stream-ordered launches, as capi.cu has them for the int8 and MXFP8 calls.
#include "capi_common.cuh"
#include "gemm_bf16.cuh"
#include "norm.cuh"

using namespace w8a8;

namespace {

w8a8_status norm_common(int form, const uint16_t* x, const uint16_t* residual, const void* weight, int64_t M,
                        int64_t K, float eps, uint32_t flags, uint16_t* residual_out, uint16_t* y, void* q,
                        void* scale, w8a8_stream_t stream) {
  if (M < 0 || M > INT32_MAX) return W8A8_ERR_SHAPE;
  if (w8a8_status s = check_k(K)) return s;
  if (form == 2 && K % 32 != 0) return W8A8_ERR_ALIGN;
  if (!(eps > 0.0f && eps <= 3.4028234663852886e38f) || (flags & ~W8A8_NORM_WEIGHT_F32) != 0u) return W8A8_ERR_SHAPE;
  if ((residual == nullptr) != (residual_out == nullptr) && M > 0) return W8A8_ERR_NULL;
  if (M == 0) return W8A8_OK;
  if (!x || !weight || !q || !scale) return W8A8_ERR_NULL;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(residual_out) || !aligned16(y) ||
      !aligned16(q))
    return W8A8_ERR_ALIGN;
  int sms = 0;
  if (w8a8_status s = device_info(sms)) return s;
  NormArgs a;
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.residual_out = residual_out;
  a.y = y;
  a.q = static_cast<uint8_t*>(q);
  a.scale = scale;
  a.M = M;
  a.K = static_cast<int>(K);
  a.eps = eps;
  a.weight_f32 = (flags & W8A8_NORM_WEIGHT_F32) != 0u;
  return cuda_status(launch_norm_quant(a, form, sms, reinterpret_cast<cudaStream_t>(stream)));
}

// (a tile's last rows lie up to 255 past the tensor's: their coordinates are 32-bit integers)
constexpr int64_t kMaxRows = INT32_MAX - 256;
static_assert(kStatusBytes + kBf16CounterBytes == W8A8_BF16_ZERO_BYTES, "what of a workspace has to be zero");

w8a8_status matmul_common(Bf16GemmArgs& a, uint32_t flags, void* ws, size_t ws_bytes, w8a8_stream_t stream) {
  if (a.E <= 0 || a.E > kMaxE || a.R < 0 || a.R > kMaxRows || a.act < W8A8_ACT_NONE || a.act > W8A8_ACT_SWIGLU ||
      (flags & ~W8A8_MM_F32) != 0u)
    return W8A8_ERR_SHAPE;
  if (a.N <= 0 || a.N > kMaxRows / a.E / (a.act == W8A8_ACT_SWIGLU ? 2 : 1)) return W8A8_ERR_SHAPE;
  if (w8a8_status s = check_k(a.K)) return s;
  if (a.R == 0) return W8A8_OK;
  if (!a.x || !a.w || !a.y) return W8A8_ERR_NULL;
  if (!ws) return W8A8_ERR_WORKSPACE;
  if (!aligned16(a.x) || !aligned16(a.w)) return W8A8_ERR_ALIGN;
  if (ws_bytes < kStatusBytes + plan_bf16_gemm(a) || !aligned16(ws)) return W8A8_ERR_WORKSPACE;
  int sms = 0;
  if (w8a8_status s = device_info(sms)) return s;  // refuses a device of another kind
  a.f32 = (flags & W8A8_MM_F32) != 0u;
  a.status = static_cast<DeviceStatus*>(ws);
  t_last_engine = W8A8_ENGINE_TC;
  return cuda_status(launch_bf16_gemm(a, static_cast<uint8_t*>(ws) + kStatusBytes, reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

w8a8_status w8a8_rms_norm_quant(const uint16_t* x, const uint16_t* residual, const void* weight, int64_t M, int64_t K,
                                float eps, uint32_t flags, uint16_t* residual_out, uint16_t* y, int8_t* q,
                                float* scale, w8a8_stream_t stream) {
  return norm_common(0, x, residual, weight, M, K, eps, flags, residual_out, y, q, scale, stream);
}

w8a8_status w8a8_fp8_rms_norm_quant(const uint16_t* x, const uint16_t* residual, const void* weight, int64_t M,
                                    int64_t K, float eps, uint32_t flags, uint16_t* residual_out, uint16_t* y,
                                    uint8_t* q, float* scale, w8a8_stream_t stream) {
  return norm_common(1, x, residual, weight, M, K, eps, flags, residual_out, y, q, scale, stream);
}

w8a8_status w8a8_mx_rms_norm_quant(const uint16_t* x, const uint16_t* residual, const void* weight, int64_t M,
                                   int64_t K, float eps, uint32_t flags, uint16_t* residual_out, uint16_t* y,
                                   uint8_t* q, uint8_t* scale, w8a8_stream_t stream) {
  return norm_common(2, x, residual, weight, M, K, eps, flags, residual_out, y, q, scale, stream);
}

size_t w8a8_bf16_matmul_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  return M < 0 || N <= 0 || K <= 0 ? 0 : kStatusBytes + bf16_gemm_ws_bytes(M, N);
}

size_t w8a8_bf16_matmul_call_bytes(int64_t M, int64_t N, int64_t K, int act) {
  if (M < 0 || M > kMaxRows || N <= 0 || N > kMaxRows || K <= 0 || K > W8A8_MAX_K || act < W8A8_ACT_NONE ||
      act > W8A8_ACT_SWIGLU)
    return 0;
  Bf16GemmArgs a;
  a.R = M;
  a.N = N;
  a.K = K;
  a.act = act;
  return kStatusBytes + (M == 0 ? 0 : plan_bf16_gemm(a));
}

size_t w8a8_bf16_grouped_matmul_workspace_bytes(int64_t E, int64_t R, int64_t N, int64_t K) {
  return E <= 0 || E > kMaxE || R < 0 || N <= 0 || K <= 0 ? 0 : kStatusBytes;
}

w8a8_status w8a8_bf16_matmul(const uint16_t* x, int64_t M, int64_t K, const uint16_t* w, int64_t N,
                             const uint16_t* bias, int act, const uint16_t* residual, uint32_t flags, void* y, void* ws,
                             size_t ws_bytes, w8a8_stream_t stream) {
  Bf16GemmArgs a;
  a.x = x;
  a.w = w;
  a.bias = bias;
  a.residual = residual;
  a.y = y;
  a.R = M;
  a.K = K;
  a.N = N;
  a.act = act;
  return matmul_common(a, flags, ws, ws_bytes, stream);
}

w8a8_status w8a8_bf16_grouped_matmul(const uint16_t* x, const int64_t* group_list, int64_t E, int64_t R, int64_t K,
                                     const uint16_t* w, int64_t N, const uint16_t* bias, int act, uint32_t flags,
                                     void* y, void* ws, size_t ws_bytes, w8a8_stream_t stream) {
  if (R > 0 && !group_list) return W8A8_ERR_NULL;
  Bf16GemmArgs a;
  a.x = x;
  a.group_list = group_list;
  a.w = w;
  a.bias = bias;
  a.y = y;
  a.E = E;
  a.R = R;
  a.K = K;
  a.N = N;
  a.act = act;
  return matmul_common(a, flags, ws, ws_bytes, stream);
}

}  // extern "C"
