// capi_bf16.cu -- the extern "C" boundary of the norm with 8-bit outputs (declared in include/w8a8.h): argument
// validation and stream-ordered launches, as capi.cu has them for the int8 and MXFP8 calls.
#include "capi_common.cuh"
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

}  // extern "C"
