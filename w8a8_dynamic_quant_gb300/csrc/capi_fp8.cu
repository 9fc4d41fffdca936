// capi_fp8.cu -- the extern "C" boundary of the expert router and of the block-scaled FP8 calls (declared in
// include/w8a8.h): argument validation, workspace layouts and stream-ordered launches, as capi.cu has them for the
// int8 and MXFP8 calls.
#include <cmath>

#include "capi_common.cuh"
#include "fp8.cuh"

using namespace w8a8;

extern "C" {

w8a8_status moe_gate_topk(const void* logits, int64_t T, int64_t E, const float* bias, int64_t n_group,
                          int64_t topk_group, int64_t k, float routed_scale, uint32_t flags, int64_t* topk_ids,
                          float* topk_weights, w8a8_stream_t stream) {
  if (T < 0 || E < 1 || E > kMaxE || n_group < 1 || n_group > W8A8_GATE_MAX_GROUPS || E % n_group != 0 ||
      topk_group < 1 || topk_group > n_group || k < 1 || k > W8A8_GATE_MAX_K || k > topk_group * (E / n_group))
    return W8A8_ERR_SHAPE;
  if (T > INT32_MAX / std::max(E, k)) return W8A8_ERR_SHAPE;
  if ((flags & ~(W8A8_GATE_SIGMOID | W8A8_GATE_GROUP_TOP2 | W8A8_GATE_RENORM | W8A8_GATE_BF16)) ||
      !(routed_scale > -INFINITY && routed_scale < INFINITY))
    return W8A8_ERR_SHAPE;
  if (T == 0) return W8A8_OK;
  if (!logits || !topk_ids || !topk_weights) return W8A8_ERR_NULL;
  int sms = 0;
  if (w8a8_status s = device_info(sms)) return s;
  return cuda_status(launch_gate(logits, (flags & W8A8_GATE_BF16) != 0u, T, static_cast<int>(E), bias,
                                 (flags & W8A8_GATE_SIGMOID) != 0u, static_cast<int>(n_group),
                                 static_cast<int>(topk_group), (flags & W8A8_GATE_GROUP_TOP2) != 0u,
                                 static_cast<int>(k), (flags & W8A8_GATE_RENORM) != 0u, routed_scale, topk_ids,
                                 topk_weights, reinterpret_cast<cudaStream_t>(stream)));
}

w8a8_status w8a8_fp8_quant(const uint16_t* x, int64_t M, int64_t K, uint8_t* q, float* scale, w8a8_stream_t stream) {
  if (M < 0 || M > INT32_MAX) return W8A8_ERR_SHAPE;
  if (w8a8_status s = check_k(K)) return s;
  if (M == 0) return W8A8_OK;
  if (!x || !q || !scale) return W8A8_ERR_NULL;
  if (!aligned16(x) || !aligned16(q)) return W8A8_ERR_ALIGN;
  int sms = 0;
  if (w8a8_status s = device_info(sms)) return s;
  return cuda_status(launch_fp8_quant(x, M, K, q, scale, reinterpret_cast<cudaStream_t>(stream), sms));
}

w8a8_status w8a8_fp8_swiglu_quant(const uint16_t* y13, int64_t R, int64_t I, uint8_t* q, float* scale,
                                  w8a8_stream_t stream) {
  if (R < 0 || R > INT32_MAX) return W8A8_ERR_SHAPE;
  if (w8a8_status s = check_k(I)) return s;
  if (R == 0) return W8A8_OK;
  if (!y13 || !q || !scale) return W8A8_ERR_NULL;
  if (!aligned16(y13) || !aligned16(q)) return W8A8_ERR_ALIGN;
  int sms = 0;
  if (w8a8_status s = device_info(sms)) return s;
  return cuda_status(launch_fp8_swiglu_quant(y13, R, I, q, scale, reinterpret_cast<cudaStream_t>(stream), sms));
}

size_t w8a8_fp8_matmul_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N <= 0 || K <= 0) return 0;
  return kStatusBytes + fp8_gemm_ws_bytes(1, M, N, K, false);
}

size_t w8a8_fp8_grouped_matmul_workspace_bytes(int64_t E, int64_t R, int64_t N, int64_t K) {
  if (E <= 0 || E > kMaxE || R < 0 || N <= 0 || K <= 0) return 0;
  return kStatusBytes + fp8_gemm_ws_bytes(E, R, N, K, true);
}

static w8a8_status fp8_common(const Fp8GemmArgs& in, void* ws, size_t ws_bytes, w8a8_stream_t stream) {
  Fp8GemmArgs a = in;
  if (a.E <= 0 || a.E > kMaxE || a.R < 0 || a.R > INT32_MAX || a.N <= 0 || a.N > INT32_MAX / a.E) return W8A8_ERR_SHAPE;
  if (w8a8_status s = check_k(a.K)) return s;
  if (a.R == 0) return W8A8_OK;
  if (!a.q || !a.x_scale || !a.w || !a.w_scale || !a.y) return W8A8_ERR_NULL;
  if (!ws) return W8A8_ERR_WORKSPACE;
  if (!aligned16(a.q) || !aligned16(a.w)) return W8A8_ERR_ALIGN;
  const size_t need = kStatusBytes + fp8_gemm_ws_bytes(a.E, a.R, a.N, a.K, a.group_list != nullptr);
  if (ws_bytes < need || !aligned16(ws)) return W8A8_ERR_WORKSPACE;
  int sms = 0;
  if (w8a8_status s = device_info(sms)) return s;  // refuses a device of another kind
  a.status = static_cast<DeviceStatus*>(ws);
  t_last_engine = W8A8_ENGINE_TC;
  return cuda_status(
      launch_fp8_gemm(a, static_cast<uint8_t*>(ws) + kStatusBytes, reinterpret_cast<cudaStream_t>(stream)));
}

w8a8_status w8a8_fp8_matmul(const uint8_t* q, const float* x_scale, int64_t M, int64_t K, const uint8_t* w,
                            const float* w_scale, int64_t N, const uint16_t* bias, uint16_t* y, void* ws,
                            size_t ws_bytes, w8a8_stream_t stream) {
  Fp8GemmArgs a;
  a.q = q;
  a.x_scale = x_scale;
  a.R = M;
  a.K = K;
  a.N = N;
  a.w = w;
  a.w_scale = w_scale;
  a.bias = bias;
  a.y = y;
  return fp8_common(a, ws, ws_bytes, stream);
}

w8a8_status w8a8_fp8_grouped_matmul(const uint8_t* q, const float* x_scale, const int64_t* group_list, int64_t E,
                                    int64_t R, int64_t K, const uint8_t* w, const float* w_scale, int64_t N,
                                    uint16_t* y, void* ws, size_t ws_bytes, w8a8_stream_t stream) {
  if (R > 0 && !group_list) return W8A8_ERR_NULL;
  Fp8GemmArgs a;
  a.q = q;
  a.x_scale = x_scale;
  a.group_list = group_list;
  a.E = E;
  a.R = R;
  a.K = K;
  a.N = N;
  a.w = w;
  a.w_scale = w_scale;
  a.y = y;
  return fp8_common(a, ws, ws_bytes, stream);
}

namespace {

// Workspace of moe_fp8_layer: status word, routing results and scratch, the routed rows' codes and scales, the
// W13 output, h's codes and scales, the routed output, and the contractions' scratch (one region for both).
struct Fp8LayerWs {
  size_t group_list, pos, counts, xq, xs, y13, hq, hs, y_routed, gemm, total;
};
Fp8LayerWs fp8_layer_layout(int64_t T, int64_t k, int64_t H, int64_t I, int64_t E) {
  Fp8LayerWs L;
  const uint64_t R = static_cast<uint64_t>(T * k);
  size_t off = kStatusBytes;
  const auto take = [&off](uint64_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes, 256);
    return at;
  };
  L.gemm = take(std::max(fp8_gemm_ws_bytes(E, T * k, 2 * I, H, true), fp8_gemm_ws_bytes(E, T * k, H, I, true)));
  L.group_list = take(static_cast<uint64_t>(E) * 8);
  L.pos = take(R * 4);
  L.counts = take(static_cast<uint64_t>(route_scratch_ints(T * k, E)) * 4);
  L.xq = take(R * H);
  L.xs = take(R * ((H + 127) / 128) * 4);
  L.y13 = take(R * 2 * I * 2);
  L.hq = take(R * I);
  L.hs = take(R * ((I + 127) / 128) * 4);
  L.y_routed = take(R * H * 2);
  L.total = off;
  return L;
}

}  // namespace

size_t moe_fp8_layer_workspace_bytes(int64_t T, int64_t k, int64_t H, int64_t I, int64_t E) {
  if (check_route_shape(T, k, E) != W8A8_OK || H <= 0 || I <= 0) return 0;
  return fp8_layer_layout(T, k, H, I, E).total;
}

w8a8_status moe_fp8_layer(const uint16_t* x, const int64_t* topk_ids, const float* topk_weights, int64_t T, int64_t k,
                          int64_t E, int64_t H, int64_t I, const uint8_t* w13, const float* w13_scale,
                          const uint8_t* w2, const float* w2_scale, void* ws, size_t ws_bytes, uint16_t* y,
                          w8a8_stream_t stream) {
  if (w8a8_status s = check_route_shape(T, k, E)) return s;
  if (H <= 0 || I <= 0 || !combine_grid_ok(T, H)) return W8A8_ERR_SHAPE;
  if (w8a8_status s = check_k(H)) return s;
  if (w8a8_status s = check_k(I)) return s;
  if (H > INT32_MAX / E || 2 * I > INT32_MAX / E) return W8A8_ERR_SHAPE;
  if (T == 0) return W8A8_OK;
  if (!x || !topk_ids || !topk_weights || !w13 || !w13_scale || !w2 || !w2_scale || !y) return W8A8_ERR_NULL;
  if (!ws) return W8A8_ERR_WORKSPACE;
  if (!aligned16(x) || !aligned16(y) || !aligned16(w13) || !aligned16(w2)) return W8A8_ERR_ALIGN;
  const Fp8LayerWs L = fp8_layer_layout(T, k, H, I, E);
  if (ws_bytes < L.total || !aligned16(ws)) return W8A8_ERR_WORKSPACE;
  int sms = 0;
  if (w8a8_status s = device_info(sms)) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* b = static_cast<uint8_t*>(ws);
  DeviceStatus* status = static_cast<DeviceStatus*>(ws);
  const int64_t R = T * k;
  const int kk = static_cast<int>(k);
  int64_t* gl = reinterpret_cast<int64_t*>(b + L.group_list);
  int32_t* pos = reinterpret_cast<int32_t*>(b + L.pos);
  uint16_t* y13 = reinterpret_cast<uint16_t*>(b + L.y13);
  uint16_t* yr = reinterpret_cast<uint16_t*>(b + L.y_routed);
  float* xs = reinterpret_cast<float*>(b + L.xs);
  float* hs = reinterpret_cast<float*>(b + L.hs);
  if (w8a8_status e = cuda_status(launch_route(topk_ids, R, static_cast<int>(E),
                                               reinterpret_cast<int32_t*>(b + L.counts), gl, pos, status, st)))
    return e;
  if (w8a8_status e = cuda_status(launch_fp8_quant_scatter(x, T, H, pos, kk, b + L.xq, xs, st, sms))) return e;
  Fp8GemmArgs a;
  a.q = b + L.xq;
  a.x_scale = xs;
  a.group_list = gl;
  a.E = E;
  a.R = R;
  a.K = H;
  a.N = 2 * I;
  a.w = w13;
  a.w_scale = w13_scale;
  a.y = y13;
  a.status = status;
  if (w8a8_status e = cuda_status(launch_fp8_gemm(a, b + L.gemm, st))) return e;
  if (w8a8_status e = cuda_status(launch_fp8_swiglu_quant(y13, R, I, b + L.hq, hs, st, sms))) return e;
  a.q = b + L.hq;
  a.x_scale = hs;
  a.K = I;
  a.N = H;
  a.w = w2;
  a.w_scale = w2_scale;
  a.y = yr;
  if (w8a8_status e = cuda_status(launch_fp8_gemm(a, b + L.gemm, st))) return e;
  t_last_engine = W8A8_ENGINE_TC;
  return cuda_status(launch_combine(yr, pos, topk_weights, T, kk, H, y, status, st, sms));
}

}  // extern "C"
