// fp8_quant.cu -- rows to E4M3 codes with one binary32 scale per 128 values.
//
// The dynamic half of the block-scaled FP8 path: a row of K values is cut
// into blocks of 128 (the last one may be shorter); per block
//   s = max |v| / 448 (binary32 divide),  q = E4M3(RN(v / s)),
// rounded to nearest, ties to even (448 is the largest E4M3 value).  A block
// of zeros gets s = 0 and codes 0.  The maximum passes NaNs over; a NaN value
// gets the NaN code.  A block holding an infinity has s = inf: its finite
// values get code 0 and its infinities the NaN code.
//
// Two sources: BF16 rows, and the SwiGLU of a BF16 row [gate | up] of 2K,
//   v = (g * sigmoid(g)) * u, sigmoid(g) = 1 / (1 + exp(-g)),
// kept in binary32 into the quantisation (one rounding, to E4M3).  And two
// destinations: the same row, or the k routed rows of a token.
//
// Memory-bound: 2 (plain) or 4 (SwiGLU) bytes read and 1 written per value,
// 1/32 byte of scale.  Eight lanes own a block, 16 values each; the block's
// maximum meets through three shuffles.  CTAs of 128 threads in many waves keep
// the tail short (measured, back to back: 8192 x 4096 18.2 us, 5.6 TB/s, where 256
// threads in eight waves took 20.3; SwiGLU of 32768 x 2048 54.6 us, 6.2 TB/s, and
// with a shorter sigmoid 52.9 against 58.7 so).  Two blocks a thread in flight
// gained nothing.
#include "fp8.cuh"

namespace w8a8 {

namespace {

constexpr int kB = 128;          // values per scale
constexpr int kLanes = 8;        // lanes per block
constexpr int kPer = kB / kLanes;

__device__ __forceinline__ void pdl_enter() {
  pdl_trigger();
  pdl_wait();
}

__device__ __forceinline__ uint4 ldg_stream16(const void* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}

// Two binary32 values -> two E4M3 bytes (nearest even, saturating), lo in the low byte.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// 16 bf16 of two 16-byte words, widened.
__device__ __forceinline__ void widen16(const uint4& a, const uint4& b, float (&v)[kPer]) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// silu(g) * u, silu(g) = g / (1 + t) for g >= 0 and t g / (1 + t) below, t = exp(-|g|) <= 1: nothing overflows, and a far
// negative gate keeps what t has down to 2^-149 (1 / (1 + exp(-g)) has no exp past -88.7, and the fast quotient gives 0
// for divisors above 2^126, from -87.3).  exp is the fast one, within 2 + 1.173 |g| units in the last place, which for
// a negative gate are the result's; the quotient is within 2.  The result is rounded to three mantissa bits next: of
// 134,217,728 codes of normal inputs 274 differ from the 64-bit formula's, 268 with expf's and the divide's rounding.
// 32768 x 2048 takes 54.6 us (1 / (1 + exp(-g)), wrong from -87.3, took 53.3; the sigmoid and its product apart 57.5;
// exp(-|g| / 2), squared, 60; a look at the gates and a second pass for the far ones 56.5).
__device__ __forceinline__ float swiglu_fast(float g, float u) {
  const float t = __expf(-fabsf(g));
  return __fdividef(g >= 0.0f ? g : t * g, 1.0f + t) * u;
}

__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}

// The codes of 16 values under scale s.  For s in [2^-100, 2^100] the quotient comes from the reciprocal
// product with one correction (Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990): y0 = RN(v * rs), y = RN(y0 + (v - y0 * s) * rs).  In that range the steps commute with
// powers of two, so whether the code equals E4M3(RN(v / s)) depends only on the mantissas of v and of the
// block's maximum and on their distance in exponent: every such triple of bf16 values agrees.
__device__ __forceinline__ uint4 codes16(const float (&v)[kPer], float s) {
  uint32_t c[4];
  if (s >= 0x1p-100f && s <= 0x1p100f) {
    const float rs = __frcp_rn(s);
    const uint64_t rs2 = pair(rs, rs), ns2 = pair(-s, -s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = 0u;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint64_t x2 = pair(v[4 * i + 2 * h], v[4 * i + 2 * h + 1]);
        uint64_t y0, r2, y2;
        asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(y0) : "l"(x2), "l"(rs2));
        asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r2) : "l"(y0), "l"(ns2), "l"(x2));
        asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(y2) : "l"(r2), "l"(rs2), "l"(y0));
        float lo, hi;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(y2));
        c[i] |= to_e4m3x2(lo, hi) << (16 * h);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = 0u;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float a = v[4 * i + 2 * h], b = v[4 * i + 2 * h + 1];
        // a block of zeros: +0, or NaN for a NaN value
        const float lo = s == 0.0f ? __fadd_rn(__fmul_rn(a, 0.0f), 0.0f) : __fdiv_rn(a, s);
        const float hi = s == 0.0f ? __fadd_rn(__fmul_rn(b, 0.0f), 0.0f) : __fdiv_rn(b, s);
        c[i] |= to_e4m3x2(lo, hi) << (16 * h);
      }
    }
  }
  return make_uint4(c[0], c[1], c[2], c[3]);
}

// Block b of the M * KB blocks: row b / KB, values [128 kb, 128 kb + 128) of it, kb = b % KB.  `dst` (or
// nullptr): the k routed rows dst[row * k + j] of a token row; an index < 0 is skipped.
template <bool SWIGLU, bool SCATTER>
__global__ void __launch_bounds__(128) fp8_quant_kernel(const uint16_t* __restrict__ x, int64_t M, int64_t K, int KB,
                                                        uint8_t* __restrict__ q, float* __restrict__ scale,
                                                        const int32_t* __restrict__ dst, int k) {
  pdl_enter();
  const int64_t nblk = M * KB;
  const int sub = threadIdx.x % kLanes;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (128 / kLanes);
  // whole warps stay in the loop together: the shuffles below take the full mask
  for (int64_t b0 = static_cast<int64_t>(blockIdx.x) * (128 / kLanes) + (threadIdx.x / 32) * (32 / kLanes); b0 < nblk;
       b0 += step) {
    const int64_t b = b0 + (threadIdx.x % 32) / kLanes;
    const bool in_blk = b < nblk;
    int64_t row;
    int kb;
    if (nblk <= 0xffffffffll) {  // 32-bit division where it fits
      const uint32_t r32 = static_cast<uint32_t>(b) / static_cast<uint32_t>(KB);
      row = r32;
      kb = static_cast<int>(static_cast<uint32_t>(b) - r32 * static_cast<uint32_t>(KB));
    } else {
      row = b / KB;
      kb = static_cast<int>(b - row * KB);
    }
    // the lane's values: 8 of the block's first half and 8 of its second, so that every load and store instruction
    // covers whole 32-byte sectors
    const int64_t col = static_cast<int64_t>(kb) * kB + sub * 8;
    const bool in0 = in_blk && col < K, in1 = in_blk && col + kB / 2 < K;  // K % 16 == 0: 8 values are in or out together
    float v[kPer];
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    if constexpr (SWIGLU) {
      const uint16_t* g = x + row * 2 * K + col;
      const uint4 g0 = in0 ? ldg_stream16(g) : zero, g1 = in1 ? ldg_stream16(g + kB / 2) : zero;
      const uint4 u0 = in0 ? ldg_stream16(g + K) : zero, u1 = in1 ? ldg_stream16(g + K + kB / 2) : zero;
      float u[kPer];
      widen16(g0, g1, v);
      widen16(u0, u1, u);
#pragma unroll
      for (int i = 0; i < kPer; ++i) v[i] = swiglu_fast(v[i], u[i]);
    } else {
      const uint16_t* p = x + row * K + col;
      const uint4 a = in0 ? ldg_stream16(p) : zero, c = in1 ? ldg_stream16(p + kB / 2) : zero;
      widen16(a, c, v);
    }
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) amax = fmaxf(amax, fabsf(v[i]));  // fmaxf passes a NaN over
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float s = __fdiv_rn(amax, 448.0f);
    const uint4 c = codes16(v, s);
    const uint2 c0 = make_uint2(c.x, c.y), c1 = make_uint2(c.z, c.w);
    if constexpr (SCATTER) {
      if (in_blk) {
        for (int j = 0; j < k; ++j) {
          const int64_t r = dst[row * k + j];
          if (r < 0) continue;
          if (in0) *reinterpret_cast<uint2*>(q + r * K + col) = c0;
          if (in1) *reinterpret_cast<uint2*>(q + r * K + col + kB / 2) = c1;
          if (sub == 0) scale[r * KB + kb] = s;
        }
      }
    } else {
      if (in0) *reinterpret_cast<uint2*>(q + row * K + col) = c0;
      if (in1) *reinterpret_cast<uint2*>(q + row * K + col + kB / 2) = c1;
      if (in_blk && sub == 0) scale[row * KB + kb] = s;
    }
  }
}

template <bool SWIGLU, bool SCATTER>
cudaError_t launch_t(const uint16_t* x, int64_t M, int64_t K, uint8_t* q, float* scale, const int32_t* dst, int k,
                     cudaStream_t stream, int num_sms) {
  if (M == 0) return cudaSuccess;
  const int KB = static_cast<int>((K + kB - 1) / kB);
  const int64_t ctas = (M * KB + 128 / kLanes - 1) / (128 / kLanes);
  const int64_t grid = std::min<int64_t>(ctas, static_cast<int64_t>(num_sms) * 64);
  return launch_pdl(fp8_quant_kernel<SWIGLU, SCATTER>, dim3(static_cast<unsigned>(grid)), dim3(128), 0, stream, x, M,
                    K, KB, q, scale, dst, k);
}

}  // namespace

cudaError_t launch_fp8_quant(const uint16_t* x, int64_t M, int64_t K, uint8_t* q, float* scale, cudaStream_t stream,
                             int num_sms) {
  return launch_t<false, false>(x, M, K, q, scale, nullptr, 0, stream, num_sms);
}

cudaError_t launch_fp8_quant_scatter(const uint16_t* x, int64_t T, int64_t K, const int32_t* dst, int k, uint8_t* q,
                                     float* scale, cudaStream_t stream, int num_sms) {
  return launch_t<false, true>(x, T, K, q, scale, dst, k, stream, num_sms);
}

cudaError_t launch_fp8_swiglu_quant(const uint16_t* y13, int64_t R, int64_t I, uint8_t* q, float* scale,
                                    cudaStream_t stream, int num_sms) {
  return launch_t<true, false>(y13, R, I, q, scale, nullptr, 0, stream, num_sms);
}

}  // namespace w8a8
