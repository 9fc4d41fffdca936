// fp8_gemm.cu -- block-scaled FP8 contraction, dense and grouped by expert.
//
//   y[m,n] = bf16( sum_b xs[m,b] * ws[n / 128, b] * sum_{k in block b} q[m,k] * w[n,k]  (+ bias[n]) )
//
// q [R,K] E4M3 rows with a binary32 scale per 128 values, w [E,N,K] E4M3 with
// a binary32 scale per 128 x 128 block.  The product of a block is summed in
// binary32 by the tensor core, scaled by xs * ws and added into binary32 sums.
//
// 64 x 64 output tiles on the warp-level FP8 instruction, one 128-deep block
// at a time through shared memory.
#include "kernels.cuh"
#include "tc_common.cuh"

namespace w8a8 {

namespace {

constexpr int F_BT = 64, F_BN = 64, F_BK = 128;
constexpr int F_STRIDE = F_BK + 16;  // padded rows: conflict-free fragment loads
constexpr int F_THREADS = 128;

__device__ __forceinline__ void mma_e4m3(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Rows [r0, r0 + rows) of a [.., K] byte matrix, columns [k0, k0 + 128), into padded shared rows; outside: 0.
__device__ __forceinline__ void load_tile(uint8_t* s, const uint8_t* p, int64_t r0, int64_t r_end, int64_t K, int k0) {
  for (int i = threadIdx.x; i < 64 * 8; i += F_THREADS) {
    const int r = i >> 3, c = (i & 7) * 16;
    const bool in = r0 + r < r_end && k0 + c < K;
    const uint4 v = in ? *reinterpret_cast<const uint4*>(p + (r0 + r) * K + k0 + c) : make_uint4(0u, 0u, 0u, 0u);
    *reinterpret_cast<uint4*>(s + r * F_STRIDE + c) = v;
  }
}

__global__ void __launch_bounds__(F_THREADS) fp8_gemm_kernel(const Fp8GemmArgs a) {
  __shared__ __align__(16) uint8_t sx[F_BT * F_STRIDE];
  __shared__ __align__(16) uint8_t sw[F_BN * F_STRIDE];
  __shared__ int64_t s_row0, s_rows;
  __shared__ int s_bad;
  const int e = blockIdx.z;
  if (threadIdx.x == 0) {
    int64_t before = 0, sum = 0, mine = a.R;
    int bad = 0;
    if (a.group_list != nullptr) {
      for (int i = 0; i < a.E; ++i) {
        const int64_t c = a.group_list[i];
        if (c < 0 || c > a.R) bad = 1;
        if (i == e) {
          before = sum;
          mine = c;
        }
        sum += c < 0 ? 0 : c;
      }
      if (sum != a.R) bad = 1;
      if (bad && blockIdx.x == 0 && blockIdx.y == 0 && e == 0) set_status(a.status, W8A8_ERR_GROUP_LIST, 0u);
    }
    s_row0 = before;
    s_rows = mine;
    s_bad = bad;
  }
  __syncthreads();
  if (s_bad) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * F_BN;
  const int KB = static_cast<int>((a.K + 127) / 128), NB = static_cast<int>((a.N + 127) / 128);
  const int wt = (warp & 1) * 32, wn = (warp >> 1) * 32;
  const uint8_t* we = a.w + static_cast<int64_t>(e) * a.N * a.K;
  const float* wse = a.w_scale + (static_cast<int64_t>(e) * NB + n0 / 128) * KB;
  for (int64_t t0 = static_cast<int64_t>(blockIdx.y) * F_BT; t0 < s_rows; t0 += static_cast<int64_t>(gridDim.y) * F_BT) {
    float acc[2][4][4] = {};
    for (int kb = 0; kb < KB; ++kb) {
      __syncthreads();
      load_tile(sx, a.q, s_row0 + t0, s_row0 + s_rows, a.K, kb * 128);
      load_tile(sw, we, n0, a.N, a.K, kb * 128);
      __syncthreads();
      float part[2][4][4] = {};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = k * 32 + (lane & 3) * 4;
        uint32_t fa[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint8_t* p = sx + (wt + i * 16 + (lane >> 2)) * F_STRIDE + c;
          fa[i][0] = *reinterpret_cast<const uint32_t*>(p);
          fa[i][1] = *reinterpret_cast<const uint32_t*>(p + 8 * F_STRIDE);
          fa[i][2] = *reinterpret_cast<const uint32_t*>(p + 16);
          fa[i][3] = *reinterpret_cast<const uint32_t*>(p + 8 * F_STRIDE + 16);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint8_t* p = sw + (wn + j * 8 + (lane >> 2)) * F_STRIDE + c;
          const uint32_t b0 = *reinterpret_cast<const uint32_t*>(p), b1 = *reinterpret_cast<const uint32_t*>(p + 16);
#pragma unroll
          for (int i = 0; i < 2; ++i) mma_e4m3(part[i][j], fa[i], b0, b1);
        }
      }
      const float w = wse[kb];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int64_t t = t0 + wt + i * 16 + h * 8 + (lane >> 2);
          const float s = t < s_rows ? a.x_scale[(s_row0 + t) * KB + kb] * w : 0.0f;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            acc[i][j][2 * h] = fmaf(part[i][j][2 * h], s, acc[i][j][2 * h]);
            acc[i][j][2 * h + 1] = fmaf(part[i][j][2 * h + 1], s, acc[i][j][2 * h + 1]);
          }
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const int64_t t = t0 + wt + i * 16 + (h >> 1) * 8 + (lane >> 2);
          const int64_t n = n0 + wn + j * 8 + (lane & 3) * 2 + (h & 1);
          if (t < s_rows && n < a.N) {
            float v = acc[i][j][h];
            if (a.bias != nullptr) v += bf16_bits_to_f32(a.bias[n]);
            a.y[(s_row0 + t) * a.N + n] = f32_to_bf16_bits(v);
          }
        }
  }
}

}  // namespace

size_t fp8_gemm_ws_bytes(int64_t, int64_t, int64_t, int64_t, bool) { return 0; }

cudaError_t launch_fp8_gemm(const Fp8GemmArgs& a, void*, int, cudaStream_t stream) {
  if (a.R == 0) return cudaSuccess;
  const int64_t tb = a.group_list != nullptr ? std::min<int64_t>(a.R, 512) : a.R;
  const dim3 g(static_cast<unsigned>((a.N + F_BN - 1) / F_BN),
               static_cast<unsigned>(std::min<int64_t>(65535, (tb + F_BT - 1) / F_BT)), static_cast<unsigned>(a.E));
  fp8_gemm_kernel<<<g, F_THREADS, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace w8a8
