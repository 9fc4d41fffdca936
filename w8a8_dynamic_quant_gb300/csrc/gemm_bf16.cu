// gemm_bf16.cu -- bf16 x bf16 products on the 5th-generation tensor cores (tcgen05.mma.cta_group::2.kind::f16) with bias,
// activation and residual in the epilogue, dense and grouped by expert: the layers that a quantised model keeps in bf16
// (the router's projection, output projections, expert stacks that are not quantised).
//
//   y[m,n] = act(sum_k x[m,k] w[n,k] + bias[n]) (+ residual[m,n])          rounded once, to bf16 or binary32
//   swiglu:  y[m,n] = silu(gate) * up,  gate = row n of the product, up = row N + n
//
// Products of bf16 are exact in binary32; the sum over K stays in the tensor core's binary32 accumulator, bias,
// activation and residual in registers.
//
// Tile.  The weights are the MMA's M side, 256 rows per CTA pair (128 in each CTA); a block of up to NT tokens is N, in
// steps of 16: the even CTA holds the first half of the block's token rows, the odd CTA the rest.  Ragged groups pad to
// 16 rows, not to a tile.  A ring stage is 64 of K: 128 weight rows and the CTA's token rows, 128 bytes each, by TMA with
// 128-byte swizzle.  Gated: each CTA's 128 rows are 64 gate rows and the 64 up rows that belong to them, so a channel's
// two sums meet inside a CTA (through the epilogue's staging buffers) and the weights need no packing.
//
// Tensor memory (512 columns): accumulators of NT columns; the epilogue of one unit runs beside the MMAs of the next.
//
// Warp roles (320 threads, one CTA per SM):
//   warp 0      TMA producer
//   warp 1      TMEM owner; the even CTA's issues the MMAs (whole warp, one lane elected)
//   warps 2-9   epilogue: warp w reads TMEM lanes 32 * (w % 4) .. (channels) and one half of the tokens, 16 at a time:
//               activation with a channel a lane, then through shared memory to rows of 32 channels for the residual's
//               loads and the stores
//
// Work.  A unit is one tile over the whole of K, and the pairs take every C-th one, 16 token blocks beside one another
// per block of weight rows (32: x does not stay in L2, 8192 x 14336 x 4096 without a pause 608 us against 552; 8: 557).
// A dense problem of few units gives each to a cluster of 2 to 8 pairs that take parts of K; every part's sums go
// straight to the CTAs that finish a share of the tokens each (bulk copies between shared memories, one barrier a warp),
// which add them in the order of K.  One with a few more units than pairs cuts the last ones' blocks into equal runs,
// whose sums meet in the workspace.  No order of arrival changes a bit.  The host chooses tiles, parts and cuts by the
// sizes alone, from the costs at make_plan().
//
// What bounds it.  Many tokens: the tensor cores, under the power cap when called without a pause (8192 x 14336 x 4096
// with gelu_tanh 563 to 569 us at 1.5 GHz, 485 to 493 in a burst; the library's product alone 557 and 478 to 497).  Tiles of fewer than about
// 230 tokens: bringing 128 weight rows and half the token rows of a block to each SM, about 58 bytes a cycle, where the
// MMAs would take twice that at 128 tokens (1141 x 4096 x 4096: 32.5 us).  Few tokens: the weight stream (128 tokens to
// 8 of 64 experts of 4096 x 7168: 541 us, 7.0 TB/s) or, for one small layer, latency: of the 10.7 us of 64 x 2048 x 7168
// the stream takes 4.3, the way of the first tiles 1.5, the parts' meeting and the epilogue 2, launch and end 2.
// Small K: the epilogue, 3.7 us a tile of 256 tokens (5.8 with a residual).
//
// Registers: 145 to 168 of the 168 that 320 threads may have, none spilled.
//
// Every mbarrier wait is bounded (2 s): on expiry the CTA sets W8A8_ERR_DEVICE_TIMEOUT, lets in-flight copies land,
// frees TMEM and returns.
#include "fp8_common.cuh"
#include "gemm_bf16.cuh"

namespace w8a8 {

namespace {

using namespace fp8;

constexpr int B_BK = 64;       // K per stage: 128 bytes
constexpr int B_HALF = 128;    // weight rows of a tile in each CTA
constexpr int B_SUPER = 16;    // token blocks per rasterisation group (32: 10 % slower at 8192 x 14336 x 4096, 8: 1 %)
constexpr int B_THREADS = 320;
constexpr int B_EPI0 = 2;
constexpr uint32_t B_W_BYTES = B_HALF * B_BK * 2;  // 16 KB
constexpr int B_LD = 36;                           // floats a staged token row: 32 channels, and 4 against conflicts
constexpr uint32_t B_STG_FLOATS = 16 * B_LD;       // per epilogue warp

struct BArgs {
  const int64_t* group_list;
  const uint16_t* bias;
  const uint16_t* residual;
  void* y;
  DeviceStatus* status;
  int64_t R, N, K;
  int E;
  int act;
  int split;   // pairs per cluster that share a unit's K
  int cut;     // the last units' blocks in sequence are cut into equal runs, one a pair
  uint32_t* counters;  // cut: [pairs][2 CTAs][epilogue warps], zero between calls
  float* pieces;       // cut: [pairs][head, tail][2 CTAs][epilogue warp][token][32 channels]
  int blocks;  // dense: token blocks of `per` tokens each
  int per;
  int chunk;         // blocks of K that an accumulator takes before its sum is added up in binary32
  int xbig, xsmall;  // token rows of the two TMA boxes (dense: one)
  bool f32;
  bool vec;    // rows of y (and the residual) start on 16-byte boundaries
};

template <int NT>
struct BCfg {
  static constexpr uint32_t kXBytes = NT / 2 * B_BK * 2;
  static constexpr uint32_t kStageBytes = B_W_BYTES + kXBytes;
  static constexpr int kStages = NT == 256 ? 6 : NT == 128 ? 8 : NT == 64 ? 9 : 10;
  static constexpr int kAcc = NT == 128 ? 3 : 2;   // accumulators of NT columns
  static constexpr uint32_t kSumCol = NT == 256 ? NT : kAcc * NT;  // NT columns of sums over chunks of K (NT = 256: in
                                                                   // the place of the second accumulator)
  static constexpr uint32_t kTmemCols = NT >= 128 ? 512 : NT == 64 ? 256 : 128;
  static constexpr int kCols = NT / 2;             // columns read by one epilogue warp, at most
  static constexpr size_t kSmem = static_cast<size_t>(kStages) * kStageBytes + F_EPI_WARPS * B_STG_FLOATS * 4 +
                                  1024;  // and the groups' offsets
  static_assert(kSmem + (F_MAX_E + 1) * 8 + 512 <= 227 * 1024, "shared memory of a CTA");
  // Where the parts of a shared unit's K come in, [part][epilogue warp][its share of the tokens][32 channels]: the
  // ring's last stages, which a launch whose units are shared does without.
  static constexpr uint32_t kRecvBytes = (kCols + F_MAX_SPLIT) * F_EPI_WARPS * 32 * 4;
  static constexpr int kRingShared = kStages - static_cast<int>((kRecvBytes + kStageBytes - 1) / kStageBytes);
  // the parts go out from the stages that remain
  static_assert(NT > 128 || static_cast<size_t>(F_EPI_WARPS) * kCols * 32 * 4 <= static_cast<size_t>(kRingShared) * kStageBytes,
                "");
};

// Instruction descriptor: binary32 accumulator, bf16 operands, both K-major, M = 256, N = n.
__device__ __forceinline__ uint32_t idesc_bf16(int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | (256u >> 4 << 24);
}

// Two binary32 values side by side, and paired operations on them.
__device__ __forceinline__ uint64_t pk(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint64_t pk(float both) { return pk(both, both); }
__device__ __forceinline__ void upk(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// x * sigmoid(z), z2 = z * log2 e: x / (1 + t) for z >= 0 and t x / (1 + t) below, t = exp(-|z|) <= 1, so nothing
// overflows and far negative values keep what t has (down to 2^-126).
__device__ __forceinline__ float times_sigmoid(float x, float z2) {
  const float t = exp2_fast(-fabsf(z2));
  return (z2 < 0.0f ? t * x : x) * rcp_fast(1.0f + t);
}
__device__ __forceinline__ float silu(float x) { return times_sigmoid(x, x * 1.4426950408889634f); }
// (1 + tanh u) / 2 = sigmoid(2u), u = sqrt(2 / pi) (x + 0.044715 x^3)
__device__ __forceinline__ void gelu_tanh2(float& x0, float& x1) {
  const uint64_t x = pk(x0, x1), z = mul2(x, fma2(mul2(x, x), pk(0.10294324f), pk(2.3022082f)));
  float z0, z1;
  upk(z, z0, z1);
  x0 = times_sigmoid(x0, z0);
  x1 = times_sigmoid(x1, z1);
}
// x Phi(x) = max(x, 0) - |x| erfc(z) / 2, z = |x| / sqrt 2, which keeps its digits far below zero.  erfc(z) =
// t exp(-z^2 + P(t)), t = 1 / (1 + z / 2), within a relative 1.2e-7: the Chebyshev fit of Press, Teukolsky, Vetterling
// and Flannery, "Numerical Recipes in C" (1992), 6.2, here with its coefficients times log2 e and the half in the
// exponent.  |x| is cut at 2^60, where erfc is 0, so that an infinity is not multiplied by it.
__device__ __forceinline__ void gelu2(float& x0, float& x1) {
  constexpr float kL = 1.4426950408889634f;
  const float a0 = fminf(fabsf(x0), 0x1p60f), a1 = fminf(fabsf(x1), 0x1p60f);
  const uint64_t a = pk(a0, a1);
  float d0, d1;
  upk(fma2(a, pk(0.35355339059327376f), pk(1.0f)), d0, d1);
  const uint64_t t = pk(rcp_fast(d0), rcp_fast(d1));
  uint64_t p = fma2(t, pk(0.17087277f * kL), pk(-0.82215223f * kL));
  p = fma2(t, p, pk(1.48851587f * kL));
  p = fma2(t, p, pk(-1.13520398f * kL));
  p = fma2(t, p, pk(0.27886807f * kL));
  p = fma2(t, p, pk(-0.18628806f * kL));
  p = fma2(t, p, pk(0.09678418f * kL));
  p = fma2(t, p, pk(0.37409196f * kL));
  p = fma2(t, p, pk(1.00002368f * kL));
  p = fma2(t, p, pk(-1.26551223f * kL - 1.0f));
  p = fma2(mul2(a, a), pk(-0.5f * kL), p);
  float p0, p1, h0, h1;
  upk(p, p0, p1);
  upk(mul2(mul2(t, pk(exp2_fast(p0), exp2_fast(p1))), a), h0, h1);
  float m0, m1;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m0) : "f"(x0), "f"(0.0f));
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m1) : "f"(x1), "f"(0.0f));
  x0 = m0 - h0;
  x1 = m1 - h1;
}
template <int N>
__device__ __forceinline__ void activate(float (&v)[N], int act) {
  switch (act) {
    case W8A8_ACT_RELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = v[i] < 0.0f ? 0.0f : v[i];  // a NaN stays
      break;
    case W8A8_ACT_SILU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = silu(v[i]);
      break;
    case W8A8_ACT_GELU:
#pragma unroll
      for (int i = 0; i < N; i += 2) gelu2(v[i], v[i + 1]);
      break;
    case W8A8_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < N; i += 2) gelu_tanh2(v[i], v[i + 1]);
      break;
    default: break;
  }
}

// Wait of a whole converged warp, bounded as wait_all; a probe sleeps in hardware for up to 20 us before it comes back:
// a role that waits for a whole tile, polled without the hint, costs power that the tensor cores then lack (8192 x 14336
// x 4096 without a pause: 3 %).
__device__ __forceinline__ bool probe(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(20000u)
      : "memory");
  return ok != 0u;
}
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int* abort_flag, DeviceStatus* st,
                                         uint32_t where) {
  if (__all_sync(0xffffffffu, probe(bar, parity))) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!__all_sync(0xffffffffu, probe(bar, parity))) {
    const bool late = globaltimer_ns() - t0 > kWaitLimitNs;
    if (__any_sync(0xffffffffu, late || *abort_flag)) {
      if ((threadIdx.x & 31) == 0 && !*abort_flag) {
        *abort_flag = 1;
        set_status(st, W8A8_ERR_DEVICE_TIMEOUT, where);
      }
      return false;
    }
  }
  return true;
}

// 16 columns of the warp's lanes to tensor memory.
__device__ __forceinline__ void tmem_store(uint32_t taddr, const float (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
      "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
      : "memory");
}

// The cluster's CTAs meet.  Relaxed: no data rides on it (barriers' initialisation has its own fence, and what a CTA
// stored for others to read in global memory is complete when the grid is), so nobody waits for stores on their way.
// What a CTA sends to a barrier or the shared memory of another one has been waited for there before they leave.
__device__ __forceinline__ void cluster_meet() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Shared memory of this CTA to that of a CTA of the cluster, whose barrier counts the bytes (cluster-window addresses).
__device__ __forceinline__ void copy_to_peer(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "r"(src),
      "r"(bytes), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// One unit of work: the tile and its K range.
struct Unit {
  int e, wb;   // expert, block of weight rows
  int row0;    // first token row (of all R)
  int tvalid;  // tokens
  int n;       // tokens rounded up to 16
};

// The segments of one pair, blocks [kb0, kb1) of a unit each.  Every role walks them on its own.
template <bool CUT>
struct Segments;
// Every step-th unit, whole or the pair's part of it: the same blocks of each (kb0 and kb1 stay as they are).
template <>
struct Segments<false> {
  int unit, units, step;
};
// Whole units, then a run of blocks.
template <>
struct Segments<true> {
  Walk units, run;
};
__device__ __forceinline__ bool next_segment(Segments<false>& w, int& unit, int&, int&) {
  unit = w.unit;
  w.unit += w.step;
  return unit < w.units;
}
__device__ __forceinline__ bool next_segment(Segments<true>& w, int& unit, int& kb0, int& kb1) {
  int u = 0, k0 = 0, k1 = 0;
  const bool more = next_unit(w.units, u, k0, k1) || next_unit(w.run, u, k0, k1);
  unit = uni(u);
  kb0 = uni(k0);
  kb1 = uni(k1);
  return uni(more);
}

// The barrier of an epilogue warp that holds gate rows and of the one that holds the up rows of the same channels and
// tokens; the AND of what they bring.
__device__ __forceinline__ void pair_sync(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool pair_and(int id, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %2, 0;\n barrier.cta.red.and.pred q, %1, 64, p;\n"
      " selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(id), "r"(static_cast<uint32_t>(ok))
      : "memory");
  return r != 0u;
}

// An epilogue warp's place: what it stages, reads back and stores.
struct Place {
  float* stg;         // its staging buffer
  const float* gate;  // gated: those of the two warps of its channels
  const float* up;
  int q, h, lane;
  int r0, c;          // the first token and channel of 16 x 32 that the lane stores
  int bar;            // gated: the two warps' barrier
};

// The residual's values that finish() adds, asked for one step ahead.
template <bool GATED>
struct Residual {
  static constexpr int kSlots = GATED ? 1 : 2;  // rows a lane stores
  uint4 v[kSlots];
};
// (at: as in finish())
template <bool GATED>
__device__ __forceinline__ void fetch_residual(const BArgs& a, const Place& p, Residual<GATED>& res, int64_t at, int rows,
                                               int ncols) {
  if (a.residual == nullptr || !a.vec) return;
#pragma unroll
  for (int i = 0; i < Residual<GATED>::kSlots; ++i)
    if (p.r0 + 8 * i < rows && p.c < ncols) res.v[i] = *reinterpret_cast<const uint4*>(a.residual + at + 8 * i * a.N);
}

// 16 tokens x 32 channels: v[i] is this lane's channel of token i.  `rows` of the tokens and ncols of the channels exist;
// at: where the value of token r0 at channel c, the lane's first one to store, stands in y and in the residual.
template <bool GATED>
__device__ __forceinline__ void finish(const BArgs& a, const Place& p, float (&v)[16], float bias,
                                       const Residual<GATED>& res, int64_t at, int rows, int ncols) {
  constexpr int kSlots = Residual<GATED>::kSlots;
  const int lane = p.lane, c = p.c, r0 = p.r0;
  const bool add = a.residual != nullptr;
  if (a.bias != nullptr) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] += bias;
  }
  if constexpr (!GATED) activate(v, a.act);
#pragma unroll
  for (int i = 0; i < 16; ++i) p.stg[i * B_LD + lane] = v[i];
  if constexpr (GATED) pair_sync(p.bar);
  else __syncwarp();
  if (a.vec) {
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      const int r = r0 + 8 * i;
      if (r < rows && c < ncols) {
        float o[8];
        const float* s = (GATED ? p.gate : p.stg) + r * B_LD + c;
        const float4 s0 = *reinterpret_cast<const float4*>(s), s1 = *reinterpret_cast<const float4*>(s + 4);
        o[0] = s0.x; o[1] = s0.y; o[2] = s0.z; o[3] = s0.w;
        o[4] = s1.x; o[5] = s1.y; o[6] = s1.z; o[7] = s1.w;
        if constexpr (GATED) {
          const float* t = p.up + r * B_LD + c;
          const float4 t0 = *reinterpret_cast<const float4*>(t), t1 = *reinterpret_cast<const float4*>(t + 4);
          const float u[8] = {t0.x, t0.y, t0.z, t0.w, t1.x, t1.y, t1.z, t1.w};
#pragma unroll
          for (int k = 0; k < 8; ++k) o[k] = silu(o[k]) * u[k];
        }
        if (add) {
          const uint32_t w[4] = {res.v[i].x, res.v[i].y, res.v[i].z, res.v[i].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            o[2 * k] += __uint_as_float(w[k] << 16);
            o[2 * k + 1] += __uint_as_float(w[k] & 0xffff0000u);
          }
        }
        const int64_t to = at + 8 * i * a.N;
        if (a.f32) {
          float4* d = reinterpret_cast<float4*>(static_cast<float*>(a.y) + to);
          d[0] = make_float4(o[0], o[1], o[2], o[3]);
          d[1] = make_float4(o[4], o[5], o[6], o[7]);
        } else {
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.y) + to) =
              make_uint4(f32x2_to_bf16x2_bits(o[0], o[1]), f32x2_to_bf16x2_bits(o[2], o[3]),
                         f32x2_to_bf16x2_bits(o[4], o[5]), f32x2_to_bf16x2_bits(o[6], o[7]));
        }
      }
    }
  } else {  // rows of y start anywhere: a channel a lane, eight rows' residuals on their way at once
    const int64_t first = at - r0 * a.N - c + lane;  // token 0, the lane's channel
#pragma unroll 1
    for (int r = GATED ? 8 * (p.q >> 1) : 0, i = 0; i < kSlots; r += 8, ++i) {
      const int64_t to = first + r * a.N;
      float o[8];
      if (add) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          o[k] = r + k < rows && lane < ncols ? bf16_bits_to_f32(a.residual[to + k * a.N]) : 0.0f;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        float u = (GATED ? p.gate : p.stg)[(r + k) * B_LD + lane];
        if constexpr (GATED) u = silu(u) * p.up[(r + k) * B_LD + lane];
        if (add) u += o[k];
        if (r + k < rows && lane < ncols) {
          if (a.f32) static_cast<float*>(a.y)[to + k * a.N] = u;
          else static_cast<uint16_t*>(a.y)[to + k * a.N] = f32_to_bf16_bits(u);
        }
      }
    }
  }
  if constexpr (GATED) pair_sync(p.bar);
  else __syncwarp();
}

// A cut unit's counter (one per epilogue warp, gated: per pair of warps): 1 the tail's sums are in the workspace, 2 the
// head's.  seen(): whether it reads `what`.  arrive(): the warp's sums are written; adds `what` and says whether the
// other's were there already, in which case it is back at zero.  The two warps of a gated pair decide together.
template <bool GATED>
__device__ __forceinline__ bool agreed(const Place& p, uint32_t answer) {
  answer = __shfl_sync(0xffffffffu, answer, 0);
  if constexpr (GATED) return pair_and(p.bar, p.q >= 2 || answer != 0u);
  return answer != 0u;
}
template <bool GATED>
__device__ __forceinline__ bool seen(const BArgs& a, const Place& p, int key, int lane, uint32_t what) {
  uint32_t v = 0;
  if (lane == 0 && (!GATED || p.q < 2))
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(a.counters + key) : "memory");
  const bool yes = agreed<GATED>(p, v == what);
  if (yes) __threadfence();
  return yes;
}
template <bool GATED>
__device__ __forceinline__ bool arrive(const BArgs& a, const Place& p, int key, int lane, uint32_t what) {
  __threadfence();
  if constexpr (GATED) pair_sync(p.bar);
  else __syncwarp();
  uint32_t before = 0;
  if (lane == 0 && (!GATED || p.q < 2)) {
    before = atomicAdd(a.counters + key, what);
    if (before != 0u) a.counters[key] = 0u;
  }
  const bool last = agreed<GATED>(p, before != 0u);
  if (last) __threadfence();
  return last;
}

// CUT: the last units' K is cut over all pairs.  (A kernel of its own: the code that joins the pieces costs every other
// launch about 1 us and the large ones up to 8 %.)
template <int NT, bool GATED, bool CUT>
__global__ void __launch_bounds__(B_THREADS, 1)
bf16_gemm_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmXbig,
                 const __grid_constant__ CUtensorMap tmXsmall, const BArgs a) {
  using C = BCfg<NT>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bar_full[C::kStages];   // even CTA: both CTAs' tiles of the stage landed
  __shared__ __align__(8) uint64_t bar_empty[C::kStages];  // the MMAs reading the stage are done
  __shared__ __align__(8) uint64_t bar_accf[C::kAcc];      // the unit's accumulator is complete
  __shared__ __align__(8) uint64_t bar_acce[C::kAcc];      // even CTA: both CTAs read it
  __shared__ uint32_t s_tmem_base;
  __shared__ volatile int s_abort;
  __shared__ int s_bad;
  __shared__ __align__(8) uint64_t bar_alloc;              // even CTA: both CTAs hold their tensor memory
  __shared__ __align__(8) uint64_t bar_recv[F_EPI_WARPS];  // the parts' sums for the warp are there
  __shared__ int s_warp[B_THREADS / 32];
  __shared__ unsigned long long s_rows;  // the counts' sum where 32 bits may not hold it

  const int tid = threadIdx.x;
  const int warp = uni(tid >> 5);
  const int lane = tid & 31;
  const int E = a.E;
  const int KB = static_cast<int>((a.K + B_BK - 1) / B_BK);
  constexpr int kRows = GATED ? 128 : 256;  // channels of y per tile
  const int WB = static_cast<int>((a.N + kRows - 1) / kRows);
  const bool grouped = a.group_list != nullptr;

  uint8_t* stages = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t stage_base = smem_u32(stages);
  float* s_part = reinterpret_cast<float*>(stages);  // [epilogue warp][token][channel], after the last block
  float* s_stg = reinterpret_cast<float*>(stages + C::kStages * C::kStageBytes);
  const int nstages = a.split > 1 && NT <= 128 ? C::kRingShared : C::kStages;
  float* s_recv = reinterpret_cast<float*>(stages + (NT <= 128 ? C::kRingShared : 0) * C::kStageBytes);
  int* s_prefix = reinterpret_cast<int*>(s_stg + F_EPI_WARPS * B_STG_FLOATS);  // [E + 1]
  int* s_off = s_prefix + E + 1;                                               // [E + 1]
  // CTAs 2i and 2i + 1 of a cluster are a pair; rank: the CTA's place in it
  uint32_t crank, cluster_id, nclusters;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(crank));
  asm volatile("mov.u32 %0, %%clusterid.x;" : "=r"(cluster_id));
  asm volatile("mov.u32 %0, %%nclusterid.x;" : "=r"(nclusters));
  const uint32_t rank = crank & 1u, even = crank & ~1u;
  const uint16_t pair_mask = static_cast<uint16_t>(3u << even);

  if (tid == 0) {
    s_abort = 0;
    s_bad = 0;
    s_rows = 0ull;
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(smem_u32(&bar_full[s]), 1);
      mbar_init(smem_u32(&bar_empty[s]), 1);
    }
    for (int b = 0; b < C::kAcc; ++b) {
      mbar_init(smem_u32(&bar_accf[b]), 1);
      mbar_init(smem_u32(&bar_acce[b]), 2 * F_EPI_WARPS);
    }
    mbar_init(smem_u32(&bar_alloc), 2);
    for (int w = 0; w < F_EPI_WARPS; ++w) mbar_init(smem_u32(&bar_recv[w]), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmXbig);
    if (grouped) tma_prefetch_desc(&tmXsmall);
  }
  int units = 0, rows_total = 0;
  const int dense_blocks = a.blocks;
  auto blocks_of = [grouped, dense_blocks](int cnt) { return grouped ? (cnt + NT - 1) / NT : dense_blocks; };
  auto scan = [&] {
    rows_total = scan_checked<B_THREADS>(
        a, [WB, blocks_of](int c) { return blocks_of(c) * WB; }, s_off, s_prefix, s_warp, &s_bad, &s_rows, &units);
  };
  if (!grouped) scan();  // reads nothing from memory
  __syncthreads();
  pdl_trigger();
  cluster_meet();  // the CTAs' barriers exist before any touches another's
  const int part = static_cast<int>(crank >> 1), me = static_cast<int>(cluster_id);
  const int chunk = a.chunk;
  const int nacc = NT == 256 && chunk < KB ? 1 : C::kAcc;
  const int part0 = KB * part / a.split, part1 = KB * (part + 1) / a.split;  // the pair's part of K (split 1: all of it)
  // Whole units, every C-th one; or the pair's part of its cluster's unit; CUT: whole units, then the pair's run of the
  // blocks of the last C to 2 C units, which ends and begins inside units.
  auto start = [&] {
    Segments<CUT> w;
    const int C = static_cast<int>(nclusters);
    if constexpr (CUT) {
      const int64_t whole = static_cast<int64_t>(units / C - 1) * C, rest = (units - whole) * KB;
      w.units = Walk{me, whole, C, KB};
      w.run = Walk{whole * KB + run_begin(rest, C, me), whole * KB + run_begin(rest, C, me + 1), 0, KB};
    } else {
      w = Segments<CUT>{me, units, C};
    }
    return w;
  };
  auto unit_of = [&](int unit) {
    Unit u;
    int tb, cnt, TB;
    unit_tile<B_SUPER>(unit, E, WB, s_prefix, s_off, blocks_of, u.e, u.wb, tb, cnt, TB);
    const int per = grouped ? ((cnt + TB - 1) / TB + 15) & ~15 : a.per;  // tokens split evenly over the blocks
    u.row0 = s_off[u.e] + tb * per;
    u.tvalid = min(per, cnt - tb * per);
    u.n = (u.tvalid + 15) & ~15;
    return u;
  };

  // rows of the weight that the CTA reads for a unit: from w_row (gated: the gate's, the up projection's N further on)
  auto w_row = [&](const Unit& u) {
    return static_cast<int>(GATED ? static_cast<int64_t>(u.e) * 2 * a.N + static_cast<int64_t>(u.wb) * 128 + rank * 64
                                  : static_cast<int64_t>(u.e) * a.N + static_cast<int64_t>(u.wb) * 256 + rank * 128);
  };
  Unit u0 = {};  // the first unit, worked out while the kernel in front still runs
  int first = -1;
  auto begin = [&] {
    Segments<CUT> w = start();
    int k0, k1;
    if (next_segment(w, first, k0, k1)) u0 = unit_of(first);
  };
  if (!grouped) begin();
  // Each role waits for the kernel in front at its first access to memory: what is before it in the code, and the
  // code's own way into the instruction cache, is behind it then.
  if (grouped) {
    pdl_wait();
    scan();
    __syncthreads();
    if (bad_list(a, rows_total, s_bad, s_rows)) {
      if (tid == 0 && blockIdx.x == 0) set_status(a.status, W8A8_ERR_GROUP_LIST, 0u);
      units = 0;
    }
    begin();
  }
  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer (both CTAs)
    const uint32_t full_even0 = smem_cluster_addr(smem_u32(&bar_full[0]), even);
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    const int xbig = uni(a.xbig), xsmall = uni(a.xsmall);
    Segments<CUT> w = start();
    int unit = 0, kb0 = part0, kb1 = part1;
    while (ok && next_segment(w, unit, kb0, kb1)) {
      const Unit u = unit == first ? u0 : unit_of(unit);
      const int yw = uni(w_row(u)), yu = uni(yw + static_cast<int>(a.N));
      const int rows = u.n >> 1;
      const int small = (rows + xsmall - 1) / xsmall;  // loads of the small box that the rows would take
      const bool few = uni(grouped && small <= 3 && rows < xbig);
      const int loads = few ? uni(small) : 1;
      const int box = few ? xsmall : xbig;
      const CUtensorMap* tmX = few ? &tmXsmall : &tmXbig;
      const int yx = uni(u.row0 + static_cast<int>(rank) * rows);
      const uint32_t bytes = 2u * B_W_BYTES + static_cast<uint32_t>(2 * loads * box) * (B_BK * 2);
      if (unit == first) pdl_wait();
      for (int kb = kb0; kb < kb1; ++kb) {
        ok = wait_for(smem_u32(&bar_empty[stage]), phase ^ 1u, &s_abort, a.status, 1u);
        if (!ok) break;
        if (rank == 0) expect_tx_elect(smem_u32(&bar_full[0]) + 8 * stage, bytes);
        const uint32_t full = full_even0 + 8 * stage;
        const uint32_t dst = stage_base + stage * C::kStageBytes;
        tma_pair_elect(dst, &tmW, kb * B_BK, yw, full);
        if constexpr (GATED) tma_pair_elect(dst + B_W_BYTES / 2, &tmW, kb * B_BK, yu, full);
        for (int i = 0; i < loads; ++i)
          tma_pair_elect(dst + B_W_BYTES + i * box * (B_BK * 2), tmX, kb * B_BK, yx + i * box, full);
        if (++stage == nstages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // Drain: the last fill of every stage has been consumed, so no copy into this CTA and no MMA arrival on its
    // barriers is still in flight when the cluster leaves.
    for (int i = 0; i < nstages && ok; ++i) {
      ok = wait_for(smem_u32(&bar_empty[stage]), phase ^ 1u, &s_abort, a.status, 5u);
      if (++stage == nstages) {
        stage = 0;
        phase ^= 1u;
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------- TMEM owner; MMA issuer (even CTA, whole warp)
    // Tensor memory is asked for after the wait: a kernel in front that has not got its own yet is never waited for by
    // a CTA that holds some.
    pdl_wait();
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem_base)),
                 "r"(C::kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    tc_fence_before();
    __syncwarp();
    asm volatile("bar.arrive 15, 288;" ::: "memory");  // the epilogue warps of this CTA
    if (lane == 0)
      asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                       smem_cluster_addr(smem_u32(&bar_alloc), even))
                   : "memory");
    __syncwarp();
    tc_fence_after();
    if (rank == 0) {
      const uint32_t tmem_base = static_cast<uint32_t>(uni(static_cast<int>(s_tmem_base)));
      int stage = 0, buf = 0;
      uint32_t phase = 0, bphase = 0;
      bool ok = wait_for(smem_u32(&bar_alloc), 0u, &s_abort, a.status, 7u);
      Segments<CUT> w = start();
      int unit = 0, kb0 = part0, kb1 = part1;
      while (ok && next_segment(w, unit, kb0, kb1)) {
        const uint32_t idesc = idesc_bf16(uni((unit == first ? u0 : unit_of(unit)).n));
        for (int c0 = kb0; ok && c0 < kb1; c0 += chunk) {
          ok = wait_for(smem_u32(&bar_acce[buf]), bphase ^ 1u, &s_abort, a.status, 2u);
          if (!ok) break;
          const uint32_t acc = tmem_base + buf * NT;
          const int c1 = min(kb1, c0 + chunk);
          for (int kb = c0; kb < c1; ++kb) {
            ok = wait_for(smem_u32(&bar_full[stage]), phase, &s_abort, a.status, 3u);
            if (!ok) break;
            tc_fence_after();
            const uint32_t sa = stage_base + stage * C::kStageBytes;
            const uint64_t adesc = smem_desc_sw128(sa);
            const uint64_t bdesc = smem_desc_sw128(sa + B_W_BYTES);
#pragma unroll
            for (int k = 0; k < B_BK / 16; ++k)
              tc_mma_pair(acc, adesc + 2u * k, bdesc + 2u * k, idesc, kb > c0 || k > 0 ? 1u : 0u);
            tc_commit_pair_mc(smem_u32(&bar_empty[stage]), pair_mask);  // frees the stage in both CTAs
            if (++stage == nstages) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (!ok) break;
          tc_commit_pair_mc(smem_u32(&bar_accf[buf]), pair_mask);
          if (++buf == nacc) {
            buf = 0;
            bphase ^= 1u;
          }
        }
      }
      // Drain: the odd CTA's last arrivals on this CTA's barriers have come, so none is in flight when the pair leaves.
      for (int i = 0; i < nacc && ok; ++i) {
        ok = wait_for(smem_u32(&bar_acce[buf]), bphase ^ 1u, &s_abort, a.status, 9u);
        if (++buf == nacc) {
          buf = 0;
          bphase ^= 1u;
        }
      }
    }
  }

  // ------------------------------------------------------------------ epilogue (both CTAs)
  Place p;
  const int ew = warp - B_EPI0;
  p.q = warp & 3;
  p.h = ew >> 2;
  p.lane = lane;
  p.bar = 1 + (p.q & 1) + 2 * p.h;
  p.r0 = (lane >> 2) + (GATED ? 8 * (p.q >> 1) : 0);
  p.c = (lane & 3) * 8;
  {
    float* mine = s_stg + (p.h * 4 + p.q) * B_STG_FLOATS;
    p.stg = mine;
    p.gate = mine - (p.q >> 1) * 2 * B_STG_FLOATS;
    p.up = p.gate + 2 * B_STG_FLOATS;
  }
  // channels of the warp in a tile (gated: the same ones for the two warps of a pair), and its bias row
  const int c_tile = GATED ? static_cast<int>(rank) * 64 + 32 * (p.q & 1) : static_cast<int>(rank) * B_HALF + 32 * p.q;
  auto bias_of = [&](const Unit& u, int64_t n0) {
    if (a.bias == nullptr || n0 + lane >= a.N) return 0.0f;
    const int64_t w_rows = GATED ? 2 * a.N : a.N;
    return bf16_bits_to_f32(a.bias[u.e * w_rows + (GATED && p.q >= 2 ? a.N : 0) + n0 + lane]);
  };
  if (warp >= B_EPI0) {
    pdl_wait();
    asm volatile("bar.sync 15, 288;" ::: "memory");
    tc_fence_after();
    const uint32_t tmem_base = static_cast<uint32_t>(uni(static_cast<int>(s_tmem_base)));
    const uint32_t lane_addr = tmem_base + (static_cast<uint32_t>(32 * p.q) << 16);
    const uint32_t acce_even = smem_cluster_addr(smem_u32(&bar_acce[0]), even);
    int buf = 0;
    uint32_t bphase = 0;
    Segments<CUT> w = start();
    int unit = 0, kb0 = part0, kb1 = part1;
    while (next_segment(w, unit, kb0, kb1)) {
      const Unit u = unit == first ? u0 : unit_of(unit);
      // the first half's warps read tokens [0, cut), the second's [cut, n)
      const int n = uni(u.n);
      const int cut = ((n >> 1) + 15) & ~15;
      const int c0 = p.h == 0 ? 0 : cut;
      const int cols = p.h == 0 ? cut : n - cut;
      const int tv = uni(min(cols, u.tvalid - c0));  // tokens of this warp that exist (may be <= 0)
      const int64_t n0 = static_cast<int64_t>(u.wb) * kRows + c_tile;
      const int ncols = static_cast<int>(min(static_cast<int64_t>(32), a.N - n0));  // (may be <= 0)
      const bool works = uni(tv > 0 && ncols > 0);
      const float bias = works ? bias_of(u, n0) : 0.0f;
      const int64_t row0 = static_cast<int64_t>(u.row0) + c0;
      Residual<GATED> res;
      // the tokens that the warp finishes: all of its own, or its part's share of them
      int t0 = 0, t1 = tv;
      if (a.split > 1) {
        t0 = uni(max(tv, 0) * part / a.split);
        t1 = uni(max(tv, 0) * (part + 1) / a.split);
      }
      const int64_t at0 = (row0 + p.r0) * a.N + n0 + p.c;
      if (works && t0 < t1) {
        if (a.residual != nullptr && a.vec)  // the rest of the tile's rows come as far as L2
          for (int t = t0 + 16 + lane; t < t1; t += 32) prefetch_l2(a.residual + (row0 + t) * a.N + n0);
        fetch_residual(a, p, res, at0 + t0 * a.N, min(16, t1 - t0), ncols);
      }
      // where this lane's share of the warp's sums goes: CTA 2 lane + rank of the cluster
      int cap = 0;  // tokens of a share, at most
      uint32_t send = 0, send_to = 0, send_from = 0, send_bar = 0;
      if (NT <= 128 && a.split > 1) cap = (C::kCols + a.split - 1) / a.split;
      if (NT <= 128 && a.split > 1 && works && lane < a.split) {
        const int from = tv * lane / a.split;
        send = static_cast<uint32_t>(tv * (lane + 1) / a.split - from) * 128u;
        send_from = smem_u32(s_part + (ew * C::kCols + from) * 32);
        send_to = smem_cluster_addr(smem_u32(s_recv + (part * F_EPI_WARPS + ew) * cap * 32), 2 * lane + rank);
        send_bar = smem_cluster_addr(smem_u32(&bar_recv[ew]), 2 * lane + rank);
      }
      float* part_at = s_part + ew * C::kCols * 32 + lane;
      // A cut unit's head (its first blocks, the end of this run) and tail (the beginning of the next pair's) are joined
      // by whichever comes last, as a rule the head: it finds the tail's sums in the workspace and adds them to its own.
      const bool head = CUT && kb1 < KB, tail = CUT && kb0 > 0;
      const int key = ((tail ? me - 1 : me) * 2 + static_cast<int>(rank)) * F_EPI_WARPS + (GATED ? (p.h * 4 + (p.q & 1)) : ew);
      auto piece = [&](bool of_tail) {
        return a.pieces + ((((static_cast<int64_t>(tail ? me - 1 : me) * 2 + (of_tail ? 1 : 0)) * 2 + rank) * F_EPI_WARPS + ew) *
                           C::kCols) * 32 + lane;
      };
      bool joined = CUT && head && works && seen<GATED>(a, p, key, lane, 1u);  // the tail was there
      float other[16];  // its sums, a step ahead of their use
      auto fetch_other = [&](int t) {
        const float* from = piece(true) + t * 32;
#pragma unroll
        for (int i = 0; i < 16; ++i) other[i] = __ldcg(from + i * 32);
      };
      if (joined) fetch_other(0);
      // The sums over chunks of K: columns of its own for each half (c0 = 0 is the first), whatever n is.  The other half may
      // be at a unit of another n, whose halves meet elsewhere.
      const uint32_t sum_at = lane_addr + (c0 != 0 ? C::kSumCol + C::kCols : C::kSumCol);
      bool ok = true;
      for (int k0 = kb0; k0 < kb1; k0 += chunk) {
        ok = wait_for(smem_u32(&bar_accf[buf]), bphase, &s_abort, a.status, 4u);
        if constexpr (GATED) ok = pair_and(p.bar, ok);  // the two warps of a pair give up together
        if (!ok) break;
        tc_fence_after();
        const uint32_t here = lane_addr + buf * NT + c0, release = acce_even + 8u * buf;
        if (++buf == nacc) {
          buf = 0;
          bphase ^= 1u;
        }
        if (!works) {
          tc_fence_before();
          arrive_lane0(release, lane);
          continue;
        }
        const bool more = k0 > kb0, last = k0 + chunk >= kb1;
        if (CUT && last && head && !joined) {
          joined = seen<GATED>(a, p, key, lane, 1u);
          if (joined) fetch_other(0);
        }
        for (int t = 0; t < tv; t += 16) {
          uint32_t r[16], s[16];
          tmem_fetch(here + t, r);
          if (more) tmem_fetch(sum_at + t, s);
          tmem_ready(r);
          if (t + 16 >= tv) {
            tc_fence_before();
            arrive_lane0(release, lane);
          }
          float v[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
          if (more) {
            tmem_ready(s);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] += __uint_as_float(s[i]);
          }
          if (!last) {
            tmem_store(sum_at + t, v);
          } else if (a.split > 1) {  // a part of K of the cluster's unit: its sums to the ring, which is at rest
#pragma unroll
            for (int i = 0; i < 16; ++i) part_at[(t + i) * 32] = v[i];
          } else if (CUT && ((head && !joined) || tail)) {
            float* to = piece(tail) + t * 32;
#pragma unroll
            for (int i = 0; i < 16; ++i) __stcg(to + i * 32, v[i]);
          } else {
            if (CUT && joined) {
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] += other[i];
              if (t + 16 < tv) fetch_other(t + 16);
            }
            Residual<GATED> next;
            if (t + 16 < tv) fetch_residual(a, p, next, at0 + (t + 16) * a.N, min(16, tv - t - 16), ncols);
            finish<GATED>(a, p, v, bias, res, at0 + t * a.N, min(16, tv - t), ncols);
            res = next;
          }
        }
        if (!last) tmem_wait_st();
      }
      if (!ok) break;
      if (CUT && works && (head || tail)) {
        if (joined) {
          if (lane == 0 && (!GATED || p.q < 2)) a.counters[key] = 0u;
        } else if (arrive<GATED>(a, p, key, lane, tail ? 1u : 2u)) {
          // the other one came while this one's sums were written: both are in the workspace
          fetch_residual(a, p, res, at0, min(16, tv), ncols);
          for (int t = 0; t < tv; t += 16) {
            const float* h = piece(false) + t * 32;
            const float* l = piece(true) + t * 32;
            float v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __ldcg(h + i * 32) + __ldcg(l + i * 32);
            if (t > 0) fetch_residual(a, p, res, at0 + t * a.N, min(16, tv - t), ncols);
            finish<GATED>(a, p, v, bias, res, at0 + t * a.N, min(16, tv - t), ncols);
          }
        }
      }
      if constexpr (NT <= 128) {
        if (a.split > 1 && works) {
          // the parts' sums meet: each goes out to the CTAs that add a share of the tokens each, in the order of K
          const uint32_t bar = smem_u32(&bar_recv[ew]);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (send != 0u) copy_to_peer(send_to, send_from, send, send_bar);
          __syncwarp();
          if (t0 < t1) {
            expect_tx_elect(bar, static_cast<uint32_t>(a.split * (t1 - t0)) * 128u);
            ok = wait_for(bar, 0u, &s_abort, a.status, 6u);
          }
          if constexpr (GATED) ok = pair_and(p.bar, ok);
          if (!ok) break;
          const float* in = s_recv + ew * cap * 32 + lane;
          for (int t = t0; t < t1; t += 16) {
            float v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = 0.0f;
            const float* at = in + (t - t0) * 32;
            for (int j = 0; j < a.split; ++j, at += F_EPI_WARPS * cap * 32) {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (t + i < t1) v[i] += at[i * 32];
              if (t + 8 < t1) {
#pragma unroll
                for (int i = 8; i < 16; ++i)
                  if (t + i < t1) v[i] += at[i * 32];
              }
            }
            if (t > t0) fetch_residual(a, p, res, at0 + t * a.N, min(16, t1 - t), ncols);
            finish<GATED>(a, p, v, bias, res, at0 + t * a.N, min(16, t1 - t), ncols);
          }
        }
      }
    }
  }

  // ---- teardown: on abort, give in-flight copies and MMAs time to land first, then the pair leaves together.
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (s_abort) {
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 20000000ull) {
    }
  }
  cluster_meet();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(s_tmem_base), "r"(C::kTmemCols)
                 : "memory");
  }
}

using BPlan = decltype(Bf16GemmArgs::plan);
constexpr int round16(int64_t n) { return static_cast<int>((n + 15) & ~int64_t(15)); }

// Cycles of one 64-deep block of a tile of n tokens: the tensor core's (four MMAs of n / 2, at least 40), or bringing
// 128 weight rows and n / 2 token rows of 128 bytes to a SM at about 58 bytes a cycle.  (The memory's rate is not in it: it
// bounds few tokens' products alike whichever way they are tiled.)
constexpr int64_t block_cost(int n) { return std::max(2 * n, (128 + n / 2) * 128 / 58); }

// The accumulator's columns for blocks of `per` tokens.
constexpr int tile_of(int per) { return per <= 32 ? 32 : per <= 64 ? 64 : per <= 128 ? 128 : 256; }

// Scratch of cut units: the counters, and two pieces a pair, [2 CTAs][128 channels][tile tokens] binary32 each.
constexpr size_t cut_bytes(int pairs, int nt) { return kBf16CounterBytes + static_cast<size_t>(pairs) * 4 * B_HALF * nt * 4; }
static_assert(kBf16CounterBytes == kCounterBytes, "[pairs][2 CTAs][epilogue warps]");

BPlan make_plan(int64_t E, int64_t R, int64_t channel_blocks, int64_t K, bool grouped) {
  BPlan p{256, 0, 0, 1, F_MAX_CLUSTERS, 0};
  if (grouped) {
    // Twice the mean rows of a group: the host knows no more of the list.  Each group's weights are read once a tile of its
    // rows.  64 experts of 2 x 2048 x 4096, top-8 by a zipf rule, tiles of 32 / 64 / 128 / 256 in us: 256 tokens (mean 32,
    // most 243) 382 / 337 / 326 / 328, 1024 tokens (128, 963) 913 / 575 / 420 / 359, 4096 (512, 3814) 3309 / 1781 / 1046 /
    // 741.  128 tokens alike (mean 16), 2 x 2048 x 7168: 541 / 544 / 550 / 566.  It is wrong where one expert has nearly all
    // rows: 1024 of 1024 in one of 64, 4096 x 4096: 100 / 60 / 34 / 27.
    const int64_t want = 2 * ((R + E - 1) / E);
    p.nt = want <= 32 ? 32 : want <= 64 ? 64 : want <= 128 ? 128 : 256;
    return p;
  }
  const int64_t KB = (K + B_BK - 1) / B_BK;
  // clusters of 2 ks CTAs (one a SM) that are resident at once on 152 SMs, as the occupancy query gives them
  constexpr int kFit[F_MAX_SPLIT + 1] = {0, 76, 36, 23, 15, 13, 8, 7, 7};
  int64_t best = INT64_MAX;
  const int widest = static_cast<int>(std::min<int64_t>(256, round16(R)));
  for (int per = widest; per >= 16; per -= 16) {
    const int64_t blocks = (R + per - 1) / per;
    const int64_t units = blocks * channel_blocks;
    auto take = [&](int64_t cost, int ks, int cut) {
      if (cost >= best) return;
      best = cost;
      p.per = per;
      p.blocks = static_cast<int>(blocks);
      p.split = ks;
      p.cut = cut;
      p.pairs = static_cast<int>(ks > 1 ? units * ks : std::min<int64_t>(units, F_MAX_CLUSTERS));
      p.nt = tile_of(per);
    };
    const int64_t waves = (units + F_MAX_CLUSTERS - 1) / F_MAX_CLUSTERS;
    take(waves * (KB * block_cost(per) + 300) + 8 * per, 1, 0);
    // Whole units in `waves` rounds, or as many blocks a pair.  The cut units' sums go through the workspace, and pairs
    // that are not at the same block of K at the same time share fewer of their reads in L2: about 3 us at 16 tokens a
    // tile, 10 at 128, 19 at 256 (64 x 20480 x 7168, 80 units: 69.0 us whole, 50.0 cut; 2483 x 2048 x 7168: 59.4 and
    // 50.4; 4096 x 4096 x 4096: 80.1 and 87.1).
    if (units > F_MAX_CLUSTERS && units < 4 * F_MAX_CLUSTERS && units % F_MAX_CLUSTERS != 0)
      take((units * KB + F_MAX_CLUSTERS - 1) / F_MAX_CLUSTERS * block_cost(per) + (waves + 1) * 300 + 2000 + 100 * per, 1, 1);
    for (int ks = 2; ks <= F_MAX_SPLIT; ++ks)
      if (units <= kFit[ks] && 2 * ks <= KB && per <= 128)
        take((KB + ks - 1) / ks * block_cost(per) + 1200 + 6 * per, ks, 0);
  }
  return p;
}

template <int NT, bool GATED, bool CUT>
cudaError_t launch_nt(const Bf16GemmArgs& g, const BArgs& a, int pairs, cudaStream_t stream) {
  using C = BCfg<NT>;
  CUtensorMap mw, mb, ms;
  const auto type = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const auto sw = CU_TENSOR_MAP_SWIZZLE_128B;
  if (!encode_map_2d(&mw, g.w, type, 2, g.E * g.N * (GATED ? 2 : 1), g.K, B_BK, GATED ? 64 : B_HALF, sw) ||
      !encode_map_2d(&mb, g.x, type, 2, g.R, g.K, B_BK, a.xbig, sw))
    return cudaErrorInvalidValue;
  if (g.group_list == nullptr) ms = mb;  // not used
  else if (!encode_map_2d(&ms, g.x, type, 2, g.R, g.K, B_BK, a.xsmall, sw)) return cudaErrorInvalidValue;
  static std::atomic<uint64_t> ready{0};
  constexpr size_t kMost = C::kSmem + (F_MAX_E + 1) * 8;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(bf16_gemm_kernel<NT, GATED, CUT>), kMost, ready);
  if (e != cudaSuccess) return e;
  return launch_pairs(bf16_gemm_kernel<NT, GATED, CUT>, pairs, a.split, B_THREADS, C::kSmem + (a.E + 1) * 8, stream, mw, mb,
                      ms, a);
}

template <bool GATED>
cudaError_t launch_gated(int nt, const Bf16GemmArgs& g, const BArgs& a, int pairs, cudaStream_t stream) {
  switch (nt) {
    case 32: return a.cut ? launch_nt<32, GATED, true>(g, a, pairs, stream) : launch_nt<32, GATED, false>(g, a, pairs, stream);
    case 64: return a.cut ? launch_nt<64, GATED, true>(g, a, pairs, stream) : launch_nt<64, GATED, false>(g, a, pairs, stream);
    case 128: return a.cut ? launch_nt<128, GATED, true>(g, a, pairs, stream) : launch_nt<128, GATED, false>(g, a, pairs, stream);
    default: return a.cut ? launch_nt<256, GATED, true>(g, a, pairs, stream) : launch_nt<256, GATED, false>(g, a, pairs, stream);
  }
}

}  // namespace

size_t plan_bf16_gemm(Bf16GemmArgs& a) {
  const int64_t width = a.act == W8A8_ACT_SWIGLU ? 128 : 256;  // channels of a tile
  a.plan = make_plan(a.E, a.R, (a.N + width - 1) / width, a.K, a.group_list != nullptr);
  return a.plan.cut ? cut_bytes(a.plan.pairs, a.plan.nt) : 0;
}

size_t bf16_gemm_ws_bytes(int64_t R, int64_t N) {
  // make_plan() cuts only between F_MAX_CLUSTERS and 4 F_MAX_CLUSTERS units: what the widest tile that R rows (fewer, with
  // fewer channels, no wider one) can be cut into so many with takes, be that plan chosen or not
  const int64_t channel_blocks = std::min<int64_t>((std::min<int64_t>(N, INT32_MAX) + 127) / 128, 4 * F_MAX_CLUSTERS - 1);
  const int64_t least = F_MAX_CLUSTERS / channel_blocks + 1;  // token blocks
  const int64_t rows = std::min<int64_t>(R, 4 * F_MAX_CLUSTERS * 256);
  int64_t per = std::min<int64_t>(256, round16(rows));
  if (least > 1) per = std::min(per, (rows - 1) / (least - 1) & ~int64_t(15));
  if (rows == 0 || per < 16) return 0;
  return cut_bytes(F_MAX_CLUSTERS, tile_of(static_cast<int>(per)));
}

cudaError_t launch_bf16_gemm(const Bf16GemmArgs& g, void* ws, cudaStream_t stream) {
  if (g.R == 0) return cudaSuccess;
  const bool grouped = g.group_list != nullptr, gated = g.act == W8A8_ACT_SWIGLU;
  const int64_t channel_blocks = (g.N + (gated ? 127 : 255)) / (gated ? 128 : 256);
  const BPlan& p = g.plan;
  if ((g.R / (grouped ? p.nt : p.per) + g.E) * channel_blocks > INT32_MAX) return cudaErrorInvalidValue;
  BArgs a;
  a.group_list = g.group_list;
  a.bias = g.bias;
  a.residual = g.residual;
  a.y = g.y;
  a.status = g.status;
  a.R = g.R;
  a.N = g.N;
  a.K = g.K;
  a.E = static_cast<int>(g.E);
  a.act = g.act;
  a.split = p.split;
  a.cut = p.cut;
  a.counters = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(ws));
  a.pieces = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kCounterBytes);
  a.blocks = p.blocks;
  a.per = p.per;
  // An accumulator's additions truncate: over the whole of K a sum comes out low by about K * 2^-30 of itself (7168:
  // 7.9e-6).  bf16 outputs round 2^-9 away; for fp32 ones an accumulator takes 512 of K (4.8e-7
  // whatever K is), or 768 where its sums are not added up beside the next MMAs.
  a.chunk = !g.f32 ? 1 << 20 : p.nt == 256 ? 12 : 8;
  a.xbig = (grouped ? p.nt : p.per) / 2;
  a.xsmall = std::max(8, (a.xbig / 4 + 7) & ~7);
  a.f32 = g.f32;
  a.vec = g.N % 8 == 0 && (reinterpret_cast<uintptr_t>(g.y) & 15u) == 0u &&
          (reinterpret_cast<uintptr_t>(g.residual) & 15u) == 0u;
  return gated ? launch_gated<true>(p.nt, g, a, p.pairs, stream) : launch_gated<false>(p.nt, g, a, p.pairs, stream);
}

}  // namespace w8a8
