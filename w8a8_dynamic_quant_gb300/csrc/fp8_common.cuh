// fp8_common.cuh -- what the two block-scaled FP8 contractions share: the work walk, tensor-memory loads, waits and
// the MMA issue.  The kernels are in fp8_gemm.cu (weights as the MMA's M side) and fp8_wide.cu (tokens as M side).
// The bf16 product (gemm_bf16.cu) takes the group scan, the waits, the elected loads and the launch from here.
#pragma once

#include <atomic>

#include "fp8.cuh"
#include "tc_common.cuh"

namespace w8a8 {
namespace fp8 {

using namespace tc;

constexpr int F_BK = 128;            // K per stage and per scale block (bytes = E4M3 values)
constexpr int F_SG = 4;              // blocks per scale group
constexpr int F_SRING = 2;           // scale groups in the ring
constexpr int F_MAX_CLUSTERS = 76;   // CTA pairs, one CTA per SM
constexpr int F_MAX_E = 1024;
constexpr int F_SUPER = 32;          // token blocks per rasterisation group
constexpr int F_MAX_SPLIT = 8;        // pairs of a cluster that share a unit's K
constexpr int F_EPI_WARPS = 8;
constexpr uint32_t F_TMEM_COLS = 512;
constexpr size_t kCounterBytes = F_MAX_CLUSTERS * 2 * F_EPI_WARPS * 4;
static_assert(kCounterBytes % 256 == 0, "pieces start 256-byte aligned");

struct KArgs {
  const float* xs;
  const int64_t* group_list;
  const float* wsc;
  const uint16_t* bias;
  uint16_t* y;
  DeviceStatus* status;
  uint32_t* counters;  // [clusters][2][epilogue warps], zero between calls
  float* pieces;       // [clusters][2 slots][2 CTAs][kPiece]
  int64_t R, N, K;
  int E;
  int split;  // pairs per cluster: 1, or the parts of K of a unit whose sums meet in distributed shared memory
  int runs;   // dense: runs of cut units (0: units are not cut); grouped: -1, chosen on the device
};

// D(tmem, both CTAs) (+)= A * B, kind::f8f6f4 with both operands E4M3, on the CTA pair (issued by the elected lane
// of a converged warp).
__device__ __forceinline__ void mma_pair_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n setp.ne.b32 p, %4, 0;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n"
      ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor: binary32 accumulator, E4M3 operands (format 0), both K-major, M = 256, N = n.
__device__ __forceinline__ uint32_t idesc_f8(int n) {
  return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (256u >> 4 << 24);
}

// The producer's steps, issued by the elected lane of a converged warp: with warp-uniform operands three loads and the
// expected bytes issue in well under 200 cycles, in over 300 from one lane of a diverged branch, which bounded the
// whole kernel (511 cycles a block of 384 cycles' MMAs).
__device__ __forceinline__ void expect_tx_elect(uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n}\n" ::"r"(bar), "r"(bytes)
      : "memory");
}
__device__ __forceinline__ void tma_pair_elect(uint32_t dst, const CUtensorMap* map, int x, int y,
                                               uint32_t mbar_cluster) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%2, %3}], [%4];\n}\n"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(mbar_cluster)
      : "memory");
}

// A shared-memory word of CTA `rank` of the cluster.
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// The value of lane 0.  Warp-uniform values and control flow (votes as loop conditions, bounds and indices passed
// through here) let the compiler keep an MMA's descriptors in uniform registers: measured, a wait, four MMAs and a
// commit issue in 184 cycles so, in 299 when each lane branches on its own probe.
__device__ __forceinline__ int uni(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// Wait of a whole converged warp for the phase of parity `parity`, bounded as mbar_wait; false when aborting.  No call
// inside: a call would cost the caller its registers.
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity, volatile int* abort_flag, DeviceStatus* st,
                                         uint32_t where) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) {
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

// Tensor-memory loads that order only against other volatile statements (no memory clobber): the scales' shared-
// memory reads may move past them.  The values are usable after tmem_ready on the same array.
__device__ __forceinline__ void tmem_fetch(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_fetch(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%2"
      "7,%28,%29,%30,%31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]),
        "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]),
        "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]),
        "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_fetch(uint32_t taddr, uint32_t (&v)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%2"
      "7,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%5"
      "2,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]),
        "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]),
        "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]),
        "=r"(v[29]), "=r"(v[30]), "=r"(v[31]), "=r"(v[32]), "=r"(v[33]), "=r"(v[34]), "=r"(v[35]),
        "=r"(v[36]), "=r"(v[37]), "=r"(v[38]), "=r"(v[39]), "=r"(v[40]), "=r"(v[41]), "=r"(v[42]),
        "=r"(v[43]), "=r"(v[44]), "=r"(v[45]), "=r"(v[46]), "=r"(v[47]), "=r"(v[48]), "=r"(v[49]),
        "=r"(v[50]), "=r"(v[51]), "=r"(v[52]), "=r"(v[53]), "=r"(v[54]), "=r"(v[55]), "=r"(v[56]),
        "=r"(v[57]), "=r"(v[58]), "=r"(v[59]), "=r"(v[60]), "=r"(v[61]), "=r"(v[62]), "=r"(v[63])
      : "r"(taddr));
}
template <int C>
__device__ __forceinline__ void tmem_ready(uint32_t (&v)[C]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;");
#pragma unroll
  for (int i = 0; i < C; ++i) asm volatile("" : "+r"(v[i]));  // no use of a value moves before the wait
}

// Arrival of lane 0 on a cluster-window mbarrier, without a branch.
__device__ __forceinline__ void arrive_lane0(uint32_t bar, int lane) {
  asm volatile("{\n .reg .pred p;\n setp.eq.s32 p, %1, 0;\n @p mbarrier.arrive.shared::cluster.b64 _, [%0];\n}\n" ::"r"(bar), "r"(lane)
               : "memory");
}
__device__ __forceinline__ void arrive_lane0_cta(uint32_t bar, int lane) {
  asm volatile("{\n .reg .pred p;\n setp.eq.s32 p, %1, 0;\n @p mbarrier.arrive.shared::cta.b64 _, [%0];\n}\n" ::"r"(bar), "r"(lane)
               : "memory");
}
__device__ __forceinline__ bool mbar_test(uint32_t a, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(ok) : "r"(a), "r"(parity) : "memory");
  return ok != 0u;
}

// The sequence of segments of one pair.  Every role walks it on its own.
struct Walk {
  int64_t x, end;  // cut: block position; else: unit number
  int step;        // 0: cut
  int KB;
};
__device__ __forceinline__ int64_t run_begin(int64_t total, int C, int c) { return total * c / C; }
// The pair whose run holds block position p.
__device__ __forceinline__ int run_owner(int64_t total, int C, int64_t p) {
  return static_cast<int>(((p + 1) * C - 1) / total);
}
// The next unit of the walk and its blocks [kb0, kb1).
__device__ __forceinline__ bool next_unit(Walk& w, int& unit, int& kb0, int& kb1) {
  if (w.x >= w.end) return false;
  if (w.step == 0) {
    unit = static_cast<int>(w.x / w.KB);
    kb0 = static_cast<int>(w.x - static_cast<int64_t>(unit) * w.KB);
    kb1 = static_cast<int>(min(static_cast<int64_t>(w.KB), kb0 + (w.end - w.x)));
    w.x += kb1 - kb0;
  } else {
    unit = static_cast<int>(w.x);
    kb0 = 0;
    kb1 = w.KB;
    w.x += w.step;
  }
  return true;
}
// Unit -> expert, channel block, token block of TB.  Token blocks go in groups of SUPER with the channel block
// outside: the pairs in flight share weight blocks, and a group's token rows stay in L2 while the weights sweep past.
template <int SUPER = F_SUPER, typename BlocksOf>
__device__ __forceinline__ void unit_tile(int unit, int E, int WB, const int* s_prefix, const int* s_off,
                                          BlocksOf blocks_of, int& e, int& wb, int& tb, int& cnt, int& TB) {
  e = expert_of(unit, E, s_prefix);
  const int local = unit - s_prefix[e];
  cnt = s_off[e + 1] - s_off[e];
  TB = blocks_of(cnt);
  const int g = local / (WB * SUPER);
  const int rem = local - g * WB * SUPER;
  const int gt = min(SUPER, TB - g * SUPER);
  wb = rem / gt;
  tb = g * SUPER + rem - wb * gt;
}

// Rows and units of the groups, and whether the list is usable: scan_groups with its sum checked in 64 bits where 32
// may not hold it.  Called by all NT threads; s_rows is 0 and s_bad set up before.  A __syncthreads (or a cluster
// barrier) follows before bad_list() is asked.
template <int NT, typename Args, typename UnitsOf>
__device__ __forceinline__ int scan_checked(const Args& a, UnitsOf units_of, int* s_off, int* s_prefix, int* s_warp,
                                            int* s_bad, unsigned long long* s_rows, int* units) {
  if (a.group_list == nullptr) {  // one group of R rows (R <= INT32_MAX)
    const int u = units_of(static_cast<int>(a.R));
    if (threadIdx.x == 0) {
      s_off[0] = s_prefix[0] = 0;
      s_off[1] = static_cast<int>(a.R);
      s_prefix[1] = u;
    }
    *units = u;
    return static_cast<int>(a.R);
  }
  GemmArgs ga;
  ga.group_list = a.group_list;
  ga.R = a.R;
  const int rows = scan_groups<NT, F_MAX_E>(ga, a.E, units_of, s_off, s_prefix, s_warp, s_bad, units);
  if (a.group_list != nullptr && a.R > INT32_MAX / a.E)
    for (int e = threadIdx.x; e < a.E; e += NT)
      atomicAdd(s_rows, static_cast<unsigned long long>(max(0ll, static_cast<long long>(a.group_list[e]))));
  return rows;
}
template <typename Args>
__device__ __forceinline__ bool bad_list(const Args& a, int rows, int s_bad, unsigned long long s_rows) {
  return s_bad != 0 || rows != a.R ||
         (a.group_list != nullptr && a.R > INT32_MAX / a.E && s_rows != static_cast<unsigned long long>(a.R));
}

// How the units' blocks are shared out over C pairs, from costs in eighths of a block's time (about 0.25 us at 64
// tokens a tile, 0.4 us at 256).  Uncut: whole units, every C-th one to a pair.  Cut: equal runs of blocks, aligned to
// units where there are fewer runs than pairs; writing, fencing and adding the pieces costs about 22 blocks (30 for
// 256 tokens, whose pieces are 128 KB a CTA) and one or three more a piece.  Measured, uncut against cut: 80 units of
// 16 blocks and 64 tokens 15.2 and 17.3 us, 96 of 32 and 128 tokens 39.6 and 38.6; with 256 tokens, 112 units of 32
// blocks 31.2 and 41.6, 336 71 and 83, 80 of 56 46.2 and 44.3.
struct RunPlan {
  int runs;      // 0: uncut
  int64_t cost;
};
__host__ __device__ inline RunPlan plan_runs(int64_t units, int KB, int C, bool wide) {
  const int64_t fixed = wide ? 240 : 180, per = wide ? 24 : 8;
  RunPlan p{0, (units + C - 1) / C * KB * 8};
  if (units <= 0) return p;
  const int64_t total = units * KB;
  const int64_t all = total < C ? total : C;
  if (units % C != 0 && units < 8 * C) {  // (many whole units in turn keep neighbouring weights in flight: 5 % faster)
    const int64_t c = (total + all - 1) / all * 8 + fixed + per * (all / units + 2);
    if (c < p.cost) p = RunPlan{static_cast<int>(all), c};
  }
  for (int64_t ks = 2; ks * units <= C && ks <= KB; ++ks) {
    const int64_t c = (KB + ks - 1) / ks * 8 + fixed + per * ks;
    if (c < p.cost) p = RunPlan{static_cast<int>(ks * units), c};
  }
  return p;
}

// The walk of pair `me` of C.  split > 1: the pair's part of K of its cluster's one unit.
__device__ __forceinline__ Walk start_walk(const KArgs& a, int units, int KB, int C, int me, bool wide, int64_t& total,
                                           int& runs) {
  total = static_cast<int64_t>(units) * KB;
  Walk w;
  w.KB = KB;
  w.step = 0;
  w.x = w.end = 0;
  if (a.split > 1) {
    runs = 0;
    const int unit = me / a.split, part = me % a.split;
    if (unit < units) {
      w.x = static_cast<int64_t>(unit) * KB + static_cast<int64_t>(KB) * part / a.split;
      w.end = static_cast<int64_t>(unit) * KB + static_cast<int64_t>(KB) * (part + 1) / a.split;
    }
    return w;
  }
  runs = a.runs >= 0 ? min(a.runs, static_cast<int>(min(total, static_cast<int64_t>(C)))) : plan_runs(units, KB, C, wide).runs;
  if (runs == 0) {
    w.step = C;
    w.x = me;
    w.end = units;
  } else if (me < runs) {
    w.x = run_begin(total, runs, me);
    w.end = run_begin(total, runs, me + 1);
  }
  return w;
}

}  // namespace fp8

// The contraction with tokens as the MMA's M side (fp8_wide.cu).
cudaError_t launch_fp8_wide(const Fp8GemmArgs& g, const fp8::KArgs& a, int pairs, cudaStream_t stream);

namespace fp8 {

// The kernel's attributes on the current device, set once (`done`: one bit a device): a call costs as much as a
// tensor map.
inline cudaError_t allow_smem(const void* k, size_t smem, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_acquire) & bit) != 0u) return cudaSuccess;
  e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// Launch of `pairs` CTA pairs in clusters of `split` pairs, with programmatic stream serialization.
template <typename... KArgsT, typename... Args>
inline cudaError_t launch_pairs(void (*k)(KArgsT...), int pairs, int split, int threads, size_t smem, cudaStream_t stream,
                                Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(2 * split);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k, args...);
}

}  // namespace fp8

}  // namespace w8a8
