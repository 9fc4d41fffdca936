// fp8_gemm.cu -- block-scaled FP8 contraction on the 5th-generation tensor
// cores (tcgen05.mma.cta_group::2.kind::f8f6f4), dense and grouped by expert.
//
//   y[m,n] = bf16( sum_b xs[m,b] * ws[n / 128, b] * sum_{k in block b} q[m,k] * w[n,k]  (+ bias[n]) )
//
// q [R,K] E4M3 rows with a binary32 scale per 128 values, w [E,N,K] E4M3 with
// a binary32 scale per 128 x 128 block.  The scales are arbitrary binary32
// numbers, so the tensor core cannot apply them (its block scales are powers
// of two): every 128-deep block is one accumulator of its own, which the
// epilogue warps drain, multiply by xs * ws and add into binary32 sums held in
// registers, while the MMAs of the next blocks fill other accumulators.
//
// This file: tiles of up to 128 tokens; fp8_wide.cu: of 256.
//
// Tile.  The weights are the MMA's M side, 256 output channels per CTA pair
// (128 in each CTA: one weight scale per CTA and block), and a block of up to
// NT tokens is N, sized to the tokens there are in steps of 16: the even CTA
// holds the first half of the block's token rows, the odd CTA the rest.  So
// ragged groups pad to 16 rows, not to a tile, and an MMA costs what its tokens
// need (N <= 32: 39 cycles, 64: 43, 128: 64).  A ring stage is one 128-deep
// block: the CTA's 128 x 128-byte weight tile and its token rows by TMA,
// 128-byte swizzle.
//
// Tensor memory (512 columns): 512 / NT accumulators of NT columns.
//
// Warp roles (384 threads, one CTA per SM):
//   warp 0       TMA producer
//   warp 1       TMEM owner; the even CTA's issues the MMAs (whole warp, one lane elected)
//   warps 2-3    scales: xs * ws of four blocks at a time, [block][token], into a shared-memory ring (half of the
//                tokens each)
//   warps 4-11   epilogue: warp w reads TMEM lanes 32 * (w % 4) .. (channels) and one half of the tokens
//
// Work.  A unit is one tile over the whole of K.  With many units the pairs
// take every C-th one.  With few in a dense call, the 2 to 8 pairs of a cluster
// take parts of K of one unit each and add their sums through distributed
// shared memory, in the order of K.  Else the units' blocks in sequence are cut
// into C equal runs, one per pair: a run ends and begins inside units, every
// piece of a cut unit leaves its partial sums in the workspace, and the warp
// that arrives last at a unit adds the pieces in the order of K and writes the
// result: no order of arrival changes a bit, and no warp waits for another.
// The cluster's sum costs about 1.2 us, a cut unit's 5 and more (64 x 2048 x 7168:
// 10.2 us in clusters of 6 pairs, 13.1 us in seven parts through the workspace), so
// units are cut only where they are few and long.
//
// What bounds it.  Many experts with few rows: the weight stream (1024 rows over
// 256 experts of 4096 x 7168: 1040 us, 7.1 TB/s).  One small layer: latency.
// 64 x 2048 x 7168 could stream its weights in 2.3 us; launch and the first
// tiles' way take about 4 (16 x 256 x 512: 4.5 us in all), ten blocks a pair
// in turn and the sum over the cluster the rest.
//
// Registers: 159 to 168 of the 168 that 384 threads may have; with tiles of 128
// tokens ptxas reports 24 bytes spilled (32 and 64: none).  That is a few values a
// thread, and these tiles are bound by the weight stream or by latency.
//
// Every mbarrier wait is bounded (2 s): on expiry the CTA sets
// W8A8_ERR_DEVICE_TIMEOUT, lets in-flight copies land, frees TMEM and returns.
#include "fp8_common.cuh"

namespace w8a8 {

namespace {

using namespace fp8;

constexpr int F_ROWS = 256;   // output channels per pair tile (MMA M)
constexpr int F_HALF = 128;   // of them in each CTA
constexpr int F_THREADS = 384;
constexpr int F_EPI0 = 4;
constexpr uint32_t F_W_BYTES = F_HALF * F_BK;  // 16 KB
constexpr uint32_t F_STG_BYTES = F_EPI_WARPS * 16 * 32 * 2;  // output staging: [16 tokens][32 channels] per warp

template <int NT>
struct Cfg {
  static constexpr uint32_t kXBytes = NT / 2 * F_BK;
  static constexpr uint32_t kStageBytes = F_W_BYTES + kXBytes;
  static constexpr int kStages = NT == 128 ? 8 : NT == 64 ? 9 : 10;
  static constexpr int kAcc = NT >= 64 ? 512 / NT : 8;  // accumulators of NT columns
  static constexpr int kCols = NT / 2;                  // of them read by one epilogue warp
  static constexpr int kBig = NT / 2;                   // token rows per large TMA box
  static constexpr uint32_t kScaleBytes = F_SRING * F_SG * NT * 4;
  static constexpr size_t kSmem = static_cast<size_t>(kStages) * kStageBytes + kScaleBytes + F_STG_BYTES + 1024;
  static constexpr size_t kPiece = static_cast<size_t>(F_EPI_WARPS) * kCols * 32;  // floats of one CTA's partial sums
};

// acc[c] += accumulator column c * sc[c], c < cols (rounded up to 16), two columns an instruction.  The warp's columns
// come in one load; once it is complete the accumulator is released (arrival on `release`) and the next one's barrier
// probed, before the sums.
template <int COLS>
__device__ __forceinline__ bool drain(uint32_t taddr, const float* sc, int cols, uint32_t release, int lane,
                                      uint32_t next_bar, uint32_t next_parity, float (&acc)[COLS]) {
  uint32_t v[COLS];
  tmem_fetch(taddr, v);
  tmem_ready(v);
  tc_fence_before();
  arrive_lane0(release, lane);
  const bool next = mbar_test(next_bar, next_parity);
#pragma unroll
  for (int j = 0; j < COLS; j += 16) {
    if (j < cols) {
#pragma unroll
      for (int i = j; i < j + 16; i += 4) {
        const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(sc + i);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint64_t a, x;
          asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(acc[i + 2 * h]), "f"(acc[i + 2 * h + 1]));
          asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "r"(v[i + 2 * h]), "r"(v[i + 2 * h + 1]));
          asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(a) : "l"(x), "l"(h == 0 ? f.x : f.y));
          asm("mov.b64 {%0, %1}, %2;" : "=f"(acc[i + 2 * h]), "=f"(acc[i + 2 * h + 1]) : "l"(a));
        }
      }
    }
  }
  return next;
}

// One run of blocks of a unit: the tile and its K range.
struct Seg {
  int e, wb;       // expert, 256-channel block
  int row0;        // first token row (of all R)
  int tvalid;      // tokens
  int n;           // tokens rounded up to 16
  int kb0, kb1;    // blocks [kb0, kb1)
  int unit;
};

template <int NT>
__device__ __forceinline__ bool next_seg(Walk& w, int E, int WB, const int* s_prefix, const int* s_off, Seg& s) {
  if (!next_unit(w, s.unit, s.kb0, s.kb1)) return false;
  int tb, cnt, TB;
  unit_tile(s.unit, E, WB, s_prefix, s_off, [](int c) { return (c + NT - 1) / NT; }, s.e, s.wb, tb, cnt, TB);
  const int per = ((cnt + TB - 1) / TB + 15) & ~15;  // tokens split evenly over the blocks
  s.row0 = s_off[s.e] + tb * per;
  s.tvalid = min(per, cnt - tb * per);
  s.n = (s.tvalid + 15) & ~15;
  return true;
}

// Rows [0, rows) of a warp's staging buffer [rows][32] bf16 to out[(row0 + r) * ld + c0 + c], c < min(32, ld - c0).
__device__ __forceinline__ void store_rows(const uint16_t* stg, uint16_t* out, int64_t row0, int64_t ld, int64_t c0,
                                           int rows, int lane) {
  const int64_t ncols = ld - c0 < 32 ? ld - c0 : 32;
  if (ncols == 32 && (ld & 7) == 0 && (reinterpret_cast<uintptr_t>(out) & 15u) == 0u) {
    const int c = (lane & 3) * 8;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = (lane >> 2) + 8 * i;
      if (r < rows)
        *reinterpret_cast<uint4*>(out + (row0 + r) * ld + c0 + c) = *reinterpret_cast<const uint4*>(stg + r * 32 + c);
    }
  } else {
    for (int r = 0; r < rows; ++r)
      if (lane < ncols) out[(row0 + r) * ld + c0 + lane] = stg[r * 32 + lane];
  }
}

template <int NT>
__global__ void __launch_bounds__(F_THREADS, 1)
fp8_gemm_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmXbig,
                const __grid_constant__ CUtensorMap tmXsmall, const KArgs a) {
  using C = Cfg<NT>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bar_full[C::kStages];   // even CTA: both CTAs' tiles of the stage landed
  __shared__ __align__(8) uint64_t bar_empty[C::kStages];  // the MMAs reading the stage are done
  __shared__ __align__(8) uint64_t bar_accf[C::kAcc];      // the block's accumulator is complete
  __shared__ __align__(8) uint64_t bar_acce[C::kAcc];      // even CTA: both CTAs drained it
  __shared__ __align__(8) uint64_t bar_scf[F_SRING];       // the group's scales are in shared memory
  __shared__ __align__(8) uint64_t bar_sce[F_SRING];       // the epilogue warps read them
  __shared__ uint32_t s_tmem_base;
  __shared__ volatile int s_abort;
  __shared__ int s_bad;
  __shared__ int s_prefix[F_MAX_E + 1];
  __shared__ int s_off[F_MAX_E + 1];
  __shared__ int s_warp[F_THREADS / 32];
  __shared__ unsigned long long s_rows;  // the counts' sum where 32 bits may not hold it

  const int tid = threadIdx.x;
  const int warp = uni(tid >> 5);
  const int lane = tid & 31;
  const int E = a.E;
  const int64_t N = a.N;
  const int KB = static_cast<int>((a.K + F_BK - 1) / F_BK);
  const int WB = static_cast<int>((N + F_ROWS - 1) / F_ROWS);

  uint8_t* stages = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t stage_base = smem_u32(stages);
  float* s_scale = reinterpret_cast<float*>(stages + C::kStages * C::kStageBytes);  // [ring][4 blocks][NT]
  float* s_part = reinterpret_cast<float*>(stages);  // [epilogue warp][token][channel], after the last block
  uint16_t* s_out = reinterpret_cast<uint16_t*>(stages + C::kStages * C::kStageBytes + C::kScaleBytes);
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
    for (int s = 0; s < F_SRING; ++s) {
      mbar_init(smem_u32(&bar_scf[s]), 2);
      mbar_init(smem_u32(&bar_sce[s]), F_EPI_WARPS);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmXbig);
    tma_prefetch_desc(&tmXsmall);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem_base)),
                 "r"(F_TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  __syncthreads();  // s_bad, before the scan may set it
  pdl_trigger();
  pdl_wait();
  int units;
  const int rows_total = scan_checked<F_THREADS>(
      a, [WB](int c) { return ((c + NT - 1) / NT) * WB; }, s_off, s_prefix, s_warp, &s_bad, &s_rows, &units);
  tc_fence_before();
  cluster_sync_all();  // both CTAs' barriers and tensor memory exist before either touches the other's
  tc_fence_after();
  const uint32_t tmem_base = static_cast<uint32_t>(uni(static_cast<int>(s_tmem_base)));
  if (bad_list(a, rows_total, s_bad, s_rows)) {
    if (tid == 0 && blockIdx.x == 0) set_status(a.status, W8A8_ERR_GROUP_LIST, 0u);
    units = 0;
  }
  const int me = static_cast<int>(cluster_id) * a.split + static_cast<int>(crank >> 1);
  int64_t total;
  int runs;
  const Walk walk0 = start_walk(a, units, KB, static_cast<int>(nclusters), me, false, total, runs);

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer (both CTAs)
    const uint32_t full_even0 = smem_cluster_addr(smem_u32(&bar_full[0]), even);
    int stage = 0;
    uint32_t phase = 0;
    Walk w = walk0;
    Seg s;
    bool ok = true;
    while (ok && uni(next_seg<NT>(w, E, WB, s_prefix, s_off, s))) {
      const int yw = uni(static_cast<int>(static_cast<int64_t>(s.e) * N) + s.wb * F_ROWS + static_cast<int>(rank) * F_HALF);
      const int rows = uni(s.n >> 1);
      const int yx = uni(s.row0 + static_cast<int>(rank) * (s.n >> 1));
      const uint32_t bytes = 2u * F_W_BYTES + static_cast<uint32_t>(2 * rows) * F_BK;
      const int kb1 = uni(s.kb1);
      for (int kb = uni(s.kb0); kb < kb1; ++kb) {
        ok = wait_all(smem_u32(&bar_empty[stage]), phase ^ 1u, &s_abort, a.status, 1u);
        if (!ok) break;
        if (rank == 0) expect_tx_elect(smem_u32(&bar_full[0]) + 8 * stage, bytes);
        const uint32_t full = full_even0 + 8 * stage;
        const uint32_t dst = stage_base + stage * C::kStageBytes;
        tma_pair_elect(dst, &tmW, kb * F_BK, yw, full);
        // the block's first n / 2 token rows go to the even CTA, the rest to the odd one
        if (rows == C::kBig) {
          tma_pair_elect(dst + F_W_BYTES, &tmXbig, kb * F_BK, yx, full);
        } else {
          for (int r = 0; r < rows; r += 8) tma_pair_elect(dst + F_W_BYTES + r * F_BK, &tmXsmall, kb * F_BK, yx + r, full);
        }
        if (++stage == C::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // Drain: the last fill of every stage has been consumed, so no copy into this CTA and no MMA arrival on its
    // barriers is still in flight when the cluster leaves.
    for (int i = 0; i < C::kStages && ok; ++i) {
      ok = wait_all(smem_u32(&bar_empty[stage]), phase ^ 1u, &s_abort, a.status, 5u);
      if (++stage == C::kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------- MMA issuer (even CTA, whole warp)
    if (rank == 0) {
      int stage = 0, buf = 0;
      uint32_t phase = 0, bphase = 0;
      Walk w = walk0;
      Seg s;
      bool ok = true;
      while (ok && uni(next_seg<NT>(w, E, WB, s_prefix, s_off, s))) {
        const uint32_t idesc = idesc_f8(uni(s.n));
        const int kb1 = uni(s.kb1);
        for (int kb = uni(s.kb0); kb < kb1; ++kb) {
          ok = wait_all(smem_u32(&bar_full[stage]), phase, &s_abort, a.status, 3u) &&
               wait_all(smem_u32(&bar_acce[buf]), bphase ^ 1u, &s_abort, a.status, 2u);
          if (!ok) break;
          tc_fence_after();
          const uint32_t sa = stage_base + stage * C::kStageBytes;
          const uint64_t adesc = smem_desc_sw128(sa);
          const uint64_t bdesc = smem_desc_sw128(sa + F_W_BYTES);
#pragma unroll
          for (int k = 0; k < F_BK / 32; ++k)
            mma_pair_f8(tmem_base + buf * NT, adesc + 2u * k, bdesc + 2u * k, idesc, k > 0 ? 1u : 0u);
          tc_commit_pair_mc(smem_u32(&bar_accf[buf]), pair_mask);
          tc_commit_pair_mc(smem_u32(&bar_empty[stage]), pair_mask);  // frees the stage in both CTAs
          if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1u;
          }
          if (++buf == C::kAcc) {
            buf = 0;
            bphase ^= 1u;
          }
        }
      }
    }
  } else if (warp < F_EPI0) {
    // ------------------------------------------------------------- scales (both CTAs)
    constexpr int kPerLane = NT >= 64 ? NT / 64 : 1;
    const int t0 = lane + (warp - 2) * (NT >= 64 ? NT / 2 : 32);  // NT = 32: the second warp has no token
    const int NB = static_cast<int>((N + 127) / 128);
    const bool vec = (KB & 3) == 0 && (reinterpret_cast<uintptr_t>(a.xs) & 15u) == 0u;
    int slot = 0;
    uint32_t phase = 0;
    Walk w = walk0;
    Seg s;
    bool ok = true;
    while (ok && uni(next_seg<NT>(w, E, WB, s_prefix, s_off, s))) {
      const int nb = s.wb * 2 + static_cast<int>(rank);
      const float* wrow = a.wsc + (static_cast<int64_t>(s.e) * NB + nb) * KB;
      for (int g = s.kb0 / F_SG; ok && g * F_SG < s.kb1; ++g) {
        const int k0 = g * F_SG;
        float wv[F_SG];
#pragma unroll
        for (int j = 0; j < F_SG; ++j) wv[j] = nb < NB && k0 + j < KB ? wrow[k0 + j] : 0.0f;
        float v[kPerLane][F_SG];
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) {
          const int t = t0 + 32 * i;
          const float* p = a.xs + (static_cast<int64_t>(s.row0) + t) * KB + k0;
          const bool in = t < s.tvalid;
          if (vec) {
            const float4 f = in ? *reinterpret_cast<const float4*>(p) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            v[i][0] = f.x; v[i][1] = f.y; v[i][2] = f.z; v[i][3] = f.w;
          } else {
#pragma unroll
            for (int j = 0; j < F_SG; ++j) v[i][j] = in && k0 + j < KB ? p[j] : 0.0f;
          }
        }
        ok = wait_all(smem_u32(&bar_sce[slot]), phase ^ 1u, &s_abort, a.status, 11u);
        if (!ok) break;
        float* d = s_scale + slot * F_SG * NT;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i)
#pragma unroll
          for (int j = 0; j < F_SG; ++j)
            if (t0 + 32 * i < NT) d[j * NT + t0 + 32 * i] = v[i][j] * wv[j];
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bar_scf[slot]));
        if (++slot == F_SRING) {
          slot = 0;
          phase ^= 1u;
        }
      }
    }
  } else {
    // ---------------------------------------------------------------- epilogue (both CTAs)
    const int ew = warp - F_EPI0;
    const int q = warp & 3;
    const int h = ew >> 2;
    const uint32_t lane_addr = tmem_base + (static_cast<uint32_t>(32 * q) << 16);
    const uint32_t acce_even = smem_cluster_addr(smem_u32(&bar_acce[0]), even);
    uint16_t* stg = s_out + ew * 16 * 32;
    int buf = 0, slot = 0;
    uint32_t bphase = 0, sphase = 0;
    bool probed = false;  // the next accumulator was seen complete
    const uint32_t accf0 = smem_u32(&bar_accf[0]);
    Walk w = walk0;
    Seg s;
    bool ok = true;
    while (ok && uni(next_seg<NT>(w, E, WB, s_prefix, s_off, s))) {
      // the first half's warps read tokens [0, split), the second's [split, n)
      const int n = uni(s.n), kb0 = uni(s.kb0), kb1 = uni(s.kb1);
      const int split = ((n >> 1) + 15) & ~15;
      const int c0 = h == 0 ? 0 : split;
      const int cols = h == 0 ? split : n - split;
      float acc[C::kCols];
#pragma unroll
      for (int i = 0; i < C::kCols; ++i) acc[i] = 0.0f;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (kb == kb0 || (kb & (F_SG - 1)) == 0)
          ok = wait_all(smem_u32(&bar_scf[slot]), sphase, &s_abort, a.status, 6u);
        if (!probed) ok = ok && wait_all(accf0 + 8 * buf, bphase, &s_abort, a.status, 4u);
        if (!ok) break;
        tc_fence_after();
        const uint32_t here = lane_addr + buf * NT + c0, release = acce_even + 8u * buf;
        if (++buf == C::kAcc) {
          buf = 0;
          bphase ^= 1u;
        }
        probed = __all_sync(0xffffffffu, drain<C::kCols>(here, s_scale + (slot * F_SG + (kb & (F_SG - 1))) * NT + c0, cols,
                                                         release, lane, accf0 + 8 * buf, bphase, acc));
        if ((kb & (F_SG - 1)) == F_SG - 1 || kb == kb1 - 1) {
          __syncwarp();
          arrive_lane0_cta(smem_u32(&bar_sce[0]) + 8 * slot, lane);
          if (++slot == F_SRING) {
            slot = 0;
            sphase ^= 1u;
          }
        }
      }
      if (!ok) break;
      const int64_t n0 = static_cast<int64_t>(s.wb) * F_ROWS + static_cast<int64_t>(rank) * F_HALF + 32 * q;
      const int tv = min(cols, s.tvalid - c0);  // tokens of this warp that exist (may be <= 0)
      if (n0 >= N || tv <= 0) continue;
      const float bias = a.bias != nullptr && n0 + lane < N ? bf16_bits_to_f32(a.bias[n0 + lane]) : 0.0f;
      const int64_t row0 = static_cast<int64_t>(s.row0) + c0;
      if (kb0 == 0 && kb1 == KB) {
#pragma unroll
        for (int t = 0; t < C::kCols; t += 16) {
          if (t < tv) {
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              float lo = acc[t + i], hi = acc[t + i + 1];
              if (a.bias != nullptr) {
                lo += bias;
                hi += bias;
              }
              const uint32_t v = f32x2_to_bf16x2_bits(lo, hi);
              stg[i * 32 + lane] = static_cast<uint16_t>(v);
              stg[(i + 1) * 32 + lane] = static_cast<uint16_t>(v >> 16);
            }
            __syncwarp();
            store_rows(stg, a.y, row0 + t, N, n0, min(16, tv - t), lane);
            __syncwarp();
          }
        }
      } else if (a.split > 1) {  // a part of K of the cluster's unit: its sums to the ring, which is at rest
        float* d = s_part + ew * C::kCols * 32 + lane;
#pragma unroll
        for (int i = 0; i < C::kCols; ++i)
          if (i < tv) d[i * 32] = acc[i];
      } else {
        // a piece of a cut unit: partial sums to this pair's slot (1: the unit begins in this run, 0: it began in an
        // earlier one), then the last warp to arrive adds the unit's pieces in the order of K
        const int64_t u0 = static_cast<int64_t>(s.unit) * KB;
        const int first = run_owner(total, runs, u0), last = run_owner(total, runs, u0 + KB - 1);
        auto piece = [&](int c) {
          return a.pieces + ((static_cast<int64_t>(c) * 2 + (c == first ? 1 : 0)) * 2 + rank) * C::kPiece +
                 static_cast<int64_t>(ew) * C::kCols * 32 + lane;
        };
        float* mine = piece(me);
#pragma unroll
        for (int i = 0; i < C::kCols; ++i)
          if (i < tv) __stcg(mine + i * 32, acc[i]);
        __threadfence();
        __syncwarp();
        uint32_t* ctr = a.counters + (first * 2 + static_cast<int>(rank)) * F_EPI_WARPS + ew;
        uint32_t arrived = 0;
        if (lane == 0) arrived = atomicAdd(ctr, 1u);
        arrived = __shfl_sync(0xffffffffu, arrived, 0);
        if (arrived == static_cast<uint32_t>(last - first)) {
          __threadfence();
          if (lane == 0) *ctr = 0u;
          for (int t = 0; t < tv; t += 16) {
            float sum[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) sum[i] = 0.0f;
            for (int c = first; c <= last; c += 4) {  // four pieces' loads in flight, added in order
              float v[4][16];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float* src = piece(min(c + j, last)) + t * 32;
#pragma unroll
                for (int i = 0; i < 16; ++i) v[j][i] = t + i < tv ? __ldcg(src + i * 32) : 0.0f;
              }
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (c + j <= last) {
#pragma unroll
                  for (int i = 0; i < 16; ++i) sum[i] += v[j][i];
                }
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) stg[i * 32 + lane] = f32_to_bf16_bits(a.bias != nullptr ? sum[i] + bias : sum[i]);
            __syncwarp();
            store_rows(stg, a.y, row0 + t, N, n0, min(16, tv - t), lane);
            __syncwarp();
          }
        }
      }
    }
  }

  if (a.split > 1) {
    // the parts' sums meet: every CTA adds its share of the tokens over its peers' shared memory, in the order of K
    __syncwarp();
    cluster_sync_all();
    Walk w = walk0;
    Seg s;
    if (warp >= F_EPI0 && uni(next_seg<NT>(w, E, WB, s_prefix, s_off, s))) {
      const int ew = warp - F_EPI0, h = ew >> 2;
      const int split = ((s.n >> 1) + 15) & ~15;
      const int tv = min(h == 0 ? split : s.n - split, s.tvalid - (h == 0 ? 0 : split));
      const int64_t n0 = static_cast<int64_t>(s.wb) * F_ROWS + static_cast<int64_t>(rank) * F_HALF + 32 * (warp & 3);
      if (n0 < N && tv > 0) {
        const int part = static_cast<int>(crank >> 1);
        const int t1 = tv * (part + 1) / a.split;
        const float bias = a.bias != nullptr && n0 + lane < N ? bf16_bits_to_f32(a.bias[n0 + lane]) : 0.0f;
        const uint32_t src = smem_u32(s_part + ew * C::kCols * 32 + lane);
        uint16_t* stg = s_out + ew * 16 * 32;
        for (int t = tv * part / a.split; t < t1; t += 4) {
          float v[F_MAX_SPLIT][4], sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int j = 0; j < F_MAX_SPLIT; ++j) {  // every peer's words in flight, added in order
            const uint32_t p = smem_cluster_addr(src, 2 * min(j, a.split - 1) + rank) + t * 128;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[j][i] = j < a.split && t + i < t1 ? ld_cluster(p + i * 128) : 0.0f;
          }
#pragma unroll
          for (int j = 0; j < F_MAX_SPLIT; ++j)
            if (j < a.split) {
#pragma unroll
              for (int i = 0; i < 4; ++i) sum[i] += v[j][i];
            }
#pragma unroll
          for (int i = 0; i < 4; ++i) stg[i * 32 + lane] = f32_to_bf16_bits(a.bias != nullptr ? sum[i] + bias : sum[i]);
          __syncwarp();
          store_rows(stg, a.y, static_cast<int64_t>(s.row0) + (h == 0 ? 0 : split) + t, N, n0, min(4, t1 - t), lane);
          __syncwarp();
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
  cluster_sync_all();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(F_TMEM_COLS)
                 : "memory");
  }
}

// Tokens per tile: the power of two from 32 to 256 that holds the rows (dense), or twice the mean rows of a group.
int tile_tokens(int64_t E, int64_t R, bool grouped) {
  const int64_t want = grouped ? 2 * ((R + E - 1) / E) : R;
  return want <= 32 ? 32 : want <= 64 ? 64 : want <= 128 ? 128 : 256;
}

struct Plan {
  int nt, pairs, split, runs;
};
// A dense problem of few tiles lets the pairs of a cluster share each tile's K (their sums meet in distributed shared
// memory: about 3 blocks' time, or 5 and 1.5 a part for 256 tokens, where 256 x 5000 x 2048 takes 11.9 us whole and 13.6
// in two parts), as far as the clusters fit the GPU at once; else plan_runs.  The plan goes by the sizes alone, so that
// the workspace's size and the launch agree on every device: no pair waits for a pair of another cluster, so a GPU with
// fewer SMs runs the same grid in two waves.
Plan make_plan(int64_t E, int64_t R, int64_t N, int64_t K, bool grouped) {
  constexpr int most = F_MAX_CLUSTERS;
  Plan p{tile_tokens(E, R, grouped), most, 1, -1};
  if (grouped) return p;
  const bool wide = p.nt == 256;
  const int64_t units = ((R + p.nt - 1) / p.nt) * ((N + F_ROWS - 1) / F_ROWS);
  const int KB = static_cast<int>((K + F_BK - 1) / F_BK);
  const RunPlan r = plan_runs(units, KB, most, wide);
  p.runs = r.runs;
  p.pairs = static_cast<int>(r.runs > 0 ? r.runs : std::min<int64_t>(units, most));
  int64_t best = r.cost;
  // clusters of 2 ks CTAs (one a SM) that are resident at once on 152 SMs, as the occupancy query gives them
  constexpr int kFit[F_MAX_SPLIT + 1] = {0, 76, 36, 23, 15, 13, 8, 7, 7};
  for (int ks = 2; ks <= F_MAX_SPLIT; ++ks) {
    const int64_t cost = (KB + ks - 1) / ks * 8 + (wide ? 40 + 12 * ks : 24);
    if (units > kFit[ks] || units * ks > most || 2 * ks > KB || cost >= best) continue;
    if (wide && 16 % ks != 0) continue;  // equal shares of a part's sixteen 8-channel chunks (three parts: slower)
    best = cost;
    p.split = ks;
    p.runs = 0;
    p.pairs = static_cast<int>(units) * ks;
  }
  return p;
}

template <int NT>
cudaError_t launch_nt(const Fp8GemmArgs& g, const KArgs& a, int pairs, cudaStream_t stream) {
  using C = Cfg<NT>;
  CUtensorMap mw, mb, ms;
  const auto type = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const auto sw = CU_TENSOR_MAP_SWIZZLE_128B;
  // token boxes of a whole tile's half and of 8 rows (for the tiles that hold fewer)
  if (!encode_map_2d(&mw, g.w, type, 1, g.E * g.N, g.K, F_BK, F_HALF, sw) ||
      !encode_map_2d(&ms, g.q, type, 1, g.R, g.K, F_BK, 8, sw))
    return cudaErrorInvalidValue;
  if (g.group_list == nullptr && g.R <= NT - 16) mb = ms;  // no tile is full: the large box is not used
  else if (!encode_map_2d(&mb, g.q, type, 1, g.R, g.K, F_BK, C::kBig, sw)) return cudaErrorInvalidValue;
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(fp8_gemm_kernel<NT>), C::kSmem, ready);
  if (e != cudaSuccess) return e;
  return launch_pairs(fp8_gemm_kernel<NT>, pairs, a.split, F_THREADS, C::kSmem, stream, mw, mb, ms, a);
}

}  // namespace

size_t fp8_gemm_ws_bytes(int64_t E, int64_t R, int64_t N, int64_t K, bool grouped) {
  // pieces of cut units: at most two a pair, [2 CTAs][128 channels or tokens][tile tokens or channels] binary32 each
  const Plan p = make_plan(E, R, N, K, grouped);
  const size_t pieces = p.runs != 0 ? static_cast<size_t>(p.pairs) * 4 * F_HALF * p.nt * 4 : 0;
  return kCounterBytes + pieces;
}

cudaError_t launch_fp8_gemm(const Fp8GemmArgs& g, void* ws, cudaStream_t stream) {
  if (g.R == 0) return cudaSuccess;
  const bool grouped = g.group_list != nullptr;
  const Plan p = make_plan(g.E, g.R, g.N, g.K, grouped);
  if ((g.R / p.nt + g.E) * ((g.N + F_ROWS - 1) / F_ROWS) > INT32_MAX) return cudaErrorInvalidValue;
  KArgs a;
  a.xs = g.x_scale;
  a.group_list = g.group_list;
  a.wsc = g.w_scale;
  a.bias = g.bias;
  a.y = g.y;
  a.status = g.status;
  a.counters = static_cast<uint32_t*>(ws);
  a.pieces = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kCounterBytes);
  a.R = g.R;
  a.N = g.N;
  a.K = g.K;
  a.E = static_cast<int>(g.E);
  a.split = p.split;
  a.runs = p.runs;
  switch (p.nt) {
    case 32: return launch_nt<32>(g, a, p.pairs, stream);
    case 64: return launch_nt<64>(g, a, p.pairs, stream);
    case 128: return launch_nt<128>(g, a, p.pairs, stream);
    default: return launch_fp8_wide(g, a, p.pairs, stream);
  }
}

}  // namespace w8a8
