// fp8_wide.cu -- block-scaled FP8 contraction for many tokens (see
// fp8_gemm.cu for the formula and for few): tokens as the MMA's M side.
//
// Tile.  256 tokens x 256 output channels per CTA pair, in two parts of 128
// channels (one weight block each); a CTA holds 128 token rows and 64 weight
// rows of each part of every 128-deep stage.  A part and block of K is one
// accumulator (128 lanes x 128 columns of tensor memory), four in all: two parts
// times two.  A thread of the epilogue owns one token row of one part, so xs * ws
// is one number for all of its 128 columns and block: a fused multiply-add a
// value with its scale in a register.  (With the weights as M side every column
// has its own scale, which comes from shared memory: four values a 16-byte load.)
//
// What bounds it.  Per 128-deep block a pair's MMAs take 512 cycles; an epilogue
// warp's round -- barrier, tensor-memory loads of 128 columns, 128 sums, release --
// takes about 660, and the end of a tile about 2200 (sums to bf16, shared memory, TMA)
// in which the MMAs are at most two blocks ahead.  On 8192 x 14336 x 4096, 332 us in
// a burst (2.90 PFLOP/s, 0.76 of twice the measured BF16 burst) and 371 without a
// pause, under the power cap (0.68).  What was kept and what not, each beside the
// step before it:
//   - few, wide rounds: 2 x 128 channels a tile 392 us, 2 x 96 452 us, one part of
//     160 with three accumulators 486 us (before the steps below); sixteen epilogue
//     warps of 64 channels 365 us against 357; one barrier for two blocks 410 us: it
//     lengthens the way above.  Without the drain the pipeline took 261 us;
//   - an issuing warp (437 -> 418 us) and four epilogue warps per part;
//   - scales of four blocks read at once, the loop unrolled by them (388 -> 357 us);
//   - overlapping accumulator loads (357 -> 349 us);
//   - registers: the segment comes with its first scales from the warp that walks
//     ahead, the walk is worked out again where it is seldom needed, and both halves
//     of a tile are staged at once at the price of the fifth stage (355 -> 338 us).
//     ptxas still reports 28 bytes a thread spilled and 128 loaded, in a kernel whose
//     epilogue holds 128 sums and 48 buffer words of 216 registers.
//
// Warp roles (384 threads, one CTA per SM):
//   warp 0       TMA producer
//   warps 1, 2   issue the MMAs of part 0, 1 (even CTA); warp 1 owns the TMEM
//   warp 3       scales: xs * ws, [block][part][token], four blocks at a time, into a shared-memory ring, with the
//                segment that they belong to
//   warps 4-11   epilogue: part (w - 4) / 4, TMEM lanes 32 * (w % 4) ..
// Whole rows of 32 tokens leave through shared memory by TMA.  Work, cut units and bounded waits as in fp8_gemm.cu.
#include "fp8_common.cuh"

namespace w8a8 {

namespace {

using namespace fp8;

constexpr int G_TOK = 256;    // tokens per pair tile (MMA M)
constexpr int G_HALF = 128;   // of them in each CTA
constexpr int G_CH = 256;     // channels per tile
constexpr int G_PART = 128;   // channels per part (MMA N)
constexpr int G_THREADS = 384;
constexpr int G_EPI0 = 4;
constexpr int G_STAGES = 4;
constexpr int G_SEGS = 4;  // the scales are at most two groups, so two segments, ahead of an epilogue warp
constexpr uint32_t G_X_BYTES = G_HALF * F_BK;       // 16 KB: the CTA's token rows
constexpr uint32_t G_P_BYTES = G_PART / 2 * F_BK;   // 8 KB: its weight rows of a part
constexpr uint32_t G_STAGE_BYTES = G_X_BYTES + 2 * G_P_BYTES;
constexpr uint32_t G_SCALE_BYTES = F_SRING * F_SG * 2 * G_HALF * 4;
constexpr uint32_t G_STG_HALF = 32 * 128;            // output staging of a warp: two of [32 tokens][64 channels] bf16
constexpr uint32_t G_STG_WARP = 2 * G_STG_HALF;
constexpr uint32_t G_STG_BYTES = F_EPI_WARPS * G_STG_WARP;
constexpr size_t kWideSmem = static_cast<size_t>(G_STAGES) * G_STAGE_BYTES + G_SCALE_BYTES + G_STG_BYTES + 1024;
constexpr size_t kWidePiece = static_cast<size_t>(F_EPI_WARPS) * G_PART * 32;  // floats of one CTA's partial sums


struct WSeg {
  int e, wb;     // expert, 256-channel block
  int row0;      // first token row (of all R)
  int tvalid;    // tokens
  int kb0, kb1;  // blocks [kb0, kb1)
  int unit;      // < 0: no more segments
};

// (c + G_TOK - 1 would pass INT32_MAX, which c may be)
__device__ __forceinline__ int wide_blocks(int c) { return c / G_TOK + (c % G_TOK != 0 ? 1 : 0); }

__device__ __forceinline__ bool next_wide(Walk& w, int E, int WB, const int* s_prefix, const int* s_off, WSeg& s) {
  if (!next_unit(w, s.unit, s.kb0, s.kb1)) return false;
  int tb, cnt, TB;
  unit_tile(s.unit, E, WB, s_prefix, s_off, [](int c) { return wide_blocks(c); }, s.e, s.wb, tb, cnt, TB);
  s.row0 = s_off[s.e] + tb * G_TOK;
  s.tvalid = min(G_TOK, cnt - tb * G_TOK);
  return true;
}

// acc[i] += s * v[i], two values an instruction.
template <int C>
__device__ __forceinline__ void fma_scaled(float* acc, const uint32_t* v, float s) {
  uint64_t s2;
  asm("mov.b64 %0, {%1, %1};" : "=l"(s2) : "f"(s));
#pragma unroll
  for (int i = 0; i < C; i += 2) {
    uint64_t a, x;
    asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(acc[i]), "f"(acc[i + 1]));
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "r"(v[i]), "r"(v[i + 1]));
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(a) : "l"(x), "l"(s2));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(acc[i]), "=f"(acc[i + 1]) : "l"(a));
  }
}

// acc += s * the warp's 128 accumulator columns, through buffers of 32 and 16: while one is added the other's load runs.
// (With 32 and 32 the block loop spilled.)  The accumulator is released once its last load is complete, and the next
// one's barrier probed while the last sums run.
__device__ __forceinline__ bool drain_wide(uint32_t taddr, float s, uint32_t release, int lane, uint32_t next_bar,
                                           uint32_t next_parity, float (&acc)[G_PART]) {
  uint32_t u[32], v[16];
  tmem_fetch(taddr, u);
  tmem_fetch(taddr + 32, v);
  tmem_ready(u);
  tmem_ready(v);
  fma_scaled<32>(acc, u, s);
  tmem_fetch(taddr + 48, u);
  fma_scaled<16>(acc + 32, v, s);
  tmem_ready(u);
  tmem_fetch(taddr + 80, v);
  fma_scaled<32>(acc + 48, u, s);
  tmem_ready(v);
  tmem_fetch(taddr + 96, u);
  fma_scaled<16>(acc + 80, v, s);
  tmem_ready(u);
  tc_fence_before();
  arrive_lane0(release, lane);
  const bool next = mbar_test(next_bar, next_parity);
  fma_scaled<32>(acc + 96, u, s);
  return next;
}

// The warp's staging buffer holds 64 channels of 32 token rows as [32][64] bf16 in the 128-byte swizzle: 16-byte chunk
// c of row r at c ^ (r & 7), so neither the row-wise writes nor the reads conflict.
__device__ __forceinline__ uint32_t stg_at(int r, int c) { return static_cast<uint32_t>(r * 128 + ((c ^ (r & 7)) << 4)); }

// 8 channels (chunk c, 16 bytes) of the lane's row into the staging buffers.
__device__ __forceinline__ void stage_chunk(uint8_t* stg, int c, int lane, const float* f) {
  *reinterpret_cast<uint4*>(stg + (c >> 3) * G_STG_HALF + stg_at(lane, c & 7)) =
      make_uint4(f32x2_to_bf16x2_bits(f[0], f[1]), f32x2_to_bf16x2_bits(f[2], f[3]), f32x2_to_bf16x2_bits(f[4], f[5]),
                 f32x2_to_bf16x2_bits(f[6], f[7]));
}
// f[i] += bias[n + i] inside N.
template <int C>
__device__ __forceinline__ void add_bias(float* f, const uint16_t* bias, int64_t n, int64_t N) {
#pragma unroll
  for (int i = 0; i < C; ++i) f[i] += n + i < N ? bf16_bits_to_f32(bias[n + i]) : 0.0f;
}

// The staged rows to y rows row0 + r < row0 + rows, channels n0 .. (16-byte chunks [c_lo, c_hi) of them).  Rows of y
// that do not start on 16-byte boundaries take a row an instruction in words of two channels, or of one where N is odd.
__device__ __forceinline__ void store_wide(const uint8_t* stg, uint16_t* y, int64_t row0, int rows, int64_t N,
                                           int64_t n0, int lane, int c_lo = 0, int c_hi = 8) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(y);
  if ((N & 7) == 0 && (at & 15u) == 0u) {
    const int c = lane & 7;
    if (c < c_lo || c >= c_hi || n0 + 8 * c >= N) return;
#pragma unroll 1
    for (int r = lane >> 3; r < rows; r += 4)
      *reinterpret_cast<uint4*>(y + (row0 + r) * N + n0 + 8 * c) = *reinterpret_cast<const uint4*>(stg + stg_at(r, c));
  } else if ((N & 1) == 0 && (at & 3u) == 0u) {
    const int c = lane >> 2;
    if (c < c_lo || c >= c_hi || n0 + 2 * lane >= N) return;
#pragma unroll 4
    for (int r = 0; r < rows; ++r)
      *reinterpret_cast<uint32_t*>(y + (row0 + r) * N + n0 + 2 * lane) =
          *reinterpret_cast<const uint32_t*>(stg + stg_at(r, c) + 4 * (lane & 3));
  } else {
#pragma unroll
    for (int k = 0; k < 64; k += 32) {
      const int n = lane + k, c = n >> 3;
      if (c < c_lo || c >= c_hi || n0 + n >= N) continue;
#pragma unroll 4
      for (int r = 0; r < rows; ++r)
        y[(row0 + r) * N + n0 + n] = *reinterpret_cast<const uint16_t*>(stg + stg_at(r, c) + 2 * (n & 7));
    }
  }
}

// The same by TMA (32 whole rows; columns past N are cut off by the map), asynchronously: the writes are fenced for it
// before, and stg_free() comes before the buffer is written again.
__device__ __forceinline__ void tma_store_rows(const CUtensorMap* map, uint32_t stg, int x, int y) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];\n"
      " @e cp.async.bulk.commit_group;\n}\n" ::"l"(reinterpret_cast<uint64_t>(map)),
      "r"(stg), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void stg_free() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  __syncwarp();
}

// This CTA's pair among all, its clusters, and the pair's walk over `units` units.
__device__ __forceinline__ Walk pair_walk(const KArgs& a, int units, int KB, int& me, int64_t& total, int& runs) {
  uint32_t crank, cluster_id, nclusters;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(crank));
  asm volatile("mov.u32 %0, %%clusterid.x;" : "=r"(cluster_id));
  asm volatile("mov.u32 %0, %%nclusterid.x;" : "=r"(nclusters));
  me = static_cast<int>(cluster_id) * a.split + static_cast<int>(crank >> 1);
  return start_walk(a, units, KB, static_cast<int>(nclusters), me, true, total, runs);
}

__global__ void __launch_bounds__(G_THREADS, 1)
fp8_wide_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                const __grid_constant__ CUtensorMap tmY, const int y_tma, const KArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bar_full[G_STAGES];   // even CTA: both CTAs' tiles of the stage landed
  __shared__ __align__(8) uint64_t bar_empty[G_STAGES];  // both parts' MMAs reading the stage are done
  __shared__ __align__(8) uint64_t bar_accf[4];          // [part][2]: the accumulator is complete
  __shared__ __align__(8) uint64_t bar_acce[4];          // even CTA: both CTAs drained it
  __shared__ __align__(8) uint64_t bar_scf[F_SRING];     // the group's scales are in shared memory
  __shared__ __align__(8) uint64_t bar_sce[F_SRING];     // the epilogue warps read them
  __shared__ uint32_t s_tmem_base;
  __shared__ volatile int s_abort;
  __shared__ int s_bad;
  __shared__ int s_prefix[F_MAX_E + 1];
  __shared__ int s_off[F_MAX_E + 1];
  __shared__ int s_warp[G_THREADS / 32];
  __shared__ WSeg s_seg[G_SEGS];         // the segments in turn, from the scales warp to the epilogue
  __shared__ unsigned long long s_rows;

  const int tid = threadIdx.x;
  const int warp = uni(tid >> 5);
  const int lane = tid & 31;
  const int E = a.E;
  const int64_t N = a.N;
  const int KB = static_cast<int>((a.K + F_BK - 1) / F_BK);
  const int WB = static_cast<int>((N + G_CH - 1) / G_CH);

  uint8_t* stages = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t stage_base = smem_u32(stages);
  float* s_scale = reinterpret_cast<float*>(stages + G_STAGES * G_STAGE_BYTES);  // [ring][4 blocks][2 parts][128]
  float* s_part = reinterpret_cast<float*>(stages);  // [epilogue warp][channel][token], after the last block
  uint8_t* s_out = stages + G_STAGES * G_STAGE_BYTES + G_SCALE_BYTES;
  // CTAs 2i and 2i + 1 of a cluster are a pair; rank: the CTA's place in it
  uint32_t crank;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(crank));
  const uint32_t rank = crank & 1u, even = crank & ~1u;
  const uint16_t pair_mask = static_cast<uint16_t>(3u << even);

  if (tid == 0) {
    s_abort = 0;
    s_bad = 0;
    s_rows = 0ull;
    for (int s = 0; s < G_STAGES; ++s) {
      mbar_init(smem_u32(&bar_full[s]), 1);
      mbar_init(smem_u32(&bar_empty[s]), 2);
    }
    for (int b = 0; b < 4; ++b) {
      mbar_init(smem_u32(&bar_accf[b]), 1);
      mbar_init(smem_u32(&bar_acce[b]), F_EPI_WARPS);  // four warps of each CTA
    }
    for (int s = 0; s < F_SRING; ++s) {
      mbar_init(smem_u32(&bar_scf[s]), 1);
      mbar_init(smem_u32(&bar_sce[s]), F_EPI_WARPS);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmW);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem_base)),
                 "r"(F_TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  __syncthreads();  // s_bad and s_rows, before the scan may set them
  pdl_trigger();
  pdl_wait();
  int units;
  const int rows_total = scan_checked<G_THREADS>(
      a, [WB](int c) { return wide_blocks(c) * WB; }, s_off, s_prefix, s_warp, &s_bad, &s_rows, &units);
  tc_fence_before();
  cluster_sync_all();  // both CTAs' barriers and tensor memory exist before either touches the other's
  tc_fence_after();
  const uint32_t tmem_base = static_cast<uint32_t>(uni(static_cast<int>(s_tmem_base)));
  if (bad_list(a, rows_total, s_bad, s_rows)) {
    if (tid == 0 && blockIdx.x == 0) set_status(a.status, W8A8_ERR_GROUP_LIST, 0u);
    units = 0;
  }
  if (warp < G_EPI0) {
    // the epilogue's 128 sums a thread take registers from these warps (384 x 168 at launch = 128 x 72 + 256 x 216)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    int me, runs;
    int64_t total;
    const Walk walk0 = pair_walk(a, units, KB, me, total, runs);
    if (warp == 0) {
      // ---------------------------------------------------------- TMA producer (both CTAs)
      const uint32_t full_even0 = smem_cluster_addr(smem_u32(&bar_full[0]), even);
      int stage = 0;
      uint32_t phase = 0;
      Walk w = walk0;
      WSeg s;
      bool ok = true;
      while (ok && uni(next_wide(w, E, WB, s_prefix, s_off, s))) {
        const int yx = uni(s.row0 + static_cast<int>(rank) * G_HALF);
        const int yw = uni(static_cast<int>(static_cast<int64_t>(s.e) * N) + s.wb * G_CH +
                           static_cast<int>(rank) * (G_PART / 2));
        const int kb1 = uni(s.kb1);
        for (int kb = uni(s.kb0); kb < kb1; ++kb) {
          ok = wait_all(smem_u32(&bar_empty[0]) + 8 * stage, phase ^ 1u, &s_abort, a.status, 1u);
          if (!ok) break;
          if (rank == 0) expect_tx_elect(smem_u32(&bar_full[0]) + 8 * stage, 2u * G_STAGE_BYTES);
          const uint32_t full = full_even0 + 8 * stage;
          const uint32_t sa = stage_base + stage * G_STAGE_BYTES;
          tma_pair_elect(sa, &tmX, kb * F_BK, yx, full);
          tma_pair_elect(sa + G_X_BYTES, &tmW, kb * F_BK, yw, full);
          tma_pair_elect(sa + G_X_BYTES + G_P_BYTES, &tmW, kb * F_BK, yw + G_PART, full);
          if (++stage == G_STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // Drain: the last fill of every stage has been consumed, so no copy into this CTA and no MMA arrival on its
      // barriers is still in flight when the cluster leaves.
      for (int i = 0; i < G_STAGES && ok; ++i) {
        ok = wait_all(smem_u32(&bar_empty[stage]), phase ^ 1u, &s_abort, a.status, 5u);
        if (++stage == G_STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    } else if (warp < 3) {
      // ----------------------------------------------------------- MMA issuers (even CTA, whole warps)
      if (rank == 0) {
        // The blocks of all segments in one sequence (the accumulators restart at every block, so tiles do not matter
        // here), unrolled over the ring: stage and accumulator are constants of each body, and the descriptors stay in
        // uniform registers.
        const int p = warp - 1;
        constexpr uint32_t idesc = (1u << 4) | (uint32_t(G_PART >> 3) << 17) | (uint32_t(G_TOK >> 4) << 24);
        const int64_t blocks = walk0.step == 0 ? walk0.end - walk0.x
                               : walk0.x < walk0.end ? (walk0.end - walk0.x + walk0.step - 1) / walk0.step * KB : 0;
        const int nblk = uni(static_cast<int>(min(blocks, static_cast<int64_t>(INT32_MAX))));
        const uint64_t adesc0 = smem_desc_sw128(stage_base);
        const uint64_t bdesc0 = smem_desc_sw128(stage_base + G_X_BYTES + p * G_P_BYTES);
        const uint32_t acc0 = tmem_base + 2 * p * G_PART;
        const uint32_t accf0 = smem_u32(&bar_accf[2 * p]), acce0 = smem_u32(&bar_acce[2 * p]);
        const uint32_t full0 = smem_u32(&bar_full[0]), empty0 = smem_u32(&bar_empty[0]);
        bool ok = true;
        uint32_t round = 0;
        for (int g = 0; ok && g < nblk; g += G_STAGES, ++round) {
#pragma unroll
          for (int s = 0; s < G_STAGES; ++s) {
            if (g + s >= nblk) break;
            const uint32_t gi = round * G_STAGES + s;
            const uint32_t b = gi & 1u;
            ok = wait_all(full0 + 8 * s, round & 1u, &s_abort, a.status, 3u) &&
                 wait_all(acce0 + 8 * b, ((gi >> 1) + 1u) & 1u, &s_abort, a.status, 2u);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < F_BK / 32; ++k)
              mma_pair_f8(acc0 + b * G_PART, adesc0 + (s * (G_STAGE_BYTES >> 4) + 2u * k),
                          bdesc0 + (s * (G_STAGE_BYTES >> 4) + 2u * k), idesc, k > 0 ? 1u : 0u);
            tc_commit_pair_mc(accf0 + 8 * b, pair_mask);
            tc_commit_pair_mc(empty0 + 8 * s, pair_mask);  // this part is done with the stage
          }
        }
      }
    } else {
      // ----------------------------------------------------------- scales (both CTAs)
      const int NB = static_cast<int>((N + 127) / 128);
      const bool vec = (KB & 3) == 0 && (reinterpret_cast<uintptr_t>(a.xs) & 15u) == 0u;
      int slot = 0, seg = 0;
      uint32_t phase = 0;
      Walk w = walk0;
      WSeg s;
      bool ok = true;
      for (; ok && uni(next_wide(w, E, WB, s_prefix, s_off, s)); ++seg) {
        const int nb = 2 * s.wb;
        const float* w0 = a.wsc + (static_cast<int64_t>(s.e) * NB + nb) * KB;
        const bool two = nb + 1 < NB;
        const int t0 = static_cast<int>(rank) * G_HALF + lane;
        for (int g = s.kb0 / F_SG; g * F_SG < s.kb1; ++g) {
          const int k0 = g * F_SG;
          float v[4][F_SG];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float* p = a.xs + (static_cast<int64_t>(s.row0) + t0 + 32 * i) * KB + k0;
            const bool in = t0 + 32 * i < s.tvalid;
            if (vec) {
              const float4 f = in ? *reinterpret_cast<const float4*>(p) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
              v[i][0] = f.x; v[i][1] = f.y; v[i][2] = f.z; v[i][3] = f.w;
            } else {
#pragma unroll
              for (int j = 0; j < F_SG; ++j) v[i][j] = in && k0 + j < KB ? p[j] : 0.0f;
            }
          }
          float wv[2][F_SG];
#pragma unroll
          for (int j = 0; j < F_SG; ++j) {
            wv[0][j] = k0 + j < KB ? w0[k0 + j] : 0.0f;
            wv[1][j] = two && k0 + j < KB ? w0[KB + k0 + j] : 0.0f;
          }
          ok = wait_all(smem_u32(&bar_sce[slot]), phase ^ 1u, &s_abort, a.status, 11u);
          if (!ok) break;
          float* d = s_scale + slot * F_SG * 2 * G_HALF + lane;
#pragma unroll
          for (int j = 0; j < F_SG; ++j)
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
              for (int i = 0; i < 4; ++i) d[(j * 2 + p) * G_HALF + 32 * i] = v[i][j] * wv[p][j];
          if (lane == 0 && k0 <= s.kb0) s_seg[seg % G_SEGS] = s;  // with its first group
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bar_scf[slot]));
          if (++slot == F_SRING) {
            slot = 0;
            phase ^= 1u;
          }
        }
      }
      if (ok && wait_all(smem_u32(&bar_sce[slot]), phase ^ 1u, &s_abort, a.status, 12u)) {  // the end, as a group
        if (lane == 0) s_seg[seg % G_SEGS].unit = -1;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bar_scf[slot]));
      }
    }
  } else {
    // ---------------------------------------------------------------- epilogue (both CTAs)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int ew = warp - G_EPI0;
    const int q = warp & 3;
    const int p = ew >> 2;
    const uint32_t lane_addr = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + 2 * p * G_PART;
    const uint32_t acce_even = smem_cluster_addr(smem_u32(&bar_acce[2 * p]), even);
    uint8_t* stg = s_out + ew * G_STG_WARP;
    uint32_t blk = 0, grp = 0;  // blocks and scale groups so far: ring places and phases follow from them
    bool probed = false;        // the next accumulator was seen complete
    const uint32_t accf0 = smem_u32(&bar_accf[2 * p]);
    const float* my_scale = s_scale + p * G_HALF + 32 * q + lane;
    const bool shares = a.split > 1;  // one segment, whose sums meet the cluster's others
    bool ok = true;
    for (int seg = 0; ok && (seg == 0 || !shares); seg = (seg + 1) % G_SEGS) {
      ok = wait_all(smem_u32(&bar_scf[0]) + 8 * (grp & 1u), (grp >> 1) & 1u, &s_abort, a.status, 6u);
      if (ok && uni(s_seg[seg].unit) < 0) break;
      const int kb0 = ok ? uni(s_seg[seg].kb0) : 0, kb1 = ok ? uni(s_seg[seg].kb1) : 0;
      float acc[G_PART];
#pragma unroll
      for (int i = 0; i < G_PART; ++i) acc[i] = 0.0f;
      for (int k4 = kb0 & ~(F_SG - 1); ok && k4 < kb1; k4 += F_SG) {
        ok = wait_all(smem_u32(&bar_scf[0]) + 8 * (grp & 1u), (grp >> 1) & 1u, &s_abort, a.status, 6u);
        if (!ok) break;
        float s4[F_SG];  // the group's scales; its slot is free again at once
#pragma unroll
        for (int j = 0; j < F_SG; ++j) s4[j] = my_scale[((grp & 1u) * F_SG + j) * 2 * G_HALF];
        __syncwarp();
        arrive_lane0_cta(smem_u32(&bar_sce[0]) + 8 * (grp & 1u), lane);
        ++grp;
#pragma unroll
        for (int j = 0; j < F_SG; ++j) {
          if (k4 + j < kb0 || k4 + j >= kb1) continue;
          const uint32_t buf = blk & 1u, phase = (blk >> 1) & 1u;
          if (!probed) ok = wait_all(accf0 + 8u * buf, phase, &s_abort, a.status, 4u);
          if (!ok) break;
          tc_fence_after();
          ++blk;
          probed = __all_sync(0xffffffffu, drain_wide(lane_addr + buf * G_PART, s4[j], acce_even + 8u * buf, lane,
                                                      accf0 + 8u * (buf ^ 1u), (blk >> 1) & 1u, acc));
        }
      }
      // every part's MMAs are done with the ring before it takes the sums of a shared unit
      if (shares) asm volatile("bar.sync 1, 256;" ::: "memory");
      if (!ok) break;
      const WSeg s = s_seg[seg];
      const int64_t n0 = static_cast<int64_t>(s.wb) * G_CH + p * G_PART;
      const int rbase = static_cast<int>(rank) * G_HALF + 32 * q;  // first token of the warp inside the tile
      const int rows = min(32, s.tvalid - rbase);
      if (n0 >= N || rows <= 0) continue;
      const int64_t row0 = static_cast<int64_t>(s.row0) + rbase;
      if (s.kb0 == 0 && s.kb1 == KB) {
        if (a.bias != nullptr) add_bias<G_PART>(acc, a.bias, n0, N);
        stg_free();
#pragma unroll
        for (int c = 0; c < G_PART / 8; ++c) stage_chunk(stg, c, lane, acc + 8 * c);
        const bool two = n0 + 64 < N;
        if (y_tma != 0 && rows == 32) {
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          tma_store_rows(&tmY, smem_u32(stg), static_cast<int>(n0), static_cast<int>(row0));
          if (two) tma_store_rows(&tmY, smem_u32(stg + G_STG_HALF), static_cast<int>(n0) + 64, static_cast<int>(row0));
        } else {
          __syncwarp();
          store_wide(stg, a.y, row0, rows, N, n0, lane);
          if (two) store_wide(stg + G_STG_HALF, a.y, row0, rows, N, n0 + 64, lane);
        }
      } else if (shares) {  // a part of K of the cluster's unit
        float* d = s_part + ew * G_PART * 32 + lane;
#pragma unroll
        for (int i = 0; i < G_PART; ++i) d[i * 32] = acc[i];
      } else {
        // a piece of a cut unit (as in fp8_gemm.cu): [channel][token] partial sums
        int me, runs;
        int64_t total;
        pair_walk(a, s_prefix[E], KB, me, total, runs);
        const int64_t u0 = static_cast<int64_t>(s.unit) * KB;
        const int first = run_owner(total, runs, u0), last = run_owner(total, runs, u0 + KB - 1);
        auto piece = [&](int c) {
          return a.pieces + ((static_cast<int64_t>(c) * 2 + (c == first ? 1 : 0)) * 2 + rank) * kWidePiece +
                 static_cast<int64_t>(ew) * G_PART * 32 + lane;
        };
        float* mine = piece(me);
#pragma unroll
        for (int i = 0; i < G_PART; ++i) __stcg(mine + i * 32, acc[i]);
        __threadfence();
        __syncwarp();
        uint32_t* ctr = a.counters + (first * 2 + static_cast<int>(rank)) * F_EPI_WARPS + ew;
        uint32_t arrived = 0;
        if (lane == 0) arrived = atomicAdd(ctr, 1u);
        arrived = __shfl_sync(0xffffffffu, arrived, 0);
        if (arrived == static_cast<uint32_t>(last - first)) {
          __threadfence();
          if (lane == 0) *ctr = 0u;
          for (int half = 0; half < 2; ++half) {
            if (n0 + half * 64 >= N) break;
            stg_free();
            for (int c = 0; c < 8; c += 2) {
              float f[2][8] = {};
              for (int r = first; r <= last; r += 4) {  // four pieces' loads in flight, added in order
                float v[4][16];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const float* src = piece(min(r + j, last)) + (half * 8 + c) * 8 * 32;
#pragma unroll
                  for (int k = 0; k < 16; ++k) v[j][k] = __ldcg(src + k * 32);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  if (r + j <= last) {
#pragma unroll
                    for (int k = 0; k < 16; ++k) f[k >> 3][k & 7] += v[j][k];
                  }
              }
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                if (a.bias != nullptr) add_bias<8>(f[j], a.bias, n0 + (half * 8 + c + j) * 8, N);
                stage_chunk(stg, half * 8 + c + j, lane, f[j]);
              }
            }
            __syncwarp();
            store_wide(stg + half * G_STG_HALF, a.y, row0, rows, N, n0 + half * 64, lane);
          }
        }
      }
    }
  }

  if (a.split > 1) {
    // the parts' sums meet: every CTA adds its share of the channels over its peers' shared memory, in the order of K
    __syncwarp();
    cluster_sync_all();
    int me, runs;
    int64_t total;
    Walk w = pair_walk(a, s_prefix[E], KB, me, total, runs);
    WSeg s;
    if (warp >= G_EPI0 && uni(next_wide(w, E, WB, s_prefix, s_off, s))) {
      const int ew = warp - G_EPI0;
      const int64_t n0 = static_cast<int64_t>(s.wb) * G_CH + (ew >> 2) * G_PART;
      const int rbase = static_cast<int>(rank) * G_HALF + 32 * (warp & 3);
      const int rows = min(32, s.tvalid - rbase);
      if (n0 < N && rows > 0) {
        const int share = G_PART / 8 / a.split, lo = share * static_cast<int>(crank >> 1);  // 8-channel chunks
        const uint32_t src = smem_u32(s_part + ew * G_PART * 32 + lane);
        uint8_t* stg = s_out + ew * G_STG_WARP;
        for (int c = lo; c < lo + share; ++c) {
          float f[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
          for (int j = 0; j < a.split; ++j) {
            const uint32_t p = smem_cluster_addr(src, 2 * j + rank) + c * 8 * 128;
#pragma unroll
            for (int k = 0; k < 8; ++k) f[k] += ld_cluster(p + k * 128);
          }
          if (a.bias != nullptr) add_bias<8>(f, a.bias, n0 + 8 * c, N);
          stage_chunk(stg, c, lane, f);
        }
        __syncwarp();
        store_wide(stg + (lo >> 3) * G_STG_HALF, a.y, static_cast<int64_t>(s.row0) + rbase, rows, N, n0 + (lo >> 3) * 64, lane, lo & 7,
                   (lo & 7) + share);
      }
    }
  }

  // (a warp's last TMA stores read their staging buffer before it exits)
  if (warp >= G_EPI0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");

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

}  // namespace

cudaError_t launch_fp8_wide(const Fp8GemmArgs& g, const fp8::KArgs& a, int pairs, cudaStream_t stream) {
  CUtensorMap mx, mw, my;
  const auto type = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const auto sw = CU_TENSOR_MAP_SWIZZLE_128B;
  if (!encode_map_2d(&mx, g.q, type, 1, g.R, g.K, F_BK, G_HALF, sw) ||
      !encode_map_2d(&mw, g.w, type, 1, g.E * g.N, g.K, F_BK, G_PART / 2, sw))
    return cudaErrorInvalidValue;
  // bf16 y in boxes of 32 rows x 64 channels, where its rows start on 16-byte boundaries
  const int y_tma = g.N % 8 == 0 && (reinterpret_cast<uintptr_t>(g.y) & 15u) == 0u ? 1 : 0;
  if (!y_tma) my = mx;
  else if (!encode_map_2d(&my, g.y, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, g.R, g.N, 64, 32, sw)) return cudaErrorInvalidValue;
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(fp8_wide_kernel), kWideSmem, ready);
  if (e != cudaSuccess) return e;
  return launch_pairs(fp8_wide_kernel, pairs, a.split, G_THREADS, kWideSmem, stream, mx, mw, my, y_tma, a);
}

}  // namespace w8a8
