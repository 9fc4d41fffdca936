// norm.cu -- root-mean-square norm of BF16 rows, with the residual's addition before it and the 8-bit quantisation
// behind it in one pass: what stands between two quantised products of a layer.
//
//   r = bf16(x + residual)                (binary32 sum; r = x without a residual)
//   g = RN(1 / sqrt(S / K + eps)),  S = sum_k r_k^2
//   v = (r * g) * w                       (binary32, kept so into the quantisation: one rounding to 8 bits)
//   INT8   s = max |v| / 127 a row,       q = rint(v / s)                 (as quant.cu)
//   FP8    s = max |v| / 448 per 128,     q = E4M3(v / s)                 (as fp8_quant.cu)
//   MXFP8  2^(floor(log2 max |v|) - 8) per 32, q = E4M3(v / 2^...)        (as mx.cu)
//
// r and bf16(v) are written where they are asked for.
//
// The sum decides every code of a row, so its bits must not hang on the order of the additions: squares of bf16 are
// exact in binary32, and they are added with their rounding errors carried in a second word (Knuth's TwoSum), in the
// threads and in the reductions.  What the second word itself loses is bounded (slack()): where the two together lie so
// close to the middle between two binary32 values that it could decide, about one row in 6000, the group adds the row's
// squares up anew as integers.  So S is the exact sum rounded once, every later step is one rounding per element, and
// codes and scales are functions of the row alone, whatever the launch shape.
//
// Bound by memory: 2 bytes in (4 with a residual), 1 out (3 with it, 2 more for y).  A row lives in the registers of G
// warps, CH chunks of 8 values a thread; two meetings of the group (the sum; INT8 the maximum), which other rows'
// loads hide.  8192 x 4096 with residual: INT8 39.2 us, FP8 39.8, MXFP8 38.7, 5.9 to 6.1 TB/s, 0.87 to 0.90 of the copy
// rate; 16384 x 2048 the same.  The first form, one chunk or two a thread, six operations a square and the residual's
// sum in binary32, issued 302 instructions a chunk and was bound by them (43.9 and 57.7 us).  One row: 2.4 us.
// Rows of more than 32768 values spill 108 to 244 bytes a thread (eight chunks in 64 registers).  What the sums' second
// look costs, without it in brackets: 16384 x 2048 39.1 us (38.7), 8192 x 1024 11.2 (11.0), 64 x 7168 FP8 4.1 (3.9).
#include "norm.cuh"

namespace w8a8 {

namespace {

enum Form : int { F_INT8 = 0, F_FP8 = 1, F_MX = 2 };

constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: y + kMagic holds rint(y), ties to even, in its low bits

__device__ __forceinline__ uint64_t pk(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void upk(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
// Paired binary32 operations: each half is the correctly rounded operation of its own operands.
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
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

// s + p in s, what its rounding lost added to c (Knuth, "The Art of Computer Programming" 2, 4.2.2).
__device__ __forceinline__ void two_sum2(uint64_t& s, uint64_t& c, uint64_t p) {
  const uint64_t t = add2(s, p), b = sub2(t, s);
  c = add2(c, add2(sub2(s, sub2(t, b)), sub2(p, b)));
  s = t;
}
// (s, e) + (so, eo).  The same bits with the two exchanged, so all lanes of a butterfly end with the same.
__device__ __forceinline__ void two_sum(float& s, float& e, float so, float eo) {
  const float t = __fadd_rn(s, so), b = __fsub_rn(t, s);
  e = __fadd_rn(__fadd_rn(e, eo), __fadd_rn(__fsub_rn(s, __fsub_rn(t, b)), __fsub_rn(so, b)));
  s = t;
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// max of |a|, |b| and |c|; NaN if one is.
__device__ __forceinline__ float max_abs3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// The same, a NaN passed over.
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
  float r;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Two bf16 of a word, widened.
__device__ __forceinline__ uint64_t wide2(uint32_t w) {
  return pk(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// The sum of the squares of a thread's values as s + e.  The sum starts at B, the power of two of the largest square,
// and B is taken off at the end (exact: s - B is a smaller multiple of what s's last place holds).  A sum whose exponent
// is never below that of what is added gives its rounding error in two operations (Dekker, "A floating-point technique
// for extending the available precision", 1971), the second an fma since squares are exact; any order of magnitudes
// takes six.
template <int CH>
__device__ __forceinline__ void sum_squares(const uint4 (&v)[CH], float& s, float& e) {
  uint32_t top = 0u;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const uint32_t q[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("max.NaN.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(top) : "r"(q[i]));
  }
  const float m = max_nan(__uint_as_float((top << 16) & 0x7fff0000u), __uint_as_float(top & 0x7fff0000u));
  const float B = __uint_as_float(__float_as_uint(__fmul_rn(m, m)) & 0x7f800000u);
  if (m < 0x1p59f) {
    uint64_t s2 = pk(B, B), c2 = 0ull;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const uint32_t q[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t r = wide2(q[i]), t = fma2(r, r, s2);
        c2 = add2(c2, fma2(r, r, sub2(s2, t)));
        s2 = t;
      }
    }
    float s1, e1;
    upk(s2, s, s1);
    upk(c2, e, e1);
    s = __fsub_rn(s, B);
    s1 = __fsub_rn(s1, B);
    two_sum(s, e, s1, e1);
  } else {  // squares near the top of binary32 or above it, infinities and NaNs
    uint64_t s2 = 0ull, c2 = 0ull;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const uint32_t q[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) two_sum2(s2, c2, mul2(wide2(q[i]), wide2(q[i])));
    }
    float s1, e1;
    upk(s2, s, s1);
    upk(c2, e, e1);
    two_sum(s, e, s1, e1);
  }
}

// How far s + e may be from the exact sum S, relative to it.  With u = 2^-24 and n = 4 CH additions to each half of a
// thread's pair, whose running sums, B among them, come to no more than X: every error is at most u X, the j-th addition
// to e rounds by at most j u^2 X, and over a row the X come to at most 3 S (the B of a thread are no larger than its
// largest square): 1.5 n (n + 1) u^2 S.  Joining the halves rounds e twice, by (6 n + 2) u^2 S at most, and each of up to
// ten steps of the reductions twice, together by (60 n + 110) u^2 S.  Squares below 2^-126 may lose 2^-149 each, with S
// above 2^-90 a relative 2^-43 in all.  n = 4: 406 u^2 < 2^-39; n = 16: 1576 u^2 < 2^-37; n = 32: 3808 u^2 < 2^-36.
template <int CH>
constexpr float slack() {
  static_assert(CH <= 8, "the bounds above");
  return CH == 1 ? 0x1p-39f : CH <= 4 ? 0x1p-37f : 0x1p-36f;
}

template <int G>
__device__ __forceinline__ void meet(int grp);

// The exact sum of a row's squares, rounded once to binary32; s is that sum as it was before, within a few of its last
// places, or infinite.  A value is an integer m < 256 times 2^(E - 134), E its exponent field.  Its square is cut into
// what is a multiple of 2^top, top 57 below s's exponent, and digits of 40 bits below that; the first parts are added up
// as integers, which no order changes.  They decide the rounding unless they come to less than 65536 units below the
// middle (a unit for each value that has digits left); then the next digits are added up, and so on.
// row: K / 8 = nchunk chunks, which this thread wrote itself as far as it reads them (t, t + threads, ...).  words: two
// a warp.
template <int G>
__device__ __noinline__ float exact_sum(const uint4* row, int nchunk, int t, int warp, int grp, unsigned long long* words, float s) {
  constexpr unsigned long long kRest = 1ull << 63, kHuge = 1ull << 62;
  const int lane = t & 31;
  const int top = (s <= 3.4028234663852886e38f ? static_cast<int>(__float_as_uint(s) >> 23) - 127 : 145) - 57;
  // the sum of the parts of one level; kRest: there is something below them; kHuge: squares of 2^128 and more
  const auto level_sum = [&](int level) {
    const int at = 268 + top - 40 * level;  // a square's m^2 stands 2 E - at places above the level's unit
    unsigned long long sum = 0ull;
    bool rest = false, huge = false;
#pragma unroll 2
    for (int c = t; c < nchunk; c += 32 * G) {
      const uint4 v = row[c];
      const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t b = (q[i >> 1] >> (16 * (i & 1))) & 0x7fffu;
        const uint32_t m = b >= 128u ? (b & 127u) | 128u : b;
        const int sh = 2 * max(static_cast<int>(b >> 7), 1) - at;
        huge = huge || b >= 191u << 7;  // 2^64
        if (sh >= 0) {
          const unsigned long long part = static_cast<unsigned long long>(m * m) << min(sh, 63);
          sum += level == 0 ? part : sh < 40 ? part & ((1ull << 40) - 1) : 0ull;
        } else {
          const int r = min(-sh, 31);
          sum += (m * m) >> r;
          rest = rest || ((m * m) & ((1u << r) - 1u)) != 0u;
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (__any_sync(0xffffffffu, rest)) sum |= kRest;
    if (__any_sync(0xffffffffu, huge)) sum |= kHuge;
    if constexpr (G > 1) {
      unsigned long long* w = words + (level & 1) * G;  // (the other half is read until the next level's barrier)
      if (lane == 0) w[warp] = sum;
      meet<G>(grp);
      unsigned long long all = 0ull, flags = 0ull;
      for (int i = 0; i < G; ++i) {
        all += w[i] & (kHuge - 1);
        flags |= w[i] & (kRest | kHuge);
      }
      sum = all | flags;
    }
    return sum;
  };
  unsigned long long w = level_sum(0);
  if ((w & kHuge) != 0ull) return s;
  bool rest = (w & kRest) != 0ull;
  w &= kHuge - 1;
  // exponent of the result's last place; 32 to 36 bits of w lie below it
  const int lsb = max(64 - __clzll(static_cast<long long>(w)) - 24 + top, -149);
  const int shift = lsb - top;
  unsigned long long q = w >> shift;
  const unsigned long long below = w & ((1ull << shift) - 1), half = 1ull << (shift - 1);
  if (below >= half) {
    q += below > half || rest || (q & 1ull) != 0ull ? 1ull : 0ull;
  } else {
    unsigned long long gap = half - below;
    for (int level = 1; rest && gap < 65536ull; ++level) {
      gap <<= 40;
      w = level_sum(level);
      rest = (w & kRest) != 0ull;
      w &= kHuge - 1;
      if (w >= gap) {
        q += w > gap || rest || (q & 1ull) != 0ull ? 1ull : 0ull;
        break;
      }
      gap -= w;
    }
  }
  // (with lsb = -149 q may be below 2^23, a number without the leading bit: the same bits)
  const long long bits = (static_cast<long long>(lsb + 150) << 23) + static_cast<long long>(q) - (1ll << 23);
  return __uint_as_float(static_cast<uint32_t>(min(bits, 0x7f800000ll)));
}

// 16 bytes read once.  Not the read-only path: residual_out may be x or residual itself.
__device__ __forceinline__ uint4 ld_once(const uint4* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
  return r;
}

__device__ __forceinline__ uint32_t e4m3x2_of(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// RN(v / s) of two values from nv = -v, s and nrs = -RN(1 / s).  Markstein ("Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990): a quotient within one unit in the last place, corrected by its exact remainder times a
// correctly rounded reciprocal, is the correctly rounded quotient.  The product v * rs may be a little more than a unit
// off, hence two corrections.  s in [2^-100, 2^100]; values so small that their remainder underflows have code 0.
// (From -v, so that -0 stays -0: its remainder 0 times -rs, added to -0, is -0.)
__device__ __forceinline__ uint64_t quotient2(uint64_t nv, uint64_t nrs, uint64_t s) {
  uint64_t y = mul2(nv, nrs);
  y = fma2(fma2(y, s, nv), nrs, y);
  return fma2(fma2(y, s, nv), nrs, y);
}
__device__ __forceinline__ bool plain_scale(float s) { return s >= 0x1p-100f && s <= 0x1p100f; }

// RN(m / 448) for m >= 0, by the same steps with a constant's reciprocal where the remainder cannot underflow.
__device__ __forceinline__ float over_448(float m) {
  if (m >= 0x1p-90f && m <= 0x1p120f) {
    constexpr float kInv = 1.0f / 448.0f;
    float y = __fmul_rn(m, kInv);
    y = __fmaf_rn(__fmaf_rn(-y, 448.0f, m), kInv, y);
    return __fmaf_rn(__fmaf_rn(-y, 448.0f, m), kInv, y);
  }
  return __fdiv_rn(m, 448.0f);
}

// The 8 int8 codes of a chunk of -v.  slow: the row holds a NaN (code 0) or its scale is out of quotient2's range.
__device__ __forceinline__ uint2 codes_int8(const uint64_t (&nv)[4], float s, float rs, bool slow) {
  uint32_t u[8];
  if (!slow) {
    const uint64_t rs2 = pk(-rs, -rs), s2 = pk(s, s), mg = pk(kMagic, kMagic);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo, hi;
      upk(add2(quotient2(nv[i], rs2, s2), mg), lo, hi);
      u[2 * i] = __float_as_uint(lo);
      u[2 * i + 1] = __float_as_uint(hi);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float f[2];
      upk(nv[i], f[0], f[1]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // s = 0: every value is zero or a NaN; s = inf: quotients 0 or NaN
        const int r = s > 0.0f ? __float2int_rn(__fdiv_rn(-f[h], s)) : 0;  // a NaN converts to 0
        u[2 * i + h] = static_cast<uint32_t>(max(-127, min(127, r)));
      }
    }
  }
  return make_uint2(__byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410),
                    __byte_perm(__byte_perm(u[4], u[5], 0x0040), __byte_perm(u[6], u[7], 0x0040), 0x5410));
}

// The 8 E4M3 codes of a chunk of -v under scale s.
__device__ __forceinline__ uint2 codes_fp8(const uint64_t (&nv)[4], float s) {
  uint32_t c[4];
  if (plain_scale(s)) {
    const float rs = __frcp_rn(s);
    const uint64_t rs2 = pk(-rs, -rs), s2 = pk(s, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo, hi;
      upk(quotient2(nv[i], rs2, s2), lo, hi);
      c[i] = e4m3x2_of(lo, hi);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      upk(nv[i], a, b);
      a = -a;
      b = -b;
      // a block of zeros: +0, or NaN for a NaN value
      const float lo = s == 0.0f ? __fadd_rn(__fmul_rn(a, 0.0f), 0.0f) : __fdiv_rn(a, s);
      const float hi = s == 0.0f ? __fadd_rn(__fmul_rn(b, 0.0f), 0.0f) : __fdiv_rn(b, s);
      c[i] = e4m3x2_of(lo, hi);
    }
  }
  return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// Group grp's barrier of 32 G threads (ids as immediates: a register id would reserve all sixteen).
template <int G>
__device__ __forceinline__ void meet(int grp) {
  switch (grp) {
    case 0: asm volatile("bar.sync 1, %0;" ::"n"(32 * G) : "memory"); break;
    case 1: asm volatile("bar.sync 2, %0;" ::"n"(32 * G) : "memory"); break;
    case 2: asm volatile("bar.sync 3, %0;" ::"n"(32 * G) : "memory"); break;
    default: asm volatile("bar.sync 4, %0;" ::"n"(32 * G) : "memory"); break;
  }
}

// max of a group's values, the same in every thread; KeepNaN: a NaN among them is the result, else it is passed over.
template <bool KeepNaN, int G>
__device__ __forceinline__ float group_max(float m, float* red, int grp, int w, int lane) {
  const auto op = [](float a, float b) { return KeepNaN ? max_nan(a, b) : fmaxf(a, b); };
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = op(m, __shfl_xor_sync(0xffffffffu, m, o));
  if constexpr (G > 1) {
    if (lane == 0) red[w] = m;
    meet<G>(grp);
    m = red[lane % G];
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) m = op(m, __shfl_xor_sync(0xffffffffu, m, o));
  }
  return m;
}

// FORM: the output.  A group of G warps holds one row, CH chunks of 8 values a thread.
template <int G>
constexpr int kCtaWarps = G > 4 ? G : 4;

// CTAs a SM that the registers have to allow: all 64 warps with a chunk a thread, 36 with four (CTAs of four warps; larger
// ones 32).  exact_sum() alone would take more registers, and spills its own in that case.
template <int CH, int G>
constexpr int kCtas = CH == 1 ? 64 / kCtaWarps<G> : G <= 4 ? 9 : 32 / G;

template <int FORM, int CH, int G>
__global__ void __launch_bounds__(32 * kCtaWarps<G>, kCtas<CH, G>) norm_quant_kernel(const NormArgs a) {
  constexpr int kWarps = kCtaWarps<G>;
  constexpr int NG = kWarps / G;
  __shared__ float red_s[kWarps], red_c[kWarps], red_m[kWarps], red_n[kWarps];
  __shared__ unsigned long long words[2 * kWarps];
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int warp = static_cast<int>(threadIdx.x >> 5);
  const int grp = warp / G, w = warp % G;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * NG + grp;
  const int nchunk = a.K / 8;
  const int t = w * 32 + lane;
  const bool f32w = a.weight_f32;
  pdl_wait();
  if (row >= a.M) return;  // whole groups: their barriers are their own

  const int64_t at = row * a.K;
  uint4 v[CH];
  {
    const uint4* x = reinterpret_cast<const uint4*>(a.x + at);
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int c = 0; c < CH; ++c) v[c] = t + 32 * G * c < nchunk ? ld_once(x + t + 32 * G * c) : zero;
    if (a.residual != nullptr) {
      const uint4* p = reinterpret_cast<const uint4*>(a.residual + at);
      uint4 res[CH];
#pragma unroll
      for (int c = 0; c < CH; ++c) res[c] = t + 32 * G * c < nchunk ? ld_once(p + t + 32 * G * c) : zero;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        uint32_t* p0 = &v[c].x;
        const uint32_t q0[4] = {res[c].x, res[c].y, res[c].z, res[c].w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          // One rounding, the bits of the binary32 sum rounded to bf16: rounding to p bits by way of 2 p + 2 or more changes
          // no sum (Figueroa, "When is double rounding innocuous?", 1995), here 8 by way of 24.
          asm("add.rn.bf16x2 %0, %0, %1;" : "+r"(p0[i]) : "r"(q0[i]));
        if (t + 32 * G * c < nchunk) reinterpret_cast<uint4*>(a.residual_out + at)[t + 32 * G * c] = v[c];
      }
    }
  }

  // the sum of squares in two words, over the thread, the warp and the group
  float s = 0.0f, e = 0.0f;
  sum_squares<CH>(v, s, e);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float so = __shfl_xor_sync(0xffffffffu, s, o), eo = __shfl_xor_sync(0xffffffffu, e, o);
    two_sum(s, e, so, eo);
  }
  if constexpr (G > 1) {
    if (lane == 0) {
      red_s[warp] = s;
      red_c[warp] = e;
    }
    meet<G>(grp);
    s = red_s[grp * G + lane % G];
    e = red_c[grp * G + lane % G];
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) {
      const float so = __shfl_xor_sync(0xffffffffu, s, o), eo = __shfl_xor_sync(0xffffffffu, e, o);
      two_sum(s, e, so, eo);
    }
  }
  // S: s + e rounded where what e lost cannot change it, else the exact sum.  Below 2^-88 a sum counts only beside an eps
  // that is as small.  (All threads of a group have the same s and e, and go the same way.)
  float sum = s;
  bool sure = a.eps >= 0x1p-60f || s != s;
  if (s >= 0x1p-89f) {
    const float lost = __fmul_ru(s, slack<CH>());
    sum = __fadd_rn(s, __fsub_rd(e, lost));
    sure = sum == __fadd_rn(s, __fadd_ru(e, lost));
  }
  if (!sure)
    sum = exact_sum<G>(reinterpret_cast<const uint4*>((a.residual != nullptr ? a.residual_out : a.x) + at), nchunk, t, w, grp,
                       words + 2 * G * grp, s);
  const float g = __frsqrt_rn(__fadd_rn(__fdiv_rn(sum, static_cast<float>(a.K)), a.eps));

  // -v = (r * -g) * w
  uint64_t f[CH][4];
  const uint64_t ng2 = pk(-g, -g);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int idx = t + 32 * G * c;
    const uint32_t q0[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
    uint64_t wt[4] = {0ull, 0ull, 0ull, 0ull};
    if (idx < nchunk) {
      if (f32w) {
        const float4 w0 = reinterpret_cast<const float4*>(a.weight)[2 * idx];
        const float4 w1 = reinterpret_cast<const float4*>(a.weight)[2 * idx + 1];
        wt[0] = pk(w0.x, w0.y);
        wt[1] = pk(w0.z, w0.w);
        wt[2] = pk(w1.x, w1.y);
        wt[3] = pk(w1.z, w1.w);
      } else {
        const uint4 wb = reinterpret_cast<const uint4*>(a.weight)[idx];
        const uint32_t w4[4] = {wb.x, wb.y, wb.z, wb.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) wt[i] = wide2(w4[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      f[c][i] = mul2(mul2(wide2(q0[i]), ng2), wt[i]);
    if (idx >= nchunk) {  // (0 * inf above)
#pragma unroll
      for (int i = 0; i < 4; ++i) f[c][i] = 0ull;
    }
    if (a.y != nullptr && idx < nchunk) {
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float lo, hi;
        upk(f[c][i], lo, hi);
        o[i] = f32x2_to_bf16x2_bits(lo, hi) ^ 0x80008000u;
      }
      reinterpret_cast<uint4*>(a.y + at)[idx] = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }

  if constexpr (FORM == F_INT8) {
    float m = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float lo, hi;
        upk(f[c][i], lo, hi);
        m = max_abs3_nan(m, lo, hi);
      }
    m = group_max<true, G>(m, red_m + grp * G, grp, w, lane);
    const bool nan = m != m;
    if (nan) {  // rare, the whole group together: the maximum over the other values
      m = 0.0f;
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float lo, hi;
          upk(f[c][i], lo, hi);
          m = max_abs3(m, lo, hi);
        }
      m = group_max<false, G>(m, red_n + grp * G, grp, w, lane);
    }
    const float sc = __fdiv_rn(m, 127.0f);
    const bool slow = nan || !plain_scale(sc);
    const float rs = slow ? 0.0f : __frcp_rn(sc);
    if (t == 0) static_cast<float*>(a.scale)[row] = sc;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const uint2 q = codes_int8(f[c], sc, rs, slow);
      if (t + 32 * G * c < nchunk) reinterpret_cast<uint2*>(a.q + at)[t + 32 * G * c] = q;
    }
  } else {
    constexpr int kLanes = FORM == F_FP8 ? 16 : 4;  // lanes that share a scale
    const int64_t sat = row * ((nchunk + kLanes - 1) / kLanes);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int idx = t + 32 * G * c;
      float m = 0.0f;
      bool nan = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float lo, hi;
        upk(f[c][i], lo, hi);
        m = max_abs3(m, lo, hi);  // passes a NaN over
        nan = nan || lo != lo || hi != hi;
      }
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      if constexpr (FORM == F_FP8) {
        const float sc = over_448(m);
        const uint2 q = codes_fp8(f[c], sc);
        if (idx < nchunk) {
          reinterpret_cast<uint2*>(a.q + at)[idx] = q;
          if ((lane & 15) == 0) static_cast<float*>(a.scale)[sat + idx / 16] = sc;
        }
      } else {
        nan = (__ballot_sync(0xffffffffu, nan) >> (lane & ~3) & 15u) != 0u;
        // floor(log2 m) - 8 of the largest magnitude: at most 120, an infinity's, and no less than E8M0's lowest (m below
        // 2^-119)
        const int sh = max(-127, static_cast<int>(__float_as_uint(m) >> 23) - 127 - 8);
        const float inv = __uint_as_float(static_cast<uint32_t>(127 - sh) << 23);
        const uint64_t inv2 = pk(-inv, -inv);
        uint32_t k[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float lo, hi;
          upk(mul2(f[c][i], inv2), lo, hi);
          k[i] = e4m3x2_of(lo, hi);
        }
        if (idx < nchunk) {
          reinterpret_cast<uint2*>(a.q + at)[idx] = make_uint2(k[0] | k[1] << 16, k[2] | k[3] << 16);
          if ((lane & 3) == 0)
            static_cast<uint8_t*>(a.scale)[sat + idx / 4] =
                nan ? 0xffu : m > 0.0f ? static_cast<uint8_t>(sh + 127) : static_cast<uint8_t>(0u);
        }
      }
    }
  }
}

template <int FORM, int CH, int G>
cudaError_t go(const NormArgs& a, cudaStream_t stream) {
  constexpr int kWarps = kCtaWarps<G>;
  const int64_t ctas = (a.M + kWarps / G - 1) / (kWarps / G);
  return launch_pdl(norm_quant_kernel<FORM, CH, G>, dim3(static_cast<unsigned>(ctas)), dim3(32 * kWarps), 0, stream, a);
}

template <int FORM>
cudaError_t pick(const NormArgs& a, int num_sms, cudaStream_t stream) {
  const int nchunk = a.K / 8;
  // Four chunks a thread where the rows then still fill the GPU (16 warps a SM): a row's reductions are a warp's work,
  // so fewer warps a row leave fewer instructions.  Else a chunk a thread: the shortest way through a row.
  if (nchunk <= 32) return go<FORM, 1, 1>(a, stream);
  if (nchunk <= 1024 && a.M * ((nchunk + 127) / 128) < 16 * num_sms) {
    if (nchunk <= 64) return go<FORM, 1, 2>(a, stream);
    if (nchunk <= 128) return go<FORM, 1, 4>(a, stream);
    if (nchunk <= 256) return go<FORM, 1, 8>(a, stream);
    if (nchunk <= 512) return go<FORM, 1, 16>(a, stream);
    return go<FORM, 1, 32>(a, stream);
  }
  if (nchunk <= 128) return go<FORM, 4, 1>(a, stream);
  if (nchunk <= 256) return go<FORM, 4, 2>(a, stream);
  if (nchunk <= 512) return go<FORM, 4, 4>(a, stream);
  if (nchunk <= 1024) return go<FORM, 4, 8>(a, stream);
  if (nchunk <= 2048) return go<FORM, 4, 16>(a, stream);
  if (nchunk <= 4096) return go<FORM, 4, 32>(a, stream);
  return go<FORM, 8, 32>(a, stream);
}

}  // namespace

cudaError_t launch_norm_quant(const NormArgs& a, int form, int num_sms, cudaStream_t stream) {
  if (a.M == 0) return cudaSuccess;
  switch (form) {
    case 0: return pick<F_INT8>(a, num_sms, stream);
    case 1: return pick<F_FP8>(a, num_sms, stream);
    default: return pick<F_MX>(a, num_sms, stream);
  }
}

}  // namespace w8a8
