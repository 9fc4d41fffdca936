// gate.cu -- expert router: logits [T,E] -> the k chosen experts of each
// token and their weights (the topk_ids and topk_weights of the MoE layers).
//
//   live     an expert whose logit is above -inf (a NaN or -inf logit masks it)
//   score    sigmoid: s = 1 / (1 + exp(-l)); softmax: s = exp(l - m) / S over
//            the live experts, m their largest logit, S the sum
//   key      s + bias where a bias is given, else s (softmax: exp(l - m), the
//            same order); a masked expert, or a key of -inf or NaN, ranks below
//            every other
//   groups   n_group runs of E / n_group experts; a group's score is its largest
//            key, or the sum of its two largest ("top2"; a second key that is
//            masked counts 0); the topk_group best groups stay
//   choice   the k largest keys of those groups in falling order, ties to the
//            lowest index; slots that only masked experts are left for take
//            them by index
//   weight   s of the chosen (0 for a masked one); renormalised: divided by
//            their sum (0 where the sum is 0); times routed_scale
//
// exp, the reciprocal and every sum that decides an order are binary32
// operations rounded as the formulas read, so that equal keys are equal
// bit for bit.  S is summed with the rounding errors carried along (Knuth's
// two-sum), so that its last bit does not depend on the order of the sum.
//
// L lanes per token (32; 8 or 16 for many tokens of few experts); lane l holds
// the experts [l * P, l * P + P), P = the experts per lane.  A choice is the
// maximum of the lanes' best keys (as order-preserving integers) at the lowest
// lane holding it.  Traffic is one read of the logits and 12 bytes per choice.
// What bounds large batches is the issue of about 190 warp instructions a token
// (65536 tokens, 64 experts, top-8: 13.8 us, issuing in 72 % of the SMs' active
// cycles); a wave of CTAs or less its latency (16384 such tokens 6.1 us at 53 %,
// top-2 of them 5.2, the reads and writes alone 0.5); small batches the chain of
// k choices (128 tokens, 256 experts in 8 groups of which 4 stay, top-8: 3.2 us).
#include "fp8.cuh"

namespace w8a8 {

namespace {

constexpr int kGateWarps = 4;
constexpr float kNegInf = -INFINITY;

// Order-preserving map of binary32 (no NaN) to unsigned: larger values get larger integers; 0 is below all.
__device__ __forceinline__ uint32_t ordered(float f) {
  const uint32_t u = __float_as_uint(f);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
constexpr uint32_t kOrderedNegInf = 0x007fffffu;  // ordered(-inf)

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
  if constexpr (BF16) return bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i]);
  else return static_cast<const float*>(p)[i];
}

// P consecutive values of a row from i0, by 16-byte loads (the caller checks the alignment).
template <int P, bool BF16>
__device__ __forceinline__ void load_row(const void* p, int64_t i0, float (&l)[P]) {
  if constexpr (BF16 && P % 8 == 0) {
#pragma unroll
    for (int i = 0; i < P; i += 8) {
      const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i0 + i);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        l[i + 2 * j] = __uint_as_float(w[j] << 16);
        l[i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
    }
  } else if constexpr (!BF16 && P % 4 == 0) {
#pragma unroll
    for (int i = 0; i < P; i += 4) {
      const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i0 + i);
      l[i] = v.x;
      l[i + 1] = v.y;
      l[i + 2] = v.z;
      l[i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i) l[i] = load_logit<BF16>(p, i0 + i);
  }
}

__device__ __forceinline__ float sigmoid_rn(float x) { return __frcp_rn(__fadd_rn(1.0f, expf(-x))); }

// a + b as the rounded sum s and its error e, exactly (Knuth, TAOCP vol. 2, 4.2.2).
__device__ __forceinline__ void two_sum(float a, float b, float& s, float& e) {
  s = __fadd_rn(a, b);
  const float t = __fsub_rn(s, a);
  e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t));
}

// A group's score from its two largest keys (a masked second counts 0), order-preserving.
__device__ __forceinline__ uint32_t group_key(uint32_t k1, uint32_t k2, bool top2) {
  if (!top2 || k1 <= kOrderedNegInf) return k1;
  return ordered(__fadd_rn(unordered(k1), k2 > kOrderedNegInf ? unordered(k2) : 0.0f));
}

struct GateArgs {
  int full;  // P divides E, and logits and bias allow 16-byte loads
  const void* logits;
  const float* bias;
  int64_t T;
  int E, k, n_group, topk_group;
  bool top2, renorm;
  float scale;
  int64_t* ids;
  float* weights;
};

// L lanes a token, P experts a lane.
template <int L, int P, bool BF16, bool SIGMOID>
__global__ void __launch_bounds__(32 * kGateWarps) gate_kernel(const GateArgs a) {
  pdl_trigger();
  pdl_wait();
  constexpr int kTokens = 32 / L;  // of a warp
  const int lane = threadIdx.x % L;           // within the token's lanes
  const int first = threadIdx.x % 32 - lane;  // the token's first lane
  int64_t t = (static_cast<int64_t>(blockIdx.x) * kGateWarps + threadIdx.x / 32) * kTokens;
  if (t >= a.T) return;
  t += first / L;
  const bool live = t < a.T;  // a warp's last tokens may not be there: they repeat the last one and store nothing
  if (!live) t = a.T - 1;
  const int E = a.E;
  const int64_t row = t * E;
  float l[P], bias[P];
  if (a.full && lane * P < E) {
    load_row<P, BF16>(a.logits, row + lane * P, l);
    if (a.bias != nullptr) load_row<P, false>(a.bias, lane * P, bias);
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int e = lane * P + i;
      l[i] = e < E ? load_logit<BF16>(a.logits, row + e) : kNegInf;
      if (a.bias != nullptr) bias[i] = e < E ? a.bias[e] : 0.0f;
    }
  }
#pragma unroll
  for (int i = 0; i < P; ++i)
    if (!(l[i] > kNegInf)) l[i] = kNegInf;  // NaN
  float m = kNegInf, S = 0.0f;
  uint32_t key[P];
  if constexpr (SIGMOID) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      float s = sigmoid_rn(l[i]);
      if (a.bias != nullptr) s = __fadd_rn(s, bias[i]);
      key[i] = (l[i] > kNegInf && s > kNegInf) ? ordered(s) : kOrderedNegInf;
    }
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i) m = fmaxf(m, l[i]);
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float ex[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const float x = expf(l[i] == m ? 0.0f : __fsub_rn(l[i], m));
      ex[i] = l[i] > kNegInf ? x : 0.0f;
    }
    if (a.bias != nullptr || !a.renorm) {
      float err = 0.0f;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        float e;
        two_sum(S, ex[i], S, e);
        err += e;
      }
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) {
        const float S2 = __shfl_xor_sync(0xffffffffu, S, o), err2 = __shfl_xor_sync(0xffffffffu, err, o);
        float e;
        two_sum(S, S2, S, e);
        err = err + err2 + e;
      }
      S = __fadd_rn(S, err);
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
      float s = ex[i];
      if (a.bias != nullptr) s = __fadd_rn(__fdiv_rn(s, S), bias[i]);
      key[i] = (l[i] > kNegInf && s > kNegInf) ? ordered(s) : kOrderedNegInf;
    }
  }
  if (E != L * P) {
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (lane * P + i >= E) key[i] = 0u;
  }

  if (a.topk_group < a.n_group) {
    const int gs = E / a.n_group;
    // group scores: every lane of group g's lanes holds its key, and then whether the group stays: fewer than
    // topk_group groups rank above it
    const int lanes = gs / P;
    if (lanes * P == gs && (lanes & (lanes - 1)) == 0) {  // a group is a power of two of whole lanes
      uint32_t k1 = key[0], k2 = 0u;
#pragma unroll
      for (int i = 1; i < P; ++i) {
        k2 = max(k2, min(k1, key[i]));
        k1 = max(k1, key[i]);
      }
      for (int o = 1; o < lanes; o <<= 1) {
        const uint32_t o1 = __shfl_xor_sync(0xffffffffu, k1, o), o2 = __shfl_xor_sync(0xffffffffu, k2, o);
        k2 = max(max(k2, o2), min(k1, o1));
        k1 = max(k1, o1);
      }
      const uint32_t gk = group_key(k1, k2, a.top2);
      const int mine = lane / lanes;
      int above = 0;
      for (int g = 0; g < a.n_group; ++g) {
        const uint32_t other = __shfl_sync(0xffffffffu, gk, first + g * lanes);
        above += other > gk || (other == gk && g < mine) ? 1 : 0;
      }
      if (above >= a.topk_group) {
#pragma unroll
        for (int i = 0; i < P; ++i) key[i] = 0u;
      }
    } else if constexpr (L == 32) {  // through shared memory: lane g scans group g's keys (n_group <= 32)
      __shared__ uint32_t s_gkey[kGateWarps][32 * P];
      uint32_t* sk = s_gkey[threadIdx.x / 32];
#pragma unroll
      for (int i = 0; i < P; ++i)
        if (lane * P + i < E) sk[lane * P + i] = key[i];
      __syncwarp();
      uint32_t gk = 0u;
      if (lane < a.n_group) {
        uint32_t k1 = 0u, k2 = 0u;
        for (int j = 0; j < gs; ++j) {
          const uint32_t v = sk[lane * gs + j];
          k2 = max(k2, min(k1, v));
          k1 = max(k1, v);
        }
        gk = group_key(k1, k2, a.top2);
      }
      int above = 0;
      for (int g = 0; g < a.n_group; ++g) {
        const uint32_t other = __shfl_sync(0xffffffffu, gk, g);
        above += other > gk || (other == gk && g < lane) ? 1 : 0;
      }
      const uint32_t keep = __ballot_sync(0xffffffffu, lane < a.n_group && above < a.topk_group);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int e = lane * P + i;
        if (e < E && !((keep >> (e / gs)) & 1u)) key[i] = 0u;
      }
    }
  }

  // The k <= L largest keys; lane j keeps choice j: the maximum of the lanes' best keys, at its lowest lane.
  int my_id = 0;
  uint32_t my_key = 0u;
  if constexpr (L == 32) {
    // A lane knows its two best (keys and places) and moves the second up when its best is taken.  Only a lane that
    // gave both looks through its keys again.
    uint32_t b1, b2, taken = 0u;
    int a1, a2;
    auto two_best = [&]() {
      b1 = b2 = 0u;
      a1 = a2 = 0;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const uint32_t v = (taken >> i) & 1u ? 0u : key[i];
        const bool best = v > b1, second = v > b2;  // places in rising order: ties stay with the lower
        b2 = best ? b1 : second ? v : b2;
        a2 = best ? a1 : second ? i : a2;
        b1 = best ? v : b1;
        a1 = best ? i : a1;
      }
    };
    two_best();
    for (int j = 0; j < a.k; ++j) {
      const uint32_t top = __reduce_max_sync(0xffffffffu, b1);
      const int w = __ffs(__ballot_sync(0xffffffffu, b1 == top)) - 1;
      const int id = __shfl_sync(0xffffffffu, lane * P + a1, w);
      if (lane == j) {
        my_id = id;
        my_key = top;
      }
      if (lane == w) {
        taken |= 1u << a1;
        b1 = b2;
        a1 = a2;
        b2 = 0u;
        if (b1 == 0u) two_best();
      }
    }
  } else {
    // A lane sorts its keys once, so that a choice costs the warp's tokens the same few steps.  Neighbours change
    // places only where the later key is larger: equal keys stay in the order of their places.
    uint32_t place[P];
#pragma unroll
    for (int i = 0; i < P; ++i) place[i] = i;
#pragma unroll
    for (int r = 0; r < P; ++r)
#pragma unroll
      for (int i = r & 1; i + 1 < P; i += 2) {
        const bool swap = key[i + 1] > key[i];
        const uint32_t k0 = key[i], p0 = place[i];
        key[i] = swap ? key[i + 1] : k0;
        place[i] = swap ? place[i + 1] : p0;
        key[i + 1] = swap ? k0 : key[i + 1];
        place[i + 1] = swap ? p0 : place[i + 1];
      }
    uint32_t places = 0u;  // four bits each, the best lowest
#pragma unroll
    for (int i = 0; i < P; ++i) places |= place[i] << (4 * i);
    for (int j = 0; j < a.k; ++j) {
      uint32_t top = key[0];
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      const uint32_t at = __ballot_sync(0xffffffffu, key[0] == top) >> first;
      const int w = __ffs(at) - 1;  // below L: one of the token's own lanes holds it
      const int id = __shfl_sync(0xffffffffu, lane * P + static_cast<int>(places & 15u), first + w);
      if (lane == j) {
        my_id = id;
        my_key = top;
      }
      if (lane == w) {
#pragma unroll
        for (int i = 0; i + 1 < P; ++i) key[i] = key[i + 1];
        key[P - 1] = 0u;
        places >>= 4;
      }
    }
  }
  float wgt = 0.0f;
  if (lane < a.k && my_key > kOrderedNegInf) {
    const float x = load_logit<BF16>(a.logits, row + my_id);
    if constexpr (SIGMOID) wgt = sigmoid_rn(x);
    else wgt = x == m ? 1.0f : expf(__fsub_rn(x, m));
  }
  if (a.renorm) {
    float d = wgt;
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    wgt = d > 0.0f ? __fdiv_rn(wgt, d) : 0.0f;
  } else if constexpr (!SIGMOID) {
    wgt = S > 0.0f ? __fdiv_rn(wgt, S) : 0.0f;
  }
  if (live && lane < a.k) {
    a.ids[t * a.k + lane] = my_id;
    a.weights[t * a.k + lane] = wgt * a.scale;
  }
}

template <int L, int P>
cudaError_t launch_p(GateArgs a, bool bf16, bool sigmoid, cudaStream_t stream) {
  constexpr int per = kGateWarps * 32 / L;  // tokens of a CTA
  const dim3 g(static_cast<unsigned>((a.T + per - 1) / per)), b(32 * kGateWarps);
  const auto aligned = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0u; };
  a.full = a.E % P == 0 && aligned(a.logits) && aligned(a.bias) ? 1 : 0;
  if (bf16) {
    return sigmoid ? launch_pdl(gate_kernel<L, P, true, true>, g, b, 0, stream, a)
                   : launch_pdl(gate_kernel<L, P, true, false>, g, b, 0, stream, a);
  }
  return sigmoid ? launch_pdl(gate_kernel<L, P, false, true>, g, b, 0, stream, a)
                 : launch_pdl(gate_kernel<L, P, false, false>, g, b, 0, stream, a);
}

}  // namespace

cudaError_t launch_gate(const void* logits, bool bf16, int64_t T, int E, const float* bias, bool sigmoid, int n_group,
                        int topk_group, bool top2, int k, bool renorm, float scale, int64_t* ids, float* weights,
                        cudaStream_t stream) {
  if (T == 0) return cudaSuccess;
  const GateArgs a{0, logits, bias, T, E, k, n_group, topk_group, top2, renorm, scale, ids, weights};
  // Many tokens of few experts: 8 or 16 lanes a token, so that the steps of a choice serve four or two tokens.  Softmax
  // without groups, top-8 (top-2), against a warp a token: E = 32 at 2048 tokens 2.4 (2.0) us against 3.7 (2.9), 16384
  // 4.8 (3.8) against 6.1 (5.4); E = 64 at 2048 3.2 (2.8) against 4.9 (3.5), 16384 6.1 (5.2) against 8.3 (6.0), 65536
  // 13.8 (11.7) against 28.6 (19.1); E = 128 at 8192 6.6 (5.3) against 5.8 (4.2), 16384 8.5 (6.8) against 9.8 (6.7),
  // 65536 27.9 (22.2) against 33.9 (22.7).  (E = 256 in 16 lanes of 16: 57.8 us at 65536, against 47.)  Groups have to
  // be whole lanes.
  const auto whole = [=](int P) {
    const int gs = E / n_group, lanes = gs / P;
    return topk_group == n_group || (lanes * P == gs && (lanes & (lanes - 1)) == 0);
  };
  if (T >= 2048 && E <= 32 && k <= 8 && whole(4)) return launch_p<8, 4>(a, bf16, sigmoid, stream);
  if (T >= 2048 && E > 32 && E <= 64 && k <= 8 && whole(8)) return launch_p<8, 8>(a, bf16, sigmoid, stream);
  if (T >= 16384 && E > 64 && E <= 128 && k <= 16 && whole(8)) return launch_p<16, 8>(a, bf16, sigmoid, stream);
  // experts per lane: as few as hold E, so that common counts (96, 160, 192, 384 and the powers of two) fill every lane
  // and their groups are whole lanes
  const int P = (E + 31) / 32;
  if (P <= 1) return launch_p<32, 1>(a, bf16, sigmoid, stream);
  if (P <= 2) return launch_p<32, 2>(a, bf16, sigmoid, stream);
  if (P <= 3) return launch_p<32, 3>(a, bf16, sigmoid, stream);
  if (P <= 4) return launch_p<32, 4>(a, bf16, sigmoid, stream);
  if (P <= 5) return launch_p<32, 5>(a, bf16, sigmoid, stream);
  if (P <= 6) return launch_p<32, 6>(a, bf16, sigmoid, stream);
  if (P <= 8) return launch_p<32, 8>(a, bf16, sigmoid, stream);
  if (P <= 12) return launch_p<32, 12>(a, bf16, sigmoid, stream);
  if (P <= 16) return launch_p<32, 16>(a, bf16, sigmoid, stream);
  return launch_p<32, 32>(a, bf16, sigmoid, stream);
}

}  // namespace w8a8
