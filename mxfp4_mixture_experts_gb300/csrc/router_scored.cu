// Router in the score domain: top-k experts by their scores plus a balance
// bias, weighted by the unbiased scores.
//
//   s_e = sigmoid(x_e), or softmax(x)_e over all E experts           fp32
//   c_e = s_e + bias_e                                               one fp32 addition
//   groups (n_group > 1): a group's score is the sum of its group_top (1 or 2)
//     largest c; the topk_group best groups (ties to the lower index) stay
//   the k largest c are chosen (ties to the lower expert); without a bias the
//     logits decide, which order as the scores do without the ties that the
//     rounding of a score near 0 or 1 would add
//   w_j = s_j, divided by the sum of the chosen s when renormalising, times
//     route_scale
// An expert whose logit or biased score is NaN or -inf is out: it is never
// chosen and a NaN or -inf logit scores 0. A slot with no expert left gets id
// -1 (padding for the layer) and weight 0; a chosen sum of 0 gives weights 0.
//
// Scores are computed as written: expf, IEEE addition and division, none of them
// contracted into another operation. A choice by logits (no bias, one group) or by
// sigmoid scores is then the same in every fp32 evaluation of the formula by the same
// expf. A softmax score has a sum in it whose last bits go by the order of its terms
// (here a lane's, then a tree): with a bias or groups, experts that lie within 2^-20
// of one another may change places against another order.
//
// One warp per token. Each group gets 32 / n_group neighbouring lanes (all of
// them without groups), each lane consecutive experts, so of equal candidates
// the lower lane holds the lower index, and the two best of every group come
// from shuffles inside its lanes, all groups at once. Candidates are compared as
// order-preserving unsigned keys (0: none): a choice is one maximum over the
// lane's keys, one over the warp, and one ballot for the lowest lane that holds it; the
// scores of the chosen are recomputed from their logits at the end. T x E
// floats are read once; small calls are bound by the launch and one token's
// chain of these rounds, large ones by their instructions.
#include <cstdint>

#include "common.cuh"
#include "ops.h"

namespace mxmoe {
namespace {

constexpr int kRsWarps = 8;

// Order-preserving map of non-NaN floats to integers >= 1 (-0 as +0), and back.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(__fadd_rn(x, 0.f));
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);   // negative: all bits, else the sign
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
// A group's key from the keys of its two largest scores (0: none).
__device__ __forceinline__ uint32_t group_key(uint32_t k1, uint32_t k2, int top) {
  if (top == 1 || k2 == 0) return k1;
  const float sum = __fadd_rn(key_value(k1), key_value(k2));
  return sum != sum ? 0u : order_key(sum);
}
__device__ __forceinline__ void top2(uint32_t& k1, uint32_t& k2, uint32_t k) {
  k2 = max(k2, min(k1, k));
  k1 = max(k1, k);
}

// NPL: experts per lane (at least `per`, those that the mapping gives a lane).
// lpg: lanes per group, 32 without groups or with a group count that does not
// divide 32.
template <int NPL>
__global__ void __launch_bounds__(kRsWarps * 32)
    router_scored_kernel(const RouterScoredArgs a, int lpg, int per, int vec) {
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kRsWarps + (threadIdx.x >> 5);
  if (t >= a.T) return;
  const int E = a.E;
  const bool by_lanes = lpg < 32;               // a group is a run of lanes
  const int gs = E / a.n_group;
  const int run = by_lanes ? gs : E;            // experts of a run of lpg lanes
  const int in_run = (lane % lpg) * per;
  const int e0 = lane / lpg * run + in_run;
  const int mine = max(0, min(per, run - in_run));
  const float* row = a.logits + (size_t)t * E;
  const bool biased = a.bias != nullptr;
  float x[NPL];
  if (NPL >= 4 && vec) {   // per, gs and E multiples of 4, rows 16-byte aligned
#pragma unroll
    for (int j = 0; j < NPL; j += 4) {
      float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (j < mine) v = __ldg(reinterpret_cast<const float4*>(row + e0 + j));
      x[j] = v.x;
      x[j + (NPL > 1 ? 1 : 0)] = v.y;
      x[j + (NPL > 2 ? 2 : 0)] = v.z;
      x[j + (NPL > 3 ? 3 : 0)] = v.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < NPL; ++j) x[j] = j < mine ? __ldg(row + e0 + j) : -INFINITY;
  }
  float m = -INFINITY, total = 0.f;   // softmax: largest logit, sum of exponentials
  if (a.scoring == 0) {
#pragma unroll
    for (int j = 0; j < NPL; ++j) m = fmaxf(m, x[j]);   // NaN passes by
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll
    for (int j = 0; j < NPL; ++j)
      total += x[j] > -INFINITY ? (x[j] == m ? 1.f : expf(x[j] - m)) : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  }
  auto score = [&](float v) -> float {
    if (!(v > -INFINITY)) return 0.f;   // NaN too
    if (a.scoring == 0) return __fdiv_rn(v == m ? 1.f : expf(v - m), total);
    return __frcp_rn(__fadd_rn(1.f, expf(-v)));   // (the rounded 1 / x, as a division gives it)
  };
  uint32_t key[NPL];   // of what the choice goes by; 0: out
  if (biased || a.n_group > 1) {
    uint32_t ck[NPL];   // of the biased scores
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
      float c = -INFINITY;
      if (x[j] > -INFINITY) {
        c = score(x[j]);
        if (biased) c = __fadd_rn(c, __ldg(a.bias + e0 + j));
      }
      ck[j] = c > -INFINITY ? order_key(c) : 0u;
      key[j] = biased || ck[j] == 0 ? ck[j] : order_key(x[j]);
    }
    if (by_lanes) {
      uint32_t k1 = 0, k2 = 0;
#pragma unroll
      for (int j = 0; j < NPL; ++j) top2(k1, k2, ck[j]);
      for (int o = 1; o < lpg; o <<= 1) {
        const uint32_t o1 = __shfl_xor_sync(0xffffffffu, k1, o);
        const uint32_t o2 = __shfl_xor_sync(0xffffffffu, k2, o);
        k2 = max(max(k2, o2), min(k1, o1));
        k1 = max(k1, o1);
      }
      const uint32_t gk = group_key(k1, k2, a.group_top);
      const int g = lane / lpg;
      int beaten = 0;   // groups before this one: larger, or equal and lower
      for (int i = 0; i < a.n_group; ++i) {
        const uint32_t other = __shfl_sync(0xffffffffu, gk, i * lpg);
        beaten += other > gk || (other == gk && i < g);
      }
      if (beaten >= a.topk_group) {
#pragma unroll
        for (int j = 0; j < NPL; ++j) key[j] = 0;
      }
    } else if (a.n_group > 1) {
      uint32_t my_g = 0;   // lane g: group g's key
      for (int g = 0; g < a.n_group; ++g) {
        uint32_t k1 = 0, k2 = 0;
#pragma unroll
        for (int j = 0; j < NPL; ++j)
          if (e0 + j >= g * gs && e0 + j < (g + 1) * gs) top2(k1, k2, ck[j]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const uint32_t o1 = __shfl_xor_sync(0xffffffffu, k1, o);
          const uint32_t o2 = __shfl_xor_sync(0xffffffffu, k2, o);
          k2 = max(max(k2, o2), min(k1, o1));
          k1 = max(k1, o1);
        }
        if (lane == g) my_g = group_key(k1, k2, a.group_top);
      }
      uint32_t kept = 0;
      for (int r = 0; r < a.topk_group; ++r) {
        const uint32_t cand = (lane < a.n_group && !((kept >> lane) & 1u)) ? my_g : 0u;
        const uint32_t best = __reduce_max_sync(0xffffffffu, cand);
        if (best == 0) break;
        const uint32_t who = __ballot_sync(0xffffffffu, cand == best);
        kept |= who & (0u - who);
      }
#pragma unroll
      for (int j = 0; j < NPL; ++j)
        if (e0 + j < E && !((kept >> ((e0 + j) / gs)) & 1u)) key[j] = 0;
    }
  } else {
#pragma unroll
    for (int j = 0; j < NPL; ++j) key[j] = x[j] > -INFINITY ? order_key(x[j]) : 0u;
  }
  int my_e = -1;
  for (int r = 0; r < a.topk; ++r) {
    uint32_t best = 0;
#pragma unroll
    for (int j = 0; j < NPL; ++j) best = max(best, key[j]);
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    if (top == 0) break;   // no candidate left
    const int src = __ffs(__ballot_sync(0xffffffffu, best == top)) - 1;
    int j0 = 0;
    if (lane == src) {   // its first expert with that key is taken
      bool found = false;
#pragma unroll
      for (int j = 0; j < NPL; ++j)
        if (!found && key[j] == top) {
          found = true;
          j0 = j;
          key[j] = 0;
        }
    }
    const int e = __shfl_sync(0xffffffffu, e0 + j0, src);
    if (lane == r) my_e = e;
  }
  const float s = my_e >= 0 ? score(__ldg(row + my_e)) : 0.f;   // 0 in lanes past the choices
  float w = s;
  if (a.renormalise) {
    float sum = s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    w = sum > 0.f ? s / sum : 0.f;
  }
  if (lane < a.topk) {
    a.ids[(size_t)t * a.topk + lane] = my_e;
    a.wts[(size_t)t * a.topk + lane] = w * a.route_scale;
  }
}

}  // namespace

cudaError_t launch_router_scored(const RouterScoredArgs& a, int num_sms, cudaStream_t stream) {
  (void)num_sms;
  const unsigned blocks = ((unsigned)a.T + kRsWarps - 1) / kRsWarps;   // (T + 7 may pass 2^31)
  const int lpg = a.n_group > 1 && 32 % a.n_group == 0 ? 32 / a.n_group : 32;
  const int run = lpg < 32 ? a.E / a.n_group : a.E;
  const int per = (run + lpg - 1) / lpg;
  const int vec = per % 4 == 0 && run % 4 == 0 && a.E % 4 == 0 &&
                  (reinterpret_cast<uintptr_t>(a.logits) & 15) == 0;
#define MXMOE_RS(N) router_scored_kernel<N><<<blocks, kRsWarps * 32, 0, stream>>>(a, lpg, per, vec)
  if (per <= 1) MXMOE_RS(1);
  else if (per <= 2) MXMOE_RS(2);
  else if (per <= 4) MXMOE_RS(4);
  else if (per <= 8) MXMOE_RS(8);
  else if (per <= 16) MXMOE_RS(16);
  else MXMOE_RS(32);
#undef MXMOE_RS
  return cudaGetLastError();
}

}  // namespace mxmoe
