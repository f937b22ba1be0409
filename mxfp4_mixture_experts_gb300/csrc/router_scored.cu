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
// The choice has to be the same wherever the fp32 scores are, so they are
// computed as written: expf, IEEE addition and division, none of them
// contracted into another operation.
//
// One warp per token; lane l holds the NPL consecutive experts from l * NPL, so
// of equal candidates the lower lane holds the lower index. Candidates are
// compared as order-preserving unsigned keys (0: none): a choice is one
// warp-wide integer maximum, one ballot for the lowest lane that holds it, and
// a rescan of that lane's share. T x E floats are read once; small calls are
// bound by the launch, large ones by these rounds.
#include <cstdint>

#include "common.cuh"
#include "ops.h"

namespace mxmoe {
namespace {

constexpr int kRsWarps = 8;

// Order-preserving map of non-NaN floats to integers >= 1 (-0 as +0).
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(__fadd_rn(x, 0.f));
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

template <int NPL>
__global__ void __launch_bounds__(kRsWarps * 32)
    router_scored_kernel(const RouterScoredArgs a) {
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kRsWarps + (threadIdx.x >> 5);
  if (t >= a.T) return;
  const int E = a.E, e0 = lane * NPL;
  const float* row = a.logits + (size_t)t * E;
  float s[NPL];
  uint32_t key[NPL];   // 0: not a candidate
  float x[NPL];
#pragma unroll
  for (int j = 0; j < NPL; ++j) x[j] = e0 + j < E ? row[e0 + j] : -INFINITY;
  if (a.scoring == 0) {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < NPL; ++j) m = fmaxf(m, x[j]);   // NaN passes by
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
      s[j] = x[j] > -INFINITY ? (x[j] == m ? 1.f : expf(x[j] - m)) : 0.f;
      sum += s[j];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
#pragma unroll
    for (int j = 0; j < NPL; ++j) s[j] = sum > 0.f ? __fdiv_rn(s[j], sum) : 0.f;
  } else {
#pragma unroll
    for (int j = 0; j < NPL; ++j)
      s[j] = x[j] > -INFINITY ? __fdiv_rn(1.f, __fadd_rn(1.f, expf(-x[j]))) : 0.f;
  }
  float c[NPL];   // the biased scores, -inf for those that are out
#pragma unroll
  for (int j = 0; j < NPL; ++j) {
    c[j] = -INFINITY;
    if (x[j] > -INFINITY) {   // false for NaN too
      const float v = a.bias != nullptr ? __fadd_rn(s[j], a.bias[e0 + j]) : s[j];
      if (v > -INFINITY) c[j] = v;
    }
    key[j] = c[j] > -INFINITY ? order_key(a.bias != nullptr ? c[j] : x[j]) : 0u;
  }
  if (a.n_group > 1) {
    const int gs = E / a.n_group;
    uint32_t my_g = 0;   // lane g: key of group g's score
    for (int g = 0; g < a.n_group; ++g) {
      // the two largest keys of the scores in the group (0: none)
      uint32_t k1 = 0, k2 = 0;
#pragma unroll
      for (int j = 0; j < NPL; ++j) {
        if (e0 + j >= g * gs && e0 + j < (g + 1) * gs && c[j] > -INFINITY) {
          const uint32_t k = order_key(c[j]);
          k2 = max(k2, min(k1, k));
          k1 = max(k1, k);
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const uint32_t o1 = __shfl_xor_sync(0xffffffffu, k1, o);
        const uint32_t o2 = __shfl_xor_sync(0xffffffffu, k2, o);
        k2 = max(max(k2, o2), min(k1, o1));
        k1 = max(k1, o1);
      }
      auto value = [](uint32_t k) {
        return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
      };
      uint32_t gk = k1;
      if (a.group_top == 2 && k2 != 0) {
        const float sum = __fadd_rn(value(k1), value(k2));
        gk = sum != sum ? 0u : order_key(sum);
      }
      if (lane == g) my_g = gk;
    }
    uint32_t kept = 0;
    for (int r = 0; r < a.topk_group; ++r) {
      const uint32_t cand = (lane < a.n_group && !((kept >> lane) & 1u)) ? my_g : 0u;
      const uint32_t m = __reduce_max_sync(0xffffffffu, cand);
      if (m == 0) break;
      const uint32_t who = __ballot_sync(0xffffffffu, cand == m);
      kept |= who & (0u - who);
    }
#pragma unroll
    for (int j = 0; j < NPL; ++j)
      if (e0 + j < E && !((kept >> ((e0 + j) / gs)) & 1u)) key[j] = 0;
  }
  int my_e = -1;
  float my_s = 0.f;
  for (int r = 0; r < a.topk; ++r) {
    uint32_t best = 0;
    int bj = 0;
    float bs = 0.f;
#pragma unroll
    for (int j = NPL - 1; j >= 0; --j)
      if (key[j] >= best) {
        best = key[j];
        bj = j;
        bs = s[j];
      }
    const uint32_t m = __reduce_max_sync(0xffffffffu, best);
    if (m == 0) break;   // no candidate left
    const int src = __ffs(__ballot_sync(0xffffffffu, best == m)) - 1;
    const int e = __shfl_sync(0xffffffffu, e0 + bj, src);
    const float sv = __shfl_sync(0xffffffffu, bs, src);
    if (lane == r) {
      my_e = e;
      my_s = sv;
    }
    if (lane == src) {
#pragma unroll
      for (int j = 0; j < NPL; ++j)
        if (j == bj) key[j] = 0;
    }
  }
  float w = my_s;   // 0 in lanes past the choices
  if (a.renormalise) {
    float sum = my_s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    w = sum > 0.f ? my_s / sum : 0.f;
  }
  if (lane < a.topk) {
    a.ids[(size_t)t * a.topk + lane] = my_e;
    a.wts[(size_t)t * a.topk + lane] = w * a.route_scale;
  }
}

}  // namespace

cudaError_t launch_router_scored(const RouterScoredArgs& a, int num_sms, cudaStream_t stream) {
  (void)num_sms;
  const unsigned blocks = (unsigned)((a.T + kRsWarps - 1) / kRsWarps);
  const int npl = (a.E + 31) / 32;
#define MXMOE_RS(N) router_scored_kernel<N><<<blocks, kRsWarps * 32, 0, stream>>>(a)
  if (npl <= 1) MXMOE_RS(1);
  else if (npl <= 2) MXMOE_RS(2);
  else if (npl <= 4) MXMOE_RS(4);
  else if (npl <= 8) MXMOE_RS(8);
  else if (npl <= 16) MXMOE_RS(16);
  else MXMOE_RS(32);
#undef MXMOE_RS
  return cudaGetLastError();
}

}  // namespace mxmoe
