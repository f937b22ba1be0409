// Host-side declarations of the operators around the MoE layer: residual
// addition with RMS norm, the norms after and before a block with its gate and
// their gradient, the router in the score domain, the balance losses and the
// gradient of a routing, the gradient of the combination of the routes, and the
// shared MXFP4 projection with low-rank adapters.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mxmoe {

// h = x (+ residual); residual_out = bf16(h); y = h * rsqrt(mean(h^2) + eps) *
// gamma; out = bf16(y); q8 / s8 = MXFP8 of y (E4M3, one E8M0 scale per 32
// values; nosat != 0: the exponent raised where the block would saturate).
// Null pointers leave a part out (addnorm.cu).
struct AddNormArgs {
  const uint16_t* x;         // bf16 [T, K]
  const uint16_t* residual;  // bf16 [T, K] or null
  const uint16_t* gamma;     // bf16 [K]
  uint16_t* residual_out;    // bf16 [T, K] or null
  uint16_t* out;             // bf16 [T, K] or null
  uint8_t* q8;               // E4M3 [T, K] or null
  uint8_t* s8;               // E8M0 [T, K/32] or null
  int T, K, nosat;
  float eps;
};
cudaError_t launch_add_rmsnorm(const AddNormArgs& a, int num_sms, cudaStream_t stream);

// The norms after and before a block with its gate and the residual's scale
// (sandwich.cu). gate_kind 0: none, 1: bf16 [K], 2: fp32 [T], 3: bf16 [T, K];
// gate_act 1: sigmoid. Null pointers leave a part out.
struct SandwichArgs {
  const uint16_t* x;         // bf16 [T, K]
  const uint16_t* residual;  // bf16 [T, K]
  const uint16_t* post;      // bf16 [K] or null
  const uint16_t* pre;       // bf16 [K] or null
  const void* gate;
  const float* rscale;       // [1] or null: 1
  uint16_t* h_out;           // bf16 [T, K] or null; may be x or residual
  uint16_t* out;             // bf16 [T, K] or null
  uint8_t *q8, *s8;          // MXFP8 of y or null
  uint8_t *x8, *xs8;         // MXFP8 of x or null
  uint8_t *h8, *hs8;         // MXFP8 of h or null
  float* rstd;               // [2, T] or null
  int T, K, gate_kind, gate_act, nosat, ck_nosat;
  float eps;
};
cudaError_t launch_sandwich_norm(const SandwichArgs& a, int num_sms, cudaStream_t stream);

constexpr int kSwMaxCtas = 512;   // rows of column sums in the gradient's workspace
struct SandwichBwdArgs {
  const uint16_t *dh, *dy;   // bf16 [T, K], either may be null
  const void* x;             // bf16 [T, K], or E4M3 with xs
  const uint8_t* xs;         // E8M0 [T, K/32] or null
  const void* h;             // likewise; null without dy
  const uint8_t* hs;
  const float* rstd;         // [2, T]
  const uint16_t *post, *pre;
  const void* gate;
  const uint16_t* residual;  // bf16 [T, K], read for dscale only
  const float* rscale;       // [1] or null: 1
  uint16_t *dx, *dres;       // bf16 [T, K] or null
  float *dpost, *dpre;       // [K] or null
  void* dgate;               // fp32 [K] or [T], bf16 [T, K], or null
  float* dscale;             // [1] or null
  float* ws;
  int T, K, gate_kind, gate_act;
};
size_t sandwich_bwd_workspace_bytes(int T, int K);
cudaError_t launch_sandwich_norm_backward(const SandwichBwdArgs& a, int num_sms, cudaStream_t stream);

// Router in the score domain (router_scored.cu).
struct RouterScoredArgs {
  const float* logits;   // [T, E]
  const float* bias;     // [E] or null
  int T, E, topk, scoring, n_group, topk_group, group_top, renormalise;
  float route_scale;
  int32_t* ids;          // [T, topk]
  float* wts;            // [T, topk]
};
cudaError_t launch_router_scored(const RouterScoredArgs& a, int num_sms, cudaStream_t stream);

// Losses and counts of a routing, and the gradient of its logits (router_grad.cu).
struct RouterBalanceArgs {
  const float* logits;       // [T, E]
  const int32_t* ids;        // [T, topk]
  const int32_t* offsets;    // [S + 1] or null: one sequence of all rows
  int T, E, topk, scoring, S;
  float* stats;              // [4]
  int32_t* counts;           // [S, E]
  float *prob, *slope;       // [S, E]
  void* ws;
};
size_t router_balance_workspace_bytes(int T, int E, int S);
cudaError_t launch_router_balance(const RouterBalanceArgs& a, int num_sms, cudaStream_t stream);

struct RouterBackwardArgs {
  const float* logits;       // [T, E]
  const int32_t* ids;        // [T, topk]
  const float* dw;           // [T, topk] or null
  const float* dloss;        // [2] or null
  const float* stats;        // [4], with dloss
  const float* slope;        // [S, E], with dloss
  const int32_t* offsets;    // [S + 1] or null
  int T, E, topk, scoring, renormalise, S;
  float route_scale;
  float* dlogits;            // [T, E]
};
cudaError_t launch_router_backward(const RouterBackwardArgs& a, cudaStream_t stream);

// Gradient of y_t = sum_j w_tj o_tj (combine_grad.cu).
struct CombineBwdArgs {
  const uint16_t* dy;        // bf16 [T, K]
  const uint16_t* routes;    // bf16 [T * topk, K]
  const int32_t* ids;        // [T, topk] or null
  const float* wts;          // [T, topk], with droutes
  int T, K, topk, ebase, E;  // E 0: any id that is not negative
  float* dw;                 // [T, topk]
  uint16_t* droutes;         // bf16 [T * topk, K] or null
};
cudaError_t launch_combine_backward(const CombineBwdArgs& a, int num_sms, cudaStream_t stream);

constexpr int kLinearMaxAdapters = 1024;
constexpr int kLinearMaxRank = 256;

// y[t] = W x[t] + scale[a] B[a] (A[a] x[t]), a = ids[t] (linear.cu).
struct LinearArgs {
  const void* x;            // bf16 [T, K], or E4M3 [T, K] with xs
  const uint8_t* xs;        // E8M0 [T, K/32] or null
  const uint8_t* w;         // [N, K/2]
  const uint8_t* s;         // [N, K/32]
  const int32_t* ids;       // [T] or null: no adapters
  const uint16_t* a;        // bf16 [L, rank, K]
  const uint16_t* b;        // bf16 [L, N, rank]
  const float* ascale;      // [L] or null: 1
  uint16_t* out;            // bf16 [T, N]
  int32_t* status;          // [4] or null
  void* ws;
  int T, K, N, L, rank;
  int skip_copy;            // test only: this CTA's first copy of weights is left out; -1: none
};
size_t linear_workspace_bytes(int T, int K, int N, int rank, bool x8);
cudaError_t launch_linear(const LinearArgs& a, int num_sms, cudaStream_t stream);

}  // namespace mxmoe
