// Host-side declarations of the operators around the MoE layer: residual
// addition with RMS norm, the router in the score domain and the shared MXFP4
// projection with low-rank adapters.
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
