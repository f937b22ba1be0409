// Gradient of the layer's combination of its routes, y_t = sum_j w_tj o_tj.
//
//   dw_tj = sum_k dy_tk o_tjk (fp32)        do_tj = bf16(w_tj dy_t)
//
// HBM-bound: k rows of o read for one of dy, and k written where the routes'
// gradients are wanted. A warp per route, a CTA of 8 warps on routes that follow one
// another, so that a token's dy leaves L2 about once; with few routes several warps
// share one. T = 4096, K = 6144, top 8: weights alone 65 us = 6.97 TB/s, with the routes'
// gradients 126 us = 6.80 TB/s, the copy rate. (Without the 4 CTAs of the launch bounds the compiler
// takes 36 registers and waits for every second load: 81 us.)
#include <cstdint>

#include "ops.h"
#include "rows.cuh"

namespace mxmoe {
namespace {

constexpr int kCbWarps = 8;

// Loads that are issued where they are written, several before the first use; stores of rows that
// pass once.
__device__ __forceinline__ uint4 ld_stream16(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ void st_stream16(uint16_t* p, const uint4& v) {
  asm volatile("st.global.cs.v4.u32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// SPLIT: warps of a route. The sum does not depend on it: a lane's chunks 32 apart go to 4 sums
// in turn, these are added up in order, and the lanes last.
template <bool ROUTES, int SPLIT>
__global__ void __launch_bounds__(32 * kCbWarps, 4) combine_backward_kernel(const CombineBwdArgs a) {
  constexpr int V = 4 / SPLIT;   // sums of a warp: chunks of 8 values loaded together
  __shared__ float part[SPLIT > 1 ? kCbWarps : 1][V][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % SPLIT;
  const unsigned routes = (unsigned)a.T * (unsigned)a.topk;   // below 2^31
  const unsigned r = blockIdx.x * (kCbWarps / SPLIT) + warp / SPLIT;
  const int n8 = a.K / 8;
  float acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.f;
  if (r < routes) {
    bool live = true;
    if (a.ids != nullptr) {
      const int id = a.ids[r];
      live = a.E == 0 ? id >= 0 : id >= a.ebase && id - a.ebase < a.E;
    }
    const uint16_t* dy = a.dy + (size_t)(r / (unsigned)a.topk) * a.K;
    const uint16_t* row = a.routes + (size_t)r * a.K;
    uint16_t* to = a.droutes + (size_t)r * a.K;
    if (live) {
      const float w = ROUTES ? a.wts[r] : 0.f;
#pragma unroll(SPLIT)
      for (int base = 32 * V * sub; base < n8; base += 128) {
        uint4 o[V], g[V];
#pragma unroll
        for (int u = 0; u < V; ++u) {
          const int c = base + 32 * u + lane;
          o[u] = g[u] = make_uint4(0u, 0u, 0u, 0u);
          if (c < n8) {
            o[u] = ld_stream16(row + 8 * c);
            g[u] = ld_stream16(dy + 8 * c);
          }
        }
#pragma unroll
        for (int u = 0; u < V; ++u) {
          const int c = base + 32 * u + lane;
          float x[8], y[8];
          unpack8(o[u], x);
          unpack8(g[u], y);
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[u] = fmaf(x[i], y[i], acc[u]);
          if (ROUTES && c < n8) {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] *= w;
            st_stream16(to + 8 * c, pack8(y));
          }
        }
      }
    } else if (ROUTES) {
      for (int c = sub * 32 + lane; c < n8; c += 32 * SPLIT) st_stream16(to + 8 * c, make_uint4(0u, 0u, 0u, 0u));
    }
  }
  float s = 0.f;
  if (SPLIT == 1) {
#pragma unroll
    for (int v = 0; v < V; ++v) s += acc[v];
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) part[SPLIT > 1 ? warp : 0][v][lane] = acc[v];
    __syncthreads();
    if (sub != 0) return;
#pragma unroll
    for (int i = 0; i < SPLIT; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) s += part[SPLIT > 1 ? warp + i : 0][v][lane];
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  if (lane == 0 && r < routes) a.dw[r] = s;
}

template <bool ROUTES>
void run(const CombineBwdArgs& a, int split, unsigned blocks, cudaStream_t stream) {
  if (split == 1) combine_backward_kernel<ROUTES, 1><<<blocks, 32 * kCbWarps, 0, stream>>>(a);
  else if (split == 2) combine_backward_kernel<ROUTES, 2><<<blocks, 32 * kCbWarps, 0, stream>>>(a);
  else combine_backward_kernel<ROUTES, 4><<<blocks, 32 * kCbWarps, 0, stream>>>(a);
}

}  // namespace

cudaError_t launch_combine_backward(const CombineBwdArgs& a, int num_sms, cudaStream_t stream) {
  // Warps of a route: as many as keep 32 warps an SM busy, each with a row's part of at least
  // 512 values.
  const unsigned routes = (unsigned)a.T * (unsigned)a.topk;
  int split = 1;
  while (split < 4 && (size_t)routes * split < (size_t)32 * num_sms && a.K >= 1024 * split) split *= 2;
  const unsigned per = kCbWarps / split, blocks = (routes + per - 1) / per;
  if (a.droutes != nullptr) run<true>(a, split, blocks, stream);
  else run<false>(a, split, blocks, stream);
  return cudaGetLastError();
}

}  // namespace mxmoe
