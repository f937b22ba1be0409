// Gradient of the layer's combination of its routes, y_t = sum_j w_tj o_tj.
//
//   dw_tj = sum_k dy_tk o_tjk (fp32)        do_tj = bf16(w_tj dy_t)
//
// HBM-bound: k rows of o read for one of dy, and k written where the routes'
// gradients are wanted. A CTA per token, a warp per route: dy is read by the
// token's warps together, so it leaves L2 once.
#include <cstdint>

#include "ops.h"
#include "rows.cuh"

namespace mxmoe {
namespace {

__global__ void __launch_bounds__(256) combine_backward_kernel(const CombineBwdArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const size_t t = blockIdx.x;
  const int n8 = a.K / 8;
  const uint16_t* dy = a.dy + t * a.K;
  for (int j = warp; j < a.topk; j += warps) {
    const size_t r = t * a.topk + j;
    bool live = true;
    if (a.ids != nullptr) {
      const int id = a.ids[r];
      live = id >= a.ebase && (a.E == 0 || id - a.ebase < a.E);
    }
    const float w = a.droutes != nullptr ? a.wts[r] : 0.f;
    float sum = 0.f;
#pragma unroll 4
    for (int c = lane; c < n8; c += 32) {
      float g[8], o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = o[i] = 0.f;
      if (live) {
        unpack8(ld_row16(dy + 8 * c), g);
        unpack8(ld_row16(a.routes + r * a.K + 8 * c), o);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(g[i], o[i], sum);
      if (a.droutes != nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = live ? w * g[i] : 0.f;
        st_row16(a.droutes + r * a.K + 8 * c, pack8(g));
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) a.dw[r] = sum;
  }
}

}  // namespace

cudaError_t launch_combine_backward(const CombineBwdArgs& a, cudaStream_t stream) {
  const int warps = a.topk < 8 ? a.topk : 8;
  combine_backward_kernel<<<a.T, 32 * warps, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace mxmoe
