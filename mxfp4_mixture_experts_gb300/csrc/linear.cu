// A shared projection from packed MXFP4 weights with the low-rank adapters of
// many requests beside it:
//   y_t = W x_t + scale_a * B_a (A_a x_t),  a = adapter of token t (or none)
// W = E2M1 * 2^(E8M0 - 127), [N, K]; A_a [rank, K] and B_a [N, rank] in bf16;
// x in bf16, or in MXFP8 (E4M3 with an E8M0 scale per 32 values). Sums in
// fp32, one rounding of y to bf16.
//
// This first form is the plain one: the adapters' inner products
// v = scale_a (A_a x_t) by one CTA per token, then a shared-memory tiled
// product in fp32 FMAs with the second adapter product in its epilogue.
#include <cstdint>

#include "common.cuh"
#include "ops.h"

namespace mxmoe {
namespace {

__device__ __forceinline__ float e4m3_to_f32(uint32_t b) {
  // sign and the 7 magnitude bits placed as a bf16: the value times 2^-120,
  // E4M3 subnormals included; 0x7F is NaN
  if ((b & 0x7Fu) == 0x7Fu) return NAN;
  return __uint_as_float(((b & 0x80u) << 24) | ((b & 0x7Fu) << 20)) * 0x1p120f;
}
__device__ __forceinline__ float bf16_to_f32(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

__device__ __forceinline__ float x_value(const LinearArgs& a, int t, int k) {
  const size_t i = (size_t)t * a.K + k;
  if (a.xs == nullptr) return bf16_to_f32(static_cast<const uint16_t*>(a.x)[i]);
  return e4m3_to_f32(static_cast<const uint8_t*>(a.x)[i]) *
         e8m0_to_f32(a.xs[(size_t)t * (a.K / 32) + k / 32]);
}

__global__ void __launch_bounds__(256) adapter_down_kernel(const LinearArgs a, float* v) {
  __shared__ float part[8];
  const int t = blockIdx.x;
  const int ad = a.ids[t];
  if (ad < 0 || ad >= a.L) return;
  for (int r = 0; r < a.rank; ++r) {
    const uint16_t* row = a.a + ((size_t)ad * a.rank + r) * a.K;
    float s = 0.f;
    for (int k = threadIdx.x; k < a.K; k += 256) s += x_value(a, t, k) * bf16_to_f32(row[k]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
      float z = 0.f;
      for (int i = 0; i < 8; ++i) z += part[i];
      v[(size_t)t * a.rank + r] = z * (a.ascale != nullptr ? a.ascale[ad] : 1.f);
    }
    __syncthreads();
  }
}

__global__ void __launch_bounds__(256) linear_kernel(const LinearArgs a, const float* v) {
  constexpr int kTile = 64, kStep = 32;
  __shared__ float xs[kStep][kTile + 1], ws[kStep][kTile + 1];
  const int n0 = blockIdx.x * kTile, t0 = blockIdx.y * kTile;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < a.K; k0 += kStep) {
    for (int i = threadIdx.x; i < kTile * kStep; i += 256) {
      const int r = i / kStep, k = i % kStep;
      xs[k][r] = t0 + r < a.T ? x_value(a, t0 + r, k0 + k) : 0.f;
    }
    for (int i = threadIdx.x; i < kTile * kStep; i += 256) {
      const int r = i / kStep, k = i % kStep, n = n0 + r;
      float w = 0.f;
      if (n < a.N) {
        const uint32_t byte = a.w[(size_t)n * (a.K / 2) + (k0 + k) / 2];
        const uint32_t c = (k & 1) ? byte >> 4 : byte & 15u;
        const uint32_t m = c & 7u;
        const float mag = m < 2 ? 0.5f * m : (1.f + 0.5f * (m & 1u)) * (float)(1 << ((m >> 1) - 1));
        w = ((c & 8u) ? -mag : mag) * e8m0_to_f32(a.s[(size_t)n * (a.K / 32) + k0 / 32]);
      }
      ws[k][r] = w;
    }
    __syncthreads();
    for (int k = 0; k < kStep; ++k)
      for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) acc[i][j] += xs[k][ty + 16 * i] * ws[k][tx + 16 * j];
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i) {
    const int t = t0 + ty + 16 * i;
    if (t >= a.T) continue;
    const int ad = a.ids != nullptr ? a.ids[t] : -1;
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + tx + 16 * j;
      if (n >= a.N) continue;
      float y = acc[i][j];
      if (ad >= 0 && ad < a.L)
        for (int r = 0; r < a.rank; ++r)
          y += v[(size_t)t * a.rank + r] * bf16_to_f32(a.b[((size_t)ad * a.N + n) * a.rank + r]);
      a.out[(size_t)t * a.N + n] = f32_to_bf16_rne(y);
    }
  }
}

// status[0] = tokens whose adapter id is >= L, the rest zero
__global__ void __launch_bounds__(256) linear_status_kernel(const int32_t* ids, int T, int L,
                                                            int32_t* status) {
  __shared__ int n;
  if (threadIdx.x == 0) n = 0;
  __syncthreads();
  int c = 0;
  if (ids != nullptr)
    for (int t = threadIdx.x; t < T; t += 256) c += ids[t] >= L;
  if (c) atomicAdd(&n, c);
  __syncthreads();
  if (threadIdx.x < 4) status[threadIdx.x] = threadIdx.x == 0 ? n : 0;
}

}  // namespace

size_t linear_workspace_bytes(int T, int K, int N, int rank, bool x8) {
  (void)K;
  (void)N;
  (void)x8;
  return ((size_t)T * rank * sizeof(float) + 255) & ~size_t(255);
}

cudaError_t launch_linear(const LinearArgs& a, int num_sms, cudaStream_t stream) {
  (void)num_sms;
  float* v = static_cast<float*>(a.ws);
  if (a.status != nullptr)
    linear_status_kernel<<<1, 256, 0, stream>>>(a.ids, a.T, a.L, a.status);
  if (a.ids != nullptr) adapter_down_kernel<<<a.T, 256, 0, stream>>>(a, v);
  const dim3 grid((a.N + 63) / 64, (a.T + 63) / 64);
  linear_kernel<<<grid, 256, 0, stream>>>(a, v);
  return cudaGetLastError();
}

}  // namespace mxmoe
