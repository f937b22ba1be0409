// Residual addition and root-mean-square norm of the rows that enter an MoE
// layer, with the normed rows in bf16, in MXFP8, or both.
//
//   h_k = x_k + res_k                        fp32 (exact operands, one rounding)
//   res'_k = bf16(h_k)                       the residual stream, may overwrite x or res
//   y_k = (h_k * rsqrt(mean(h^2) + eps)) * gamma_k    fp32, from the unrounded h
//   out_k = bf16(y_k)
//   MXFP8 per 32 values: X = floor(log2(amax)) - 8 (E4M3's largest exponent is
//   8), raised by one under "nosat" where amax / 2^X > 448, clamped to
//   [-127, 127]; code = E4M3(y / 2^X), nearest even, saturating; an all-zero
//   block has byte 0, a block with a NaN or infinity byte 255 and codes 0.
//
// HBM-bound: 4 bytes read, 4 written per value, and 33/32 more for MXFP8. One
// CTA per row, 16 bytes (8 values) per thread and step; the fp32 row stays in
// registers between the sum of squares and the scaling, so every byte moves
// once. The 4 threads of a 32-value block share its maximum by two shuffles.
#include <cstdint>

#include "ops.h"
#include "ops_common.cuh"

namespace mxmoe {
namespace {

// Two fp32 -> two E4M3 bytes (first value in the low byte), nearest even, saturating.
__device__ __forceinline__ uint32_t e4m3x2_rn_sat(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// An fp32 value and its remainder. The warps' sums are added and the scaling is
// applied with remainders: y then carries one rounding instead of the sums',
// the root's and two products' (about 4 ulp apart at worst), so the codes made
// of it are those of the exact y but where that lies within an ulp of a tie.
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two add(Two a, Two b) {
  const float s = __fadd_rn(a.hi, b.hi);
  const float t = __fsub_rn(s, a.hi);
  const float e = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, t)), __fsub_rn(b.hi, t));
  return Two{s, e + (a.lo + b.lo)};
}
// 1 / sqrt(sum / n + eps): the root's approximation and one Newton step.
__device__ __forceinline__ Two rsqrt_mean(Two sum, float n, float eps) {
  const float m = __fdiv_rn(sum.hi, n);
  const Two v = add(Two{m, (fmaf(-m, n, sum.hi) + sum.lo) / n}, Two{eps, 0.f});
  const float r = rsqrtf(v.hi);
  const float p = __fmul_rn(v.hi, r);
  const float e = fmaf(-p, r, 1.f) - r * (fmaf(v.hi, r, -p) + v.lo * r);
  const float c = 0.5f * r * e;
  if (!(fabsf(c) < r)) return Two{r, 0.f};   // sum 0, infinite or NaN: the root as it is
  const float hi = __fadd_rn(r, c);
  return Two{hi, c - __fsub_rn(hi, r)};
}
// (h * r) * g
__device__ __forceinline__ float scaled(float h, Two r, float g) {
  const float t = __fmul_rn(h, r.hi);
  const float e = fmaf(h, r.hi, -t) + h * r.lo;
  const float y = fmaf(t, g, e * g);
  return fabsf(t) < INFINITY ? y : t * g;   // infinite products leave no remainder
}

// CH: 16-byte chunks per thread (K / 8 <= CH * blockDim.x).
template <int CH>
__global__ void __launch_bounds__(CH <= 2 ? 1024 : 256) add_rmsnorm_kernel(const AddNormArgs a) {
  __shared__ float part[32];
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
  const int n8 = a.K / 8;
  const size_t row = (size_t)blockIdx.x * a.K;
  float h[CH][8];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = tid + i * nt;
    if (c >= n8) {
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] = 0.f;
      continue;
    }
    const uint4 u = *reinterpret_cast<const uint4*>(a.x + row + 8 * c);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      h[i][2 * j] = __uint_as_float(w[j] << 16);
      h[i][2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
    if (a.residual != nullptr) {
      const uint4 v = *reinterpret_cast<const uint4*>(a.residual + row + 8 * c);
      const uint32_t z[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        h[i][2 * j] += __uint_as_float(z[j] << 16);
        h[i][2 * j + 1] += __uint_as_float(z[j] & 0xFFFF0000u);
      }
    }
    if (a.residual_out != nullptr) {
      uint4 o;
      o.x = bf16x2_rn(h[i][0], h[i][1]);
      o.y = bf16x2_rn(h[i][2], h[i][3]);
      o.z = bf16x2_rn(h[i][4], h[i][5]);
      o.w = bf16x2_rn(h[i][6], h[i][7]);
      *reinterpret_cast<uint4*>(a.residual_out + row + 8 * c) = o;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) ss += h[i][j] * h[i][j];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if (lane == 0) part[warp] = ss;
  __syncthreads();
  Two r = {lane < (nt >> 5) ? part[lane] : 0.f, 0.f};
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    r = add(r, Two{__shfl_xor_sync(0xffffffffu, r.hi, o), __shfl_xor_sync(0xffffffffu, r.lo, o)});
  r = rsqrt_mean(r, (float)a.K, a.eps);
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = tid + i * nt;
    const bool valid = c < n8;
    float y[8];
    uint32_t m = 0;
    if (valid) {
      const uint4 u = *reinterpret_cast<const uint4*>(a.gamma + 8 * c);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        y[2 * j] = scaled(h[i][2 * j], r, __uint_as_float(w[j] << 16));
        y[2 * j + 1] = scaled(h[i][2 * j + 1], r, __uint_as_float(w[j] & 0xFFFF0000u));
      }
      if (a.out != nullptr) {
        uint4 o;
        o.x = bf16x2_rn(y[0], y[1]);
        o.y = bf16x2_rn(y[2], y[3]);
        o.z = bf16x2_rn(y[4], y[5]);
        o.w = bf16x2_rn(y[6], y[7]);
        *reinterpret_cast<uint4*>(a.out + row + 8 * c) = o;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = 0.f;
    }
    if (a.q8 != nullptr) {
      // magnitude bits: integer order is magnitude order, NaN above infinity
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(y[j]) & 0x7FFFFFFFu);
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const bool nonfinite = m >= 0x7F800000u;
      int X = max((int)(m >> 23) - 135, -127);
      // 448 = 1.75 * 2^8: past it the block saturates (never where X is clamped)
      if (a.nosat && (int)(m >> 23) >= 8 && (m & 0x7FFFFFu) > 0x600000u) ++X;
      const float inv = __uint_as_float((uint32_t)(127 - X) << 23);   // 2^-X, exact
      uint2 q;
      q.x = e4m3x2_rn_sat(y[0] * inv, y[1] * inv) | (e4m3x2_rn_sat(y[2] * inv, y[3] * inv) << 16);
      q.y = e4m3x2_rn_sat(y[4] * inv, y[5] * inv) | (e4m3x2_rn_sat(y[6] * inv, y[7] * inv) << 16);
      if (nonfinite) q = make_uint2(0u, 0u);
      if (valid) {
        *reinterpret_cast<uint2*>(a.q8 + row + 8 * c) = q;
        if ((c & 3) == 0)
          a.s8[(size_t)blockIdx.x * (a.K / 32) + (c >> 2)] = nonfinite ? 255u : (uint8_t)(X + 127);
      }
    }
  }
}

}  // namespace

cudaError_t launch_add_rmsnorm(const AddNormArgs& a, int num_sms, cudaStream_t stream) {
  // One row's latency counts for few rows: one chunk a thread, up to 1024
  // threads. Many rows go faster in CTAs of 128 to 256 threads with up to 8
  // chunks each, eight or more to an SM, so that some rows load while others wait
  // at their barrier (T = 8192, K = 6144 with MXFP8: 768 threads 80 us, 256
  // threads 73 us, the copy rate allows 67).
  const int n8 = a.K / 8;
  int nt = ((n8 + 31) / 32) * 32;
  if (a.T > 2 * num_sms && n8 > 128) {
    const int ch = n8 <= 1024 ? 4 : 8;
    nt = ((n8 + ch - 1) / ch + 31) / 32 * 32;
  } else if (nt > 1024) {
    nt = 1024;
  }
  const int ch = (n8 + nt - 1) / nt;
#define MXMOE_NORM(C) add_rmsnorm_kernel<C><<<a.T, nt, 0, stream>>>(a)
  if (ch <= 1) MXMOE_NORM(1);
  else if (ch <= 2) MXMOE_NORM(2);
  else if (ch <= 3) MXMOE_NORM(3);
  else if (ch <= 4) MXMOE_NORM(4);
  else MXMOE_NORM(8);
#undef MXMOE_NORM
  return cudaGetLastError();
}

}  // namespace mxmoe
