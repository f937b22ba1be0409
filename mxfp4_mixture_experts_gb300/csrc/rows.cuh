// Device helpers of the operators that work on whole rows, 8 values a thread
// and step: bf16 and MXFP8 rows in and out, the root of a norm.
#pragma once

#include "ops_common.cuh"

namespace mxmoe {

// Row data (no read-only path: an output may be the same rows as an input).
__device__ __forceinline__ uint4 ld_row16(const uint16_t* p) {
  return *reinterpret_cast<const uint4*>(p);
}
__device__ __forceinline__ void st_row16(uint16_t* p, const uint4& v) {
  *reinterpret_cast<uint4*>(p) = v;
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(bf16x2_rn(v[0], v[1]), bf16x2_rn(v[2], v[3]), bf16x2_rn(v[4], v[5]),
                    bf16x2_rn(v[6], v[7]));
}
__device__ __forceinline__ void unpack8(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
}
// Two fp32 -> two E4M3 bytes (first value in the low byte), nearest even, saturating.
__device__ __forceinline__ uint32_t e4m3x2_rn_sat(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two E4M3 bytes (low byte first) -> their values, exact.
__device__ __forceinline__ float2 e4m3x2_values(uint16_t q) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(q));
  float2 r;
  asm("{\n .reg .b16 l, u;\n mov.b32 {l, u}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, u;\n}"
      : "=f"(r.x), "=f"(r.y) : "r"(h));
  return r;
}

// 1 / sqrt(v) as a value and its remainder: the approximation and a Newton step.
struct Root {
  float hi, lo;
};
__device__ __forceinline__ Root rsqrt2(float v) {
  const float r = rsqrtf(v);
  const float p = __fmul_rn(v, r);
  const float c = 0.5f * r * (fmaf(-p, r, 1.f) - r * fmaf(v, r, -p));
  if (!(fabsf(c) < r)) return Root{r, 0.f};   // v zero, infinite or NaN: the root as it is
  const float hi = __fadd_rn(r, c);
  return Root{hi, c - __fsub_rn(hi, r)};
}
// h * r * g with one rounding: the remainders of the root and of the first
// product go into the second. (Three more operations a value, hidden behind the
// memory; y is then exact but for the sum's error and half an ulp, and the codes made of it
// are those of the exact y except next to a tie.)
__device__ __forceinline__ float scaled(float h, Root r, float g) {
  const float t = __fmul_rn(h, r.hi);
  return fmaf(t, g, (fmaf(h, r.hi, -t) + h * r.lo) * g);
}

// A thread's 8 values of a 32-value MXFP8 block that it shares with the 3 lanes
// beside it (all 32 lanes call; m: its largest magnitude as bits, integer order being
// magnitude order with NaN above infinity): 8 codes and the block's scale byte.
struct Mx8 {
  uint2 q;
  uint32_t s;
};
__device__ __forceinline__ Mx8 mx8_block(const float (&y)[8], uint32_t m, int nosat) {
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const bool nonfinite = m >= 0x7F800000u;
  int X = max((int)(m >> 23) - 135, -127);
  // 448 = 1.75 * 2^8: past it the block saturates (never where X is clamped)
  if (nosat && (int)(m >> 23) >= 8 && (m & 0x7FFFFFu) > 0x600000u) ++X;
  const float inv = __uint_as_float((uint32_t)(127 - X) << 23);   // 2^-X, exact
  Mx8 r;
  r.q.x = e4m3x2_rn_sat(y[0] * inv, y[1] * inv) | (e4m3x2_rn_sat(y[2] * inv, y[3] * inv) << 16);
  r.q.y = e4m3x2_rn_sat(y[4] * inv, y[5] * inv) | (e4m3x2_rn_sat(y[6] * inv, y[7] * inv) << 16);
  if (nonfinite) r.q = make_uint2(0u, 0u);
  r.s = nonfinite ? 255u : (uint32_t)(X + 127);
  return r;
}

// Largest magnitude of 8 values as bits.
__device__ __forceinline__ uint32_t max_bits8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
  return m;
}

}  // namespace mxmoe
