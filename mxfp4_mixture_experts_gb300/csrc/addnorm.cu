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
// HBM-bound: 4 bytes read, 4 written per value, and 33/32 more for MXFP8. A CTA
// takes a row, 16 bytes (8 values) per thread and step; the fp32 row stays in
// registers between the sum of squares and the scaling, so every byte moves
// once, and with many rows a CTA goes on to further ones, whose loads are under way
// while it waits for the sum of the row before. The 4 threads of a 32-value
// block share its maximum by two shuffles.
#include <cstdint>

#include "ops.h"
#include "rows.cuh"

namespace mxmoe {
namespace {

template <int CH>
struct RowLoads {
  uint4 x[CH], res[CH];
};

// CH: 16-byte chunks per thread (K / 8 <= CH * blockDim.x).
template <int CH>
__global__ void __launch_bounds__(1024) add_rmsnorm_kernel(const AddNormArgs a) {
  __shared__ float part[2][32];
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
  const int n8 = a.K / 8;
  const unsigned T = (unsigned)a.T;   // unsigned: T + gridDim.x may pass 2^31
  RowLoads<CH> d;
  auto load = [&](unsigned t) {
    const size_t row = (size_t)t * a.K;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = tid + i * nt;
      if (t < T && c < n8) {
        d.x[i] = ld_row16(a.x + row + 8 * c);
        if (a.residual != nullptr) d.res[i] = ld_row16(a.residual + row + 8 * c);
      }
    }
  };
  load(blockIdx.x);
  int odd = 0;
  for (unsigned t = blockIdx.x; t < T; t += gridDim.x, odd ^= 1) {
    const size_t row = (size_t)t * a.K;
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
      const uint32_t w[4] = {d.x[i].x, d.x[i].y, d.x[i].z, d.x[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        h[i][2 * j] = __uint_as_float(w[j] << 16);
        h[i][2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      }
      if (a.residual != nullptr) {
        const uint32_t z[4] = {d.res[i].x, d.res[i].y, d.res[i].z, d.res[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          h[i][2 * j] += __uint_as_float(z[j] << 16);
          h[i][2 * j + 1] += __uint_as_float(z[j] & 0xFFFF0000u);
        }
      }
      if (a.residual_out != nullptr) st_row16(a.residual_out + row + 8 * c, pack8(h[i]));
#pragma unroll
      for (int j = 0; j < 8; ++j) ss += h[i][j] * h[i][j];
    }
    load(t + gridDim.x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (lane == 0) part[odd][warp] = ss;   // two sets: the row before may still be read
    __syncthreads();
    ss = lane < (nt >> 5) ? part[odd][lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const Root r = rsqrt2(ss / (float)a.K + a.eps);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = tid + i * nt;
      const bool valid = c < n8;
      float y[8];
      uint32_t m = 0;   // largest magnitude bits: integer order is magnitude order, NaN above infinity
      if (valid) {
        const uint4 u = *reinterpret_cast<const uint4*>(a.gamma + 8 * c);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          y[2 * j] = scaled(h[i][2 * j], r, __uint_as_float(w[j] << 16));
          y[2 * j + 1] = scaled(h[i][2 * j + 1], r, __uint_as_float(w[j] & 0xFFFF0000u));
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(y[j]) & 0x7FFFFFFFu);
        if (__builtin_expect(m >= 0x7F800000u, 0)) {   // infinities leave no remainder: the plain products
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float g = __uint_as_float((j & 1) ? w[j >> 1] & 0xFFFF0000u : w[j >> 1] << 16);
            y[j] = (h[i][j] * r.hi) * g;
          }
        }
        if (a.out != nullptr) st_row16(a.out + row + 8 * c, pack8(y));
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = 0.f;
      }
      if (a.q8 != nullptr) {
        const Mx8 e = mx8_block(y, m, a.nosat);
        if (valid) {
          *reinterpret_cast<uint2*>(a.q8 + row + 8 * c) = e.q;
          if ((c & 3) == 0) a.s8[(size_t)t * (a.K / 32) + (c >> 2)] = (uint8_t)e.s;
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_add_rmsnorm(const AddNormArgs& a, int num_sms, cudaStream_t stream) {
  // Few rows: a CTA each, one chunk a thread where 1024 threads suffice (its
  // latency counts). Many rows: two chunks a thread and as many persistent CTAs as
  // fill an SM's threads. T = 8192, K = 6144 with MXFP8 (454.6 MB): 8192 CTAs of
  // 768 threads 129 us, 608 persistent ones of 384 threads 72 us = 6.3 TB/s; the
  // copy engine moves as many bytes in 72 us. Short rows fill neither a CTA nor, eight
  // to an SM, its threads: T = 8192 in a graph reaches 5.6 TB/s at K = 2048, 4.7 at
  // 1024, 3.2 at 512 (12 us) and 2.4 at 256, where half of the CTA's one warp has no chunk.
  const int n8 = a.K / 8;
  const bool many = a.T > 2 * num_sms;
  const int ch = many || n8 > 1024 ? 2 : 1;
  const int nt = ((n8 + ch - 1) / ch + 31) / 32 * 32;
  int grid = a.T;
  if (many) {
    int per_sm = 1536 / nt;
    if (per_sm > 8) per_sm = 8;
    if (per_sm < 1) per_sm = 1;
    if (grid > per_sm * num_sms) grid = per_sm * num_sms;
  }
  if (ch == 1) add_rmsnorm_kernel<1><<<grid, nt, 0, stream>>>(a);
  else add_rmsnorm_kernel<2><<<grid, nt, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace mxmoe
