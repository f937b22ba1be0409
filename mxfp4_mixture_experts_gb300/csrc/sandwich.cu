// The norms after and before a block, with the block's gate and the residual's
// scale between them, and their gradient from bf16 or 8-bit activations.
//
//   n = x * r1 * post_gamma     r1 = 1 / sqrt(mean(x^2) + eps)   (no post_gamma: n = x)
//   h = scale * res + act(gate) * n                              fp32, bf16(h) is the new stream
//   y = h * r2 * pre_gamma      r2 = 1 / sqrt(mean(h^2) + eps), from the unrounded h
//
// Gradient, from the kept x, h, r1 and r2 (hats: times r), v = pre_gamma * dy:
//   dh_total = dh + r2 (v - h^ mean(v h^))
//   dres = scale * dh_total             dscale = sum dh_total * res
//   dn = act(gate) * dh_total           dgate = act'(gate) * dh_total * n
//   dx = r1 (u - x^ mean(u x^)),  u = post_gamma * dn
//   dpre_gamma = sum_t dy * h^          dpost_gamma = sum_t dn * x^
// The second mean is linear in the first, mean(u x^) = B - c2 C with
//   c2 = r2 mean(v h^), B = mean(w x^ (dh + r2 v)), C = mean(w x^ h^),
//   w = post_gamma * act(gate),
// so that one pass over the row and one sum over the CTA give all of it. Every
// sum is fp32; what is rounded to bf16 is rounded once, on its way out.
#include <cstdint>

#include "ops.h"
#include "rows.cuh"

namespace mxmoe {
namespace {

constexpr int kSwThreads = 512;   // most threads of a row

__device__ __forceinline__ float gate_value(float g, int act) {
  return act ? __frcp_rn(__fadd_rn(1.f, expf(-g))) : g;
}

// Sum over the CTA of N values, the same in every thread; part: [2][N][16], the
// two sets in turn.
template <int N>
__device__ __forceinline__ void cta_sums(float (&v)[N], float (*part)[16], int lane, int warp, int warps) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
  if (lane == 0) {
#pragma unroll
    for (int n = 0; n < N; ++n) part[n][warp] = v[n];
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = lane < warps ? part[n][lane] : 0.f;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1)
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = __shfl_sync(0xffffffffu, v[n], 0);
}

// CH: 16-byte chunks per thread (K / 8 <= CH * blockDim.x).
template <int CH>
__global__ void __launch_bounds__(kSwThreads) sandwich_norm_kernel(const SandwichArgs a) {
  __shared__ float part[2][2][16];
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
  const int n8 = a.K / 8;
  const unsigned T = (unsigned)a.T;   // unsigned: T + gridDim.x may pass 2^31
  const float scale = a.rscale != nullptr ? *a.rscale : 1.f;
  int odd = 0;
  for (unsigned t = blockIdx.x; t < T; t += gridDim.x, odd ^= 1) {
    const size_t row = (size_t)t * a.K;
    float h[CH][8];
    float ss[1] = {0.f};
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = tid + i * nt;
      const bool valid = c < n8;
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] = 0.f;
      if (valid) unpack8(ld_row16(a.x + row + 8 * c), h[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss[0] += h[i][j] * h[i][j];
      if (a.x8 != nullptr) {
        const Mx8 e = mx8_block(h[i], max_bits8(h[i]), a.ck_nosat);
        if (valid) {
          *reinterpret_cast<uint2*>(a.x8 + row + 8 * c) = e.q;
          if ((c & 3) == 0) a.xs8[(size_t)t * (a.K / 32) + (c >> 2)] = (uint8_t)e.s;
        }
      }
    }
    Root r1 = {1.f, 0.f};
    if (a.post != nullptr) {
      cta_sums<1>(ss, part[odd], lane, warp, nt >> 5);
      r1 = rsqrt2(ss[0] / (float)a.K + a.eps);
    }
    const float gt = a.gate_kind == 2 ? gate_value(static_cast<const float*>(a.gate)[t], a.gate_act) : 1.f;
    ss[0] = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = tid + i * nt;
      const bool valid = c < n8;
      if (valid) {
        if (a.post != nullptr) {
          float g[8], n[8];
          unpack8(ld_row16(a.post + 8 * c), g);
#pragma unroll
          for (int j = 0; j < 8; ++j) n[j] = scaled(h[i][j], r1, g[j]);
          if (__builtin_expect(max_bits8(n) >= 0x7F800000u, 0)) {   // infinities leave no remainder
#pragma unroll
            for (int j = 0; j < 8; ++j) n[j] = (h[i][j] * r1.hi) * g[j];
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) h[i][j] = n[j];
        }
        float z[8];
        unpack8(ld_row16(a.residual + row + 8 * c), z);
        if (a.rscale != nullptr) {
#pragma unroll
          for (int j = 0; j < 8; ++j) z[j] = __fmul_rn(z[j], scale);
        }
        if (a.gate_kind == 0) {
#pragma unroll
          for (int j = 0; j < 8; ++j) h[i][j] += z[j];
        } else if (a.gate_kind == 2) {
#pragma unroll
          for (int j = 0; j < 8; ++j) h[i][j] = fmaf(gt, h[i][j], z[j]);
        } else {
          float g[8];
          unpack8(ld_row16(static_cast<const uint16_t*>(a.gate) + (a.gate_kind == 3 ? row : 0) + 8 * c), g);
#pragma unroll
          for (int j = 0; j < 8; ++j) h[i][j] = fmaf(gate_value(g[j], a.gate_act), h[i][j], z[j]);
        }
        if (a.h_out != nullptr) st_row16(a.h_out + row + 8 * c, pack8(h[i]));
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ss[0] += h[i][j] * h[i][j];
      if (a.h8 != nullptr) {
        const Mx8 e = mx8_block(h[i], max_bits8(h[i]), a.ck_nosat);
        if (valid) {
          *reinterpret_cast<uint2*>(a.h8 + row + 8 * c) = e.q;
          if ((c & 3) == 0) a.hs8[(size_t)t * (a.K / 32) + (c >> 2)] = (uint8_t)e.s;
        }
      }
    }
    Root r2 = {1.f, 0.f};
    if (a.pre != nullptr) {
      cta_sums<1>(ss, part[odd] + 1, lane, warp, nt >> 5);
      r2 = rsqrt2(ss[0] / (float)a.K + a.eps);
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = tid + i * nt;
        const bool valid = c < n8;
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = 0.f;
        if (valid) {
          float g[8];
          unpack8(ld_row16(a.pre + 8 * c), g);
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = scaled(h[i][j], r2, g[j]);
          if (__builtin_expect(max_bits8(y) >= 0x7F800000u, 0)) {
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = (h[i][j] * r2.hi) * g[j];
          }
          if (a.out != nullptr) st_row16(a.out + row + 8 * c, pack8(y));
        }
        if (a.q8 != nullptr) {
          const Mx8 e = mx8_block(y, max_bits8(y), a.nosat);
          if (valid) {
            *reinterpret_cast<uint2*>(a.q8 + row + 8 * c) = e.q;
            if ((c & 3) == 0) a.s8[(size_t)t * (a.K / 32) + (c >> 2)] = (uint8_t)e.s;
          }
        }
      }
    }
    if (a.rstd != nullptr && tid == 0) {
      a.rstd[t] = r1.hi;
      a.rstd[(size_t)T + t] = r2.hi;
    }
  }
}

// ---------------------------------------------------------------- gradient
// 8 values of a row in bf16, or in E4M3 with the row's scale bytes.
__device__ __forceinline__ void load8(const void* rows, const uint8_t* scale, size_t t, int K, int c, float (&v)[8]) {
  if (scale == nullptr) {
    unpack8(ld_row16(static_cast<const uint16_t*>(rows) + t * K + 8 * c), v);
    return;
  }
  const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(rows) + t * K + 8 * c);
  const float f = e8m0_to_f32(scale[t * (K / 32) + (c >> 2)]);
  const uint32_t w[2] = {q.x, q.y};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 p = e4m3x2_values((uint16_t)(w[j >> 1] >> (16 * (j & 1))));
    v[2 * j] = p.x * f;
    v[2 * j + 1] = p.y * f;
  }
}

// Column sums of the CTA's rows go to ws [gridDim.x][2][K]: 0 dy * h^, 1 d x^ with
// d = dn, or dh_total where the gate is a channel's (its gate and post_gamma take
// their gradients from the one sum). After them ws holds a float a CTA, sum dh_total * res.
template <int CH>
__global__ void __launch_bounds__(kSwThreads) sandwich_bwd_kernel(const SandwichBwdArgs a) {
  __shared__ float part[2][3][16];
  __shared__ float last[16];
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
  const int n8 = a.K / 8;
  const unsigned T = (unsigned)a.T;
  const float scale = a.rscale != nullptr ? *a.rscale : 1.f;
  const uint16_t* gate16 = static_cast<const uint16_t*>(a.gate);
  float s_pre[CH][8], s_x[CH][8], s_res = 0.f;
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) s_pre[i][j] = s_x[i][j] = 0.f;
  int odd = 0;
  for (unsigned t = blockIdx.x; t < T; t += gridDim.x, odd ^= 1) {
    const size_t row = (size_t)t * a.K;
    const float r1 = a.post != nullptr ? a.rstd[t] : 1.f;
    const float r2 = a.pre != nullptr ? a.rstd[(size_t)T + t] : 0.f;
    const float g_raw = a.gate_kind == 2 ? static_cast<const float*>(a.gate)[t] : 1.f;
    const float gt = a.gate_kind == 2 ? gate_value(g_raw, a.gate_act) : 1.f;
    float s[3] = {0.f, 0.f, 0.f};   // v h, w x (dh + r2 v), w x h; w without a token's gate
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = tid + i * nt;
      if (c >= n8) continue;
      float q[8], h[8], w[8], x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) q[j] = h[j] = 0.f;
      if (a.dh != nullptr) unpack8(ld_row16(a.dh + row + 8 * c), q);
      if (a.dy != nullptr) {
        float v[8], g[8];
        unpack8(ld_row16(a.dy + row + 8 * c), v);
        unpack8(ld_row16(a.pre + 8 * c), g);
        load8(a.h, a.hs, t, a.K, c, h);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[j] *= g[j];
          s[0] = fmaf(v[j], h[j], s[0]);
          q[j] = fmaf(r2, v[j], q[j]);
        }
      }
      load8(a.x, a.xs, t, a.K, c, x);
      if (a.post != nullptr) unpack8(ld_row16(a.post + 8 * c), w);
      else {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = 1.f;
      }
      if (a.gate_kind & 1) {
        float g[8];
        unpack8(ld_row16(gate16 + (a.gate_kind == 3 ? row : 0) + 8 * c), g);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] *= gate_value(g[j], a.gate_act);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float wx = w[j] * x[j];
        s[1] = fmaf(wx, q[j], s[1]);
        s[2] = fmaf(wx, h[j], s[2]);
      }
    }
    cta_sums<3>(s, part[odd], lane, warp, nt >> 5);
    const float inv_k = 1.f / (float)a.K;
    const float c2 = s[0] * r2 * inv_k * r2;              // r2 mean(v h^)
    const float dot = r1 * (s[1] - c2 * (r2 * s[2]));     // sum of w x^ dh_total
    const float c1 = a.post != nullptr ? gt * dot * inv_k : 0.f;
    if (a.gate_kind == 2 && a.dgate != nullptr && tid == 0)
      static_cast<float*>(a.dgate)[t] = a.gate_act ? dot * gt * gate_value(-g_raw, 1) : dot;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = tid + i * nt;
      if (c >= n8) continue;
      float d[8], x[8];   // dh_total
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = 0.f;
      if (a.dh != nullptr) unpack8(ld_row16(a.dh + row + 8 * c), d);
      if (a.dy != nullptr) {
        float v[8], g[8], h[8];
        unpack8(ld_row16(a.dy + row + 8 * c), v);
        unpack8(ld_row16(a.pre + 8 * c), g);
        load8(a.h, a.hs, t, a.K, c, h);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float hn = h[j] * r2;
          s_pre[i][j] = fmaf(v[j], hn, s_pre[i][j]);
          d[j] = fmaf(-c2, hn, fmaf(r2, v[j] * g[j], d[j]));
        }
      }
      if (a.dscale != nullptr) {
        float z[8];
        unpack8(ld_row16(a.residual + row + 8 * c), z);
#pragma unroll
        for (int j = 0; j < 8; ++j) s_res = fmaf(d[j], z[j], s_res);
      }
      if (a.dres != nullptr) {
        float z[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = d[j] * scale;
        st_row16(a.dres + row + 8 * c, pack8(z));
      }
      load8(a.x, a.xs, t, a.K, c, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] *= r1;
      float g[8], p[8];   // the gate's values; post_gamma
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = gt, p[j] = 1.f;
      if (a.post != nullptr) unpack8(ld_row16(a.post + 8 * c), p);
      if (a.gate_kind & 1) {
        float raw[8];
        unpack8(ld_row16(gate16 + (a.gate_kind == 3 ? row : 0) + 8 * c), raw);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = gate_value(raw[j], a.gate_act);
        if (a.gate_kind == 3 && a.dgate != nullptr) {
          float o[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            o[j] = d[j] * (x[j] * p[j]);
            if (a.gate_act) o[j] *= g[j] * gate_value(-raw[j], 1);
          }
          st_row16(static_cast<uint16_t*>(a.dgate) + row + 8 * c, pack8(o));
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float dn = d[j] * g[j];
        s_x[i][j] = fmaf(a.gate_kind == 1 ? d[j] : dn, x[j], s_x[i][j]);
        d[j] = a.post != nullptr ? r1 * fmaf(-c1, x[j], dn * p[j]) : dn;
      }
      if (a.dx != nullptr) st_row16(a.dx + row + 8 * c, pack8(d));
    }
  }
  float* mine = a.ws + (size_t)blockIdx.x * 2 * a.K;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = tid + i * nt;
    if (c >= n8) continue;
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
      *reinterpret_cast<float4*>(mine + 8 * c + j) =
          make_float4(s_pre[i][j], s_pre[i][j + 1], s_pre[i][j + 2], s_pre[i][j + 3]);
      *reinterpret_cast<float4*>(mine + a.K + 8 * c + j) =
          make_float4(s_x[i][j], s_x[i][j + 1], s_x[i][j + 2], s_x[i][j + 3]);
    }
  }
  if (a.dscale != nullptr) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s_res += __shfl_xor_sync(0xffffffffu, s_res, o);
    if (lane == 0) last[warp] = s_res;
    __syncthreads();
    if (tid == 0) {
      float sum = 0.f;
      for (int w = 0; w < (nt >> 5); ++w) sum += last[w];
      a.ws[(size_t)gridDim.x * 2 * a.K + blockIdx.x] = sum;
    }
  }
}

// The columns' sums over the CTAs' rows of ws, in the order of the CTAs; 32
// columns a CTA, a row group a warp.
__global__ void __launch_bounds__(256) sandwich_columns_kernel(const SandwichBwdArgs a, int rows) {
  __shared__ float part[2][8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int k = blockIdx.x * 32 + lane;   // K is a multiple of 32
  float s0 = 0.f, s1 = 0.f;
  for (int r = warp; r < rows; r += 8) {
    const float* p = a.ws + (size_t)r * 2 * a.K + k;
    s0 += p[0];
    s1 += p[a.K];
  }
  part[0][warp][lane] = s0;
  part[1][warp][lane] = s1;
  __syncthreads();
  if (warp == 0) {
    s0 = s1 = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      s0 += part[0][w][lane];
      s1 += part[1][w][lane];
    }
    if (a.dpre != nullptr) a.dpre[k] = s0;
    float gv = 1.f, dv = 1.f;
    if (a.gate_kind == 1) {
      const float g = __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.gate)[k] << 16);
      gv = gate_value(g, a.gate_act);
      if (a.gate_act) dv = gv * gate_value(-g, 1);
    }
    if (a.dpost != nullptr) a.dpost[k] = gv * s1;
    if (a.gate_kind == 1 && a.dgate != nullptr) {
      const float p = a.post != nullptr ? __uint_as_float((uint32_t)a.post[k] << 16) : 1.f;
      static_cast<float*>(a.dgate)[k] = dv * (p * s1);
    }
  }
  if (a.dscale != nullptr && blockIdx.x == 0 && warp == 1) {
    float s = 0.f;
    for (int r = lane; r < rows; r += 32) s += a.ws[(size_t)rows * 2 * a.K + r];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) *a.dscale = s;
  }
}

// Chunks a thread and threads a row.
int row_chunks(int n8) { return n8 > 2 * kSwThreads ? 4 : n8 > kSwThreads ? 2 : 1; }
int row_threads(int n8, int ch) { return ((n8 + ch - 1) / ch + 31) / 32 * 32; }

int bwd_grid(int T, int num_sms) { return T < 2 * num_sms ? T : 2 * num_sms; }

}  // namespace

cudaError_t launch_sandwich_norm(const SandwichArgs& a, int num_sms, cudaStream_t stream) {
  const int n8 = a.K / 8, ch = row_chunks(n8), nt = row_threads(n8, ch);
  int per_sm = 1024 / nt;
  if (per_sm > 8) per_sm = 8;
  const int grid = a.T < per_sm * num_sms ? a.T : per_sm * num_sms;
  if (ch == 1) sandwich_norm_kernel<1><<<grid, nt, 0, stream>>>(a);
  else if (ch == 2) sandwich_norm_kernel<2><<<grid, nt, 0, stream>>>(a);
  else sandwich_norm_kernel<4><<<grid, nt, 0, stream>>>(a);
  return cudaGetLastError();
}

size_t sandwich_bwd_workspace_bytes(int T, int K) {
  const size_t rows = T < kSwMaxCtas ? T : kSwMaxCtas;
  return rows * (2 * (size_t)K + 1) * sizeof(float);
}

cudaError_t launch_sandwich_norm_backward(const SandwichBwdArgs& a, int num_sms, cudaStream_t stream) {
  const int n8 = a.K / 8, ch = row_chunks(n8), nt = row_threads(n8, ch);
  int grid = bwd_grid(a.T, num_sms);
  if (grid > kSwMaxCtas) grid = kSwMaxCtas;
  if (grid > 0) {   // (no rows: the sums are zero)
    if (ch == 1) sandwich_bwd_kernel<1><<<grid, nt, 0, stream>>>(a);
    else if (ch == 2) sandwich_bwd_kernel<2><<<grid, nt, 0, stream>>>(a);
    else sandwich_bwd_kernel<4><<<grid, nt, 0, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (a.dpre != nullptr || a.dpost != nullptr || a.dscale != nullptr || (a.gate_kind == 1 && a.dgate != nullptr))
    sandwich_columns_kernel<<<a.K / 32, 256, 0, stream>>>(a, grid);
  return cudaGetLastError();
}

}  // namespace mxmoe
