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
// so that one pass over the row and one sum over its warps give all of it. Every
// sum is fp32, dscale's with a remainder; what is rounded to bf16 is rounded once, on its way out.
//
// Both are HBM-bound in kind: forward 4 bytes read and 4 written a value, 33/32 for each
// 8-bit copy; gradient 4 (or 2 and 2 x 33/32) and 4 more read, 4 written. What they
// have to hide is a row's waits (two forward, one in the gradient) and 250 to 300 instructions
// for 8 values of a lane. So rows come through rings in shared memory (cp.async, no register
// held by a load under way), a team of warps takes a row and several teams an SM, and
// products run in pairs (fma.rn.f32x2). T = 8192, K = 6144, a channel's gate, 8-bit x and h
// (506 MB either way), in a graph: forward 84 us = 6.0 TB/s, gradient 88 us = 5.7 TB/s; a plain
// copy moves 6.8.
#include <cstdint>
#include <mutex>

#include "ops.h"
#include "rows.cuh"

namespace mxmoe {
namespace {

// Rows of a gradient that one CTA takes, without the second kernel (two rows of K = 2880 in a graph 7.7 us for
// 6.7, and 3 us less of the host).
constexpr int kSwOneCta = 2;
constexpr int kSwRingBytes = 224 * 1024;   // shared memory of a gradient call, beside 1.7 KB of sums

// A gate's value and its derivative, (s, s (1 - s)) of a sigmoid: one exponential of -|g|, so that
// neither overflows nor cancels.
struct Gate {
  float v, d;
};
__device__ __forceinline__ Gate gate_of(float g, int act) {
  if (!act) return Gate{g, 1.f};
  const float e = expf(-fabsf(g)), hi = __frcp_rn(1.f + e), lo = e * hi;
  return Gate{g < 0.f ? lo : hi, hi * lo};
}
__device__ __forceinline__ float gate_value(float g, int act) { return gate_of(g, act).v; }
// The same for a full gate's bf16 values, a thread's 8 of every row: both steps approximate, a relative
// error below 2^-21 + |g| 2^-23 (the exponent's rounding), far under the half step of 2^-8 that the gate
// itself carries. (The gradient of T = 4096, K = 2880 with a full gate and a trained scale: 78 us with expf, 44.)
__device__ __forceinline__ Gate full_gate(float g, bool act) {
  if (!act) return Gate{g, 1.f};
  const float e = fast_exp(-fabsf(g)), hi = fast_rcp(1.f + e), lo = e * hi;
  return Gate{g < 0.f ? lo : hi, hi * lo};
}

__device__ __forceinline__ float2 dup(float v) { return make_float2(v, v); }
__device__ __forceinline__ void unpack4(const uint4& u, float2 (&v)[4]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    v[j] = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
}
__device__ __forceinline__ uint4 pack4(const float2 (&v)[4]) {
  return make_uint4(bf16x2_rn(v[0].x, v[0].y), bf16x2_rn(v[1].x, v[1].y), bf16x2_rn(v[2].x, v[2].y),
                    bf16x2_rn(v[3].x, v[3].y));
}
// 16 (8) bytes, or zeros where n is 0: nothing is read then.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void* src, int n) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
// All but the latest n (0..3) groups of this thread's copies have landed.
__device__ __forceinline__ void copies_wait(int n) {
  if (n == 0) asm volatile("cp.async.wait_group 0;" ::: "memory");
  else if (n == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
  else if (n == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
  else asm volatile("cp.async.wait_group 3;" ::: "memory");
}

// Loads that stay where they are written, ahead of their use.
__device__ __forceinline__ float ldg_ahead(const float* p) {
  float v;
  asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}

// Sum of v over a team of nt threads of the CTA (its own named barrier, none for one
// warp); part: [32], a place a warp of the CTA.
__device__ __forceinline__ float team_sum(float v, float* part, int team, int nt, int lane, int warp, int warps) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (warps == 1) return v;
  const int base = team * warps;
  if (lane == 0) part[base + warp] = v;
  named_barrier(team + 1, nt);
  v = lane < warps ? part[base + lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Shared memory of a forward call: the gammas (bf16), a channel's gate (fp32, in two halves of 4
// values a chunk), then for every team a ring of rows. A row's slots lie by warp and chunk,
// [x][residual][gate] of 32 lanes each; a thread fills and reads its own slots alone.
struct FwdPlan {
  int nt, teams, depth;   // threads of a team, teams, rows of a ring (1..4)
  int pre, gate, ring;    // byte offsets (post_gamma at 0)
  int slot, row;          // bytes of a warp's slots of a chunk, of a row
  int smem;
};

// MXFP8 of 8 values: the 4 lanes of a block call together. The largest magnitude comes from
// maxima of three magnitudes that keep a NaN (its bits are above infinity's).
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ void store_mx8(const float2 (&v)[4], int nosat, bool valid, uint8_t* q, uint8_t* scale,
                                          bool first) {
  float m = max3_abs(v[0].x, v[0].y, v[1].x);
  m = max3_abs(m, v[1].y, v[2].x);
  m = max3_abs(m, v[2].y, v[3].x);
  const float f[8] = {v[0].x, v[0].y, v[1].x, v[1].y, v[2].x, v[2].y, v[3].x, v[3].y};
  const Mx8 e = mx8_block(f, max(__float_as_uint(m), __float_as_uint(v[3].y) & 0x7FFFFFFFu), nosat);
  if (valid) *reinterpret_cast<uint2*>(q) = e.q;
  if (first && valid) *scale = (uint8_t)e.s;
}

// A team of warps to a row, CH * 32 chunks in a row to a warp; short rows share a CTA.
// A CTA has a row's two waits in each of its teams, the other teams and the other CTA of the SM
// fill them (24 warps an SM at K = 6144; T = 8192 with 8-bit copies 84 us, a CTA a row 161).
template <int CH, int MAXT, int PER_SM, bool FULL>   // FULL: a gate for every value
__global__ void __launch_bounds__(MAXT, PER_SM) sandwich_norm_kernel(const SandwichArgs a, const FwdPlan p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float part[2][2][32];
  const int nt = p.nt, team = threadIdx.x / nt, tid = threadIdx.x - team * nt;
  const int lane = tid & 31, warp = tid >> 5, warps = nt >> 5;
  const int n8 = a.K / 8, c0 = warp * (32 * CH) + lane;   // this thread's chunks: c0 + 32 i
  const unsigned T = (unsigned)a.T;   // unsigned: T + the step may pass 2^31
  const bool has_post = a.post != nullptr, has_pre = a.pre != nullptr, scaled_res = a.rscale != nullptr;
  const float scale = scaled_res ? *a.rscale : 1.f;
  const uint16_t* gate16 = static_cast<const uint16_t*>(a.gate);
  uint8_t* mine = smem + p.ring + (size_t)team * p.depth * p.row + warp * (CH * p.slot) + 16 * lane;
  const uint32_t mine_addr = smem_u32(mine);
  uint4* post = reinterpret_cast<uint4*>(smem);
  uint4* pre = reinterpret_cast<uint4*>(smem + p.pre);
  float4* gch = reinterpret_cast<float4*>(smem + p.gate);
  const int half = CH * nt;
  bool valid[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = c0 + 32 * i;
    valid[i] = c < n8;
    if (team != 0) continue;
    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
    if (has_post) post[c] = valid[i] ? ld_row16(a.post + 8 * c) : z;
    if (has_pre) pre[c] = valid[i] ? ld_row16(a.pre + 8 * c) : z;
    if (a.gate_kind == 1) {
      float g[8];
      unpack8(valid[i] ? ld_row16(gate16 + 8 * c) : z, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = gate_value(g[j], a.gate_act);
      gch[c] = make_float4(g[0], g[1], g[2], g[3]);
      gch[half + c] = make_float4(g[4], g[5], g[6], g[7]);
    }
  }
  // row t into stage st; lanes past its end copy nothing
  auto fetch = [&](unsigned t, int st) {
    const size_t at = (size_t)min(t, T - 1) * a.K + 8 * c0;
    const uint32_t to = mine_addr + st * p.row;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int n = t < T && valid[i] ? 16 : 0;
      copy16(to + i * p.slot, a.x + at + 256 * i, n);
      copy16(to + i * p.slot + 512, a.residual + at + 256 * i, n);
      if (FULL) copy16(to + i * p.slot + 1024, gate16 + at + 256 * i, n);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  const unsigned step = gridDim.x * p.teams;
  const unsigned first = blockIdx.x * p.teams + team;
  for (int d = 0; d < p.depth; ++d) fetch(first + d * step, d);
  float g_next = a.gate_kind == 2 && first < T ? ldg_ahead(static_cast<const float*>(a.gate) + first) : 1.f;
  __syncthreads();
  const float inv_k = 1.f / (float)a.K;
  int odd = 0, st = 0;
  for (unsigned t = first; t < T; t += step, odd ^= 1) {
    const size_t out = (size_t)t * a.K + 8 * c0;
    const size_t sout = (size_t)t * (a.K / 32) + (c0 >> 2);
    const float g_raw = g_next;
    if (a.gate_kind == 2 && t + step < T) g_next = ldg_ahead(static_cast<const float*>(a.gate) + t + step);
    copies_wait(p.depth - 1);
    const uint8_t* slot = mine + st * p.row;
    float2 h[CH][4], ss = dup(0.f);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      unpack4(*reinterpret_cast<const uint4*>(slot + i * p.slot), h[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) ss = __ffma2_rn(h[i][j], h[i][j], ss);
      if (a.x8 != nullptr)
        store_mx8(h[i], a.ck_nosat, valid[i], a.x8 + out + 256 * i, a.xs8 + sout + 8 * i, (lane & 3) == 0);
    }
    float r1 = 1.f;
    if (has_post) r1 = rsqrt2(team_sum(ss.x + ss.y, part[odd][0], team, nt, lane, warp, warps) * inv_k + a.eps).hi;
    const float gt = a.gate_kind == 2 ? gate_value(g_raw, a.gate_act) : 1.f;
    ss = dup(0.f);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      float2 z[4];
      unpack4(*reinterpret_cast<const uint4*>(slot + i * p.slot + 512), z);
      if (has_post) {
        float2 g[4];
        unpack4(post[c0 + 32 * i], g);
#pragma unroll
        for (int j = 0; j < 4; ++j) h[i][j] = __fmul2_rn(__fmul2_rn(h[i][j], dup(r1)), g[j]);
      }
      if (scaled_res) {
#pragma unroll
        for (int j = 0; j < 4; ++j) z[j] = __fmul2_rn(z[j], dup(scale));
      }
      float2 g[4] = {dup(gt), dup(gt), dup(gt), dup(gt)};
      if (!FULL && a.gate_kind == 1) {
        const float4 g0 = gch[c0 + 32 * i], g1 = gch[half + c0 + 32 * i];
        g[0] = make_float2(g0.x, g0.y);
        g[1] = make_float2(g0.z, g0.w);
        g[2] = make_float2(g1.x, g1.y);
        g[3] = make_float2(g1.z, g1.w);
      } else if (FULL) {
        unpack4(*reinterpret_cast<const uint4*>(slot + i * p.slot + 1024), g);
        if (a.gate_act) {
#pragma unroll
          for (int j = 0; j < 4; ++j) g[j] = make_float2(full_gate(g[j].x, true).v, full_gate(g[j].y, true).v);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        h[i][j] = __ffma2_rn(g[j], h[i][j], z[j]);
        ss = __ffma2_rn(h[i][j], h[i][j], ss);
      }
      if (a.h_out != nullptr && valid[i]) st_row16(a.h_out + out + 256 * i, pack4(h[i]));
      if (a.h8 != nullptr)
        store_mx8(h[i], a.ck_nosat, valid[i], a.h8 + out + 256 * i, a.hs8 + sout + 8 * i, (lane & 3) == 0);
    }
    fetch(t + p.depth * step, st);
    if (++st == p.depth) st = 0;
    float r2 = 1.f;
    if (has_pre) {
      r2 = rsqrt2(team_sum(ss.x + ss.y, part[odd][1], team, nt, lane, warp, warps) * inv_k + a.eps).hi;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        float2 g[4];
        unpack4(pre[c0 + 32 * i], g);
#pragma unroll
        for (int j = 0; j < 4; ++j) h[i][j] = __fmul2_rn(__fmul2_rn(h[i][j], dup(r2)), g[j]);
        if (a.out != nullptr && valid[i]) st_row16(a.out + out + 256 * i, pack4(h[i]));
        if (a.q8 != nullptr)
          store_mx8(h[i], a.nosat, valid[i], a.q8 + out + 256 * i, a.s8 + sout + 8 * i, (lane & 3) == 0);
      }
    }
    if (a.rstd != nullptr && tid == 0) {
      a.rstd[t] = r1;
      a.rstd[(size_t)T + t] = r2;
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// ---------------------------------------------------------------- gradient
// Three sums at once: lanes give up one of two values where a butterfly step would
// carry both (13 shuffles for 27). Lane 0 ends with the first, 16 the second, 8 the third.
__device__ __forceinline__ float merge3(float a, float b, float c, int lane) {
  const bool hi = lane & 16, mid = lane & 8;
  float k = (hi ? b : a) + __shfl_xor_sync(0xffffffffu, hi ? a : b, 16);
  c += __shfl_xor_sync(0xffffffffu, c, 16);
  return (mid ? c : k) + __shfl_xor_sync(0xffffffffu, mid ? k : c, 8);
}
__device__ __forceinline__ float fold8(float v) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Over a team of nt threads of the CTA (its own named barrier, none for one warp), or over a pair of CTAs,
// each of which writes its parts into both; part: [3 ROWS][32], a place a warp.
template <int ROWS, bool PAIR>
__device__ __forceinline__ void team_sum3(float (&v)[ROWS][3], float (*part)[32], int team, int nt, int lane,
                                          int warp, int warps) {
  float m[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) m[r] = fold8(merge3(v[r][0], v[r][1], v[r][2], lane));
  if (PAIR || warps > 1) {
    const uint32_t rank = PAIR ? cluster_rank() : 0;
    const int base = PAIR ? 16 * rank : team * warps;
    if ((lane & 7) == 0 && lane < 24) {
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        float* to = &part[3 * r + (lane == 0 ? 0 : lane == 16 ? 1 : 2)][base + warp];
        *to = m[r];
        if (PAIR)
          asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_addr(to, rank ^ 1)), "f"(m[r]) : "memory");
      }
    }
    if (PAIR) cluster_sync();
    else named_barrier(team + 1, nt);
    const bool there = (PAIR ? lane & 15 : lane) < warps;
    const int at = PAIR ? lane : base + lane;
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
      m[r] = fold8(merge3(there ? part[3 * r][at] : 0.f, there ? part[3 * r + 1][at] : 0.f,
                          there ? part[3 * r + 2][at] : 0.f, lane));
  }
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    v[r][0] = __shfl_sync(0xffffffffu, m[r], 0);
    v[r][1] = __shfl_sync(0xffffffffu, m[r], 16);
    v[r][2] = __shfl_sync(0xffffffffu, m[r], 8);
  }
}

// A sum as a value and its remainder, so that what cancels in the value is kept. The gradient of the residual's scale
// adds up T K products of both signs: T = 777, K = 2880, magnitudes of 5000 that come to about 4. One fp32 value
// a thread, a warp and a CTA left that off by 6.8e-7 in the median and 3.1e-6 at worst of 300 input sets, a
// relative 2e-5 where little is left; with remainders 2.0e-7 and 0.9e-6, what the roundings of
// dh + r2 v and of the row's mean come to (calls that ask for this gradient take 1 to 5% longer).
struct Sum {
  float hi, lo;
  __device__ __forceinline__ void add(const Sum& v) {
    const float t = __fadd_rn(hi, v.hi), w = __fsub_rn(t, hi);
    const float e = __fadd_rn(__fsub_rn(hi, __fsub_rn(t, w)), __fsub_rn(v.hi, w));
    lo = __fadd_rn(__fadd_rn(lo, v.lo), e);
    hi = t;
  }
  __device__ __forceinline__ void add_lanes() {   // lane 0: of the warp
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      add(Sum{__shfl_xor_sync(0xffffffffu, hi, o), __shfl_xor_sync(0xffffffffu, lo, o)});
  }
  // (the remainder of a sum that is not finite is none)
  __device__ __forceinline__ float value() const { return fabsf(hi) < INFINITY ? __fadd_rn(hi, lo) : hi; }
};
__device__ __forceinline__ float2 sub2(const float2& a, const float2& b) { return __ffma2_rn(b, dup(-1.f), a); }
// sum += a b, and e += what that rounds off: exactly where the sum is the larger part, else to a rounding of a b, as
// a itself has one.
__device__ __forceinline__ void add_product(float2& sum, float2& e, const float2& a, const float2& b) {
  const float2 to = __ffma2_rn(a, b, sum);
  e = __fadd2_rn(e, __ffma2_rn(a, b, sub2(sum, to)));
  sum = to;
}

// 8 values from shared memory: bf16, or E4M3 without their block's factor.
__device__ __forceinline__ void slot8(const uint8_t* p, bool e4m3, float2 (&v)[4]) {
  if (!e4m3) {
    unpack4(*reinterpret_cast<const uint4*>(p), v);
    return;
  }
  const uint2 q = *reinterpret_cast<const uint2*>(p);
  v[0] = e4m3x2_values((uint16_t)q.x);
  v[1] = e4m3x2_values((uint16_t)(q.x >> 16));
  v[2] = e4m3x2_values((uint16_t)q.y);
  v[3] = e4m3x2_values((uint16_t)(q.y >> 16));
}
// Shared memory of the gradient: post_gamma, times a channel's gate (fp32, in two halves of
// 4 values a chunk), then for every team a ring of rows. A row's slots lie by warp and
// chunk, [dh][dy][x][h][gate] of 32 lanes each, the residual's after the warp's chunks; a
// thread fills and reads its own slots alone. What is not there (a gradient, lanes past
// the row, rows past the last) is filled with zeros.
struct BwdPlan {
  int nt, teams, depth;        // threads of a team, teams, stages of a ring (1..4)
  int gate_bytes, row, stage;  // bytes before the rings; of a row; of a team's rows of one step
  int smem;
  bool has_dh, has_dy;         // (a gradient that is not there has the other's address)
};
// E8 0: x and h in bf16, 1: both in E4M3, 2: as the scales tell.
template <int GATE, int E8>
struct Slots {   // byte offsets
  static constexpr int dh = 0, dy = 512, x = 1024, h = x + (E8 == 1 ? 256 : 512), gate = h + (E8 == 1 ? 256 : 512),
                       size = gate + (GATE >= 2 ? 512 : 0);
};
constexpr int kSwChunks = 2;   // chunks of a thread in the gradient
// Chunks of the first half of a row whose columns a pair of CTAs shares (whole 32-value blocks).
__host__ __device__ constexpr int half_chunks(int K) { return (K / 16 + 3) & ~3; }
// Bytes of a warp's slots of one chunk.
int slots_bytes(bool full_gate, int e8, bool res) {
  return 1024 + (e8 == 1 ? 512 : 1024) + (full_gate ? 512 : 0) + (res ? 512 : 0);
}

// What a column's second sum comes to, of post_gamma's (x) and of a channel gate's (y) gradient; its
// gate and post_gamma as bits.
__device__ __forceinline__ float2 finish_column(const SandwichBwdArgs& a, uint32_t gate, uint32_t post, float s1) {
  const Gate g = a.gate_kind == 1 ? gate_of(__uint_as_float(gate << 16), a.gate_act) : Gate{1.f, 1.f};
  return make_float2(g.v * s1, g.d * ((a.post != nullptr ? __uint_as_float(post << 16) : 1.f) * s1));
}
// Four neighbouring sums, the e-th four of a row of ws: finished where one CTA holds all rows.
__device__ __forceinline__ void put_sums(const SandwichBwdArgs& a, float* row, bool all, int e, const float4& v) {
  if (!all) {
    reinterpret_cast<float4*>(row)[e] = v;
    return;
  }
  const int k = 4 * e;
  if (k < a.K) {
    if (a.dpre != nullptr) *reinterpret_cast<float4*>(a.dpre + k) = v;
    return;
  }
  const int c = k - a.K;
  const uint2 g = a.gate_kind == 1 ? __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.gate) + c))
                                   : make_uint2(0u, 0u);
  const uint2 p = a.post != nullptr ? __ldg(reinterpret_cast<const uint2*>(a.post + c)) : make_uint2(0u, 0u);
  const float2 o[4] = {finish_column(a, g.x & 0xFFFFu, p.x & 0xFFFFu, v.x), finish_column(a, g.x >> 16, p.x >> 16, v.y),
                       finish_column(a, g.y & 0xFFFFu, p.y & 0xFFFFu, v.z), finish_column(a, g.y >> 16, p.y >> 16, v.w)};
  if (a.dpost != nullptr) *reinterpret_cast<float4*>(a.dpost + c) = make_float4(o[0].x, o[1].x, o[2].x, o[3].x);
  if (a.gate_kind == 1 && a.dgate != nullptr)
    *reinterpret_cast<float4*>(static_cast<float*>(a.dgate) + c) = make_float4(o[0].y, o[1].y, o[2].y, o[3].y);
}

// Column sums of the CTA's (the pair's) rows go to ws [CTAs or pairs][2][K]: 0 dy * h^, 1 d x^ with
// d = dn, or dh_total where the gate is a channel's (its gate and post_gamma take
// their gradients from the one sum). After them ws holds a Sum a CTA, of dh_total * res.
// GATE 0: none or a token's, 1: a channel's, 2: one for every value, 3: the same through a sigmoid.
// A warp holds CH * 32 chunks in a row, lane after lane, so that the chunks of a thread lie
// at fixed distances. ROWS: rows that a team takes together, two independent chains of
// work for a warp and half the waits (T = 8192, K = 6144, 8-bit x and h: 93 us for 117).
// PAIR: a row is the work of a cluster of two CTAs, half its columns each, whose sums meet in both CTAs'
// shared memory (T = 2048, K = 16384: 92 us from bf16, 89 from 8 bits; four chunks a thread in one CTA spill, 110 and
// 130).
template <int GATE, int E8, int ROWS, int MAXT, bool PAIR>
__global__ void __launch_bounds__(MAXT, 1)
    sandwich_bwd_kernel(const SandwichBwdArgs a, const BwdPlan p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float part[2][3 * ROWS][32];
  __shared__ Sum last[32];
  using L = Slots<GATE, E8>;
  // pre_gamma is in registers, the weights are in shared memory as fp32; where registers are short and no
  // channel's gate is in the weights, both gammas are there as bf16, the same bytes. A spilled register is dear
  // here: beside the ring L1 is a few KB, so that it comes back from L2 (a full gate's sigmoid with 8-bit x and h,
  // T = 4096, K = 7168: 124 us with 20 bytes spilled, 87 without; K = 16384: 159, 111).
  constexpr bool kBf16 = GATE >= 2 || (GATE == 0 && (PAIR || E8 == 2));
  constexpr int CH = kSwChunks;
  const int nt = p.nt, team = threadIdx.x / nt, tid = threadIdx.x - team * nt;
  const int lane = tid & 31, warp = tid >> 5, warps = nt >> 5;
  // this CTA's columns: n8 chunks of 8 from chunk b0 on; this thread's: c0 + 32 i of them
  const uint32_t rank = PAIR ? cluster_rank() : 0;
  const unsigned unit = PAIR ? blockIdx.x >> 1 : blockIdx.x, units = PAIR ? gridDim.x >> 1 : gridDim.x;
  const int b0 = rank * half_chunks(a.K), n8 = !PAIR ? a.K / 8 : rank == 0 ? half_chunks(a.K) : a.K / 8 - b0;
  const int c0 = warp * (32 * CH) + lane, g0 = b0 + c0;
  const unsigned T = (unsigned)a.T;   // unsigned: T + the step may pass 2^31
  const bool scaled_res = a.rscale != nullptr;
  const float scale = scaled_res ? *a.rscale : 1.f;
  const uint16_t* gate16 = static_cast<const uint16_t*>(a.gate);
  const bool has_dy = p.has_dy, has_dh = p.has_dh, has_post = a.post != nullptr;
  const bool has_res = a.dscale != nullptr;
  const bool x8 = E8 == 1 || (E8 == 2 && a.xs != nullptr), h8 = E8 == 1 || (E8 == 2 && a.hs != nullptr);
  uint8_t* mine = smem + p.gate_bytes + (size_t)team * p.depth * p.stage + warp * (CH * (L::size + (has_res ? 512 : 0)));
  const int lane16 = 16 * lane, lane_x = (x8 ? 8 : 16) * lane, lane_h = (h8 ? 8 : 16) * lane;
  const int res0 = CH * L::size + lane16;
  float4* gch = reinterpret_cast<float4*>(smem);   // [2][chunks of a team]
  const int gch_half = CH * nt;
  uint4* wbf = reinterpret_cast<uint4*>(smem);     // or [post_gamma, pre_gamma][chunks of a team]
  bool valid[CH];
  uint4 gn[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = c0 + 32 * i;
    valid[i] = c < n8;
    gn[i] = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);   // 1
    if (kBf16 && team == 0) {
      wbf[c] = valid[i] && has_post ? ld_row16(a.post + 8 * (b0 + c)) : gn[i];
      wbf[gch_half + c] = valid[i] && has_dy ? ld_row16(a.pre + 8 * (b0 + c)) : gn[i];
    }
    if (!kBf16 && team == 0) {
      float g[8], w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = w[j] = 1.f;
      if (valid[i]) {
        if (GATE == 1) unpack8(ld_row16(gate16 + 8 * (b0 + c)), g);
        if (has_post) unpack8(ld_row16(a.post + 8 * (b0 + c)), w);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = GATE == 1 ? gate_value(g[j], a.gate_act) * w[j] : w[j];
      gch[c] = make_float4(g[0], g[1], g[2], g[3]);
      gch[gch_half + c] = make_float4(g[4], g[5], g[6], g[7]);
    }
    if (!kBf16 && valid[i] && has_dy) gn[i] = ld_row16(a.pre + 8 * (b0 + c));
  }
  __syncthreads();
  if (PAIR) cluster_sync();   // the other CTA has begun: its shared memory may be written
  // post_gamma, times the channel's gate
  auto weight_of = [&](int i, float2 (&v)[4]) {
    if (kBf16) {
      unpack4(wbf[c0 + 32 * i], v);
      return;
    }
    const float4 w0 = gch[c0 + 32 * i], w1 = gch[gch_half + c0 + 32 * i];
    v[0] = make_float2(w0.x, w0.y);
    v[1] = make_float2(w0.z, w0.w);
    v[2] = make_float2(w1.x, w1.y);
    v[3] = make_float2(w1.z, w1.w);
  };
  // Rows t .. t + ROWS - 1 into stage st. Addresses stay inside the arrays' last row but for
  // lanes past its end, whose copies read nothing.
  const uint32_t mine_addr = smem_u32(mine);
  const int n_dh = has_dh ? 16 : 0, n_dy = has_dy ? 16 : 0;
  auto fetch = [&](unsigned t, int st) {
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const int there = t + r < T ? 16 : 0;
      const size_t at = (size_t)min(t + r, T - 1) * a.K + 8 * g0;
      const uint32_t to = mine_addr + st * p.stage + r * p.row;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int n = valid[i] ? there : 0;
        const uint32_t base = to + i * L::size;
        copy16(base + L::dh + lane16, a.dh + at + 256 * i, n & n_dh);
        copy16(base + L::dy + lane16, a.dy + at + 256 * i, n & n_dy);
        if (h8) copy8(base + L::h + lane_h, static_cast<const uint8_t*>(a.h) + at + 256 * i, (n & n_dy) >> 1);
        else copy16(base + L::h + lane_h, static_cast<const uint16_t*>(a.h) + at + 256 * i, n & n_dy);
        if (x8) copy8(base + L::x + lane_x, static_cast<const uint8_t*>(a.x) + at + 256 * i, n >> 1);
        else copy16(base + L::x + lane_x, static_cast<const uint16_t*>(a.x) + at + 256 * i, n);
        if (GATE >= 2) copy16(base + L::gate + lane16, gate16 + at + 256 * i, n);
        if (has_res) copy16(to + res0 + 512 * i, a.residual + at + 256 * i, n);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // What is not worth a slot, one step ahead: the rows' factors and scale bytes (of the last
  // row, where a row is not there: its values are zeros).
  struct RowScalars {
    float r1[ROWS], r2[ROWS], g[ROWS];
    uint32_t xs[ROWS][CH], hs[ROWS][CH];
  };
  int sc[CH];   // this thread's scale bytes
#pragma unroll
  for (int i = 0; i < CH; ++i) sc[i] = (b0 + min(c0 + 32 * i, n8 - 1)) >> 2;
  auto scalars = [&](unsigned t0, RowScalars& s) {
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const unsigned t = min(t0 + r, T - 1);
      s.r1[r] = s.g[r] = 1.f;
      s.r2[r] = 0.f;
      if (has_post) s.r1[r] = ldg_ahead(a.rstd + t);
      if (has_dy) s.r2[r] = ldg_ahead(a.rstd + (size_t)T + t);
      if (GATE == 0 && a.gate_kind == 2) s.g[r] = ldg_ahead(static_cast<const float*>(a.gate) + t);
      if (E8 != 0) {
        const size_t row = (size_t)t * (a.K / 32);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          s.xs[r][i] = x8 ? ldg_u8(a.xs + row + sc[i]) : 127u;
          s.hs[r][i] = h8 && has_dy ? ldg_u8(a.hs + row + sc[i]) : 127u;
        }
      }
    }
  };
  float2 s_pre[CH][4], s_x[CH][4];
  // dscale = sum dh_total res, with q = dh + r2 v sum q res - c2 r2 sum h res. The first pass adds up both, so that
  // the rounding of dh_total stays out of it (the same for every value of an 8-bit code: T = 1151, K = 3008 off by
  // 3.7e-7 for 7.2e-7). Channel gates of pairs and of mixed types and sigmoids of pairs leave it no
  // register for that: the second pass adds up dh_total res.
  constexpr bool kFirst = PAIR ? GATE == 0 || GATE == 2 : GATE != 1 || E8 != 2;
  float2 s_res = dup(0.f);
  Sum s_all = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s_pre[i][j] = s_x[i][j] = dup(0.f);
  const unsigned step = units * p.teams * ROWS;
  const unsigned first = (unit * p.teams + team) * ROWS;
  grid_launch_dependents();
  RowScalars now = {}, next = {};
  scalars(first, next);
  for (int d = 0; d < p.depth; ++d) fetch(first + d * step, d);
  const float inv_k = 1.f / (float)a.K;
  int odd = 0, st = 0;
  for (unsigned t = first; t < T; t += step, odd ^= 1) {
    now = next;
    scalars(t + step, next);
    float fx[ROWS][CH], fh[ROWS][CH];
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        fx[r][i] = E8 != 0 ? e8m0_to_f32(now.xs[r][i]) : 1.f;
        fh[r][i] = E8 != 0 ? e8m0_to_f32(now.hs[r][i]) : 1.f;
      }
    copies_wait(p.depth - 1);
    uint8_t* slot = mine + st * p.stage;
    // v h, w x (dh + r2 v), w x h; w without a token's gate. An 8-bit block's factor is taken
    // into the sums of its chunk and into the row's factors, not into every value.
    float2 s2[ROWS][3];
    float s_h[ROWS];   // h * res of this thread's part of the row
#pragma unroll
    for (int r = 0; r < ROWS; ++r) s_h[r] = 0.f;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) s2[r][0] = s2[r][1] = s2[r][2] = dup(0.f);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      float2 g[4], w0[4];
      unpack4(kBf16 ? wbf[gch_half + c0 + 32 * i] : gn[i], g);
      weight_of(i, w0);
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        uint8_t* at = slot + r * p.row + i * L::size;
        float2 q[4], h[4], w[4], x[4], v[4];
        unpack4(*reinterpret_cast<const uint4*>(at + L::dh + lane16), q);
        unpack4(*reinterpret_cast<const uint4*>(at + L::dy + lane16), v);
        slot8(at + L::h + lane_h, h8, h);
        slot8(at + L::x + lane_x, x8, x);
        const float2 r2 = dup(now.r2[r]), hr2 = dup(now.r2[r] * fh[r][i]);
        float2 c2[3] = {dup(0.f), dup(0.f), dup(0.f)};
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = w0[j];
        if (GATE >= 2) {
          float2 f[4];
          unpack4(*reinterpret_cast<const uint4*>(at + L::gate + lane16), f);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            w[j] = __fmul2_rn(w[j], make_float2(full_gate(f[j].x, GATE == 3).v, full_gate(f[j].y, GATE == 3).v));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s_pre[i][j] = __ffma2_rn(v[j], __fmul2_rn(h[j], hr2), s_pre[i][j]);
          v[j] = __fmul2_rn(v[j], g[j]);
          q[j] = __ffma2_rn(r2, v[j], q[j]);
          const float2 wx = __fmul2_rn(w[j], x[j]);
          float2(&to)[3] = E8 != 0 ? c2 : s2[r];
          to[0] = __ffma2_rn(v[j], h[j], to[0]);
          to[1] = __ffma2_rn(wx, q[j], to[1]);
          to[2] = __ffma2_rn(wx, h[j], to[2]);
        }
        if (E8 != 0) {
          s2[r][0] = __ffma2_rn(c2[0], dup(fh[r][i]), s2[r][0]);
          s2[r][1] = __ffma2_rn(c2[1], dup(fx[r][i]), s2[r][1]);
          s2[r][2] = __ffma2_rn(__fmul2_rn(c2[2], dup(fx[r][i])), dup(fh[r][i]), s2[r][2]);
        }
        if (kFirst && has_res) {
          float2 z[4], e = dup(0.f), hz = dup(0.f);
          unpack4(*reinterpret_cast<const uint4*>(slot + r * p.row + res0 + 512 * i), z);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            add_product(s_res, e, q[j], z[j]);
            hz = __ffma2_rn(h[j], z[j], hz);
          }
          s_all.lo += e.x + e.y;
          s_h[r] = fmaf(hz.x + hz.y, fh[r][i], s_h[r]);
        }
        // dh + r2 v goes where dh and dy were, for the second pass
        *reinterpret_cast<float4*>(at + L::dh + lane16) = make_float4(q[0].x, q[0].y, q[1].x, q[1].y);
        *reinterpret_cast<float4*>(at + L::dy + lane16) = make_float4(q[2].x, q[2].y, q[3].x, q[3].y);
      }
    }
    float s[ROWS][3];
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
      for (int n = 0; n < 3; ++n) s[r][n] = s2[r][n].x + s2[r][n].y;
    team_sum3<ROWS, PAIR>(s, part[odd], team, nt, lane, warp, warps);
    float kh[ROWS], k1[ROWS], xr[ROWS];   // of h^, of x^ times the token's gate, of x
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const float r1 = now.r1[r], r2 = now.r2[r];
      const float gt = GATE == 0 && a.gate_kind == 2 ? gate_value(now.g[r], a.gate_act) : 1.f;
      const float c2 = s[r][0] * r2 * inv_k * r2;                 // r2 mean(v h^)
      const float dot = r1 * (s[r][1] - c2 * (r2 * s[r][2]));     // sum of w x^ dh_total
      if (GATE == 0 && a.gate_kind == 2 && a.dgate != nullptr && tid == 0 && rank == 0 && t + r < T)
        static_cast<float*>(a.dgate)[t + r] = dot * gate_of(now.g[r], a.gate_act).d;
      kh[r] = -c2;
      if (kFirst && has_res) {   // (an infinite residual is in the first sum, with its sign)
        const bool in = fabsf(s_h[r]) < INFINITY || !(fabsf(c2) < INFINITY);
        s_all.add(Sum{in ? -(c2 * s_h[r]) * r2 : 0.f, 0.f});
      }
      k1[r] = has_post ? -r1 * (dot * inv_k) : 0.f;
      xr[r] = r1 * gt;
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const size_t out = (size_t)(t + r) * a.K + 8 * g0;
      const bool there = t + r < T;
      const bool st_res = there && a.dres != nullptr, st_x = there && a.dx != nullptr;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const uint8_t* at = slot + r * p.row + i * L::size;
        float2 d[4], x[4], v[4], h[4], w[4];   // d: dh_total
        const float2 hr2 = dup(now.r2[r] * fh[r][i]), xrf = dup(xr[r] * fx[r][i]);
        weight_of(i, w);
        const float4 q0 = *reinterpret_cast<const float4*>(at + L::dh + lane16);
        const float4 q1 = *reinterpret_cast<const float4*>(at + L::dy + lane16);
        d[0] = make_float2(q0.x, q0.y);
        d[1] = make_float2(q0.z, q0.w);
        d[2] = make_float2(q1.x, q1.y);
        d[3] = make_float2(q1.z, q1.w);
        slot8(at + L::h + lane_h, h8, h);
        slot8(at + L::x + lane_x, x8, x);
#pragma unroll
        for (int j = 0; j < 4; ++j) d[j] = __ffma2_rn(dup(kh[r]), __fmul2_rn(h[j], hr2), d[j]);
        if (!kFirst && has_res) {
          unpack4(*reinterpret_cast<const uint4*>(slot + r * p.row + res0 + 512 * i), v);
          float2 e = dup(0.f);
#pragma unroll
          for (int j = 0; j < 4; ++j) add_product(s_res, e, d[j], v[j]);
          s_all.lo += e.x + e.y;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = __fmul2_rn(d[j], dup(scale));
        uint4 o = pack4(v);
        if (st_res && valid[i]) st_row16(a.dres + out + 256 * i, o);
        // d becomes the gated gradient but for a channel's gate, whose sums take it without
        if (GATE >= 2) {
          unpack4(*reinterpret_cast<const uint4*>(at + L::gate + lane16), v);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const Gate gx = full_gate(v[j].x, GATE == 3), gy = full_gate(v[j].y, GATE == 3);
            h[j] = __fmul2_rn(__fmul2_rn(d[j], make_float2(gx.d, gy.d)),
                              __fmul2_rn(__fmul2_rn(x[j], xrf), w[j]));
            d[j] = __fmul2_rn(d[j], make_float2(gx.v, gy.v));
          }
          o = pack4(h);
          if (a.dgate != nullptr && there && valid[i])
            st_row16(static_cast<uint16_t*>(a.dgate) + out + 256 * i, o);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 xn = __fmul2_rn(x[j], xrf);
          s_x[i][j] = __ffma2_rn(d[j], xn, s_x[i][j]);
          // (no post_gamma: r1 = 1, k1 = 0)
          d[j] = __ffma2_rn(dup(k1[r]), xn, __fmul2_rn(__fmul2_rn(d[j], w[j]), dup(xr[r])));
        }
        o = pack4(d);
        if (st_x && valid[i]) st_row16(a.dx + out + 256 * i, o);
      }
    }
    fetch(t + p.depth * step, st);
    if (++st == p.depth) st = 0;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  float* sums = a.ws + (size_t)unit * 2 * a.K;
  if (p.teams > 1) __syncthreads();
  // one team: straight out; several: through shared memory, added up in order
  const bool all = gridDim.x == 1;   // (never a pair)
  float4* const own = reinterpret_cast<float4*>(smem) + (size_t)team * (a.K / 2);
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = c0 + 32 * i;
    if (c >= n8) continue;
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      const float4 v0 = make_float4(s_pre[i][j].x, s_pre[i][j].y, s_pre[i][j + 1].x, s_pre[i][j + 1].y);
      const float4 v1 = make_float4(s_x[i][j].x, s_x[i][j].y, s_x[i][j + 1].x, s_x[i][j + 1].y);
      const int e = 2 * (b0 + c) + j / 2;
      if (p.teams > 1) {
        own[e] = v0;
        own[a.K / 4 + e] = v1;
      } else {
        put_sums(a, sums, all, e, v0);
        put_sums(a, sums, all, a.K / 4 + e, v1);
      }
    }
  }
  if (has_res) {
    Sum sr = s_all;
    sr.add(Sum{s_res.x, 0.f});
    sr.add(Sum{s_res.y, 0.f});
    sr.add_lanes();
    if (lane == 0) last[threadIdx.x >> 5] = sr;
  }
  __syncthreads();
  if (p.teams > 1) {
    const float4* from = reinterpret_cast<const float4*>(smem);
    for (int e = threadIdx.x; e < a.K / 2; e += blockDim.x) {
      float4 v = from[e];
      for (int m = 1; m < p.teams; ++m) {
        const float4 o = from[(size_t)m * (a.K / 2) + e];
        v.x += o.x;
        v.y += o.y;
        v.z += o.z;
        v.w += o.w;
      }
      put_sums(a, sums, all, e, v);
    }
  }
  if (has_res && threadIdx.x < 32) {
    Sum sr = lane < (int)(blockDim.x >> 5) ? last[lane] : Sum{0.f, 0.f};
    sr.add_lanes();
    if (lane == 0) {
      if (all) *a.dscale = sr.value();
      else reinterpret_cast<Sum*>(a.ws + (size_t)units * 2 * a.K)[blockIdx.x] = sr;
    }
  }
}

// The columns' sums over the CTAs' rows of ws, in the order of the CTAs; 32
// columns a CTA, every 16th row a warp, so that few loads follow one another. Launched
// while the rows' kernel still runs; waits for its end before it reads.
constexpr int kColWarps = 16;
__global__ void __launch_bounds__(32 * kColWarps) sandwich_columns_kernel(const SandwichBwdArgs a, int rows, int scalars) {
  __shared__ float part[2][kColWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int k = blockIdx.x * 32 + lane;   // K is a multiple of 32
  grid_dependency_wait();
  float s0 = 0.f, s1 = 0.f;
#pragma unroll 8
  for (int r = warp; r < rows; r += kColWarps) {
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
    for (int w = 0; w < kColWarps; ++w) {
      s0 += part[0][w][lane];
      s1 += part[1][w][lane];
    }
    if (a.dpre != nullptr) a.dpre[k] = s0;
    // (no rows: 0, whatever the weights hold)
    const float2 o = rows == 0 ? dup(0.f)
                               : finish_column(a, a.gate_kind == 1 ? static_cast<const uint16_t*>(a.gate)[k] : 0u,
                                               a.post != nullptr ? a.post[k] : 0u, s1);
    if (a.dpost != nullptr) a.dpost[k] = o.x;
    if (a.gate_kind == 1 && a.dgate != nullptr) static_cast<float*>(a.dgate)[k] = o.y;
  }
  if (a.dscale != nullptr && blockIdx.x == 0 && warp == 1) {
    Sum s = {0.f, 0.f};
    for (int r = lane; r < scalars; r += 32) s.add(reinterpret_cast<const Sum*>(a.ws + (size_t)rows * 2 * a.K)[r]);
    s.add_lanes();
    if (lane == 0) *a.dscale = s.value();
  }
}

// Threads of a row of n8 chunks, ch a thread.
int row_threads(int n8, int ch) { return ((n8 + ch - 1) / ch + 31) / 32 * 32; }

// Lets a kernel have this much dynamic shared memory, once a device.
cudaError_t grant_smem(const void* kernel, int bytes, bool (&granted)[kGrantDevices], std::mutex& mu) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kGrantDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(mu);
  if (granted[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  granted[dev] = e == cudaSuccess;
  return e;
}

template <int CH, int MAXT, int PER_SM, bool FULL>
cudaError_t run_fwd(const SandwichArgs& a, int num_sms, cudaStream_t stream) {
  constexpr int kRing = PER_SM == 2 ? 110 * 1024 : kSwRingBytes;
  static bool granted[kGrantDevices] = {};
  static std::mutex mu;
  const auto kernel = sandwich_norm_kernel<CH, MAXT, PER_SM, FULL>;
  const cudaError_t e = grant_smem(reinterpret_cast<const void*>(kernel), kRing, granted, mu);
  if (e != cudaSuccess) return e;
  FwdPlan p = {};
  p.nt = row_threads(a.K / 8, CH);
  p.teams = MAXT / p.nt;
  const int ctas = PER_SM * num_sms, most = (int)(((unsigned)a.T + ctas - 1) / ctas);
  if (p.teams > most) p.teams = most;
  if (p.teams > 15 && p.nt > 32) p.teams = 15;   // named barriers 1 .. 15
  const int chunks = CH * p.nt;
  p.pre = a.post != nullptr ? 16 * chunks : 0;
  p.gate = p.pre + (a.pre != nullptr ? 16 * chunks : 0);
  p.ring = p.gate + (a.gate_kind == 1 ? 32 * chunks : 0);
  p.slot = a.gate_kind == 3 ? 1536 : 1024;
  p.row = chunks / 32 * p.slot;
  p.depth = (kRing - p.ring) / (p.teams * p.row);
  if (p.depth > 4) p.depth = 4;
  p.smem = p.ring + p.teams * p.depth * p.row;
  const unsigned want = ((unsigned)a.T + p.teams - 1) / p.teams;
  const int grid = want < (unsigned)ctas ? (int)want : ctas;
  kernel<<<grid, p.teams * p.nt, p.smem, stream>>>(a, p);
  return cudaGetLastError();
}

// Threads, rows at a time and ring of a gradient call. One CTA a SM, so that an SM
// leaves one row of column sums; short rows share it, several teams to a CTA.
BwdPlan bwd_plan(const SandwichBwdArgs& a, int num_sms, int e8, int rows, int maxt, bool pair) {
  BwdPlan p = {};
  p.nt = row_threads(pair ? half_chunks(a.K) : a.K / 8, kSwChunks);
  p.teams = pair ? 1 : maxt / p.nt;   // (at most 16, and of one warp each where above 8: named barriers 1 .. 15)
  const int most = (int)(((unsigned)a.T + rows * num_sms - 1) / (rows * num_sms));
  if (p.teams > most) p.teams = most;
  p.row = p.nt / 32 * kSwChunks * slots_bytes(a.gate_kind == 3, e8, a.dscale != nullptr);
  p.stage = rows * p.row;
  p.gate_bytes = 32 * kSwChunks * p.nt;
  p.depth = (kSwRingBytes - p.gate_bytes) / (p.teams * p.stage);
  if (p.depth > 4) p.depth = 4;
  p.has_dh = a.dh != nullptr;
  p.has_dy = a.dy != nullptr;
  if (p.depth < 1) p.depth = 1;   // (never: every form has room for a row; the launch would be refused)
  p.smem = p.gate_bytes + p.teams * p.depth * p.stage;
  const int sums = p.teams > 1 ? p.teams * 8 * a.K : 0;
  if (p.smem < sums) p.smem = sums;
  return p;
}

// Rows of column sums that a call leaves in ws (CTAs or pairs), and the CTAs.
struct BwdGrid {
  int units, ctas;
};

template <int GATE, int E8, int ROWS, int MAXT, bool PAIR>
cudaError_t run_bwd(const SandwichBwdArgs& a, int num_sms, BwdGrid* grid, cudaStream_t stream) {
  static bool granted[kGrantDevices] = {};
  static int resident[kGrantDevices] = {};   // pairs at a time
  static std::mutex mu;
  const auto kernel = sandwich_bwd_kernel<GATE, E8, ROWS, MAXT, PAIR>;
  cudaError_t e = grant_smem(reinterpret_cast<const void*>(kernel), kSwRingBytes, granted, mu);
  if (e != cudaSuccess) return e;
  const BwdPlan p = bwd_plan(a, num_sms, E8, ROWS, MAXT, PAIR);
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(p.teams * p.nt);
  cfg.dynamicSmemBytes = p.smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = PAIR ? 1 : 0;
  int most = num_sms;
  if (PAIR) {   // (whatever the size, one CTA an SM: rows past 8192 values have more than 8 warps of 128 registers)
    int dev = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    std::lock_guard<std::mutex> lk(mu);
    if (resident[dev] == 0) {
      cfg.gridDim = dim3(num_sms / 2 * 2);
      e = cudaOccupancyMaxActiveClusters(&resident[dev], kernel, &cfg);
      if (e != cudaSuccess) return e;
      if (resident[dev] < 1) return cudaErrorInvalidConfiguration;
    }
    most = resident[dev] < num_sms / 2 ? resident[dev] : num_sms / 2;
  }
  const unsigned want = ((unsigned)a.T + ROWS * p.teams - 1) / (ROWS * p.teams);   // (T + 15 may pass 2^31)
  grid->units = want < (unsigned)most ? (int)want : most;
  if (!PAIR && ROWS == 1 && a.T <= kSwOneCta) grid->units = 1;
  if (grid->units > kSwMaxCtas) grid->units = kSwMaxCtas;
  grid->ctas = PAIR ? 2 * grid->units : grid->units;
  // copies that read nothing still name rows that are there
  SandwichBwdArgs k = a;
  if (!p.has_dh) k.dh = a.dy;
  if (!p.has_dy) {
    k.dy = a.dh;
    if (E8 == 1) k.h = a.x;
    else k.h = a.dh, k.hs = nullptr;
  }
  cfg.gridDim = dim3(grid->ctas);
  return cudaLaunchKernelEx(&cfg, kernel, k, p);
}

template <int E8, int MAXT, bool PAIR>
cudaError_t run_bwd_gate(const SandwichBwdArgs& a, int num_sms, BwdGrid* grid, cudaStream_t stream) {
  if (a.gate_kind == 1) return run_bwd<1, E8, 1, MAXT, PAIR>(a, num_sms, grid, stream);
  if (a.gate_kind != 3) return run_bwd<0, E8, 1, MAXT, PAIR>(a, num_sms, grid, stream);
  return a.gate_act ? run_bwd<3, E8, 1, MAXT, PAIR>(a, num_sms, grid, stream)
                    : run_bwd<2, E8, 1, MAXT, PAIR>(a, num_sms, grid, stream);
}
template <bool PAIR>
cudaError_t run_bwd_rows(const SandwichBwdArgs& a, bool x8, bool h8, int num_sms, BwdGrid* grid, cudaStream_t stream) {
  if (x8 != h8) return run_bwd_gate<2, 512, PAIR>(a, num_sms, grid, stream);
  return x8 ? run_bwd_gate<1, 512, PAIR>(a, num_sms, grid, stream)
            : run_bwd_gate<0, 512, PAIR>(a, num_sms, grid, stream);
}
cudaError_t run_bwd_form(const SandwichBwdArgs& a, int num_sms, BwdGrid* grid, cudaStream_t stream) {
  const bool x8 = a.xs != nullptr, h8 = a.dy != nullptr ? a.hs != nullptr : x8;   // (without dy h is not read)
  if (a.K > 16 * 512) return run_bwd_rows<true>(a, x8, h8, num_sms, grid, stream);
  // Two rows a team, 168 registers a thread, for many long rows whose ring is then still two deep: no
  // full gate, no residual, the same type of x and h. One row (16 warps of 128 registers) else. In a graph, one
  // row / two: T = 4000, K = 6144 from bf16 58.8 / 54.9, with the residual 65.6 / 70.9, a full gate 76 / 83; K = 2880
  // 32.4 / 30.5, T = 777 11.5 / 13.1; K = 512 11.3 / 12.2; T = 777, K = 6144 22.2 / 20.5.
  if (a.gate_kind != 3 && a.dscale == nullptr && x8 == h8 && a.K > 2048 && a.K <= 16 * 384 &&
      (size_t)a.T * a.K >= (size_t)9 << 19) {
    if (a.gate_kind == 1)
      return x8 ? run_bwd<1, 1, 2, 384, false>(a, num_sms, grid, stream)
                : run_bwd<1, 0, 2, 384, false>(a, num_sms, grid, stream);
    return x8 ? run_bwd<0, 1, 2, 384, false>(a, num_sms, grid, stream)
              : run_bwd<0, 0, 2, 384, false>(a, num_sms, grid, stream);
  }
  return run_bwd_rows<false>(a, x8, h8, num_sms, grid, stream);
}

cudaError_t run_columns(const SandwichBwdArgs& a, int rows, int scalars, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.K / 32);
  cfg.blockDim = dim3(32 * kColWarps);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = rows > 0 ? 1 : 0;   // (no rows: nothing of this call runs before it)
  return cudaLaunchKernelEx(&cfg, sandwich_columns_kernel, a, rows, scalars);
}

template <bool FULL>
cudaError_t run_fwd_form(const SandwichArgs& a, int num_sms, cudaStream_t stream) {
  // One row an SM at most: a chunk a thread, so that the row's chain is short (T = 32, K = 7168 with 8-bit
  // copies 5.7 us for 6.2, T = 1 with a full gate 5.4 for 6.9). Else two chunks a thread and two CTAs an SM,
  // or for rows past 6144 values four and one.
  if (a.T <= num_sms && a.K <= 8 * 1024) return run_fwd<1, 1024, 1, FULL>(a, num_sms, stream);
  if (a.K <= 16 * 384) return run_fwd<2, 384, 2, FULL>(a, num_sms, stream);
  return run_fwd<4, 512, 1, FULL>(a, num_sms, stream);
}

}  // namespace

cudaError_t launch_sandwich_norm(const SandwichArgs& a, int num_sms, cudaStream_t stream) {
  return a.gate_kind == 3 ? run_fwd_form<true>(a, num_sms, stream) : run_fwd_form<false>(a, num_sms, stream);
}

size_t sandwich_bwd_workspace_bytes(int T, int K) {
  const size_t rows = T < kSwMaxCtas ? T : kSwMaxCtas;
  return rows * (2 * (size_t)K * sizeof(float) + 2 * sizeof(Sum));   // (a Sum each, of a pair two)
}

cudaError_t launch_sandwich_norm_backward(const SandwichBwdArgs& a, int num_sms, cudaStream_t stream) {
  BwdGrid grid = {};
  if (a.T > 0) {   // (no rows: the sums are zero)
    const cudaError_t e = run_bwd_form(a, num_sms, &grid, stream);
    if (e != cudaSuccess) return e;
  }
  if (grid.ctas == 1) return cudaSuccess;   // its CTA has finished the columns itself
  if (a.dpre != nullptr || a.dpost != nullptr || a.dscale != nullptr || (a.gate_kind == 1 && a.dgate != nullptr))
    return run_columns(a, grid.units, grid.ctas, stream);
  return cudaSuccess;
}

}  // namespace mxmoe
