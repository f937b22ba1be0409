// Balance losses and expert counts of a routing, and the gradient of the
// router's logits.
//
//   s_e = softmax(x)_e or sigmoid(x_e) as the score router computes them; masked
//     experts (x NaN or -inf) have s = 0
//   p_e = s_e / sum s              lse = log sum exp(x)
// A sequence's tokens are its rows with an id in [0, E) and a logit that is not
// masked; over its n tokens
//   c_e = routes to e, C = sum c, P_e = mean p_e
//   balance = E sum_e (c_e / C) P_e      slope_e = dbalance / dp_(t,e) = E c_e / (C n)
// and over all of them balance = the mean over the sequences that have tokens,
// z = mean lse^2. c is a count and has no gradient.
//
//   dx_e, from the weights w_j = scale s_j (or scale q_j, q = s / sum of the chosen):
//     softmax, renormalised  scale q_j (dw_j - sum q dw)           at the chosen
//     sigmoid, renormalised  the same times (1 - s_j)
//     softmax                scale (s_j dw_j at the chosen - p_e sum s dw)
//     sigmoid                scale s_j (1 - s_j) dw_j
//   from the losses:  gb p_e (slope_e - sum p slope) [sigmoid: times 1 - s_e] / sequences
//                     + 2 gz lse softmax(x)_e / tokens
// Nothing is divided by a sum that could have gone to zero before the product:
// q and p are at most 1.
//
// One warp per token, its logits in registers, four neighbours a lane and 16-byte load where rows
// allow it: the logits are read once, 4 T E bytes and as many written by the gradient. Both
// kernels are bound by their instructions, so exponentials and reciprocals are the
// hardware's (a score below 2^-126 is 0; rows of nothing else go through the logits), a sigmoid and its
// complement come from one exponential, and a chosen expert's gradient is put
// together in its slot's lane and written over the rest's, not searched for in the registers.
// The losses' sums are per tile of tokens and sequence (a piece), written to scratch and added
// up in a fixed order: no floating-point atomics, every repeat gives the same bits.
// 8192 tokens, 256 experts, 12 sequences, sigmoid, in a graph: losses 13.1 us (two kernels, the
// first a chain of 3 or 4 tokens a warp), gradient 8.0 us; the launch alone is 2.
#include <cfloat>
#include <cstdint>

#include "common.cuh"
#include "ops.h"
#include "ops_common.cuh"

namespace mxmoe {
namespace {

constexpr int kMostTileTokens = 2048;   // keeps a warp's fp32 sums short

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// sigmoid(x) and sigmoid(-x), neither of which loses its last bits where the other is near 1
struct Sigmoid {
  float s, rest;
};
__device__ __forceinline__ Sigmoid sigmoid(float x) {
  const float e = fast_exp(-fabsf(x)), hi = fast_rcp(1.f + e), lo = e * hi;
  return x < 0.f ? Sigmoid{lo, hi} : Sigmoid{hi, lo};
}

// Rows whose scores all leave fp32's range. Below kFaint a sigmoid is e^x to fp32's last bit, so that its quotients are a
// softmax's, from the logits. They count where the router's own score of the largest logit is not 0.
constexpr float kFaint = -17.f;
__device__ __forceinline__ bool faint_scored(float x) { return expf(-x) < INFINITY; }

// A token's logits in registers, masked ones as -inf, and what its softmax needs. Values
// 4 i .. 4 i + 3 are neighbours (VEC), or 32 experts apart.
template <int NPL, bool VEC>
struct Token {
  float x[NPL];
  float m;   // largest logit, an infinite one as the largest number
  static __device__ __forceinline__ int expert(int j, int lane) {
    return VEC ? (j / 4) * 128 + lane * 4 + j % 4 : lane + 32 * j;
  }
  __device__ __forceinline__ void load(const float* row, int E, int lane) {
#pragma unroll
    for (int j = 0; j < NPL; j += VEC ? 4 : 1) {
      const int e = expert(j, lane);
      if (VEC) {
        float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (e < E) v = __ldg(reinterpret_cast<const float4*>(row + e));
        x[j] = v.x;
        x[j + (VEC ? 1 : 0)] = v.y;
        x[j + (VEC ? 2 : 0)] = v.z;
        x[j + (VEC ? 3 : 0)] = v.w;
      } else {
        x[j] = e < E ? __ldg(row + e) : -INFINITY;
      }
    }
  }
  __device__ __forceinline__ void largest() {
    m = -INFINITY;
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
      x[j] = fmaxf(x[j], -INFINITY);   // NaN becomes -inf
      m = fmaxf(m, x[j]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (m == INFINITY) {
      m = FLT_MAX;
#pragma unroll
      for (int j = 0; j < NPL; ++j) x[j] = fminf(x[j], FLT_MAX);
    }
  }
  __device__ __forceinline__ float power(float v) const { return fast_exp(v - m); }
};

__device__ __forceinline__ unsigned clamp_row(int v, unsigned T) { return v < 0 ? 0u : min((unsigned)v, T); }
// The last sequence that begins at or before row t (the first one is taken as such); 32
// offsets at a time, the whole warp calls.
__device__ __forceinline__ int sequence_of(const int32_t* offsets, int S, unsigned t, unsigned T, int lane) {
  int lo = 0, n = S;   // the answer is one of lo .. lo + n - 1
  while (n > 1) {
    const int stride = (n + 31) / 32, i = (lane + 1) * stride;
    const bool past = i < n && clamp_row(__ldg(offsets + lo + i), T) <= t;
    const int c = __popc(__ballot_sync(0xffffffffu, past));
    lo += c * stride;
    n = min(stride, n - c * stride);
  }
  return lo;
}

// Scratch: a piece's row is (tile + sequence), which no two pieces share.
struct BalanceScratch {
  float* p;          // [rows, E] sums of p
  int* c;            // [rows, E] counts
  float* z;          // [rows] sums of lse^2
  int *n, *ct;       // [rows] tokens, routes
  float *loss, *zs;  // [S, blocks of columns], [S]
  int* ns;           // [S]
  unsigned* done;    // CTAs that have finished
};
constexpr int kColumns = 32;   // experts of a CTA of the second kernel
__host__ __device__ inline size_t column_blocks(size_t E) { return (E + kColumns - 1) / kColumns; }
__host__ __device__ inline size_t balance_layout(size_t rows, size_t E, size_t S, char* base, BalanceScratch* b) {
  size_t o = 0;
  auto take = [&](size_t n) { const size_t at = o; o += (n * 4 + 255) & ~size_t(255); return base + at; };
  b->done = reinterpret_cast<unsigned*>(take(1));
  b->p = reinterpret_cast<float*>(take(rows * E));
  b->c = reinterpret_cast<int*>(take(rows * E));
  b->z = reinterpret_cast<float*>(take(rows));
  b->n = reinterpret_cast<int*>(take(rows));
  b->ct = reinterpret_cast<int*>(take(rows));
  b->loss = reinterpret_cast<float*>(take(S * column_blocks(E)));
  b->zs = reinterpret_cast<float*>(take(S));
  b->ns = reinterpret_cast<int*>(take(S));
  return o;
}
// Tokens of a tile: as many CTAs as fill the SMs twice, and no more than kMostTileTokens.
unsigned tile_tokens(int T) {
  unsigned n = ((unsigned)T + 303) / 304;
  if (n < 8) n = 8;
  return n < (unsigned)kMostTileTokens ? n : (unsigned)kMostTileTokens;
}
unsigned tile_count(int T) { return ((unsigned)T + tile_tokens(T) - 1) / tile_tokens(T); }

template <int NPL>
constexpr int kBalanceWarps = NPL > 16 ? 4 : 8;   // 32 KB of shared memory either way

// A warp's sums over tokens: of p by expert, of lse^2, tokens and routes.
template <int NPL, bool VEC>
struct Sums {
  float acc[NPL], z;
  int n, routes;
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < NPL; ++j) acc[j] = 0.f;
    z = 0.f;
    n = routes = 0;
  }
  // Rows first, first + step, ... below last, the next one's loads under way; counts into hist.
  __device__ __forceinline__ void rows(const RouterBalanceArgs& a, unsigned first, unsigned last, unsigned step,
                                       int lane, int* hist) {
    Token<NPL, VEC> next;
    int next_id = -1;
    auto load = [&](unsigned t) {
      if (t >= last) return;
      next.load(a.logits + (size_t)t * a.E, a.E, lane);
      next_id = lane < a.topk ? __ldg(a.ids + (size_t)t * a.topk + lane) : -1;
    };
    load(first);
    for (unsigned t = first; t < last; t += step) {
      Token<NPL, VEC> k = next;
      const int id = next_id;
      load(t + step);
      const unsigned hit = __ballot_sync(0xffffffffu, id >= 0 && id < a.E);
      k.largest();
      if (hit == 0 || k.m == -INFINITY) continue;
      if (id >= 0 && id < a.E) atomicAdd(&hist[id], 1);
      routes += __popc(hit);
      ++n;
      float s[NPL], total = 0.f, inv;
#pragma unroll
      for (int j = 0; j < NPL; ++j) total += s[j] = k.power(k.x[j]);
      if (a.scoring == 0) {
        total = warp_sum(total);
        inv = fast_rcp(total);
      } else {
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < NPL; ++j) sum += s[j] = fast_rcp(1.f + fast_exp(-k.x[j]));   // (0 at -inf)
        // both sums in one butterfly: the lower half of the warp ends with the first, the upper with the second
        const bool hi = lane & 16;
        float v = (hi ? sum : total) + __shfl_xor_sync(0xffffffffu, hi ? total : sum, 16);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        total = __shfl_sync(0xffffffffu, v, 0);
        sum = __shfl_sync(0xffffffffu, v, 16);
        inv = fast_rcp(sum);
        if (k.m < kFaint) {
          inv = faint_scored(k.m) ? fast_rcp(total) : 0.f;
#pragma unroll
          for (int j = 0; j < NPL; ++j) s[j] = k.power(k.x[j]);
        }
      }
      const float lse = k.m + logf(total);   // (near 1 the hardware's logarithm is off by more than the sum is)
      z = fmaf(lse, lse, z);
#pragma unroll
      for (int j = 0; j < NPL; ++j) acc[j] = fmaf(s[j], inv, acc[j]);
    }
  }
};

// What a sequence's sums of an expert come to: its count, mean and slope written, its part of the
// loss returned.
__device__ __forceinline__ float finish_expert(const RouterBalanceArgs& a, int s, int e, float p, int c, int n,
                                               int routes) {
  const size_t at = (size_t)s * a.E + e;
  const float share = n > 0 ? (float)a.E * (float)c / (float)routes : 0.f;
  const float prob = n > 0 ? p / (float)n : 0.f;
  a.counts[at] = c;
  a.prob[at] = prob;
  a.slope[at] = n > 0 ? share / (float)n : 0.f;
  return share * prob;
}
__device__ __forceinline__ void finish_stats(const RouterBalanceArgs& a, float loss, float z, int n, int seen) {
  a.stats[0] = seen > 0 ? loss / (float)seen : 0.f;
  a.stats[1] = n > 0 ? z / (float)n : 0.f;
  a.stats[2] = (float)n;
  a.stats[3] = (float)seen;
}

// All of it in one CTA, for few tokens in one or two sequences: one launch in place of two
// (32 tokens, 128 experts in a graph 3.6 us for 6.1, 64 tokens, 256 experts 5.6 for 6.9; the host 3 us less).
constexpr int kSmallTokens = 64, kSmallSequences = 2, kSmallWarps = 16;
template <int NPL, bool VEC>
__global__ void __launch_bounds__(32 * kSmallWarps) balance_small_kernel(const RouterBalanceArgs a) {
  constexpr int W = kSmallWarps;
  __shared__ float sp[W][32 * NPL];
  __shared__ int sc[32 * NPL];
  __shared__ float sz[W], sl[W];
  __shared__ int sn[W], sr[W];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned T = (unsigned)a.T;
  float loss = 0.f, z = 0.f;
  int tokens = 0, seen = 0;
  for (int s = 0; s < a.S; ++s) {
    unsigned lo = 0, hi = T;
    if (a.offsets != nullptr) {
      lo = clamp_row(__ldg(a.offsets + s), T);
      hi = clamp_row(__ldg(a.offsets + s + 1), T);
    }
    for (int e = threadIdx.x; e < a.E; e += 32 * W) sc[e] = 0;
    __syncthreads();
    Sums<NPL, VEC> k;
    k.clear();
    k.rows(a, lo + warp, hi, W, lane, sc);
#pragma unroll
    for (int j = 0; j < NPL; ++j) sp[warp][Token<NPL, VEC>::expert(j, lane)] = k.acc[j];
    if (lane == 0) {
      sz[warp] = k.z;
      sn[warp] = k.n;
      sr[warp] = k.routes;
    }
    __syncthreads();
    int n = 0, routes = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      z += sz[w];
      n += sn[w];
      routes += sr[w];
    }
    for (int e = threadIdx.x; e < a.E; e += 32 * W) {
      float p = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) p += sp[w][e];
      loss += finish_expert(a, s, e, p, sc[e], n, routes);
    }
    tokens += n;
    seen += n > 0;
    __syncthreads();
  }
  loss = warp_sum(loss);
  if (lane == 0) sl[warp] = loss;
  __syncthreads();
  if (threadIdx.x == 0) {
    loss = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) loss += sl[w];
    finish_stats(a, loss, z, tokens, seen);
  }
}

// CTAs an SM: three to 8 logits a lane (80 registers; 12 ragged sequences of 256 experts 13.1 us, with 116
// registers 2 us more), two past that, where three would spill (8192 tokens, 12 sequences, three / two: 384 experts
// 16.4 / 15.5, 1024 20.7 / 18.9; softmax of 1024 in one sequence 14.4 / 15.2).
template <int NPL>
constexpr int kBalanceCtas = NPL > 8 ? 2 : 3;
template <int NPL, bool VEC>
__global__ void __launch_bounds__(kBalanceWarps<NPL> * 32, kBalanceCtas<NPL>)
    balance_pieces_kernel(const RouterBalanceArgs a, const BalanceScratch b, unsigned tile) {
  using Tok = Token<NPL, VEC>;
  constexpr int W = kBalanceWarps<NPL>;
  __shared__ float sp[W][32 * NPL];
  __shared__ int sc[W][32 * NPL];
  __shared__ float sz[W];
  __shared__ int sn[W], sr[W];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = a.E;
  const unsigned T = (unsigned)a.T;
  if (blockIdx.x == 0 && threadIdx.x == 0) *b.done = 0;
  grid_launch_dependents();
#pragma unroll
  for (int j = 0; j < NPL; ++j) sc[warp][lane + 32 * j] = 0;
  __syncwarp();
  const unsigned t0 = blockIdx.x * tile, t1 = min(T, t0 + tile);
  Sums<NPL, VEC> k;
  auto piece = [&](int s, unsigned lo, unsigned hi) {
    const size_t at = (size_t)blockIdx.x + s;
    if (a.offsets != nullptr && hi - lo < W) {   // short: one warp's, no waiting
      if (s % W != warp) return;
      k.clear();
      k.rows(a, lo, hi, 1, lane, sc[warp]);
      __syncwarp();
#pragma unroll
      for (int j = 0; j < NPL; ++j) {
        const int e = Tok::expert(j, lane);
        if (e < E) {
          b.p[at * E + e] = k.acc[j];
          b.c[at * E + e] = sc[warp][e];
          sc[warp][e] = 0;
        }
      }
      __syncwarp();
      if (lane == 0) {
        b.z[at] = k.z;
        b.n[at] = k.n;
        b.ct[at] = k.routes;
      }
      return;
    }
    k.clear();
    k.rows(a, lo + warp, hi, W, lane, sc[warp]);
#pragma unroll
    for (int j = 0; j < NPL; ++j) sp[warp][Tok::expert(j, lane)] = k.acc[j];
    if (lane == 0) {
      sz[warp] = k.z;
      sn[warp] = k.n;
      sr[warp] = k.routes;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += 32 * W) {
      float p = 0.f;
      int c = 0;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        p += sp[w][e];
        c += sc[w][e];
        sc[w][e] = 0;
      }
      b.p[at * E + e] = p;
      b.c[at * E + e] = c;
    }
    if (threadIdx.x == 0) {
      float zz = 0.f;
      int nn = 0, rr = 0;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        zz += sz[w];
        nn += sn[w];
        rr += sr[w];
      }
      b.z[at] = zz;
      b.n[at] = nn;
      b.ct[at] = rr;
    }
    __syncthreads();
  };
  if (a.offsets == nullptr) {
    piece(0, t0, t1);
    return;
  }
  // 32 sequences a step, so that runs of empty ones cost little
  for (int s0 = sequence_of(a.offsets, a.S, t0, T, lane); s0 < a.S; s0 += 32) {
    const int s = s0 + lane;
    unsigned lo = T, hi = 0;
    if (s < a.S) {
      lo = max(clamp_row(__ldg(a.offsets + s), T), t0);
      hi = min(clamp_row(__ldg(a.offsets + s + 1), T), t1);
    }
    unsigned some = __ballot_sync(0xffffffffu, lo < hi);
    while (some != 0) {
      const int i = __ffs(some) - 1;
      some &= some - 1;
      piece(s0 + i, __shfl_sync(0xffffffffu, lo, i), __shfl_sync(0xffffffffu, hi, i));
    }
    if (__any_sync(0xffffffffu, s < a.S && clamp_row(__ldg(a.offsets + s), T) >= t1)) break;
  }
}

// A CTA per sequence and 32 experts: the sequence's pieces added up in order (every 16th a
// warp), the share, mean, slope and loss of its experts; the last CTA to finish adds up
// the losses, in order again. Launched while the first kernel still runs.
constexpr int kSeqWarps = 16;
__global__ void __launch_bounds__(32 * kSeqWarps)
    balance_sequences_kernel(const RouterBalanceArgs a, const BalanceScratch b, unsigned tile) {
  __shared__ float part[kSeqWarps][32], pz[kSeqWarps], pl[kSeqWarps];
  __shared__ int partc[kSeqWarps][32], pn[kSeqWarps], pr[kSeqWarps];
  __shared__ bool last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = a.E, blocks = (int)column_blocks(E), s = blockIdx.x / blocks, cb = blockIdx.x % blocks;
  const int e = cb * kColumns + lane;
  const unsigned T = (unsigned)a.T;
  unsigned lo = 0, hi = T;
  if (a.offsets != nullptr) {
    lo = clamp_row(__ldg(a.offsets + s), T);
    hi = clamp_row(__ldg(a.offsets + s + 1), T);
  }
  const unsigned b0 = lo / tile, b1 = lo < hi ? (hi - 1) / tile + 1 : b0;   // its tiles
  grid_dependency_wait();
  float p = 0.f, z = 0.f;
  int c = 0, n = 0, routes = 0;
  for (unsigned r = b0 + threadIdx.x; r < b1; r += 32 * kSeqWarps) {
    z += b.z[(size_t)r + s];
    n += b.n[(size_t)r + s];
    routes += b.ct[(size_t)r + s];
  }
  if (e < E) {
#pragma unroll 8
    for (unsigned r = b0 + warp; r < b1; r += kSeqWarps) {
      const size_t at = ((size_t)r + s) * E + e;
      p += b.p[at];
      c += b.c[at];
    }
  }
  part[warp][lane] = p;
  partc[warp][lane] = c;
  z = warp_sum(z);
  n = __reduce_add_sync(0xffffffffu, n);
  routes = __reduce_add_sync(0xffffffffu, routes);
  if (lane == 0) {
    pz[warp] = z;
    pn[warp] = n;
    pr[warp] = routes;
  }
  __syncthreads();
  if (warp == 0) {
    p = z = 0.f;
    c = n = routes = 0;
#pragma unroll
    for (int w = 0; w < kSeqWarps; ++w) {
      p += part[w][lane];
      c += partc[w][lane];
      z += pz[w];
      n += pn[w];
      routes += pr[w];
    }
    float loss = e < E ? finish_expert(a, s, e, p, c, n, routes) : 0.f;
    loss = warp_sum(loss);
    if (lane == 0) {
      b.loss[(size_t)s * blocks + cb] = loss;
      if (cb == 0) {
        b.zs[s] = z;
        b.ns[s] = n;
      }
      __threadfence();
      last = atomicAdd(b.done, 1u) == gridDim.x - 1;
    }
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  float l = 0.f;
  int seen = 0;
  z = 0.f;
  n = 0;
  for (int i = threadIdx.x; i < a.S * blocks; i += 32 * kSeqWarps) l += __ldcg(b.loss + i);
  for (int i = threadIdx.x; i < a.S; i += 32 * kSeqWarps) {
    z += __ldcg(b.zs + i);
    const int ni = __ldcg(b.ns + i);
    n += ni;   // (at most T)
    seen += ni > 0;
  }
  l = warp_sum(l);
  z = warp_sum(z);
  n = __reduce_add_sync(0xffffffffu, n);
  seen = __reduce_add_sync(0xffffffffu, seen);
  if (lane == 0) {
    pz[warp] = z;
    pl[warp] = l;
    pn[warp] = n;
    pr[warp] = seen;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    l = z = 0.f;
    n = seen = 0;
#pragma unroll
    for (int w = 0; w < kSeqWarps; ++w) {
      z += pz[w];
      l += pl[w];
      n += pn[w];
      seen += pr[w];
    }
    finish_stats(a, l, z, n, seen);
  }
}

constexpr int kRbWarps = 8;

template <int NPL, bool VEC>
__global__ void __launch_bounds__(kRbWarps * 32) router_backward_kernel(const RouterBackwardArgs a) {
  using Tok = Token<NPL, VEC>;
  const int lane = threadIdx.x & 31;
  const unsigned T = (unsigned)a.T;
  const unsigned t = blockIdx.x * kRbWarps + (threadIdx.x >> 5);
  if (t >= T) return;
  const int E = a.E;
  const float* row = a.logits + (size_t)t * E;
  float* out = a.dlogits + (size_t)t * E;
  Tok k;
  k.load(row, E, lane);
  int id = lane < a.topk ? __ldg(a.ids + (size_t)t * a.topk + lane) : -1;
  if (id >= E) id = -1;
  const float w = a.dw != nullptr && id >= 0 ? __ldg(a.dw + (size_t)t * a.topk + lane) : 0.f;
  float v = id >= 0 ? __ldg(row + id) : -INFINITY;   // lane r: slot r's logit
  // the losses' parts: gb, gz 0 where they do not count
  float gb = 0.f, gz = 0.f;
  const float* slope = a.slope;
  if (a.dloss != nullptr) {
    int s = 0;
    bool inside = true;
    if (a.offsets != nullptr) {
      s = sequence_of(a.offsets, a.S, t, T, lane);
      inside = t >= clamp_row(__ldg(a.offsets + s), T) && t < clamp_row(__ldg(a.offsets + s + 1), T);
    }
    if (inside) {
      gb = __ldg(a.dloss) / fmaxf(__ldg(a.stats + 3), 1.f);
      gz = 2.f * __ldg(a.dloss + 1) / fmaxf(__ldg(a.stats + 2), 1.f);
      slope += (size_t)s * E;
    }
  }
  const bool losses = gb != 0.f || gz != 0.f;   // (the same in the whole warp)
  k.largest();
  v = fminf(fmaxf(v, -INFINITY), k.m);   // masked: -inf; an infinite one as in the registers
  float d[NPL];
#pragma unroll
  for (int j = 0; j < NPL; ++j) d[j] = 0.f;
  const bool live = __any_sync(0xffffffffu, id >= 0) && k.m > -INFINITY;
  float val = 0.f;   // lane r: slot r's part of the gradient of its expert, then all of it
  if (live) {
    float ex[NPL], total = 0.f;
    const float vx = k.power(v);
#pragma unroll
    for (int j = 0; j < NPL; ++j) total += ex[j] = k.power(k.x[j]);
    total = warp_sum(total);
    const float inv = fast_rcp(total);
    const Sigmoid sv = sigmoid(v);   // (-inf: 0 and 1)
    const bool soft = a.scoring == 0, there = v > -INFINITY;
    float common = 0.f;
    if (a.dw != nullptr) {
      float s = soft ? vx * inv : sv.s;
      const float wv = there ? w : 0.f;   // (what is no part's gradient may be anything)
      if (a.renormalise) {
        float D = warp_sum(s);
        if (D < 0x1p-60f) {   // faint scores alone (a bias chose them): their quotients from the logits too
          float most = v;
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
          const bool scored = soft ? __fdiv_rn(expf(most - k.m), total) > 0.f : faint_scored(most);
          s = scored && there ? fast_exp(v - most) : 0.f;
          D = warp_sum(s);
        }
        const float q = D > 0.f ? s / D : 0.f;
        val = q * (wv - warp_sum(q * wv));
      } else {
        val = s * wv;
      }
      if (!soft) val *= sv.rest;
      val *= a.route_scale;
      if (soft && !a.renormalise) common = warp_sum(val) * inv;
    }
    // the same expert in several slots: the first one takes all
    const unsigned twins = __match_any_sync(0xffffffffu, id);
    if (__any_sync(0xffffffffu, id >= 0 && (twins & (twins - 1)) != 0)) {
      float sum = 0.f;
      for (int r = 0; r < a.topk; ++r) {
        const float o = __shfl_sync(0xffffffffu, val, r);
        if ((twins >> r) & 1u) sum += o;
      }
      val = sum;
    }
    float vbase = -common * vx;
#pragma unroll
    for (int j = 0; j < NPL; ++j) d[j] = -common * ex[j];
    if (losses) {
      float sl[NPL], p[NPL], rest[NPL], dot = 0.f, is = inv;
      if (VEC) {
#pragma unroll
        for (int j = 0; j < NPL; j += VEC ? 4 : 1) {
          const int e = Tok::expert(j, lane);
          float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
          if (e < E) q = __ldg(reinterpret_cast<const float4*>(slope + e));
          sl[j] = q.x;
          sl[j + (VEC ? 1 : 0)] = q.y;
          sl[j + (VEC ? 2 : 0)] = q.z;
          sl[j + (VEC ? 3 : 0)] = q.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < NPL; ++j) {
          const int e = Tok::expert(j, lane);
          sl[j] = e < E ? __ldg(slope + e) : 0.f;
        }
      }
      const float vsl = id >= 0 ? __ldg(slope + id) : 0.f;
      const bool faint = !soft && k.m < kFaint, powers = soft || faint;
      if (powers) {
        if (faint && !faint_scored(k.m)) is = 0.f;
#pragma unroll
        for (int j = 0; j < NPL; ++j) {
          p[j] = ex[j];
          rest[j] = 1.f;
        }
      } else {
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < NPL; ++j) {
          const Sigmoid g = sigmoid(k.x[j]);
          sum += p[j] = g.s;
          rest[j] = g.rest;
        }
        sum = warp_sum(sum);
        is = fast_rcp(sum);
      }
#pragma unroll
      for (int j = 0; j < NPL; ++j) dot = fmaf(p[j], sl[j], dot);
      dot = warp_sum(dot) * is;
      const float gp = gb * is;
      const float zc = gz != 0.f ? gz * (k.m + logf(total)) * inv : 0.f;
#pragma unroll
      for (int j = 0; j < NPL; ++j) {
        const float u = gp * p[j] * (sl[j] - dot);
        d[j] = fmaf(u, rest[j], d[j]);
        d[j] = ex[j] > 0.f ? fmaf(zc, ex[j], d[j]) : d[j];   // (an infinite zc stays at the logits that have a part)
      }
      const float u = gp * (powers ? vx : sv.s) * (vsl - dot);
      vbase = fmaf(u, powers ? 1.f : sv.rest, vbase);
      vbase = vx > 0.f ? fmaf(zc, vx, vbase) : vbase;
    }
    val = there ? val + vbase : 0.f;
  }
#pragma unroll
  for (int j = 0; j < NPL; j += VEC ? 4 : 1) {
    const int e = Tok::expert(j, lane);
    if (e >= E) continue;
    if (VEC) {
      *reinterpret_cast<float4*>(out + e) =
          make_float4(d[j], d[j + (VEC ? 1 : 0)], d[j + (VEC ? 2 : 0)], d[j + (VEC ? 3 : 0)]);
    } else {
      out[e] = d[j];
    }
  }
  __syncwarp();
  if (live && id >= 0) out[id] = val;   // after the rest's
}

// Rows that four neighbours of a lane can be read from.
bool rows_vec(int E, const void* a, const void* b, const void* c) {
  return E % 4 == 0 && ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) |
                         reinterpret_cast<uintptr_t>(c)) & 15) == 0;
}

}  // namespace

size_t router_balance_workspace_bytes(int T, int E, int S) {
  BalanceScratch b;
  return balance_layout((size_t)tile_count(T) + S, E, S, nullptr, &b);
}

cudaError_t launch_router_balance(const RouterBalanceArgs& a, int num_sms, cudaStream_t stream) {
  (void)num_sms;
  const unsigned tile = tile_tokens(a.T), tiles = tile_count(a.T);
  BalanceScratch b;
  balance_layout((size_t)tiles + a.S, a.E, a.S, static_cast<char*>(a.ws), &b);
  const int per = (a.E + 31) / 32;
  const bool vec = rows_vec(a.E, a.logits, nullptr, nullptr);
  if (a.T <= kSmallTokens && a.S <= kSmallSequences && per <= 8) {
#define MXMOE_BS(N, V) balance_small_kernel<N, V><<<1, 32 * kSmallWarps, 0, stream>>>(a)
    if (per <= 4) { if (vec) MXMOE_BS(4, true); else MXMOE_BS(4, false); }
    else { if (vec) MXMOE_BS(8, true); else MXMOE_BS(8, false); }
#undef MXMOE_BS
    return cudaGetLastError();
  }
  const unsigned grid = tiles > 0 ? tiles : 1;   // (no rows: the counter all the same)
#define MXMOE_BP(N, V) balance_pieces_kernel<N, V><<<grid, kBalanceWarps<N> * 32, 0, stream>>>(a, b, tile)
  if (per <= 1) MXMOE_BP(1, false);
  else if (per <= 2) MXMOE_BP(2, false);
  else if (per <= 4) { if (vec) MXMOE_BP(4, true); else MXMOE_BP(4, false); }
  else if (per <= 8) { if (vec) MXMOE_BP(8, true); else MXMOE_BP(8, false); }
  else if (per <= 16) { if (vec) MXMOE_BP(16, true); else MXMOE_BP(16, false); }
  else { if (vec) MXMOE_BP(32, true); else MXMOE_BP(32, false); }
#undef MXMOE_BP
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.S * column_blocks(a.E)));
  cfg.blockDim = dim3(32 * kSeqWarps);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, balance_sequences_kernel, a, b, tile);
}

cudaError_t launch_router_backward(const RouterBackwardArgs& a, cudaStream_t stream) {
  const unsigned blocks = ((unsigned)a.T + kRbWarps - 1) / kRbWarps;
  const int per = (a.E + 31) / 32;
  const bool vec = rows_vec(a.E, a.logits, a.slope, a.dlogits);
#define MXMOE_RB(N, V) router_backward_kernel<N, V><<<blocks, kRbWarps * 32, 0, stream>>>(a)
  if (per <= 1) MXMOE_RB(1, false);
  else if (per <= 2) MXMOE_RB(2, false);
  else if (per <= 4) { if (vec) MXMOE_RB(4, true); else MXMOE_RB(4, false); }
  else if (per <= 8) { if (vec) MXMOE_RB(8, true); else MXMOE_RB(8, false); }
  else if (per <= 16) { if (vec) MXMOE_RB(16, true); else MXMOE_RB(16, false); }
  else { if (vec) MXMOE_RB(32, true); else MXMOE_RB(32, false); }
#undef MXMOE_RB
  return cudaGetLastError();
}

}  // namespace mxmoe
