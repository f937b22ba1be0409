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
// One warp per token, lane l holding experts l, l + 32, ... in registers: the
// logits are read once (coalesced 128 bytes a load), 4 T E bytes and as many
// written by the gradient. The losses' sums are per tile of tokens and sequence (a
// piece), written to scratch and added up in a fixed order: no floating-point
// atomics, every repeat gives the same bits.
#include <cstdint>

#include "common.cuh"
#include "ops.h"

namespace mxmoe {
namespace {

constexpr int kMostTileTokens = 2048;   // keeps a warp's fp32 sums short

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float sigmoid(float x) { return __frcp_rn(__fadd_rn(1.f, expf(-x))); }

// A token's logits in registers, masked ones as -inf, and what its softmax needs.
template <int NPL>
struct Token {
  float x[NPL];
  float m, total;   // largest logit; sum of exp(x - m)
  __device__ __forceinline__ void load(const float* row, int E, int lane) {
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
      const int e = lane + 32 * j;
      x[j] = e < E ? __ldg(row + e) : -INFINITY;
    }
  }
  __device__ __forceinline__ void largest() {
    m = -INFINITY;
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
      if (!(x[j] > -INFINITY)) x[j] = -INFINITY;   // NaN too
      m = fmaxf(m, x[j]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  }
  // exp(x - m): 1 at the largest, also where it is infinite
  __device__ __forceinline__ float power(float v) const {
    return v == m ? 1.f : v > -INFINITY ? expf(v - m) : 0.f;
  }
  // the exponentials into ex, their sum into total
  __device__ __forceinline__ void powers(float (&ex)[NPL]) {
    total = 0.f;
#pragma unroll
    for (int j = 0; j < NPL; ++j) total += ex[j] = power(x[j]);
    total = warp_sum(total);
  }
  __device__ __forceinline__ float lse() const { return m + logf(total); }
};

__device__ __forceinline__ unsigned clamp_row(int v, unsigned T) { return v < 0 ? 0u : min((unsigned)v, T); }
// The last sequence that begins at or before row t (offsets[0] is taken as such).
__device__ __forceinline__ int sequence_of(const int32_t* offsets, int S, unsigned t, unsigned T) {
  int lo = 0, hi = S - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (clamp_row(__ldg(offsets + mid), T) <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Scratch: a piece's row is (tile + sequence), which no two pieces share.
struct BalanceScratch {
  float* p;          // [rows, E] sums of p
  int* c;            // [rows, E] counts
  float* z;          // [rows] sums of lse^2
  int* n;            // [rows] tokens
  float *loss, *zs;  // [S]
  int* ns;           // [S]
  unsigned* done;    // sequences finished
};
__host__ __device__ inline size_t balance_layout(size_t rows, size_t E, size_t S, char* base, BalanceScratch* b) {
  size_t o = 0;
  auto take = [&](size_t n) { const size_t at = o; o += (n * 4 + 255) & ~size_t(255); return base + at; };
  b->done = reinterpret_cast<unsigned*>(take(1));
  b->p = reinterpret_cast<float*>(take(rows * E));
  b->c = reinterpret_cast<int*>(take(rows * E));
  b->z = reinterpret_cast<float*>(take(rows));
  b->n = reinterpret_cast<int*>(take(rows));
  b->loss = reinterpret_cast<float*>(take(S));
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

template <int NPL>
__global__ void __launch_bounds__(kBalanceWarps<NPL> * 32)
    balance_pieces_kernel(const RouterBalanceArgs a, const BalanceScratch b, unsigned tile) {
  constexpr int W = kBalanceWarps<NPL>;
  __shared__ float sp[W][32 * NPL];
  __shared__ int sc[W][32 * NPL];
  __shared__ float sz[W];
  __shared__ int sn[W];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = a.E;
  const unsigned T = (unsigned)a.T;
  if (blockIdx.x == 0 && threadIdx.x == 0) *b.done = 0;
#pragma unroll
  for (int j = 0; j < NPL; ++j) sc[warp][lane + 32 * j] = 0;
  __syncwarp();
  const unsigned t0 = blockIdx.x * tile, t1 = min(T, t0 + tile);
  float acc[NPL], z = 0.f;
  int n = 0;
  auto clear = [&]() {
#pragma unroll
    for (int j = 0; j < NPL; ++j) acc[j] = 0.f;
    z = 0.f;
    n = 0;
  };
  // rows first, first + step, ... below last into this warp's sums
  auto rows = [&](unsigned first, unsigned last, unsigned step) {
    for (unsigned t = first; t < last; t += step) {
      Token<NPL> k;
      k.load(a.logits + (size_t)t * E, E, lane);
      const int id = lane < a.topk ? __ldg(a.ids + (size_t)t * a.topk + lane) : -1;
      const bool hit = id >= 0 && id < E;
      k.largest();
      if (!__any_sync(0xffffffffu, hit) || k.m == -INFINITY) continue;
      if (hit) atomicAdd(&sc[warp][id], 1);
      float ex[NPL];
      k.powers(ex);
      const float lse = k.lse();
      z = fmaf(lse, lse, z);
      ++n;
      if (a.scoring == 0) {
        const float inv = __frcp_rn(k.total);
#pragma unroll
        for (int j = 0; j < NPL; ++j) acc[j] = fmaf(ex[j], inv, acc[j]);
      } else {
        float s[NPL], sum = 0.f;
#pragma unroll
        for (int j = 0; j < NPL; ++j) sum += s[j] = sigmoid(k.x[j]);   // (0 at -inf)
        sum = warp_sum(sum);
        const float inv = sum > 0.f ? __frcp_rn(sum) : 0.f;
#pragma unroll
        for (int j = 0; j < NPL; ++j) acc[j] = fmaf(s[j], inv, acc[j]);
      }
    }
  };
  auto piece = [&](int s, unsigned lo, unsigned hi) {
    const size_t at = (size_t)blockIdx.x + s;
    if (a.offsets != nullptr && hi - lo < W) {   // short: one warp's, no waiting
      if (s % W != warp) return;
      clear();
      rows(lo, hi, 1);
      __syncwarp();
#pragma unroll
      for (int j = 0; j < NPL; ++j) {
        const int e = lane + 32 * j;
        if (e < E) {
          b.p[at * E + e] = acc[j];
          b.c[at * E + e] = sc[warp][e];
          sc[warp][e] = 0;
        }
      }
      __syncwarp();
      if (lane == 0) {
        b.z[at] = z;
        b.n[at] = n;
      }
      return;
    }
    clear();
    rows(lo + warp, hi, W);
#pragma unroll
    for (int j = 0; j < NPL; ++j) sp[warp][lane + 32 * j] = acc[j];
    if (lane == 0) {
      sz[warp] = z;
      sn[warp] = n;
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
      int nn = 0;
      for (int w = 0; w < W; ++w) {
        zz += sz[w];
        nn += sn[w];
      }
      b.z[at] = zz;
      b.n[at] = nn;
    }
    __syncthreads();
  };
  if (a.offsets == nullptr) {
    piece(0, t0, t1);
    return;
  }
  // 32 sequences a step, so that runs of empty ones cost little
  for (int s0 = sequence_of(a.offsets, a.S, t0, T); s0 < a.S; s0 += 32) {
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

// A CTA per sequence: its pieces added up in order, its share, slope and loss;
// the last CTA to finish adds up the sequences, in order again.
__global__ void __launch_bounds__(1024)
    balance_sequences_kernel(const RouterBalanceArgs a, const BalanceScratch b, unsigned tile, unsigned tiles) {
  __shared__ float tp[1024], part[32][32];
  __shared__ int tc[1024], partc[32][32];
  __shared__ float red[3][32];
  __shared__ long long redn[2][32];
  __shared__ bool last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int E = a.E, s = blockIdx.x;
  const unsigned T = (unsigned)a.T;
  unsigned lo = 0, hi = T;
  if (a.offsets != nullptr) {
    lo = clamp_row(__ldg(a.offsets + s), T);
    hi = clamp_row(__ldg(a.offsets + s + 1), T);
  }
  const unsigned b0 = lo / tile, b1 = lo < hi ? (hi - 1) / tile + 1 : b0;   // its tiles
  const int blocks = (E + 31) / 32;                      // of 32 columns
  const int across = blocks < warps ? blocks : warps;    // taken at a time
  const int groups = warps / across;                     // row groups of each
  const int cb = warp % across, rg = warp / across;
  for (int c0 = 0; c0 < blocks; c0 += across) {
    const int e = (c0 + cb) * 32 + lane;
    float p = 0.f;
    int c = 0;
    if (e < E && rg < groups) {
#pragma unroll 4
      for (unsigned r = b0 + rg; r < b1; r += groups) {
        const size_t at = ((size_t)r + s) * E + e;
        p += b.p[at];
        c += b.c[at];
      }
    }
    part[warp][lane] = p;
    partc[warp][lane] = c;
    __syncthreads();
    if (rg == 0 && e < E) {
      for (int g = 1; g < groups; ++g) {
        p += part[g * across + cb][lane];
        c += partc[g * across + cb][lane];
      }
      tp[e] = p;
      tc[e] = c;
    }
    __syncthreads();
  }
  float z = 0.f;
  long long n = 0, total = 0;
  for (unsigned r = b0 + threadIdx.x; r < b1; r += blockDim.x) {
    z += b.z[(size_t)r + s];
    n += b.n[(size_t)r + s];
  }
  for (int e = threadIdx.x; e < E; e += blockDim.x) total += tc[e];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    z += __shfl_xor_sync(0xffffffffu, z, o);
    n += __shfl_xor_sync(0xffffffffu, n, o);
    total += __shfl_xor_sync(0xffffffffu, total, o);
  }
  if (lane == 0) {
    red[0][warp] = z;
    redn[0][warp] = n;
    redn[1][warp] = total;
  }
  __syncthreads();
  z = 0.f;
  n = total = 0;
  for (int w = 0; w < warps; ++w) {
    z += red[0][w];
    n += redn[0][w];
    total += redn[1][w];
  }
  float loss = 0.f;
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    const size_t at = (size_t)s * E + e;
    const float share = n > 0 ? (float)E * (float)tc[e] / (float)total : 0.f;
    const float prob = n > 0 ? tp[e] / (float)n : 0.f;
    a.counts[at] = tc[e];
    a.prob[at] = prob;
    a.slope[at] = n > 0 ? share / (float)n : 0.f;
    loss = fmaf(share, prob, loss);
  }
  loss = warp_sum(loss);
  if (lane == 0) red[1][warp] = loss;
  __syncthreads();
  if (threadIdx.x == 0) {
    loss = 0.f;
    for (int w = 0; w < warps; ++w) loss += red[1][w];
    b.loss[s] = loss;
    b.zs[s] = z;
    b.ns[s] = (int)n;
    __threadfence();
    last = atomicAdd(b.done, 1u) == (unsigned)a.S - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  float l = 0.f;
  long long seen = 0;
  z = 0.f;
  n = 0;
  for (int i = threadIdx.x; i < a.S; i += blockDim.x) {
    l += __ldcg(b.loss + i);
    z += __ldcg(b.zs + i);
    const int ni = __ldcg(b.ns + i);
    n += ni;
    seen += ni > 0;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    l += __shfl_xor_sync(0xffffffffu, l, o);
    z += __shfl_xor_sync(0xffffffffu, z, o);
    n += __shfl_xor_sync(0xffffffffu, n, o);
    seen += __shfl_xor_sync(0xffffffffu, seen, o);
  }
  __syncthreads();
  if (lane == 0) {
    red[0][warp] = z;
    red[1][warp] = l;
    redn[0][warp] = n;
    redn[1][warp] = seen;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    l = z = 0.f;
    n = seen = 0;
    for (int w = 0; w < warps; ++w) {
      z += red[0][w];
      l += red[1][w];
      n += redn[0][w];
      seen += redn[1][w];
    }
    a.stats[0] = seen > 0 ? l / (float)seen : 0.f;
    a.stats[1] = n > 0 ? z / (float)n : 0.f;
    a.stats[2] = (float)n;
    a.stats[3] = (float)seen;
  }
}

constexpr int kRbWarps = 8;

template <int NPL>
__global__ void __launch_bounds__(kRbWarps * 32) router_backward_kernel(const RouterBackwardArgs a) {
  const int lane = threadIdx.x & 31;
  const unsigned T = (unsigned)a.T;
  const unsigned t = blockIdx.x * kRbWarps + (threadIdx.x >> 5);
  if (t >= T) return;
  const int E = a.E;
  const float* row = a.logits + (size_t)t * E;
  Token<NPL> k;
  k.load(row, E, lane);
  int id = lane < a.topk ? __ldg(a.ids + (size_t)t * a.topk + lane) : -1;
  if (id >= E) id = -1;
  k.largest();
  float d[NPL];
#pragma unroll
  for (int j = 0; j < NPL; ++j) d[j] = 0.f;
  if (__any_sync(0xffffffffu, id >= 0) && k.m > -INFINITY) {
    float ex[NPL];
    k.powers(ex);
    const float inv = __frcp_rn(k.total);
    if (a.dw != nullptr) {
      // lane r: slot r's score and its part of the gradient
      float s = 0.f, val = 0.f, w = 0.f;
      if (id >= 0) {
        const float v = __ldg(row + id);
        if (v > -INFINITY) {
          s = a.scoring == 0 ? k.power(v) * inv : sigmoid(v);
          w = __ldg(a.dw + (size_t)t * a.topk + lane);
          if (a.scoring == 1) val = sigmoid(-v);   // 1 - s
          else val = 1.f;
        }
      }
      if (a.renormalise) {
        const float D = warp_sum(s);
        const float q = D > 0.f ? s / D : 0.f;
        val *= q * (w - warp_sum(q * w));
      } else {
        val *= s * w;
      }
      val *= a.route_scale;
      const float common = a.scoring == 0 && !a.renormalise ? warp_sum(val) * inv : 0.f;
#pragma unroll
      for (int j = 0; j < NPL; ++j) d[j] = -common * ex[j];
      for (int r = 0; r < a.topk; ++r) {   // also the same expert twice
        const int e = __shfl_sync(0xffffffffu, id, r);
        const float v = __shfl_sync(0xffffffffu, val, r);
        if (e >= 0 && (e & 31) == lane) {
#pragma unroll
          for (int j = 0; j < NPL; ++j)
            if (j == (e >> 5)) d[j] += v;
        }
      }
    }
    if (a.dloss != nullptr) {
      int s = 0;
      bool inside = true;
      if (a.offsets != nullptr) {
        s = sequence_of(a.offsets, a.S, t, T);
        inside = t >= clamp_row(__ldg(a.offsets + s), T) && t < clamp_row(__ldg(a.offsets + s + 1), T);
      }
      if (inside) {
        const float gb = __ldg(a.dloss) / fmaxf(__ldg(a.stats + 3), 1.f);
        const float gz = 2.f * __ldg(a.dloss + 1) / fmaxf(__ldg(a.stats + 2), 1.f);
        const float* slope = a.slope + (size_t)s * E;
        float sl[NPL], p[NPL], dot = 0.f;
#pragma unroll
        for (int j = 0; j < NPL; ++j) sl[j] = lane + 32 * j < E ? __ldg(slope + lane + 32 * j) : 0.f;
        if (a.scoring == 0) {
#pragma unroll
          for (int j = 0; j < NPL; ++j) p[j] = ex[j] * inv;
        } else {
          float sum = 0.f;
#pragma unroll
          for (int j = 0; j < NPL; ++j) sum += p[j] = sigmoid(k.x[j]);
          sum = warp_sum(sum);
          const float is = sum > 0.f ? __frcp_rn(sum) : 0.f;
#pragma unroll
          for (int j = 0; j < NPL; ++j) p[j] *= is;
        }
#pragma unroll
        for (int j = 0; j < NPL; ++j) dot = fmaf(p[j], sl[j], dot);
        dot = warp_sum(dot);
        const float zc = gz * k.lse() * inv;
#pragma unroll
        for (int j = 0; j < NPL; ++j) {
          float u = gb * p[j] * (sl[j] - dot);
          if (a.scoring == 1 && p[j] > 0.f) u *= sigmoid(-k.x[j]);
          d[j] += u;
          if (gz != 0.f && ex[j] > 0.f) d[j] = fmaf(zc, ex[j], d[j]);
        }
      }
    }
  }
  float* out = a.dlogits + (size_t)t * E;
#pragma unroll
  for (int j = 0; j < NPL; ++j)
    if (lane + 32 * j < E) out[lane + 32 * j] = d[j];
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
  const unsigned grid = tiles > 0 ? tiles : 1;   // (no rows: the counter all the same)
#define MXMOE_BP(N) balance_pieces_kernel<N><<<grid, kBalanceWarps<N> * 32, 0, stream>>>(a, b, tile)
  if (per <= 1) MXMOE_BP(1);
  else if (per <= 2) MXMOE_BP(2);
  else if (per <= 4) MXMOE_BP(4);
  else if (per <= 8) MXMOE_BP(8);
  else if (per <= 16) MXMOE_BP(16);
  else MXMOE_BP(32);
#undef MXMOE_BP
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  balance_sequences_kernel<<<a.S, a.S < 128 ? 1024 : 256, 0, stream>>>(a, b, tile, tiles);
  return cudaGetLastError();
}

cudaError_t launch_router_backward(const RouterBackwardArgs& a, cudaStream_t stream) {
  const unsigned blocks = ((unsigned)a.T + kRbWarps - 1) / kRbWarps;
  const int per = (a.E + 31) / 32;
#define MXMOE_RB(N) router_backward_kernel<N><<<blocks, kRbWarps * 32, 0, stream>>>(a)
  if (per <= 1) MXMOE_RB(1);
  else if (per <= 2) MXMOE_RB(2);
  else if (per <= 4) MXMOE_RB(4);
  else if (per <= 8) MXMOE_RB(8);
  else if (per <= 16) MXMOE_RB(16);
  else MXMOE_RB(32);
#undef MXMOE_RB
  return cudaGetLastError();
}

}  // namespace mxmoe
