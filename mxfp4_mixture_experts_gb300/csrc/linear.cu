// A shared projection from packed MXFP4 weights with the low-rank adapters of
// many requests beside it:
//   y_t = W x_t + scale_a * B_a (A_a x_t),  a = adapter of token t (or none)
// W = E2M1 * 2^(E8M0 - 127), [N, K]; A_a [rank, K] and B_a [N, rank] in bf16;
// x in bf16, or in MXFP8 (E4M3 with an E8M0 scale per 32 values). Sums in
// fp32, one rounding of y to bf16.
//
//   down    v_t = scale_a * A_a x_t: the tokens of a window grouped by adapter, up to 32 of one adapter to a pass of m16n8k16 tiles, K split
//           over the warps of a CTA and, for few tokens, over the CTAs of a
//           cluster. MXFP8 rows are converted on the way, once, to the bf16 rows
//           that the projection reads (exact but for products beyond bf16's
//           range). T = 8192, K = 6144, rank 16: 34 us for the 150 MB of the
//           conversion, 4.5 TB/s
//   linear  the projection on the 5th-generation tensor cores, the second adapter
//           product as further columns of the same reduction; or, for up to 16
//           tokens, register tiles without any of that
//
// The two launches overlap: the projection starts beside the kernel before it
// and waits for it only where it takes its results.
//
// v is summed in fp32 and rounded to 17 significant bits (2^-17 of each product
// |B_a[n][r] v_t[r]|): the sum of two bf16 values hi and lo, which the tile kernel's
// tensor cores take one after the other into the same fp32 accumulators, so both
// forms multiply the same v. (hi alone leaves 2^-9 of the products, which where
// they or W x cancel is more than y's own rounding; a third part, for all 24 bits,
// would cost half as many MMAs again.)
//
// Tile kernel: a pair of CTAs holds a tile of 256 weight rows x up to 256
// tokens. The MMA computes D[weight row][token] with the dequantised weights as
// operand A in tensor memory and the tokens as operand B in shared memory, half
// of them in each CTA. After the K values, the adapters that the tile's tokens
// name follow as columns: column c stands for (c / rp)-th adapter of the tile,
// rank index c % rp (rp = rank rounded up to 16); operand A holds B_a[n][r],
// operand B hi and, in a second tile, lo of v_t[r] for the tokens of that adapter
// and 0 for the others. So
// tokens need no sorting, and a tile pays for the adapters it has. A B_a value
// that is not finite would turn the others' zeros into NaN; such values are
// left out of the tile and added in the epilogue to the tokens of their adapter
// alone.
//
// Why pairs: with one CTA per tile (128 rows x 256 tokens) every stage of 64 K
// values brought 32 KB of tokens into an SM per 512 clocks of MMAs, the most
// that the path from L2 carries, and the kernel waited on it; in a pair each SM
// takes half of the tokens.
//
// Warp roles: 0 token copies, 1 MMA issue (the even CTA's), 2 copies of packed
// weights, 4..11 adapter columns and epilogue, 12..23 dequantisation in three
// groups that take the stages in turn. Pairs are persistent: the next tile's
// operands are made while the epilogue empties the accumulators, and its MMAs
// run while the output rows go out. Few tiles (small T) split K over up to 4
// pairs of a cluster, whose partial sums meet in shared memory, added in rank
// order.
//
// Measured (T = 8192, K = 6144, N = 4096, rank 16): the tile kernel alone 204 us =
// 2.0 PFLOP/s, its MMAs back to back (1024 clocks for a stage's eight); with the
// down kernel and MXFP8 rows 235 us in a graph. Between 33 and about 1000 tokens the
// dequantisation bounds a stage (its ALU instructions: 350 to 470 clocks of a
// stage at best, 570 to 750 beside the other warps), below that the fixed
// steps of a tile: start 3 us, first operands 2 us, the cluster's addition 2 us.
#include <cuda.h>
#include <cstdint>
#include <mutex>

#include "kernels.h"
#include "ops.h"
#include "ops_common.cuh"

namespace mxmoe {
namespace {

// bf16 rows in pair order (values 0 4 1 5 2 6 3 7 of each group of 8), the order
// in which the bit placement of dequant32_bf16_pairs makes the weights: saves
// the projection a quarter of its dequantisation (470 -> 346 clocks a stage)
__device__ __forceinline__ uint4 pair_order(const uint4& u) {
  return make_uint4(prmt(u.x, u.z, 0x5410u), prmt(u.x, u.z, 0x7632u), prmt(u.y, u.w, 0x5410u),
                    prmt(u.y, u.w, 0x7632u));
}
// 16 E4M3 values of one scale block -> bf16, in row order.
__device__ __forceinline__ void e4m3x16_to_bf16(const uint4& u, uint32_t scale, uint4& a, uint4& b) {
  const ScaleMul sm = e4m3_scale_mul(scale);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  uint32_t o[8], nan = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    e4m3x4_place(w[i], o[2 * i], o[2 * i + 1]);
    nan |= (w[i] & 0x7F7F7F7Fu) + 0x01010101u;   // code 0x7F carries into bit 7
  }
  if (__builtin_expect((nan & 0x80808080u) != 0u, 0)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) e4m3x4_nan(w[i], o[2 * i], o[2 * i + 1]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = bf16x2_mul(o[i], sm.m1);
  if (__builtin_expect(sm.two, 0)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = bf16x2_mul(o[i], sm.m2);
  }
  a = make_uint4(o[0], o[1], o[2], o[3]);
  b = make_uint4(o[4], o[5], o[6], o[7]);
}

// v = hi + lo in bf16 but for 2^-17 |v|: hi the nearest bf16 (the next towards 0 where that
// is infinite), lo the rest, rounded. Infinities and NaN have no rest.
__device__ __forceinline__ void split_bf16(float v, float& hi, float& lo) {
  hi = __uint_as_float((uint32_t)f32_to_bf16_rne(v) << 16);
  lo = 0.f;
  if (fabsf(v) < INFINITY) {
    if (!(fabsf(hi) < INFINITY)) hi = __uint_as_float(__float_as_uint(v) & 0xFFFF0000u);
    lo = __uint_as_float((uint32_t)f32_to_bf16_rne(v - hi) << 16);
  }
}
// v as the sum of its parts: exact, and split into the same sum again.
__device__ __forceinline__ float two_bf16(float v) {
  float hi, lo;
  split_bf16(v, hi, lo);
  return hi + lo;
}
// Two values' parts as bf16 pairs.
__device__ __forceinline__ void split_bf16x2(float a, float b, uint32_t& hi, uint32_t& lo) {
  float ha, la, hb, lb;
  split_bf16(a, ha, la);
  split_bf16(b, hb, lb);
  hi = bf16x2_rn(ha, hb);
  lo = bf16x2_rn(la, lb);
}

__device__ __forceinline__ uint4 ldg16(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
// 32 bytes a lane in one instruction: whole sectors (as two 16-byte halves every
// sector went through L1 twice).
__device__ __forceinline__ void ldg32(const void* p, uint4& a, uint4& b) {
  asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z),
                 "=r"(b.w)
               : "l"(p));
}
__device__ __forceinline__ void stg32(void* p, const uint4& a, const uint4& b) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(a.x), "r"(a.y),
               "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

// 16 bytes of fp32 from L2: written by a kernel that may still run when this one starts.
__device__ __forceinline__ float4 ldcg_f4(const float* p) {
  const uint4 u = ldcg16(p);
  return make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z),
                     __uint_as_float(u.w));
}

// MXFP8 rows -> bf16 rows in pair order, 16 values a thread (calls without adapters).
__global__ void __launch_bounds__(256) mx8_to_bf16_kernel(const uint4* __restrict__ q,
                                                          const uint8_t* __restrict__ s, int64_t n16,
                                                          uint4* __restrict__ out) {
  grid_launch_dependents();
  for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < n16; i += (int64_t)gridDim.x * 256) {
    uint4 a, b;
    e4m3x16_to_bf16(q[i], ldg_u8(s + (i >> 1)), a, b);
    stg32(out + 2 * i, pair_order(a), pair_order(b));
  }
}

// ---------------------------------------------------------------------------
// v = scale A x, in fp32 of two bf16 values: windows of tokens, items of up to 32 tokens of one
// adapter (with MXFP8 rows also of none: those are only converted). gridDim.y
// CTAs take a window's items in turn; the gridDim.z CTAs of a cluster split K
// and add their parts in rank order through shared memory.
// ---------------------------------------------------------------------------
constexpr int kDownWin = 128;     // tokens per window
constexpr int kDownTok = 32;      // tokens per item (two m16 tiles)
constexpr int kDownMaxParts = 8;
constexpr int kDownStep = 64;     // K values per step: 16 a lane
constexpr int kDownSum = 64;      // ranks whose parts a cluster adds at once

// NT: n-tiles of 8 ranks per pass. From 17 ranks on one CTA to an SM: its loads and
// sums want more than 128 registers. With two, and 64 ranks in two passes over x,
// K = 7168, N = 4096, T = 16 took 19.8 us where this takes 13.9, T = 128 26.8 and
// 21.1, T = 512 57.1 and 35.5, T = 8192 314 and 298 (of MXFP8 rows 331 and 307); of 32
// ranks (K = 4096, N = 2048) T = 64 12.2 either way, 15.2 and 13.9 of MXFP8 rows, T = 512
// 22.8 and 20.1, T = 8192 99.7 and 104, the one size that it loses. Eight ranks have one
// n-tile: K = 2048, N = 1024, MXFP8, T = 16 6.2 us, with two (half of them unused) 6.8;
// K = 2880, N = 5760, T = 64 13.9 and 14.6; nothing at T = 8192 (all in graphs).
template <int NT, bool X8>
__global__ void __launch_bounds__(256, NT <= 2 ? 2 : 1)
    adapter_down_kernel(const LinearArgs a, uint16_t* __restrict__ xb /* null: not converted */,
                        float* __restrict__ v) {
  __shared__ int s_cid[kDownWin / 32][32], s_cn[kDownWin / 32][32], s_nc[kDownWin / 32];
  __shared__ int s_base[kDownWin], s_warp[kDownWin / 32], s_items;
  __shared__ int s_tok[kDownWin][kDownTok];   // [item][slot]: token of the window, -1 empty
  __shared__ int s_ad[kDownWin];              // [item]: adapter, -1 none
  constexpr int NP = NT < 4 ? NT : 4;         // n-tiles that the warps add at once
  __shared__ float part[8][16][NP * 8 + 4];
  __shared__ __align__(16) float s_sum[kDownTok][kDownSum];   // this CTA's part of an item
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int w0 = blockIdx.x * kDownWin;
  const int parts = gridDim.z;
  grid_launch_dependents();

  // group the window's tokens by adapter: id -1 (no adapter) is a class of its
  // own where rows are converted; -2 stays out
  const int kNone = X8 && xb != nullptr ? -1 : -2;
  int id = -2;
  if (tid < kDownWin) {
    if (w0 + tid < a.T) {
      id = a.ids[w0 + tid];
      if (id >= a.L) {
        if (a.status != nullptr && blockIdx.y == 0 && blockIdx.z == 0) atomicAdd(a.status, 1);
        id = kNone;
      }
      if (id < 0) id = kNone;
    }
    // the warp's classes: id and count, listed by their first lanes
    const uint32_t same = __match_any_sync(0xffffffffu, id);
    const int first = __ffs(same) - 1;
    const bool lead = lane == first && id > -2;
    const uint32_t leads = __ballot_sync(0xffffffffu, lead);
    const int slot = __popc(leads & lanemask_lt());
    if (lead) {
      s_cid[warp][slot] = id;
      s_cn[warp][slot] = __popc(same);
    }
    if (lane == 0) s_nc[warp] = __popc(leads);
    named_barrier(1, kDownWin);
    // a class's first warp lists its items; other warps find it there
    int before = 0, after = 0, root = warp * 32 + slot;
    if (lead) {
      for (int w = kDownWin / 32 - 1; w >= 0; --w)
        for (int j = 0; j < s_nc[w]; ++j)
          if (w != warp && s_cid[w][j] == id) {
            if (w < warp) {
              before += s_cn[w][j];
              root = w * 32 + j;   // descending: the lowest warp stays
            } else {
              after += s_cn[w][j];
            }
          }
    }
    const int mine =
        lead && before == 0 ? (__popc(same) + after + kDownTok - 1) / kDownTok : 0;
    int sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    if (lane == 31) s_warp[warp] = sum;
    named_barrier(1, kDownWin);
    int base = sum - mine, all = 0;
    for (int w = 0; w < kDownWin / 32; ++w) {
      if (w < warp) base += s_warp[w];
      all += s_warp[w];
    }
    if (mine > 0) {
      s_base[root] = base;
      for (int j = 0; j < mine; ++j) s_ad[base + j] = id;
    }
    if (tid == 0) s_items = all;
    for (int i = tid; i < all * kDownTok; i += kDownWin) s_tok[i / kDownTok][i % kDownTok] = -1;
    named_barrier(1, kDownWin);
    const int rank = __shfl_sync(0xffffffffu, before, first) + __popc(same & lanemask_lt());
    const int at = __shfl_sync(0xffffffffu, lead ? s_base[root] : 0, first);
    if (id > -2) s_tok[at + rank / kDownTok][rank % kDownTok] = tid;
  }
  __syncthreads();
  const int items = s_items;

  const int g = lane >> 2, q = lane & 3;
  const int slices = 8 * parts, slice = blockIdx.z * 8 + warp;
  const int steps = a.K / kDownStep;
  const int k0 = steps * slice / slices, k1 = steps * (slice + 1) / slices;
  for (int it = blockIdx.y; it < items; it += gridDim.y) {
    const int ad = s_ad[it];
    const bool two = s_tok[it][16] >= 0;   // a second m-tile
    int tk[4];
    size_t xo[4];                          // value offsets of this lane's rows
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      tk[i] = s_tok[it][g + 8 * i];
      xo[i] = (size_t)(w0 + max(tk[i], 0)) * a.K + 16 * q;
    }
    const int passes = ad < 0 ? 1 : (a.rank + NT * 8 - 1) / (NT * 8);
    for (int pass = 0; pass < passes; ++pass) {
      const int r0 = pass * NT * 8;
      const int nt = ad < 0 ? 0 : min(NT, (a.rank - r0) / 8);
      const uint16_t* ar = a.a + ((size_t)max(ad, 0) * a.rank + r0 + g) * a.K + 16 * q;
      float acc[2][NT][4] = {};
      // each lane holds 16 consecutive values of its rows; both operands take
      // them in the same order, so the products are those of row order
#pragma unroll NT <= 4 ? 2 : 1
      for (int k = k0; k < k1; ++k) {
        uint4 u[4][2], w[NT][2], e[4];
        uint32_t sc[4];
        if (ad >= 0) {
#pragma unroll
          for (int j = 0; j < NT; ++j)   // (past the rank: the last rows again, never stored)
            ldg32(ar + (size_t)(8 * (j < nt ? j : nt - 1)) * a.K + kDownStep * k, w[j][0], w[j][1]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          u[i][0] = u[i][1] = e[i] = make_uint4(0u, 0u, 0u, 0u);
          sc[i] = 0;
          if (tk[i] < 0) continue;
          if (X8) {
            e[i] = ldg16(static_cast<const uint8_t*>(a.x) + xo[i] + kDownStep * k);
            sc[i] = ldg_u8(a.xs + (xo[i] + kDownStep * k) / kScaleBlock);
          } else {
            ldg32(static_cast<const uint16_t*>(a.x) + xo[i] + kDownStep * k, u[i][0], u[i][1]);
          }
        }
        if (X8) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (tk[i] < 0) continue;
            e4m3x16_to_bf16(e[i], sc[i], u[i][0], u[i][1]);
            if (xb != nullptr && pass == 0)
              stg32(xb + xo[i] + kDownStep * k, pair_order(u[i][0]), pair_order(u[i][1]));
          }
        }
        if (ad < 0) continue;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          if (m == 1 && !two) break;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              const uint4 ua = u[2 * m][h], ub = u[2 * m + 1][h];
              mma_bf16_16816(acc[m][j], ua.x, ub.x, ua.y, ub.y, w[j][h].x, w[j][h].y);
              mma_bf16_16816(acc[m][j], ua.z, ub.z, ua.w, ub.w, w[j][h].z, w[j][h].w);
            }
        }
      }
      if (ad < 0) break;
      const float scale = a.ascale != nullptr ? a.ascale[ad] : 1.f;
#pragma unroll
      for (int mj = 0; mj < 2 * NT / NP; ++mj) {
        const int m = mj / (NT / NP), j0 = mj % (NT / NP) * NP;
        if (m == 1 && !two) break;
        if (j0 >= nt) continue;
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          float* dst = &part[warp][g][8 * j + 2 * q];
          dst[0] = acc[m][j0 + j][0];
          dst[1] = acc[m][j0 + j][1];
          dst[8 * (NP * 8 + 4)] = acc[m][j0 + j][2];
          dst[8 * (NP * 8 + 4) + 1] = acc[m][j0 + j][3];
        }
        __syncthreads();
        const int n = 8 * min(NP, nt - j0), f = r0 + 8 * j0;
        for (int i = tid; i < 16 * n; i += 256) {
          const int row = i / n, r = i - row * n;
          const int t = s_tok[it][16 * m + row];
          float z = 0.f;
#pragma unroll
          for (int w = 0; w < 8; ++w) z += part[w][row][r];
          if (parts > 1)
            s_sum[16 * m + row][f % kDownSum + r] = z;
          else if (t >= 0)
            v[(size_t)(w0 + t) * a.rank + f + r] = two_bf16(z * scale);
        }
        __syncthreads();
      }
      const int f0 = r0 / kDownSum * kDownSum;   // ranks f0 .. r0 + 8 nt - 1 are complete here
      if (parts > 1 && (r0 + NT * 8 - f0 == kDownSum || pass == passes - 1)) {
        // tokens rank, rank + parts, .. of the item: the cluster's parts in order
        cluster_sync();
        const int quads = (r0 + 8 * nt - f0) / 4;
        const int rows = two ? 32 : 16, me = (int)cluster_rank();
        for (int i = tid; i < rows / parts * quads; i += 256) {
          const int row = i / quads * parts + me, r = i % quads * 4;
          const int t = s_tok[it][row];
          if (t < 0) continue;
          float4 z[kDownMaxParts];
#pragma unroll
          for (int c = 0; c < kDownMaxParts; ++c)
            if (c < parts) z[c] = ld_cluster16(smem_u32(&s_sum[row][r]), c);
          float4 y = z[0];
#pragma unroll
          for (int c = 1; c < kDownMaxParts; ++c)
            if (c < parts) {
              y.x += z[c].x;
              y.y += z[c].y;
              y.z += z[c].z;
              y.w += z[c].w;
            }
          *reinterpret_cast<float4*>(v + (size_t)(w0 + t) * a.rank + f0 + r) =
              make_float4(two_bf16(y.x * scale), two_bf16(y.y * scale), two_bf16(y.z * scale),
                          two_bf16(y.w * scale));
        }
        cluster_sync();   // s_sum is read by the whole cluster until here
      }
    }
  }
}

// ---------------------------------------------------------------------------
// The projection
// ---------------------------------------------------------------------------
constexpr int kThreads = 768;
constexpr int kBM = 128;              // weight rows per CTA (half of the pair's MMA M)
constexpr int kBK = 64;               // K values of a 128-byte swizzled row
constexpr int kStageK = 2 * kBK;      // K values per stage
constexpr int kMaxTok = 256;          // tokens per tile (MMA N)
constexpr int kBTile = kBM * 128;     // adapter columns of operand A: 128 rows x 64 bf16
constexpr int kPStage = kBM * kStageK / 2;       // packed bytes of a stage
constexpr int kMaxS = 8, kMaxSP = 8, kMaxL = 4;  // ring depths
constexpr int kWCols = kStageK / 2;   // tensor-memory columns of a stage's weights
constexpr int kTmemCols = 512;
constexpr int kWarpX = 0, kWarpMma = 1, kWarpW = 2, kWarpEpi = 4, kWarpDeq = 12, kWarps = kThreads / 32;
constexpr int kEpiWarps = kWarpDeq - kWarpEpi, kEpiThreads = kEpiWarps * 32;
constexpr int kDeqGroups = (kWarps - kWarpDeq) / 4;
constexpr int kEpiBar = 1;            // named barrier of the adapter and epilogue warps
constexpr int kOutPitch = kBM * 2 + 16;   // bytes of a staged output row (128 bf16 and a bank shift)
constexpr int kListMax = kMaxTok;     // adapters that one tile can name
constexpr int kDynSmem = 227 * 1024 - 4096;   // dynamic shared memory of a CTA, one per SM (the rest is static)
constexpr int kMaxSplit = 4;          // pairs of a cluster that share a tile's K

struct LinearParams {
  CUtensorMap tmapX;   // x as bytes {128, T, K / 64}, box {128, cs / 2, 2}, 128-byte swizzle
  CUtensorMap tmapW;   // packed weights u8 [N][K/2], box {64, 128}, 64-byte swizzle
  LinearArgs a;
  const float* v;      // [T][rank]: scale_a A_a x_t, from the kernel before
  int cs;              // tokens per tile (multiple of 16, at most 256)
  int S, SP, SL;       // ring depths: operand stages, packed weights, adapter columns
  int split;           // pairs of a cluster that share a tile's K
  int rp;              // rank rounded up to 16
  int tiles;           // (pair of weight blocks, token tile)
};

// Whether a bf16 of the pair is not finite.
__device__ __forceinline__ bool nonfinite_bf16x2(uint32_t w) {
  return ((w & 0x7F80u) == 0x7F80u) || ((w & 0x7F800000u) == 0x7F800000u);
}
__device__ __forceinline__ uint32_t ldg_u16(const uint8_t* p) {
  uint16_t v;
  asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ void tmem_st16_nowait(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// PAIR: x's rows come in pair order from the kernel before this one (MXFP8);
// otherwise they are the caller's, in row order.
template <bool PAIR>
__global__ void __launch_bounds__(kThreads, 1) linear_kernel(const __grid_constant__ LinearParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[kMaxS], empty[kMaxS], p_full[kMaxSP], p_empty[kMaxSP], l_full[kMaxL],
      l_empty[kMaxL], l_list, d_full, d_empty, drain;
  __shared__ uint32_t tmem_slot, s_bits[kLinearMaxAdapters / 32];
  __shared__ int s_list[kListMax], s_tokad[kMaxTok], s_count, s_anybad, s_fail, s_efail[2];
  __shared__ uint8_t s_bad[kListMax];
  static_assert(kEpiThreads == kMaxTok, "one thread per token of a tile");
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int hb = p.cs / 2;                           // tokens of the tile in this CTA
  const int xchunk = hb * 128, xstage = 2 * xchunk;
  const int lstage = kBTile + xstage;
  uint8_t* sX = smem;                                // [S][2 chunks][hb][128 bytes]
  uint8_t* sP = sX + p.S * xstage;                   // [SP][128 rows][64 bytes]
  uint8_t* sL = sP + p.SP * kPStage;                 // [SL] of {kBTile, 2 x hb x 128 bytes: v's hi and lo};
                                                     // then the output tile [cs][kOutPitch]

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t crank = cluster_rank();
  const int half = crank & 1, part = crank >> 1;     // CTA of the pair, K part of the tile
  const uint32_t lead = crank & ~1u;                 // rank of the pair's issuing CTA
  const uint16_t pair = (uint16_t)(3u << lead);
  const int N = p.a.N, K = p.a.K;
  const int npair = (N + 2 * kBM - 1) / (2 * kBM);
  const int cluster = blockIdx.x / (2 * p.split), clusters = gridDim.x / (2 * p.split);
  // a tile's first token, and this CTA's first weight row
  auto tile_t0 = [&](int tile) { return tile / npair * p.cs; };
  auto tile_n0 = [&](int tile) { return tile % npair * 2 * kBM + half * kBM; };
  const int nSall = (K + kStageK - 1) / kStageK;
  const int st0 = nSall * part / p.split;
  const int nS = nSall * (part + 1) / p.split - st0;
  const bool adapters = p.a.ids != nullptr;
  int fail = 0;

  // full and l_full of the issuing CTA count both CTAs' warps; one thread's
  // expect covers both CTAs' token copies
  if (warp == kWarpX) {
    if (lane < p.S) { mbar_init(&full[lane], 1 + 2 * 4); mbar_init(&empty[lane], 1); }
    if (lane < p.SL) { mbar_init(&l_full[lane], 2 * kEpiWarps); mbar_init(&l_empty[lane], 1); }
    if (lane == 8) mbar_init(&l_list, 1);
    if (lane == 9) mbar_init(&d_full, 1);
    if (lane == 10) mbar_init(&d_empty, 2 * kEpiWarps);
    if (lane == 11) mbar_init(&drain, 1);
    if (lane == 12) {
      prefetch_tensormap(&p.tmapX);
      s_fail = s_efail[0] = s_efail[1] = 0;
    }
    fence_barrier_init();
  }
  // the first packed weights need this CTA's barriers alone: under way before
  // the cluster has met (skip_copy: the failure test's call leaves the first one out)
  int wk = 0;   // stages of them issued
  if (warp == kWarpW) {
    if (lane < p.SP) { mbar_init(&p_full[lane], 1); mbar_init(&p_empty[lane], 4); }
    fence_barrier_init();
    fence_proxy_async_smem();
    __syncwarp();
    for (; wk < p.SP && wk < nS && cluster < p.tiles; ++wk) {
      if (elect_one() && !(wk == 0 && p.a.skip_copy == (int)blockIdx.x)) {
        mbar_arrive_expect_tx(&p_full[wk], kPStage);
        tma_load_2d(sP + wk * kPStage, &p.tmapW, (st0 + wk) * (kStageK / 2), tile_n0(cluster),
                    &p_full[wk]);
      }
      __syncwarp();
    }
  }
  if (warp == kWarpMma) tmem2_alloc(&tmem_slot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  cluster_sync_relaxed();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const uint32_t wcol0 = tmem + (uint32_t)((p.cs + 31) & ~31);   // operand-A ring

  if (warp == kWarpX) {
    // ------------------------------------------------------------ token copies
    int s = 0, k = 0;
    uint32_t ph = 0;
    if (PAIR) grid_dependency_wait();
    for (int tile = cluster; tile < p.tiles && !fail; tile += clusters) {
      const int row = tile_t0(tile) + half * hb;
      for (int i = 0; i < nS; ++i, ++k) {
        if (k >= p.S && !warp_wait_cluster(&empty[s], ph ^ 1u)) { fail = 1; break; }
        if (elect_one()) {
          if (half == 0) mbar_arrive_expect_tx(&full[s], 2 * xstage);
          tma2_load_3d(sX + s * xstage, &p.tmapX, 0, row, 2 * (st0 + i),
                       cluster_addr(&full[s], lead));
        }
        __syncwarp();
        if (++s == p.S) { s = 0; ph ^= 1u; }
      }
    }
  } else if (warp == kWarpW) {
    // ------------------------------------------------------------ packed-weight copies
    int s = wk == p.SP ? 0 : wk, k = wk, first = wk;
    uint32_t ph = wk == p.SP ? 1 : 0;
    for (int tile = cluster; tile < p.tiles && !fail; tile += clusters) {
      const int n0 = tile_n0(tile);
      for (int i = first; i < nS; ++i, ++k) {
        if (k >= p.SP && !warp_wait_cta(&p_empty[s], ph ^ 1u)) { fail = 1; break; }
        if (elect_one()) {
          mbar_arrive_expect_tx(&p_full[s], kPStage);
          tma_load_2d(sP + s * kPStage, &p.tmapW, (st0 + i) * (kStageK / 2), n0, &p_full[s]);
        }
        __syncwarp();
        if (++s == p.SP) { s = 0; ph ^= 1u; }
      }
      first = 0;
    }
  } else if (warp == kWarpMma) {
    // ------------------------------------------------------------ MMA issue
    if (half == 0) {
      const uint64_t desc0 = umma_desc_sw128(smem_u32(sX));
      const uint32_t idesc = umma_idesc_bf16(2 * kBM, p.cs);
      int s = 0, ls = 0, it = 0;
      uint32_t ph = 0, lph = 0;
      for (int tile = cluster; tile < p.tiles && !fail; tile += clusters, ++it) {
        // the epilogues of both CTAs have read the tile before
        if (it > 0 && !warp_wait_cluster(&d_empty, (it - 1) & 1)) { fail = 1; break; }
        for (int i = 0; i < nS; ++i) {
          if (!warp_wait_cluster(&full[s], ph)) { fail = 1; break; }
          tc_fence_after();
          if (elect_one()) {
            const uint64_t d = desc0 + (uint64_t)(s * (xstage >> 4));
            const uint32_t a = wcol0 + s * kWCols;
            umma2_bf16_ts(tmem, a, d, idesc, i > 0);
            umma2_bf16_ts(tmem, a + 8, d + 2, idesc, true);
            umma2_bf16_ts(tmem, a + 16, d + 4, idesc, true);
            umma2_bf16_ts(tmem, a + 24, d + 6, idesc, true);
            if ((st0 + i) * kStageK + kBK < K) {   // K may end inside the stage
              const uint64_t e = d + (uint64_t)(xchunk >> 4);
              umma2_bf16_ts(tmem, a + 32, e, idesc, true);
              umma2_bf16_ts(tmem, a + 40, e + 2, idesc, true);
              umma2_bf16_ts(tmem, a + 48, e + 4, idesc, true);
              umma2_bf16_ts(tmem, a + 56, e + 6, idesc, true);
            }
            umma2_commit(&empty[s], pair);
          }
          __syncwarp();
          if (++s == p.S) { s = 0; ph ^= 1u; }
        }
        if (adapters && !fail) {
          if (!warp_wait_cta(&l_list, it & 1)) { fail = 1; break; }
          const int lcols = s_count * p.rp;
          for (int i = part; i * kBK < lcols; i += p.split) {
            if (!warp_wait_cluster(&l_full[ls], lph)) { fail = 1; break; }
            tc_fence_after();
            if (elect_one()) {
              const uint64_t da = umma_desc_sw128(smem_u32(sL + ls * lstage));
              const uint64_t db = umma_desc_sw128(smem_u32(sL + ls * lstage + kBTile));
              const uint64_t dl = db + (uint64_t)(xchunk >> 4);   // v's lo
              const int k16n = min(kBK, lcols - i * kBK) / 16;
              for (int k16 = 0; k16 < k16n; ++k16) {   // nS > 0 came before
                umma2_bf16_ss(tmem, da + 2 * k16, db + 2 * k16, idesc, true);
                umma2_bf16_ss(tmem, da + 2 * k16, dl + 2 * k16, idesc, true);
              }
              umma2_commit(&l_empty[ls], pair);
            }
            __syncwarp();
            if (++ls == p.SL) { ls = 0; lph ^= 1u; }
          }
        }
        if (elect_one() && !fail) umma2_commit(&d_full, pair);
        __syncwarp();
      }
      if (elect_one()) umma2_commit(&drain, pair);
      __syncwarp();
    }
  } else if (warp >= kWarpDeq) {
    // ------------------------------------------------------------ dequantisation
    // A group of four warps takes a whole stage; a thread holds one weight row
    // (TMEM lane), its 64 packed bytes of the stage from shared memory and its
    // four scale bytes straight from global memory, two of its stages early.
    // (The packed bytes too, straight into registers, cost 3000 clocks a stage:
    // 32 rows a warp load are 32 requests each.)
    const int dg = (warp - kWarpDeq) >> 2;   // group: stages dg, dg + kDeqGroups, .. of all tiles
    const int m = (warp & 3) * 32 + lane;
    const uint32_t wlane = wcol0 + ((uint32_t)((warp & 3) * 32) << 16);
    const bool words = K % kStageK == 0;     // a stage's four scale bytes are one aligned word
    int s = dg, sp = dg, k = dg;
    uint32_t ph = 0, pp = 0;
    if (s >= p.S) { s -= p.S; ph = 1; }
    if (sp >= p.SP) { sp -= p.SP; pp = 1; }
    int i0 = dg;   // this group's first stage of the tile
    for (int tile = cluster; tile < p.tiles && !fail; tile += clusters) {
      const uint8_t* srow = p.a.s + (size_t)min(tile_n0(tile) + m, N - 1) * (K / kScaleBlock) +
                            st0 * (kStageK / kScaleBlock);   // rows past N: the last row, never stored
      auto scales = [&](int i) -> uint32_t {
        if (i >= nS) return 0u;
        if (words) return __ldg(reinterpret_cast<const uint32_t*>(srow + 4 * i));
        uint32_t v = ldg_u16(srow + 4 * i);
        if ((st0 + i) * kStageK + kBK < K) v |= ldg_u16(srow + 4 * i + 2) << 16;
        return v;
      };
      int i = i0;
      uint32_t sc = scales(i), sc1 = scales(i + kDeqGroups);
#pragma unroll 1
      for (; i < nS; i += kDeqGroups) {
        // A wait by parity tells a phase from the one before it, not from the one
        // before that, so nobody may wait a whole round of a ring ahead. Order
        // and depths see to it: the MMAs that read this operand slot (stage k - S)
        // have completed, and by their order all stages before, so S >= the groups
        // keeps `empty` in step; the packed slot's fill before this one (stage
        // k - SP) has then been used too where SP >= S, and was this group's own
        // where SP is the number of groups.
        if (k >= p.S) {
          if (!warp_wait_cluster(&empty[s], ph ^ 1u)) { fail = 1; break; }
          tc_fence_after();
        }
        if (!warp_wait_cta(&p_full[sp], pp)) { fail = 1; break; }
        const uint8_t* src = sP + sp * kPStage + m * 64;
        const int swz = (m >> 1) & 3;
        const int blocks = (st0 + i) * kStageK + kBK < K ? 4 : 2;   // K may end inside the stage
        const uint32_t dst = wlane + s * kWCols;
        uint4 w = *reinterpret_cast<const uint4*>(src + (swz << 4));
        // one block's code, run four times: unrolled, the groups' loops outgrew
        // the instruction cache
#pragma unroll 1
        for (int z = 0; z < blocks; ++z) {
          const uint32_t wd[4] = {w.x, w.y, w.z, w.w};
          w = *reinterpret_cast<const uint4*>(src + ((((z + 1) & 3) ^ swz) << 4));
          uint32_t o[16];
          if (PAIR)
            dequant32_bf16_pairs(wd, scale_mul((sc >> (8 * z)) & 255u), o);
          else
            dequant32_bf16(wd, scale_mul((sc >> (8 * z)) & 255u), o);
          tmem_st16_nowait(dst + 16 * z, o);
        }
        // the generic reads above are ordered before the stage's refill by a tensor copy
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_empty[sp]);
        sc = sc1;
        sc1 = scales(i + 2 * kDeqGroups);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(cluster_addr(&full[s], lead));
        k += kDeqGroups;
        s += kDeqGroups;
        while (s >= p.S) { s -= p.S; ph ^= 1u; }
        sp += kDeqGroups;
        while (sp >= p.SP) { sp -= p.SP; pp ^= 1u; }
      }
      i0 = i - nS;
    }
  } else if (warp >= kWarpEpi) {
    const int et = threadIdx.x - kWarpEpi * 32;
    bool waited = false;
    int ls = 0, use = 0, it = 0;
    uint32_t lph = 0;
    for (int tile = cluster; tile < p.tiles && !fail; tile += clusters, ++it) {
      const int t0 = tile_t0(tile), n0 = tile_n0(tile);
      const int n = min(p.cs, p.a.T - t0);   // tokens of this tile
      if (adapters) {
        // ---------------------------------------------------------- adapter columns
        // the adapters that the tile's tokens name, in ascending order
        if (et < kLinearMaxAdapters / 32) s_bits[et] = 0;
        if (et == 0) s_anybad = 0;
        named_barrier(kEpiBar, kEpiThreads);
        {
          int id = et < n ? p.a.ids[t0 + et] : -1;
          if (id >= p.a.L) id = -1;
          s_tokad[et] = id;
          s_bad[et] = 0;
          if (id >= 0) atomicOr(&s_bits[id >> 5], 1u << (id & 31));
        }
        named_barrier(kEpiBar, kEpiThreads);
        if (warp == kWarpEpi) {
          uint32_t bits = s_bits[lane];
          int x = __popc(bits);
          const int mine = x;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
          }
          int at = x - mine;
          while (bits) {
            s_list[at++] = lane * 32 + __ffs(bits) - 1;
            bits &= bits - 1;
          }
          if (lane == 31) s_count = x;
        }
        named_barrier(kEpiBar, kEpiThreads);
        if (et == 0) mbar_arrive(&l_list);
        const int count = s_count, lcols = count * p.rp;
        // stages of 64 columns, taken in turn by the pairs of the cluster
        for (int i = part; i * kBK < lcols; i += p.split, ++use) {
          uint8_t* tb = sL + ls * lstage;
          uint8_t* tv = tb + kBTile;
          // 16-byte chunk j of a row: columns 64 i + 8 j .., one adapter's ranks r ..
          const int j = et & 7;
          const int c = i * kBK + 8 * j;
          const int ai = c / p.rp, r = c - ai * p.rp;
          const bool live = ai < count && r < p.a.rank;
          const int ad = live ? s_list[ai] : -1;
          constexpr int kPer = kBM * 8 / kEpiThreads;
          uint4 b[kPer];   // in flight together
#pragma unroll
          for (int u = 0; u < kPer; ++u) {
            const int row = (et >> 3) + kEpiThreads / 8 * u;
            b[u] = make_uint4(0u, 0u, 0u, 0u);
            if (live && n0 + row < N)
              b[u] = *reinterpret_cast<const uint4*>(p.a.b + ((size_t)ad * N + n0 + row) * p.a.rank + r);
          }
          // (their way from memory is beside the MMAs that free the slot)
          if (use >= p.SL && !warp_wait_cluster(&l_empty[ls], lph ^ 1u)) { fail = 1; break; }
#pragma unroll
          for (int u = 0; u < kPer; ++u) {
            const int row = (et >> 3) + kEpiThreads / 8 * u;
            uint32_t q[4] = {b[u].x, b[u].y, b[u].z, b[u].w};
            if (nonfinite_bf16x2(q[0]) || nonfinite_bf16x2(q[1]) || nonfinite_bf16x2(q[2]) ||
                nonfinite_bf16x2(q[3])) {
              s_bad[ai] = 1;
              s_anybad = 1;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if ((q[e] & 0x7F80u) == 0x7F80u) q[e] &= 0xFFFF0000u;
                if ((q[e] & 0x7F800000u) == 0x7F800000u) q[e] &= 0xFFFFu;
              }
            }
            *reinterpret_cast<uint4*>(tb + row * 128 + ((j ^ (row & 7)) << 4)) =
                make_uint4(q[0], q[1], q[2], q[3]);
          }
          if (!waited) {   // v comes from the kernel before this one
            grid_dependency_wait();
            waited = true;
          }
          for (int t = et >> 3; t < hb; t += kEpiThreads / 8) {
            uint4 hi = make_uint4(0u, 0u, 0u, 0u), lo = hi;
            if (live && s_tokad[half * hb + t] == ad) {
              const float* src = p.v + (size_t)(t0 + half * hb + t) * p.a.rank + r;
              const float4 x = ldcg_f4(src), y = ldcg_f4(src + 4);
              split_bf16x2(x.x, x.y, hi.x, lo.x);
              split_bf16x2(x.z, x.w, hi.y, lo.y);
              split_bf16x2(y.x, y.y, hi.z, lo.z);
              split_bf16x2(y.z, y.w, hi.w, lo.w);
            }
            uint8_t* dst = tv + t * 128 + ((j ^ (t & 7)) << 4);
            *reinterpret_cast<uint4*>(dst) = hi;
            *reinterpret_cast<uint4*>(dst + xchunk) = lo;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(cluster_addr(&l_full[ls], lead));
          if (++ls == p.SL) { ls = 0; lph ^= 1u; }
        }
        if (!waited) {
          grid_dependency_wait();
          waited = true;
        }
        named_barrier(kEpiBar, kEpiThreads);   // s_bad and s_anybad are complete
      }
      // ------------------------------------------------------------ epilogue
      // accumulators -> a shared-memory tile [token][128 rows]: bf16, or, where K
      // is split over the cluster, fp32 in the token ring (free by then)
      if (!warp_wait_cluster(&d_full, it & 1)) fail = 1;
      tc_fence_after();
      const int q = warp & 3;                 // TMEM lane quarter
      const int row = n0 + q * 32 + lane;
      const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16);
      float* red = reinterpret_cast<float*>(sX);
      const bool fix = adapters && s_anybad != 0;
#pragma unroll 1
      for (int c0 = (et >> 7) * 32; c0 < n && !fail; c0 += kEpiThreads / 128 * 32) {
        float v[32];
        tmem_ld32(taddr + c0, v);
        if (__builtin_expect(fix, 0) && row < N) {
          for (int t = 0; t < 32 && c0 + t < n; ++t) {
            const int ad = s_tokad[c0 + t];
            int ai = 0;
            while (ai < s_count && s_list[ai] != ad) ++ai;
            if (ad < 0 || !s_bad[ai]) continue;
            float z = 0.f;
            for (int r = 0; r < p.a.rank; ++r) {
              const uint32_t bw = p.a.b[((size_t)ad * N + row) * p.a.rank + r];
              if ((bw & 0x7F80u) == 0x7F80u)
                z += __uint_as_float(bw << 16) * p.v[(size_t)(t0 + c0 + t) * p.a.rank + r];
            }
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (e == t) v[e] += z;
          }
        }
        const int nv = min(32, n - c0);
        if (p.split > 1) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (e < nv) red[(c0 + e) * kBM + q * 32 + lane] = v[e];
        } else {
          uint8_t* dst = sL + c0 * kOutPitch + (q * 32 + lane) * 2;
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (e < nv) *reinterpret_cast<uint16_t*>(dst + e * kOutPitch) = f32_to_bf16_rne(v[e]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(cluster_addr(&d_empty, lead));
      if (p.split == 1) {
        // whole 256-byte rows to global memory, while the next tile's MMAs run
        named_barrier(kEpiBar, kEpiThreads);
        const int col = n0 + (et & 15) * 8;
        if (col < N && !fail)
          for (int t = et >> 4; t < n; t += kEpiThreads / 16)
            *reinterpret_cast<uint4*>(p.a.out + (size_t)(t0 + t) * N + col) =
                *reinterpret_cast<const uint4*>(sL + t * kOutPitch + (et & 15) * 16);
        // the next tile's adapter columns go there; these warps go on or leave together
        if (fail) s_efail[it & 1] = 1;
        named_barrier(kEpiBar, kEpiThreads);
        if (s_efail[it & 1]) fail = 1;
      }
    }
  }
  __syncwarp();
  auto report = [&] {
    if (p.a.status == nullptr) return;
    if (adapters || PAIR) grid_dependency_wait();   // the status words belong to that kernel until then
    atomicOr(&p.a.status[2], 1);
    atomicCAS(&p.a.status[3], 0, blockIdx.x + 1);
  };
  if (fail) {
    s_fail = 1;
    report();
  }
  tc_fence_before();
  __syncthreads();
  // after a wait that gave up, copies may still be on their way to this CTA's
  // shared memory: they land within microseconds, a millisecond is waited
  if (s_fail)
    for (int i = 0; i < 1000; ++i) __nanosleep(1000);
  cluster_sync();
  tc_fence_after();
  if (warp == kWarpMma) {
    // no MMA may still read the pair's memory when it is released: all have been
    // issued by now, and this wait's bound covers their end alone (it began with the
    // kernel for the warps without a role, which reported a call of more than 0.19 s)
    if (!warp_wait_cluster(&drain, 0)) report();
    __syncwarp();
    tmem2_dealloc(tmem, kTmemCols);
  }
  if (p.split > 1) {
    // y of tokens part, part + split, ..: the pairs' partial sums in rank order
    const uint32_t red = smem_u32(sX);
    const int t0 = tile_t0(cluster), n0 = tile_n0(cluster);   // one tile per cluster
    const int n = min(p.cs, p.a.T - t0);
    for (int t = part + p.split * warp; t < n; t += p.split * kWarps) {
      float4 z[kMaxSplit];   // all in flight before the first is used
#pragma unroll
      for (int c = 0; c < kMaxSplit; ++c)
        if (c < p.split) z[c] = ld_cluster16(red + (t * kBM + lane * 4) * 4, 2 * c + half);
      float4 y = z[0];
#pragma unroll
      for (int c = 1; c < kMaxSplit; ++c)
        if (c < p.split) {
          y.x += z[c].x;
          y.y += z[c].y;
          y.z += z[c].z;
          y.w += z[c].w;
        }
      if (n0 + lane * 4 < N)
        *reinterpret_cast<uint2*>(p.a.out + (size_t)(t0 + t) * N + n0 + lane * 4) =
            make_uint2(bf16x2_rn(y.x, y.y), bf16x2_rn(y.z, y.w));
    }
    cluster_sync();   // no CTA leaves while another reads its shared memory
  }
}

// ---------------------------------------------------------------------------
// The projection for few tokens
// ---------------------------------------------------------------------------
// Up to 16 tokens the packed weights are all there is to move, and the tile
// kernel's start, its stages one after another and its cluster-wide sums were
// most of the time (T = 1, K = 6144, N = 4096, rank 16, in a graph: 14.3 us, here
// 7.5; T = 16: 17 and 10.9). At 32 tokens, which no longer stay in registers over
// a step, this form took 16 to 45 us where the tiles take 15 to 19.
//
// A CTA takes 32 weight rows, its warps the K values in steps of 128 (4 scale
// blocks, one per lane of a quad): a lane loads 32 consecutive values of four
// rows and of its tokens, the weights two steps early, and the bf16 products run
// on m16n8k16 tiles straight from registers -- the order of K in them is free as
// long as both operands take the same, so pair order costs nothing. The warps' sums meet in shared memory in order; the epilogue adds the
// adapter's second product from its 32 rows of B_a.
constexpr int kFewTok = 16;
constexpr int kFewRows = 32;

struct FewStep {
  uint4 w[4];        // rows g, g + 8, g + 16, g + 24
  uint32_t sc[4];
};

// TT: token tiles of 8. WARPS: 16 where the CTAs do not outnumber the SMs, 8 (two
// CTAs to an SM) where they do.
template <int TT, bool X8, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 16 / WARPS)
    linear_few_kernel(const LinearArgs a, const float* __restrict__ v) {
  __shared__ float part[WARPS][kFewRows][8 * TT + 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, q = lane & 3;
  const int n0 = blockIdx.x * kFewRows;
  const int blocks = a.K / kScaleBlock, steps = (blocks + 3) / 4;
  const uint8_t* wr[4];
  const uint8_t* sr[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {   // rows past N: the last row again, never stored
    const size_t row = (size_t)min(n0 + g + 8 * i, a.N - 1);
    wr[i] = a.w + row * (a.K / 2);
    sr[i] = a.s + row * blocks;
  }
  auto fetch = [&](FewStep& d, int step) {
    const int b = 4 * step + q;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      d.w[i] = make_uint4(0u, 0u, 0u, 0u);   // past K: zeros
      d.sc[i] = 0;
      if (b < blocks) {
        d.w[i] = ldg16(wr[i] + (size_t)b * 16);
        d.sc[i] = ldg_u8(sr[i] + b);
      }
    }
  };
  float acc[2][TT][4] = {};
  FewStep buf[2];
  fetch(buf[0], warp);
  fetch(buf[1], warp + WARPS);
  for (int s0 = warp; s0 < steps; s0 += 2 * WARPS) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int step = s0 + h * WARPS;
      if (step >= steps) break;
      const int b = 4 * step + q;
      // this lane's 32 values of token 8 t + g, in pair order
      auto token = [&](int t, uint4 (&x)[4]) {
        const int tok = g + 8 * t;
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = make_uint4(0u, 0u, 0u, 0u);
        if (tok >= a.T || b >= blocks) return;
        const size_t at = (size_t)tok * a.K + (size_t)b * kScaleBlock;
        if (X8) {
          const uint8_t* src = static_cast<const uint8_t*>(a.x) + at;
          const uint4 e0 = ldg16(src), e1 = ldg16(src + 16);
          const uint32_t sc = ldg_u8(a.xs + (size_t)tok * blocks + b);
          e4m3x16_to_bf16(e0, sc, x[0], x[1]);
          e4m3x16_to_bf16(e1, sc, x[2], x[3]);
        } else {
          const uint16_t* src = static_cast<const uint16_t*>(a.x) + at;
          ldg32(src, x[0], x[1]);
          ldg32(src + 16, x[2], x[3]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = pair_order(x[j]);
      };
      uint4 x[TT][4];
#pragma unroll
      for (int t = 0; t < TT; ++t) token(t, x[t]);
      const FewStep& d = buf[h];
#pragma unroll
      for (int m = 0; m < 2; ++m) {   // rows 16 m + g and 16 m + g + 8
        uint32_t lo[16], hi[16];
        const uint4 wl = d.w[2 * m], wh = d.w[2 * m + 1];
        const uint32_t dl[4] = {wl.x, wl.y, wl.z, wl.w}, dh[4] = {wh.x, wh.y, wh.z, wh.w};
        dequant32_bf16_pairs(dl, scale_mul(d.sc[2 * m]), lo);
        dequant32_bf16_pairs(dh, scale_mul(d.sc[2 * m + 1]), hi);
#pragma unroll
        for (int t = 0; t < TT; ++t) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            mma_bf16_16816(acc[m][t], lo[4 * j], hi[4 * j], lo[4 * j + 1], hi[4 * j + 1], x[t][j].x,
                           x[t][j].y);
            mma_bf16_16816(acc[m][t], lo[4 * j + 2], hi[4 * j + 2], lo[4 * j + 3], hi[4 * j + 3],
                           x[t][j].z, x[t][j].w);
          }
        }
      }
      fetch(buf[h], step + 2 * WARPS);
    }
  }
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      part[warp][16 * m + g][8 * t + 2 * q] = acc[m][t][0];
      part[warp][16 * m + g][8 * t + 2 * q + 1] = acc[m][t][1];
      part[warp][16 * m + g + 8][8 * t + 2 * q] = acc[m][t][2];
      part[warp][16 * m + g + 8][8 * t + 2 * q + 1] = acc[m][t][3];
    }
  if (a.ids != nullptr) grid_dependency_wait();   // v comes from the kernel before this one
  __syncthreads();
  for (int i = tid; i < kFewRows * 8 * TT; i += WARPS * 32) {
    const int row = i % kFewRows, t = i / kFewRows, n = n0 + row;
    if (t >= a.T || n >= a.N) continue;
    float y = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) y += part[w][row][t];
    const int ad = a.ids != nullptr ? a.ids[t] : -1;
    if (ad >= 0 && ad < a.L) {
      const uint16_t* br = a.b + ((size_t)ad * a.N + n) * a.rank;
      const float* vr = v + (size_t)t * a.rank;
      float z = 0.f;
#pragma unroll 2
      for (int r = 0; r < a.rank; r += 8) {
        const uint4 bb = ldg16(br + r);
        const float4 v0 = ldcg_f4(vr + r), v1 = ldcg_f4(vr + r + 4);
        const uint32_t bw[4] = {bb.x, bb.y, bb.z, bb.w};
        const float vw[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          z = fmaf(__uint_as_float(bw[j] << 16), vw[2 * j], z);
          z = fmaf(__uint_as_float(bw[j] & 0xFFFF0000u), vw[2 * j + 1], z);
        }
      }
      y += z;
    }
    a.out[(size_t)t * a.N + n] = f32_to_bf16_rne(y);
  }
}

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

}  // namespace

size_t linear_workspace_bytes(int T, int K, int N, int rank, bool x8) {
  (void)N;
  return up256((size_t)T * rank * sizeof(float)) + (x8 && T > kFewTok ? up256((size_t)T * K * 2) : 0);
}

// Grid of the adapters' first product: CTAs over windows, slots for their items
// (more items are taken in turns, CTAs past a window's items leave after grouping
// it) and parts of K, with its end in clocks.
struct DownPlan {
  int parts, slots;   // parts 0: none
  double end;
};
struct DownWork {
  int win = 0, most = 0;   // windows; the items of one, at most
  int items = 0;   // the same, as a rule: the adapters that its tokens draw, or runs of 32
  int total = 0;   // items in all: those of 32 tokens, and where runs end
  int parts = 0;   // at most: a step or two to a warp; 0: no adapters
  DownWork() = default;
  explicit DownWork(const LinearArgs& a) {   // (of a call with adapters)
    win = (a.T + kDownWin - 1) / kDownWin;
    most = a.T < kDownWin ? a.T : kDownWin;
    double none = 1;   // the share of the adapters that no token draws
    for (int t = 0; t < most; ++t) none *= 1 - 1.0 / a.L;
    items = (int)(a.L * (1 - none));
    if (items < 1) items = 1;
    if (win > 1 || items < most / kDownTok) items = most / kDownTok + 1;
    total = (a.T + kDownTok - 1) / kDownTok + (win < 3 ? 0 : win < a.L ? win : a.L);
    for (parts = 1; parts < kDownMaxParts && a.K / kDownStep >= 2 * 8 * parts;) parts *= 2;
  }
};
// Clocks until `turns` items after one another end: a warp's steps of each and, in
// parts, the cluster's sums.
static double down_end(const LinearArgs& a, int parts, int turns) {
  const int steps = (a.K / kDownStep + 8 * parts - 1) / (8 * parts);
  return 5000 + turns * ((parts > 1 ? 4500 : 2000) + steps * (a.rank <= 16 ? 700.0 : 1200.0));
}
// On all SMs: parts of K while their CTAs run at once (eight parts' sums only from
// 65 tokens on: T = 32, K = 6144, MXFP8 rows 17.5 us with four, 19.1 with eight).
// One or two windows are a decode batch, up to an item per token, more are prompts,
// whose runs make 4 to 8 items a window.
static DownPlan down_alone(const LinearArgs& a, const DownWork& w, int num_sms) {
  const int fit = a.rank <= 16 ? 2 * num_sms : num_sms;   // CTAs at once
  int parts = w.parts;
  while (parts > 1 && (w.total * parts > fit || (parts > 4 && w.total <= 2))) parts /= 2;
  const int slots = w.win <= 2 ? fit / (w.win * parts) : 8;
  return {parts, slots < w.most ? slots : w.most,
          down_end(a, parts, (w.total * parts + fit - 1) / fit)};
}
// Beside a projection that needs nothing but the sums, and these after `clocks`:
// in the `room` CTAs that leave it its SMs, if a grid of them has a slot for each
// of a window's items (or one for two, without parts) and ends in time. The most
// parts, or, for the tiles, the fewest that end well before (T = 64, K = 6144: one
// part 15.4 us, four 15.8). Both kernels then start together, and the projection's
// last steps find the sums ready. us in graphs, against all SMs always (N = 4096;
// 5760 at K = 2880):
//   K = 6144, rank 16: T =  8  8.2  (8.8), T = 64 15.2 (17.3), T = 1024 37.7 (42.6)
//   K = 2880, rank 16: T =  8  8.3  (8.5), T = 64 14.4 (16.7), T = 1024 32.3 (36.0)
//   K = 7168, rank 64: T = 16 13.9 (19.6), T = 32 17.3 (17.7), T =  512 35.5 (39.4)
static DownPlan down_beside(const LinearArgs& a, const DownWork& w, double clocks, int room) {
  const bool few = a.T <= kFewTok;
  DownPlan best = {0, 0, 0};
  for (int p = w.parts; p >= 1; p /= 2) {
    int slots = room / (w.win * p);
    const bool one = slots >= w.items, two = !few && p == 1 && 2 * slots >= w.items;
    if (!one && (!two || best.parts > 0)) continue;
    const double end = down_end(a, p, one ? 1 : 2);
    if (end > 1.25 * clocks || (best.parts > 0 && (few || end > 0.76 * clocks))) continue;
    if (one && w.win > 1) slots = 12;   // (a window of more runs than that)
    best = {p, slots < w.most ? slots : w.most, end};
  }
  return best;
}

template <int NT, bool X8>
static cudaError_t launch_down(const LinearArgs& a, uint16_t* xb, float* v, const DownPlan& plan,
                               cudaStream_t stream) {
  const int win = (a.T + kDownWin - 1) / kDownWin;
  const int parts = plan.parts, slots = plan.slots;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(win, slots, parts);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = parts;
  cfg.attrs = at;
  cfg.numAttrs = parts > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, adapter_down_kernel<NT, X8>, a, xb, v);
}

// Clusters of 2 * split CTAs that are resident at once (a cluster stays inside a
// group of SMs, and those groups are not multiples of every size): asked of the
// driver once per device, under a lock: a first call from another thread must not
// see some of them, which would choose it other tiles.
static cudaError_t resident_clusters(int dev, int (&out)[kMaxSplit + 1]) {
  struct Known {
    bool set;
    int n[kMaxSplit + 1];
  };
  static Known known[kGrantDevices] = {};
  static std::mutex mu;
  std::lock_guard<std::mutex> lk(mu);
  Known& d = known[dev];
  if (!d.set) {
    for (auto* k : {linear_kernel<false>, linear_kernel<true>}) {
      const cudaError_t e =
          cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kDynSmem);
      if (e != cudaSuccess) return e;
    }
    for (int sp = 1; sp <= kMaxSplit; ++sp) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(2 * sp * 64);
      cfg.blockDim = dim3(kThreads);
      cfg.dynamicSmemBytes = kDynSmem;
      cudaLaunchAttribute at[1];
      at[0].id = cudaLaunchAttributeClusterDimension;
      at[0].val.clusterDim.x = 2 * sp;
      at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
      cfg.attrs = at;
      cfg.numAttrs = 1;
      const cudaError_t e = cudaOccupancyMaxActiveClusters(&d.n[sp], linear_kernel<false>, &cfg);
      if (e != cudaSuccess) return e;
    }
    if (d.n[1] < 1) return cudaErrorInvalidConfiguration;
    d.set = true;
  }
  for (int sp = 1; sp <= kMaxSplit; ++sp) out[sp] = d.n[sp];
  return cudaSuccess;
}

// Tokens per tile and pairs per tile that a call takes, and the grid of the
// adapters' first product before it (`alone`: on all SMs): the
// smallest estimate of waves x (stages x clocks of a stage + clocks of a tile's
// start and end), and of that kernel before or beside it. A stage costs the larger
// of its dequantisation (measured in the running kernel: 750 clocks in row order,
// 680 in pair order; alone 470 and 346) and its eight MMAs (cs / 2 clocks each);
// the cluster's addition goes by the tile's tokens. Without adapters this choice
// was within 5% of the best of all sizes and splits tried by hand (6 shapes, T = 20
// to 4096), within 11% at N = 512.
static DownPlan linear_plan(const LinearArgs& a, bool pair_order, const DownWork& w,
                            const DownPlan& alone, const int (&resident)[kMaxSplit + 1],
                            int num_sms, int& cs, int& split) {
  const int npair = (a.N + 2 * kBM - 1) / (2 * kBM), nS = (a.K + kStageK - 1) / kStageK;
  const double deq = pair_order ? 680 : 750;
  DownPlan plan = alone;
  double best = 0;
  cs = 0;
  const int c0 = (a.T + kMaxTok - 1) / kMaxTok;
  for (int c = c0; c <= c0 + 8; ++c) {
    const int tok = ((a.T + c - 1) / c + 15) & ~15;
    const int64_t tiles = (int64_t)npair * ((a.T + tok - 1) / tok);
    for (int sp = 1; sp <= kMaxSplit; ++sp) {
      // split tiles take one pass; parts of at least two stages
      if (sp > 1 && (tiles > resident[sp] || nS < 2 * sp)) continue;
      const double stage = 4.0 * tok > deq ? 4.0 * tok : deq;
      const int64_t waves = (tiles + resident[sp] - 1) / resident[sp];
      const double clocks = 6000 + (double)waves * ((double)((nS + sp - 1) / sp) * stage + 2500);
      double t = clocks + alone.end;
      DownPlan d = alone;
      if (w.parts > 0 && !pair_order) {   // (pair order: it waits for the converted rows)
        // clusters that can start a tile late; of larger clusters what no cluster
        // fits into may lie next to them
        const int spare = (int)(waves * resident[sp] - tiles) * sp;
        const int rest = num_sms / 2 - resident[sp] * sp;
        const DownPlan b = down_beside(
            a, w, clocks, sp <= 2 ? 2 * (spare + rest) : spare > 0 ? spare + rest : (rest + 1) / 2);
        if (b.parts > 0) {
          d = b;
          t = clocks > b.end ? clocks : b.end;
        }
      }
      if (sp > 1) t += 500 + 25 * tok;
      if (cs == 0 || t < best) {
        best = t;
        plan = d;
        cs = tok;
        split = sp;
      }
    }
    if (tok <= 16) break;
  }
  return plan;
}

template <int TT, bool X8>
static cudaError_t launch_few(const LinearArgs& a, const float* v, bool wide, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.N + kFewRows - 1) / kFewRows);
  cfg.blockDim = dim3((wide ? 8 : 16) * 32);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = a.ids != nullptr ? 1 : 0;
  return wide ? cudaLaunchKernelEx(&cfg, linear_few_kernel<TT, X8, 8>, a, v)
              : cudaLaunchKernelEx(&cfg, linear_few_kernel<TT, X8, 16>, a, v);
}

cudaError_t launch_linear(const LinearArgs& a, int num_sms, cudaStream_t stream) {
  cudaError_t e;
  char* ws = static_cast<char*>(a.ws);
  const bool adapters = a.ids != nullptr;
  float* v = reinterpret_cast<float*>(ws);
  uint16_t* xb = reinterpret_cast<uint16_t*>(ws + up256((size_t)a.T * a.rank * sizeof(float)));
  const bool x8 = a.xs != nullptr, few = a.T <= kFewTok;
  if (few) xb = nullptr;
  if (a.status != nullptr &&
      (e = cudaMemsetAsync(a.status, 0, 4 * sizeof(int32_t), stream)) != cudaSuccess)
    return e;
  LinearParams p = {};
  const int few_ctas = (a.N + kFewRows - 1) / kFewRows;
  const bool wide = few_ctas > num_sms;
  int resident[kMaxSplit + 1];
  const DownWork w = adapters ? DownWork(a) : DownWork();
  DownPlan plan = adapters ? down_alone(a, w, num_sms) : DownPlan{0, 0, 0};
  if (!few) {
    int dev = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if (dev < 0 || dev >= kGrantDevices) return cudaErrorInvalidDevice;
    if ((e = resident_clusters(dev, resident)) != cudaSuccess) return e;
    plan = linear_plan(a, x8, w, plan, resident, num_sms, p.cs, p.split);
  } else if (adapters) {
    // 18500 clocks: both kernels, one after the other (this one waits for the sums
    // at its end; its CTAs of 8 warps leave half an SM)
    const int room = wide ? 2 * num_sms - few_ctas : num_sms - few_ctas;
    const DownPlan beside = down_beside(a, w, 18500, room);
    if (beside.parts > 0) plan = beside;
  }
  if (adapters) {
    if (a.rank <= 8)
      e = x8 ? launch_down<1, true>(a, xb, v, plan, stream)
             : launch_down<1, false>(a, xb, v, plan, stream);
    else if (a.rank <= 16)
      e = x8 ? launch_down<2, true>(a, xb, v, plan, stream)
             : launch_down<2, false>(a, xb, v, plan, stream);
    else if (a.rank <= 32)
      e = x8 ? launch_down<4, true>(a, xb, v, plan, stream)
             : launch_down<4, false>(a, xb, v, plan, stream);
    else
      e = x8 ? launch_down<8, true>(a, xb, v, plan, stream)
             : launch_down<8, false>(a, xb, v, plan, stream);
    if (e != cudaSuccess) return e;
  } else if (x8 && !few) {
    const int64_t n16 = (int64_t)a.T * a.K / 16;
    const int64_t blocks = (n16 + 255) / 256;
    mx8_to_bf16_kernel<<<(unsigned)(blocks < num_sms * 8 ? blocks : num_sms * 8), 256, 0, stream>>>(
        static_cast<const uint4*>(a.x), a.xs, n16, reinterpret_cast<uint4*>(xb));
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if (few) {
    if (a.T <= 8)
      return x8 ? launch_few<1, true>(a, v, wide, stream) : launch_few<1, false>(a, v, wide, stream);
    return x8 ? launch_few<2, true>(a, v, wide, stream) : launch_few<2, false>(a, v, wide, stream);
  }
  const void* x = x8 ? xb : a.x;

  p.a = a;
  p.v = v;
  const int xstage = p.cs / 2 * 256;
  p.S = (kTmemCols - ((p.cs + 31) & ~31)) / kWCols;   // 4 at 256 tokens, 7 at 16
  p.rp = (a.rank + 15) & ~15;
  const uint64_t dims[3] = {128, (uint64_t)a.T, (uint64_t)a.K / kBK};
  const uint64_t strides[2] = {(uint64_t)a.K * 2, 128};
  const uint32_t box[3] = {128, (uint32_t)p.cs / 2, 2};
  if (!encode_tiled_u8(&p.tmapX, x, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_tiled_2d(&p.tmapW, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w, (uint64_t)a.K / 2, (uint64_t)a.N,
                       (uint64_t)a.K / 2, kStageK / 2, kBM, CU_TENSOR_MAP_SWIZZLE_64B))
    return cudaErrorInvalidValue;
  p.tiles = (a.N + 2 * kBM - 1) / (2 * kBM) * ((a.T + p.cs - 1) / p.cs);
  // The adapter columns take the stages (4 up to 80 tokens, 1 at 256) that leave a
  // packed-weight ring as deep as the operands', or two with the shortest such ring:
  // with one, several adapters of a tile followed one another (K = 2880, N = 5760,
  // rank 16, 48 adapters, MXFP8: T = 1024 46.3 us, here 42.4). Packed weights take what
  // is left, 3 stages to 8.
  const size_t obytes = p.split == 1 ? (size_t)p.cs * kOutPitch : 0;
  size_t fixed = 0;
  for (p.SL = adapters ? kMaxL : 0;; --p.SL) {
    const size_t lbytes = (size_t)p.SL * (kBTile + xstage);
    fixed = 1024 + (size_t)p.S * xstage + (obytes > lbytes ? obytes : lbytes);
    p.SP = fixed < kDynSmem ? (int)((kDynSmem - fixed) / kPStage) : 0;
    if (p.SP >= p.S || p.SL <= 1 || (p.SL == 2 && p.SP >= kDeqGroups)) break;
  }
  if (p.SP > kMaxSP) p.SP = kMaxSP;
  if (p.SP < p.S) p.SP = kDeqGroups;   // (see the dequantising warps' waits)
  if (p.S < kDeqGroups || fixed + (size_t)p.SP * kPStage > kDynSmem) return cudaErrorInvalidConfiguration;
  const size_t smem = fixed + (size_t)p.SP * kPStage;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.tiles < resident[p.split] ? p.tiles : resident[p.split]) * p.split * 2));   // persistent
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  int na = 0;
  at[na].id = cudaLaunchAttributeClusterDimension;
  at[na].val.clusterDim.x = 2 * p.split;
  at[na].val.clusterDim.y = at[na].val.clusterDim.z = 1;
  ++na;
  if (adapters || x8) {   // starts beside the kernel before, whose results it waits for
    at[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[na].val.programmaticStreamSerializationAllowed = 1;
    ++na;
  }
  cfg.attrs = at;
  cfg.numAttrs = na;
  return cudaLaunchKernelEx(&cfg, x8 ? linear_kernel<true> : linear_kernel<false>, p);
}

}  // namespace mxmoe
