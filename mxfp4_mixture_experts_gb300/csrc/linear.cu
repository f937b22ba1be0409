// A shared projection from packed MXFP4 weights with the low-rank adapters of
// many requests beside it:
//   y_t = W x_t + scale_a * B_a (A_a x_t),  a = adapter of token t (or none)
// W = E2M1 * 2^(E8M0 - 127), [N, K]; A_a [rank, K] and B_a [N, rank] in bf16;
// x in bf16, or in MXFP8 (E4M3 with an E8M0 scale per 32 values). Sums in
// fp32, one rounding of y to bf16.
//
//   convert  (MXFP8 only) x as bf16 rows: exact but for products beyond bf16's range
//   down     v_t = bf16(scale_a * A_a x_t): the tokens of a window grouped by
//            adapter, 16 of one adapter to an m16n8k16 tile, K split over the
//            warps of a CTA
//   linear   the projection on the 5th-generation tensor cores, the second
//            adapter product as further columns of the same reduction
//
// The one rounding of v to bf16 (relative 2^-8 of the adapter's share of y,
// below the rounding of y itself) is what lets that product run on the same
// tensor-core accumulators.
//
// linear kernel: a tile is 128 weight rows x up to 256 tokens. The MMA computes
// D[weight row][token] with the dequantised weights as operand A in tensor
// memory and the tokens as operand B in shared memory. After the K values, the
// adapters that the tile's tokens name follow as columns: column c stands for
// (c / rp)-th adapter of the tile, rank index c % rp (rp = rank rounded up to
// 16); operand A holds B_a[n][r], operand B v_t[r] for the tokens of that
// adapter and 0 for the others. So tokens need no sorting, and a tile pays for
// the adapters it has. A B_a value that is not finite would turn the others'
// zeros into NaN; such values are left out of the tile and added in the
// epilogue to the tokens of their adapter alone.
//
// Warp roles: 0 token copies, 1 MMA issue, 2 packed-weight copies, 8..15
// dequantisation, 4..7 and 16..19 adapter columns, then the epilogue.
// Few tiles (small T) split K over a cluster of up to 8 CTAs, whose partial sums meet
// in shared memory, added in rank order.
#include <cuda.h>
#include <cstdint>

#include "kernels.h"
#include "ops.h"
#include "ops_common.cuh"

namespace mxmoe {
namespace {

// ---------------------------------------------------------------------------
// MXFP8 rows -> bf16 rows, 16 values a thread
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) mx8_to_bf16_kernel(const uint4* __restrict__ q,
                                                          const uint8_t* __restrict__ s, int64_t n16,
                                                          uint4* __restrict__ out) {
  for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < n16; i += (int64_t)gridDim.x * 256) {
    const uint4 u = q[i];
    const ScaleMul sm = e4m3_scale_mul(ldg_u8(s + (i >> 1)));
    uint4 a, b;
    e4m3x4_to_bf16(u.x, sm, a.x, a.y);
    e4m3x4_to_bf16(u.y, sm, a.z, a.w);
    e4m3x4_to_bf16(u.z, sm, b.x, b.y);
    e4m3x4_to_bf16(u.w, sm, b.z, b.w);
    out[2 * i] = a;
    out[2 * i + 1] = b;
  }
}

// ---------------------------------------------------------------------------
// v = bf16(scale * A x): windows of tokens, items of up to 16 tokens of one
// adapter; gridDim.y CTAs take a window's items in turn.
// ---------------------------------------------------------------------------
constexpr int kDownWin = 128;     // tokens per window
constexpr int kDownRanks = 64;    // ranks per pass (8 n-tiles)

__global__ void __launch_bounds__(256) adapter_down_kernel(const uint16_t* __restrict__ x,
                                                           const LinearArgs a,
                                                           uint16_t* __restrict__ v) {
  __shared__ int s_id[kDownWin], s_item[kDownWin], s_leader[kDownWin], s_warp[8];
  __shared__ int s_tok[kDownWin][16];   // [item][slot]: token of the window, -1 empty
  __shared__ int s_ad[kDownWin];
  __shared__ float part[8][16][kDownRanks + 4];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int w0 = blockIdx.x * kDownWin;
  grid_launch_dependents();

  // group the window's tokens by adapter
  int id = -1;
  if (tid < kDownWin) {
    if (w0 + tid < a.T) id = a.ids[w0 + tid];
    if (id >= a.L) {
      if (a.status != nullptr && blockIdx.y == 0) atomicAdd(a.status, 1);
      id = -1;
    }
    s_id[tid] = id < 0 ? -1 : id;
    for (int j = 0; j < 16; ++j) s_tok[tid][j] = -1;
  }
  __syncthreads();
  int rank = 0, leader = tid;   // earlier tokens of this adapter; first token of this one's item
  if (tid < kDownWin && id >= 0) {
    for (int j = 0; j < tid; ++j)
      if (s_id[j] == id) {
        if ((rank & 15) == 0) leader = j;
        ++rank;
      }
    if ((rank & 15) == 0) leader = tid;
  }
  const bool lead = tid < kDownWin && id >= 0 && leader == tid;
  const uint32_t bal = __ballot_sync(0xffffffffu, lead);
  if (lane == 0) s_warp[warp] = __popc(bal);
  __syncthreads();
  int base = 0, items = 0;
  for (int i = 0; i < 8; ++i) {
    if (i < warp) base += s_warp[i];
    items += s_warp[i];
  }
  if (lead) {
    const int it = base + __popc(bal & lanemask_lt());
    s_item[tid] = it;
    s_ad[it] = id;
  }
  if (tid < kDownWin) s_leader[tid] = leader;
  __syncthreads();
  if (tid < kDownWin && id >= 0) s_tok[s_item[leader]][rank & 15] = tid;
  __syncthreads();

  const int g = lane >> 2, q = lane & 3;
  const int steps = a.K / 32;
  const int k0 = steps * warp / 8, k1 = steps * (warp + 1) / 8;
  for (int it = blockIdx.y; it < items; it += gridDim.y) {
    const int ad = s_ad[it];
    const int ta = s_tok[it][g], tb = s_tok[it][g + 8];
    const uint16_t* xa = x + (size_t)(w0 + (ta < 0 ? 0 : ta)) * a.K + 8 * q;
    const uint16_t* xb = x + (size_t)(w0 + (tb < 0 ? 0 : tb)) * a.K + 8 * q;
    for (int r0 = 0; r0 < a.rank; r0 += kDownRanks) {
      const int nt = min(kDownRanks, a.rank - r0) / 8;
      const uint16_t* ar = a.a + ((size_t)ad * a.rank + r0 + g) * a.K + 8 * q;
      float acc[8][4] = {};
      // each lane holds 8 consecutive values of its rows; both operands take
      // them in the same order, so the products are those of row order
#pragma unroll 2
      for (int k = k0; k < k1; ++k) {
        uint4 ua = make_uint4(0u, 0u, 0u, 0u), ub = ua;
        if (ta >= 0) ua = *reinterpret_cast<const uint4*>(xa + 32 * k);
        if (tb >= 0) ub = *reinterpret_cast<const uint4*>(xb + 32 * k);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (j < nt) {
            const uint4 w = *reinterpret_cast<const uint4*>(ar + (size_t)(8 * j) * a.K + 32 * k);
            mma_bf16_16816(acc[j], ua.x, ub.x, ua.y, ub.y, w.x, w.y);
            mma_bf16_16816(acc[j], ua.z, ub.z, ua.w, ub.w, w.z, w.w);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j < nt) {
          part[warp][g][8 * j + 2 * q] = acc[j][0];
          part[warp][g][8 * j + 2 * q + 1] = acc[j][1];
          part[warp][g + 8][8 * j + 2 * q] = acc[j][2];
          part[warp][g + 8][8 * j + 2 * q + 1] = acc[j][3];
        }
      }
      __syncthreads();
      const float sc = a.ascale != nullptr ? a.ascale[ad] : 1.f;
      for (int i = tid; i < 16 * 8 * nt; i += 256) {
        const int row = i / (8 * nt), r = i - row * (8 * nt);
        const int t = s_tok[it][row];
        float z = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) z += part[w][row][r];
        if (t >= 0) v[(size_t)(w0 + t) * a.rank + r0 + r] = f32_to_bf16_rne(z * sc);
      }
      __syncthreads();
    }
  }
}

// ---------------------------------------------------------------------------
// The projection
// ---------------------------------------------------------------------------
constexpr int kThreads = 640;
constexpr int kBM = 128;              // weight rows per tile (MMA M)
constexpr int kBK = 64;               // K values per stage
constexpr int kMaxTok = 256;          // tokens per tile (MMA N)
constexpr int kXBox = 64;             // token rows per tensor copy
constexpr int kPStage = kBM * kBK / 2;
constexpr int kPBoxRows = 64;
constexpr int kBTile = kBM * 128;     // adapter columns of operand A: 128 rows x 64 bf16
constexpr int kMaxS = 8, kMaxSP = 16, kMaxL = 4;   // ring depths
constexpr int kWCols = kBK / 2;
constexpr int kTmemCols = 512;
constexpr int kWarpX = 0, kWarpMma = 1, kWarpW = 2, kWarpEpi = 4, kWarpDeq = 8, kWarpEpi2 = 16;
constexpr int kDeqWarps = 8, kEpiWarps = 8, kEpiThreads = 256;
constexpr int kEpiBar = 1;            // named barrier of the epilogue warps
constexpr int kScaleAhead = 8;
constexpr int kListMax = kMaxTok;     // adapters that one tile can name

struct LinearParams {
  CUtensorMap tmapX;   // bf16 [T][K], box {64, xbox}, 128-byte swizzle
  CUtensorMap tmapW;   // u8 [N][K/2], box {32, 64}
  LinearArgs a;
  const uint16_t* v;   // bf16 [T][rank]
  int cs;              // tokens per tile (multiple of 16, at most 256)
  int xbox;            // rows per token copy
  int xstage;          // bytes of a token stage (cs * 128)
  int S, SP, SL;       // ring depths: operand stages, packed bytes, adapter columns
  int split;           // CTAs of a cluster that share a tile's K
  int rp;              // rank rounded up to 16
};

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}
// NaN in either half when a bf16 of the pair is not finite, else +-0.
__device__ __forceinline__ bool nonfinite_bf16x2(uint32_t w) {
  return ((w & 0x7F80u) == 0x7F80u) || ((w & 0x7F800000u) == 0x7F800000u);
}

__global__ void __launch_bounds__(kThreads, 1) linear_kernel(const __grid_constant__ LinearParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[kMaxS], empty[kMaxS], p_full[kMaxSP], p_empty[kMaxSP], l_full[kMaxL],
      l_empty[kMaxL], d_full, drain;
  __shared__ uint32_t tmem_slot, s_bits[kLinearMaxAdapters / 32];
  __shared__ int s_list[kListMax], s_tokad[kMaxTok], s_count, s_anybad;
  __shared__ uint8_t s_bad[kListMax];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sX = smem;
  uint8_t* sL = sX + p.S * p.xstage;                 // [SL] of {kBTile, xstage}
  const int lstage = kBTile + p.xstage;
  uint8_t* sP = sL + p.SL * lstage;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = p.split > 1 ? (int)cluster_rank() : 0;
  const int N = p.a.N, K = p.a.K;
  const int ntile = (N + kBM - 1) / kBM;
  const int tile = blockIdx.x / p.split;
  const int nt = tile % ntile;
  const int t0 = (tile / ntile) * p.cs;
  const int n = min(p.cs, p.a.T - t0);               // tokens of this tile
  const int n16 = (n + 15) & ~15;
  const int n0 = nt * kBM;
  const int nKall = K / kBK;
  const int kc0 = nKall * rank / p.split;
  const int nK = nKall * (rank + 1) / p.split - kc0;
  const bool adapters = p.a.ids != nullptr;
  int fail = 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.S; ++i) { mbar_init(&full[i], 1 + kDeqWarps); mbar_init(&empty[i], 1); }
    for (int i = 0; i < p.SP; ++i) { mbar_init(&p_full[i], 1); mbar_init(&p_empty[i], kDeqWarps); }
    for (int i = 0; i < kMaxL; ++i) { mbar_init(&l_full[i], kEpiWarps); mbar_init(&l_empty[i], 1); }
    mbar_init(&d_full, 1);
    mbar_init(&drain, 1);
    fence_barrier_init();
    prefetch_tensormap(&p.tmapX);
    prefetch_tensormap(&p.tmapW);
  }
  if (warp == kWarpMma) tmem_alloc(&tmem_slot, kTmemCols);
  if (warp == 3) {
    s_bits[lane] = 0;
    if (lane == 0) { s_count = 0; s_anybad = 0; }
  }
  __syncthreads();
  // the adapters that the tile's tokens name, in ascending order
  if (adapters) {
    if (threadIdx.x < kMaxTok) {
      int id = (int)threadIdx.x < n ? p.a.ids[t0 + threadIdx.x] : -1;
      if (id >= p.a.L) id = -1;
      s_tokad[threadIdx.x] = id;
      s_bad[threadIdx.x] = 0;
      if (id >= 0) atomicOr(&s_bits[id >> 5], 1u << (id & 31));
    }
    __syncthreads();
    if (warp == 3) {
      uint32_t w = s_bits[lane];
      int x = __popc(w);
      const int mine = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      int at = x - mine;
      while (w) {
        s_list[at++] = lane * 32 + __ffs(w) - 1;
        w &= w - 1;
      }
      if (lane == 31) s_count = x;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const uint32_t wcol0 = tmem + (uint32_t)((p.cs + 31) & ~31);   // operand-A ring
  // adapter columns: stages of 64, taken in turn by the CTAs of the cluster
  const int lcols = adapters ? s_count * p.rp : 0;
  const int lstages = (lcols + kBK - 1) / kBK;

  if (warp == kWarpX && lane == 0) {
    // ------------------------------------------------------------ token copies
    int s = 0, k = 0;
    uint32_t ph = 0, par = 0;   // parity of each stage's last fill
    const int nbox = (n16 + p.xbox - 1) / p.xbox;
    const int boxbytes = p.xbox * 128;
    for (int kc = 0; kc < nK; ++kc, ++k) {
      if (k >= p.S && !mbar_wait(&empty[s], ph ^ 1u)) { fail = 1; break; }
      par = (par & ~(1u << s)) | (ph << s);
      mbar_arrive_expect_tx(&full[s], nbox * boxbytes);
      for (int b = 0; b < nbox; ++b)
        tma_load_2d(sX + s * p.xstage + b * boxbytes, &p.tmapX, (kc0 + kc) * kBK, t0 + b * p.xbox,
                    &full[s]);
      if (++s == p.S) { s = 0; ph ^= 1u; }
    }
    // no copy may still be landing in shared memory when the CTA exits
    for (int i = 0; i < p.S && i < k; ++i) mbar_wait(&full[i], (par >> i) & 1u);
  } else if (warp == kWarpW && lane == 0) {
    // ------------------------------------------------------------ packed-weight copies
    int s = 0, k = 0;
    uint32_t ph = 0, par = 0;
    for (int kc = 0; kc < nK; ++kc, ++k) {
      if (k >= p.SP && !mbar_wait(&p_empty[s], ph ^ 1u)) { fail = 1; break; }
      par = (par & ~(1u << s)) | (ph << s);
      mbar_arrive_expect_tx(&p_full[s], kPStage);
      tma_load_2d(sP + s * kPStage, &p.tmapW, (kc0 + kc) * (kBK / 2), n0, &p_full[s]);
      tma_load_2d(sP + s * kPStage + kPStage / 2, &p.tmapW, (kc0 + kc) * (kBK / 2), n0 + kPBoxRows,
                  &p_full[s]);
      if (++s == p.SP) { s = 0; ph ^= 1u; }
    }
    for (int i = 0; i < p.SP && i < k; ++i) mbar_wait(&p_full[i], (par >> i) & 1u);
  } else if (warp == kWarpMma && lane == 0) {
    // ------------------------------------------------------------ MMA issue
    const uint64_t desc0 = umma_desc_sw128(smem_u32(sX));
    const uint32_t idesc = umma_idesc_bf16(kBM, n16);
    int s = 0;
    uint32_t ph = 0;
    bool acc = false;
    for (int kc = 0; kc < nK; ++kc) {
      if (!mbar_wait(&full[s], ph)) { fail = 1; break; }
      tc_fence_after();
      const uint64_t dsc = desc0 + (uint64_t)(s * (p.xstage >> 4));
#pragma unroll
      for (int k16 = 0; k16 < kBK / 16; ++k16) {
        umma_bf16_ts(tmem, wcol0 + s * kWCols + k16 * 8, dsc + 2 * k16, idesc, acc);
        acc = true;
      }
      umma_commit(&empty[s]);
      if (++s == p.S) { s = 0; ph ^= 1u; }
    }
    int ls = 0;
    uint32_t lph = 0;
    for (int i = rank; i < lstages && !fail; i += p.split) {
      if (!mbar_wait(&l_full[ls], lph)) { fail = 1; break; }
      tc_fence_after();
      const uint64_t da = umma_desc_sw128(smem_u32(sL + ls * lstage));
      const uint64_t db = umma_desc_sw128(smem_u32(sL + ls * lstage + kBTile));
      const int k16n = min(kBK, lcols - i * kBK) / 16;
      for (int k16 = 0; k16 < k16n; ++k16) {
        umma_bf16_ss(tmem, da + 2 * k16, db + 2 * k16, idesc, acc);
        acc = true;
      }
      umma_commit(&l_empty[ls]);
      if (++ls == p.SL) { ls = 0; lph ^= 1u; }
    }
    if (!fail) umma_commit(&d_full);
    // every issued MMA has finished before tensor memory is released
    umma_commit(&drain);
    mbar_wait(&drain, 0);
  } else if (warp >= kWarpDeq && warp < kWarpDeq + kDeqWarps) {
    // ------------------------------------------------------------ dequantisation
    const int q = warp & 3;                    // lane quarter
    const int h = (warp - kWarpDeq) >> 2;      // which 32 of the stage's 64 K values
    const int m = q * 32 + lane;               // weight row of the tile = TMEM lane
    const uint32_t wlane = wcol0 + ((uint32_t)(q * 32) << 16) + h * 16;
    const uint8_t* srow =
        p.a.s + (size_t)min(n0 + m, N - 1) * (K / kScaleBlock) + 2 * kc0 + h;
    int sp = 0, sw = 0;
    uint32_t pp = 0, pw = 0;
    uint32_t sc[kScaleAhead];
#pragma unroll
    for (int i = 0; i < kScaleAhead; ++i) sc[i] = i < nK ? ldg_u8(srow + 2 * i) : 0u;
    for (int k0 = 0; k0 < nK && !fail; k0 += kScaleAhead) {
      uint32_t nx[kScaleAhead];   // the next window's scale bytes, loaded one window early
#pragma unroll
      for (int i = 0; i < kScaleAhead; ++i)
        nx[i] = k0 + kScaleAhead + i < nK ? ldg_u8(srow + 2 * (k0 + kScaleAhead + i)) : 0u;
#pragma unroll
      for (int i = 0; i < kScaleAhead; ++i) {
        if (k0 + i >= nK || fail) break;
        if (!warp_wait(&p_full[sp], pp)) { fail = 1; break; }
        const uint4 qv = *reinterpret_cast<const uint4*>(sP + sp * kPStage + m * (kBK / 2) + h * 16);
        // the generic read above is ordered before the stage's refill by a tensor copy
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_empty[sp]);
        if (++sp == p.SP) { sp = 0; pp ^= 1u; }
        const uint32_t wd[4] = {qv.x, qv.y, qv.z, qv.w};
        uint32_t o[16];
        dequant32_bf16(wd, scale_mul(sc[i]), o);
        if (k0 + i >= p.S) {   // the MMAs that read this ring slot have completed
          if (!warp_wait(&empty[sw], pw ^ 1u)) { fail = 1; break; }
          tc_fence_after();
        }
        tmem_st16(wlane + sw * kWCols, o);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[sw]);
        if (++sw == p.S) { sw = 0; pw ^= 1u; }
      }
#pragma unroll
      for (int i = 0; i < kScaleAhead; ++i) sc[i] = nx[i];
    }
  } else if ((warp >= kWarpEpi && warp < kWarpEpi + 4) || warp >= kWarpEpi2) {
    // ------------------------------------------------------------ adapter columns
    const int q = warp & 3;
    const int half = warp >= kWarpEpi2;
    const int et = (half * 4 + q) * 32 + lane;   // 0..255
    if (adapters) {
      bool waited = false;
      int ls = 0, use = 0;
      uint32_t lph = 0;
      for (int i = rank; i < lstages && !fail; i += p.split, ++use) {
        if (use >= p.SL && !warp_wait(&l_empty[ls], lph ^ 1u)) { fail = 1; break; }
        uint8_t* tb = sL + ls * lstage;
        uint8_t* tv = tb + kBTile;
        // 16-byte chunk j of a row: columns 64 i + 8 j .., one adapter's ranks r ..
        const int j = et & 7;
        const int c = i * kBK + 8 * j;
        const int ai = c / p.rp, r = c - ai * p.rp;
        const bool live = ai < s_count && r < p.a.rank;
        const int ad = live ? s_list[ai] : -1;
        for (int row = et >> 3; row < kBM; row += kEpiThreads / 8) {
          uint4 w = make_uint4(0u, 0u, 0u, 0u);
          if (live && n0 + row < N)
            w = *reinterpret_cast<const uint4*>(p.a.b + ((size_t)ad * N + n0 + row) * p.a.rank + r);
          if (nonfinite_bf16x2(w.x) || nonfinite_bf16x2(w.y) || nonfinite_bf16x2(w.z) ||
              nonfinite_bf16x2(w.w)) {
            s_bad[ai] = 1;
            s_anybad = 1;
            uint32_t z[4] = {w.x, w.y, w.z, w.w};
            for (int e = 0; e < 4; ++e) {
              if ((z[e] & 0x7F80u) == 0x7F80u) z[e] &= 0xFFFF0000u;
              if ((z[e] & 0x7F800000u) == 0x7F800000u) z[e] &= 0xFFFFu;
            }
            w = make_uint4(z[0], z[1], z[2], z[3]);
          }
          *reinterpret_cast<uint4*>(tb + row * 128 + ((j ^ (row & 7)) << 4)) = w;
        }
        if (!waited) {   // v comes from the kernel before this one
          grid_dependency_wait();
          waited = true;
        }
        for (int t = et >> 3; t < n16; t += kEpiThreads / 8) {
          uint4 w = make_uint4(0u, 0u, 0u, 0u);
          if (live && s_tokad[t] == ad)
            w = *reinterpret_cast<const uint4*>(p.v + (size_t)(t0 + t) * p.a.rank + r);
          *reinterpret_cast<uint4*>(tv + t * 128 + ((j ^ (t & 7)) << 4)) = w;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&l_full[ls]);
        if (++ls == p.SL) { ls = 0; lph ^= 1u; }
      }
      if (!waited) grid_dependency_wait();
      named_barrier(kEpiBar, kEpiThreads);   // s_bad and s_anybad are complete
    }
    // ------------------------------------------------------------ epilogue
    if (!warp_wait(&d_full, 0)) fail = 1;
    tc_fence_after();
    if (!fail) {
      const int row = n0 + q * 32 + lane;
      const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16);
      const int n32 = (n16 + 31) >> 5, lo32 = (n32 + 1) >> 1;
      float* red = reinterpret_cast<float*>(sX);   // [token][128], the token ring is free
      const bool fix = adapters && s_anybad != 0;
#pragma unroll 1
      for (int c0 = (half ? lo32 : 0) * 32; c0 < (half ? n32 : lo32) * 32; c0 += 32) {
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
                z += __uint_as_float(bw << 16) *
                     __uint_as_float((uint32_t)p.v[(size_t)(t0 + c0 + t) * p.a.rank + r] << 16);
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
        } else if (row < N) {
          uint16_t* dst = p.a.out + (size_t)(t0 + c0) * N + row;
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (e < nv) dst[(size_t)e * N] = f32_to_bf16_rne(v[e]);
        }
      }
    }
  }
  __syncwarp();
  if (fail && p.a.status != nullptr) {
    if (adapters) grid_dependency_wait();   // the status words belong to that kernel until then
    atomicOr(&p.a.status[2], 1);
    atomicCAS(&p.a.status[3], 0, blockIdx.x + 1);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (p.split > 1) {
    // y of tokens rank, rank + split, ..: the cluster's partial sums in rank order
    cluster_sync();
    const uint32_t red = smem_u32(sX);
    for (int t = rank + p.split * warp; t < n; t += p.split * (kThreads / 32)) {
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int c = 0; c < p.split; ++c) {
        const float4 z = ld_cluster16(red + (t * kBM + lane * 4) * 4, c);
        y.x += z.x;
        y.y += z.y;
        y.z += z.z;
        y.w += z.w;
      }
      if (n0 + lane * 4 < N)
        *reinterpret_cast<uint2*>(p.a.out + (size_t)(t0 + t) * N + n0 + lane * 4) =
            make_uint2(bf16x2_rn(y.x, y.y), bf16x2_rn(y.z, y.w));
    }
    cluster_sync();   // no CTA leaves while another reads its shared memory
  }
}

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

}  // namespace

size_t linear_workspace_bytes(int T, int K, int N, int rank, bool x8) {
  (void)N;
  return up256((size_t)T * rank * 2) + (x8 ? up256((size_t)T * K * 2) : 0);
}

cudaError_t launch_linear(const LinearArgs& a, int num_sms, cudaStream_t stream) {
  cudaError_t e;
  char* ws = static_cast<char*>(a.ws);
  const bool adapters = a.ids != nullptr;
  uint16_t* v = reinterpret_cast<uint16_t*>(ws);
  const uint16_t* x = static_cast<const uint16_t*>(a.x);
  if (a.status != nullptr &&
      (e = cudaMemsetAsync(a.status, 0, 4 * sizeof(int32_t), stream)) != cudaSuccess)
    return e;
  if (a.xs != nullptr) {
    uint16_t* xb = reinterpret_cast<uint16_t*>(ws + up256((size_t)a.T * a.rank * 2));
    const int64_t n16 = (int64_t)a.T * a.K / 16;
    const int64_t blocks = (n16 + 255) / 256;
    mx8_to_bf16_kernel<<<(unsigned)(blocks < num_sms * 8 ? blocks : num_sms * 8), 256, 0, stream>>>(
        static_cast<const uint4*>(a.x), a.xs, n16, reinterpret_cast<uint4*>(xb));
    x = xb;
  }
  if (adapters) {
    const int win = (a.T + kDownWin - 1) / kDownWin;
    int slots = (2 * num_sms + win - 1) / win;
    if (slots < 8) slots = 8;
    if (slots > kDownWin) slots = kDownWin;
    if (slots > a.T) slots = a.T;
    adapter_down_kernel<<<dim3(win, slots), 256, 0, stream>>>(x, a, v);
  }
  if ((e = cudaGetLastError()) != cudaSuccess) return e;

  LinearParams p = {};
  p.a = a;
  p.v = v;
  const int chunks = (a.T + kMaxTok - 1) / kMaxTok;
  p.cs = ((a.T + chunks - 1) / chunks + 15) & ~15;
  p.xbox = p.cs < kXBox ? p.cs : kXBox;
  const int xrows = (p.cs + p.xbox - 1) / p.xbox * p.xbox;   // whole copies fill a stage
  p.xstage = xrows * 128;
  p.S = 96 * 1024 / p.xstage;
  if (p.S < 4) p.S = 4;
  if (p.S > kMaxS) p.S = kMaxS;
  p.SP = p.cs > 32 ? 8 : kMaxSP;
  p.SL = !adapters ? 0 : p.cs > 128 ? 1 : p.cs > 64 ? 2 : kMaxL;
  p.rp = (a.rank + 15) & ~15;
  const int ntile = (a.N + kBM - 1) / kBM, ttile = (a.T + p.cs - 1) / p.cs;
  const int64_t tiles = (int64_t)ntile * ttile;
  // a cluster splits K while that still gives every CTA an SM of its own and
  // at least four stages
  p.split = 1;
  while (p.split < 8 && tiles * p.split * 2 <= num_sms && a.K / kBK >= 4 * p.split * 2) p.split *= 2;
  if (!encode_tiled_2d(&p.tmapX, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, x, (uint64_t)a.K, (uint64_t)a.T,
                       (uint64_t)a.K * 2, kBK, p.xbox, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_tiled_2d(&p.tmapW, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w, (uint64_t)a.K / 2, (uint64_t)a.N,
                       (uint64_t)a.K / 2, kBK / 2, kPBoxRows, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorInvalidValue;
  const size_t smem = 1024 + (size_t)p.S * p.xstage + (size_t)p.SL * (kBTile + p.xstage) +
                      (size_t)p.SP * kPStage;
  static size_t granted[kGrantDevices] = {};
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if (dev < 0 || dev >= kGrantDevices) return cudaErrorInvalidDevice;
  if (smem > granted[dev]) {
    e = cudaFuncSetAttribute(linear_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    granted[dev] = smem;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * p.split));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  int na = 0;
  if (p.split > 1) {
    at[na].id = cudaLaunchAttributeClusterDimension;
    at[na].val.clusterDim.x = p.split;
    at[na].val.clusterDim.y = at[na].val.clusterDim.z = 1;
    ++na;
  }
  if (adapters) {   // starts beside the down kernel, whose results it waits for
    at[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[na].val.programmaticStreamSerializationAllowed = 1;
    ++na;
  }
  cfg.attrs = at;
  cfg.numAttrs = na;
  return cudaLaunchKernelEx(&cfg, linear_kernel, p);
}

}  // namespace mxmoe
