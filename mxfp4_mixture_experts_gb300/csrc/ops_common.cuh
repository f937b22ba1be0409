// Device helpers of the operators around the MoE layer (sm_103a).
#pragma once

#include "common.cuh"

namespace mxmoe {

// Two fp32 -> bf16 pair (first value in the low half), nearest even.
__device__ __forceinline__ uint32_t bf16x2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Lets the next kernel of the stream, launched with programmatic
// serialisation, start before this one has finished.
__device__ __forceinline__ void grid_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Multipliers that turn the placed bits of an E4M3 pair (value * 2^-120, see
// below) into value * 2^(s - 127): one exact step up to s = 134, two above.
__device__ __forceinline__ ScaleMul e4m3_scale_mul(uint32_t s) {
  ScaleMul r;
  if (s <= 134u) {
    const uint32_t b = (s + 120u) << 7;   // bf16 bits of 2^(s - 7)
    r.m1 = b | (b << 16);
    r.m2 = 0;
    r.two = false;
  } else {
    r.m1 = 0x7B807B80u;                   // 2^120
    const uint32_t b = (s == 255u) ? 0x7FC0u : (s << 7);
    r.m2 = b | (b << 16);
    r.two = true;
  }
  return r;
}

// Four E4M3 bytes (low byte first) -> two bf16 pairs of the values times 2^-120:
// the sign and the 7 magnitude bits of a code at bit 15 and bits 4..10 of a
// half, subnormal codes included. Multiplied by e4m3_scale_mul's factors they
// are rounded once (exact inside bf16's range).
__device__ __forceinline__ void e4m3x4_place(uint32_t w, uint32_t& o0, uint32_t& o1) {
  const uint32_t p0 = prmt(w, 0u, 0x4140u), p1 = prmt(w, 0u, 0x4342u);
  o0 = ((p0 << 8) & 0x80008000u) | ((p0 << 4) & 0x07F007F0u);
  o1 = ((p1 << 8) & 0x80008000u) | ((p1 << 4) & 0x07F007F0u);
}
// Code 0x7F (either sign), which the placement above turns into a number, as NaN.
__device__ __forceinline__ void e4m3x4_nan(uint32_t w, uint32_t& o0, uint32_t& o1) {
  if ((w & 0x7Fu) == 0x7Fu) o0 |= 0x7FC0u;
  if ((w & 0x7F00u) == 0x7F00u) o0 |= 0x7FC00000u;
  if ((w & 0x7F0000u) == 0x7F0000u) o1 |= 0x7FC0u;
  if ((w & 0x7F000000u) == 0x7F000000u) o1 |= 0x7FC00000u;
}

// D += A * B for one m16n8k16 tile, bf16 inputs, fp32 accumulators.
__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                               uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// ---------------------------------------------------------------------------
// CTA pairs: one tcgen05.mma of 256 rows over two SMs. Each CTA holds its 128
// rows of A and D in its own tensor memory and half of B's rows in its own
// shared memory; the even CTA of the pair issues.
// ---------------------------------------------------------------------------
// D[tmem] (+)= A[tmem] * B[smem]^T
__device__ __forceinline__ void umma2_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                              uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
// D[tmem] (+)= A[smem] * B[smem]^T, both operands K-major with the 128-byte swizzle.
__device__ __forceinline__ void umma2_bf16_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                              uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
// Arrive on the barrier at this offset in every CTA of the mask (ranks in the
// cluster) once all MMAs issued so far by this thread have completed.
__device__ __forceinline__ void umma2_commit(uint64_t* bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(smem_u32(bar)),
      "h"(mask)
      : "memory");
}
// Tensor memory for the pair: one warp of each of the two CTAs.
__device__ __forceinline__ void tmem2_alloc(uint32_t* dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(dst)),
               "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem2_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}
// 3-D tensor copy into this CTA, counted on a barrier of the pair's even CTA.
__device__ __forceinline__ void tma2_load_3d(void* dst, const void* tmap, int x, int y, int z,
                                             uint32_t bar_cluster) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(bar_cluster)
      : "memory");
}
// Address of a shared variable in another CTA of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
// The arrival of a thread whose results are in tensor memory (after tcgen05.wait and
// the fence before a thread synchronisation; the waiter, which acquires at cluster scope,
// has the fence after one). Relaxed: those two fences order tensor memory, and a release at
// cluster scope would also wait for the thread's prefetches from global memory (1000 to
// 10000 clocks a stage).
__device__ __forceinline__ void mbar_arrive_remote(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Bounded wait of a whole warp, which also acquires what other CTAs of the
// cluster released. The warp sleeps in the hardware until the phase completes or
// its time runs out (at most the hint of 20 us; 3.7 us measured), so waiting warps
// leave the issue slots to the others; it gives up after 0.19 s (measured: a call
// whose first copy never comes ends then).
constexpr uint32_t kSleepHintNs = 20000, kSleepLimit = 50000;
__device__ __forceinline__ bool warp_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok = 0;
  for (uint32_t i = 0; i < kSleepLimit && !ok; ++i)
    asm volatile(
        "{\n .reg .pred p;\n"
        " mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(kSleepHintNs)
        : "memory");
  return __all_sync(0xffffffffu, ok != 0);
}
// The same for barriers of this CTA alone.
__device__ __forceinline__ bool warp_wait_cta(uint64_t* bar, uint32_t parity) {
  uint32_t ok = 0;
  for (uint32_t i = 0; i < kSleepLimit && !ok; ++i)
    asm volatile(
        "{\n .reg .pred p;\n"
        " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(kSleepHintNs)
        : "memory");
  return __all_sync(0xffffffffu, ok != 0);
}

// One lane of a converged warp. The single-thread roles run their loops in the
// whole warp and only issue under this predicate: their addresses, barriers and
// descriptors then stay in uniform registers. Under a lane == 0 branch around
// the loop every tcgen05 and tensor-copy instruction had its operands moved
// there first, about 850 clocks for the four MMAs of a stage.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(ok));
  return ok != 0;
}

// Thread-block clusters: rank, barrier over all threads of the cluster, and
// 16-byte reads of another CTA's shared memory.
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// The same as a start-up barrier: no release of the threads' memory operations
// (loads under way would be waited for); barrier inits are fenced by their thread.
__device__ __forceinline__ void cluster_sync_relaxed() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n barrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
__device__ __forceinline__ float4 ld_cluster16(uint32_t smem_addr, uint32_t rank) {
  uint32_t a;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

}  // namespace mxmoe
