// tcgen05 over a pair of CTAs (cta_group::2): the two CTAs of a cluster hold
// the halves of A's rows and of B's rows at the same shared-memory offsets,
// one thread of the leader (cluster rank 0) issues, and each CTA's tensor
// memory receives its part of D.
#pragma once

#include "common.cuh"

namespace csa2 {

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Every thread of both CTAs.
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address of a shared variable of this CTA in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// Arrive on a barrier of either CTA (address from map_rank).  It announces
// operands that this CTA wrote to its OWN shared memory, where its own tensor
// core reads them: the writers' fence.proxy.async and the arrival's release at
// CTA scope order those writes.  A release to the cluster would add nothing but
// a wait for every load that the SM has in flight (about 1,000 cycles here).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Descriptor of a K-major operand stored as rows of 32 bytes with the 32-byte
// swizzle (16-byte chunk c of row r lives at chunk c ^ ((r / 4) % 2)); 8-row
// groups are 256 bytes apart.
__device__ __forceinline__ uint64_t sw32_kmajor_desc(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu);   // start address
  d |= static_cast<uint64_t>(1) << 16;                        // LBO (unused here)
  d |= static_cast<uint64_t>(256 >> 4) << 32;                 // SBO: 8 rows x 32 B
  d |= static_cast<uint64_t>(1) << 46;                        // descriptor version
  d |= static_cast<uint64_t>(6) << 61;                        // 32-byte swizzle
  return d;
}
// Byte offset of (row, byte c) in a 32-byte-swizzled tile of 32-byte rows.
__host__ __device__ __forceinline__ uint32_t sw32_offset(uint32_t row, uint32_t c) {
  return row * 32u + ((((c >> 4) ^ (row >> 2)) & 1u) << 4) + (c & 15u);
}

// 32 lanes x 16 consecutive columns of tensor memory.
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// Store a word into the other CTA's shared memory (address from map_rank), and
// an arrival that releases such stores.
__device__ __forceinline__ void st_cluster(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void mbar_arrive_release_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// mbar_try_wait that acquires what the other CTA released.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// Waits of a whole warp, bounded like mbar_wait.  Every lane polls and the
// outcome is a vote, so the warp stays converged and the compiler sees that it
// does: with one polling lane the attention kernel took 25 % longer, the weight
// kernel 60 %.  A limit of zero looks once and does not wait.
__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
template <class Try>
__device__ __forceinline__ bool wait_all(Try done, uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  if (limit_ns == 0) return __all_sync(0xffffffffu, mbar_test_wait(bar, parity));
  if (__all_sync(0xffffffffu, done(bar, parity))) return true;
  const uint64_t t0 = globaltimer();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (__all_sync(0xffffffffu, done(bar, parity))) return true;
    if (__any_sync(0xffffffffu, globaltimer() - t0 > limit_ns)) return false;
  }
}
__device__ __forceinline__ bool mbar_wait_all(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  return wait_all(mbar_try_wait, bar, parity, limit_ns);
}
__device__ __forceinline__ bool mbar_wait_cluster_all(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  return wait_all(mbar_try_wait_cluster, bar, parity, limit_ns);
}

// True in one lane of a converged warp.  The warp that issues MMAs runs its
// loop in all lanes and issues under this predicate: descriptors then stay in
// uniform registers.  Under `if (lane == 0)` every MMA took about 180 cycles to
// issue, of the 64 that it takes to run.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void tmem_alloc_pair(uint32_t* smem_dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(smem_dst)), "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tmem_release_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// D (+)= A B^T over both CTAs; 16-bit operands of one type, fp32 D.
__device__ __forceinline__ void umma_f16_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive on `bar` (the same offset) of both CTAs once every tcgen05 operation
// issued so far by this thread has completed.
__device__ __forceinline__ void umma_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
// Instruction descriptor of kind::f16: A = B = fp16 (bf16 when `bf16`), fp32
// D, shape M x N; A K-major, B K-major or (b_mn) MN-major.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool bf16, bool b_mn) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((b_mn ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

}  // namespace csa2
