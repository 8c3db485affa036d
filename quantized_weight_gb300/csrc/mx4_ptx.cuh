// mx4_ptx.cuh -- the block-scaled tensor-core instructions of the microscaled 4-bit product.
#pragma once
#include <cstdint>

#include "sm100_ptx.cuh"

namespace qmm {
namespace sm100 {

// CTAS: the CTAs whose tensor memory and tensor cores an instruction uses (cta_group::1 or ::2).

// D[tmem] (+)= A * B^T, e2m1 operands in shared memory (K-major, 64 elements = 32 bytes of a row), a scale for each 32
// elements in TMEM (sfa, sfb; idesc says which two of a column's four bytes), f32 out.  Of a pair, each CTA has half of A's
// rows, of D's rows and of B's rows.
template <int CTAS>
__device__ __forceinline__ void umma_mxf4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t sfa,
                                          uint32_t sfb, uint32_t accumulate) {
  if constexpr (CTAS == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// 32 rows of 16 bytes from shared memory to 4 columns of TMEM, the same in each of its four lane quarters (of a pair, in
// each CTA from its own shared memory).  In order with the same thread's MMAs.
template <int CTAS>
__device__ __forceinline__ void tmem_cp_32x16b(uint32_t taddr, uint64_t desc) {
  if constexpr (CTAS == 1)
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// Arrive (once) on `bar`, of a pair on both CTAs' barriers at that offset, when every MMA issued so far has completed.
template <int CTAS>
__device__ __forceinline__ void commit_mxf4(uint32_t bar) {
  if constexpr (CTAS == 1)
    umma_commit(bar);
  else
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
                 "h"((uint16_t)3)
                 : "memory");
}

// Executed by one full warp, of a pair by one of each CTA.
template <int CTAS>
__device__ __forceinline__ void tmem_alloc_for(uint32_t slot, uint32_t ncols) {
  if constexpr (CTAS == 1) {
    tmem_alloc(slot, ncols);
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(ncols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int CTAS>
__device__ __forceinline__ void tmem_dealloc_for(uint32_t taddr, uint32_t ncols) {
  if constexpr (CTAS == 1)
    tmem_dealloc(taddr, ncols);
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// Arrive on a barrier of another CTA of the cluster (mapa_shared's address); what the thread has seen before is seen by who
// waits there with mbar_try_wait_cluster.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}

// Counts `bytes` as landed on a barrier of this CTA.
__device__ __forceinline__ void mbar_complete_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// Bulk copy global -> shared: `bytes` and both addresses multiples of 16, completion as transaction bytes on `bar`.
__device__ __forceinline__ void bulk_copy(uint32_t dst, uint64_t src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar)
               : "memory");
}

// tma_load_2d of one CTA of a pair, completing on a barrier of either (mapa_shared's address).
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const void *tmap, int32_t c0, int32_t c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}

// The box at (c0, c1) into L2.
__device__ __forceinline__ void tma_prefetch_2d(const void *tmap, int32_t c0, int32_t c1) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(tmap)),
               "r"(c0), "r"(c1)
               : "memory");
}

// Descriptor of 512 bytes in that order: no swizzle, 8 rows of 16 bytes after 8 rows.
__device__ __forceinline__ uint64_t smem_desc_scales(uint32_t addr) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)(128u >> 4) << 32 | (uint64_t)1 << 46;
}

// Instruction descriptor, kind::mxf4: e2m1 operands, power-of-two scales, M x N, the scales' bytes 0 and 1 of a column.
__host__ __device__ constexpr uint32_t idesc_mxf4(int M, int N) {
  return (1u << 7) | (1u << 10)          // A, B: e2m1
         | (uint32_t)(N >> 3) << 17      // N / 8
         | (1u << 23)                    // scales: e8m0
         | (uint32_t)(M >> 7) << 27;     // M / 128
}
constexpr uint32_t kSecondScales = 2u << 4 | 2u << 29;   // bytes 2 and 3, of B's and A's scales

// One thread of a converged warp, the same each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}

// The two halves of a barrier of the cluster's threads, by whole warps.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

}  // namespace sm100
}  // namespace qmm
