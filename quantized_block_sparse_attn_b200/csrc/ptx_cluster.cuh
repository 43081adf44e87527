// Inline-PTX building blocks of the 8-bit linear layers, beside those of ptx_sm100.cuh: waits of a
// ring's threads, thread-block clusters, pairs of CTAs that share an MMA, 2-D and untiled loads.
//
// As there, every wait on an mbarrier is bounded, and no load is a multicast.
#pragma once

#include <cstdint>
#include <cuda.h>

#include "ptx_sm100.cuh"

namespace qbsa {

// mbar_wait for the threads that hand the stages of a ring to each other: one instruction in the
// common case (the thread is suspended until the phase completes, for up to 1 ms), and the rest out
// of line.  A lone thread pays some twenty cycles for each branch that it takes, so that with the
// loop of mbar_wait in line a slab of a product took 390 ns instead of 340, and with short polls 410.
// kCluster: the barrier is one that threads of other CTAs arrive on.
template <bool kCluster>
__device__ __forceinline__ bool mbar_try_wait_long(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  if constexpr (kCluster)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(1000000u)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(1000000u)
        : "memory");
  return ok != 0;
}
template <bool kCluster>
__device__ __noinline__ bool mbar_wait_rest(uint32_t bar, uint32_t parity, volatile int* abort) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait_long<kCluster>(bar, parity)) {
    if (*abort) return false;
    if (global_timer_ns() - t0 > QBSA_WAIT_TIMEOUT_NS) {
      *abort = 1;
      atomicCAS(&g_device_error, 0u, static_cast<unsigned int>(kErrTimeout));
      return false;
    }
  }
  return true;
}
template <bool kCluster = false>
__device__ __forceinline__ bool mbar_wait_hot(uint32_t bar, uint32_t parity, volatile int* abort) {
  if (__builtin_expect(mbar_try_wait_long<kCluster>(bar, parity), 1)) return true;
  return mbar_wait_rest<kCluster>(bar, parity, abort);
}

// ---------------------------------------------------------------------------------
// thread-block clusters
// ---------------------------------------------------------------------------------

__device__ __forceinline__ uint32_t cluster_ctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// Address in the cluster's shared-memory window of CTA `rank`'s copy of `addr`.
__device__ __forceinline__ uint32_t cluster_map(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

// Every thread of every CTA of the cluster; shared-memory writes before it are seen after it.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

__device__ __forceinline__ void st_cluster_b32(uint32_t cluster_addr, uint32_t v) {
  asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(cluster_addr), "r"(v) : "memory");
}

// ---------------------------------------------------------------------------------
// loads
// ---------------------------------------------------------------------------------

// A 2- or 4-byte value of shared memory, as bits.
template <int kBytes>
__device__ __forceinline__ uint32_t lds_value(uint32_t addr) {
  if constexpr (kBytes == 2) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
    return v;
  } else {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
  }
}

// `bytes` contiguous bytes (a multiple of 16, both ends 16-byte aligned) into this CTA's shared
// memory; completes on an mbarrier.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// 2-D tiled load into this CTA's shared memory; completes on an mbarrier of this CTA.
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const void* map, uint32_t bar, int c0, int c1,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(dst),
      "l"(map), "r"(bar), "r"(c0), "r"(c1), "l"(policy)
      : "memory");
}

// The same in a pair of CTAs that work on one tile (cta_group::2): the data goes to this CTA's
// shared memory, and `bar`, a shared::cluster address, may be the other CTA's mbarrier.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const void* map, uint32_t bar, int c0, int c1,
                                                 uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(dst),
      "l"(map), "r"(bar), "r"(c0), "r"(c1), "l"(policy)
      : "memory");
}

// ---------------------------------------------------------------------------------
// tcgen05
// ---------------------------------------------------------------------------------

// The pair forms (cta_group::2): issued in the even CTA of a pair, on both CTAs' shared memory and
// TMEM; the allocation is made by one warp of each CTA.
__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish_pair() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// Four MMAs over 128 bytes of K (32 bytes, 2 descriptor units, each); the operands' descriptors
// share their upper words, and their lower words start with the address.
__device__ __forceinline__ void mma_i8_ss_pair_x4(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                                  uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, one;\n\t.reg .b64 a0, a1, a2, a3, b0, b1, b2, b3;\n\t.reg .b32 x, y;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tsetp.eq.b32 one, %3, %3;\n\t"
      "mov.b64 a0, {%1, %3};\n\tmov.b64 b0, {%2, %3};\n\t"
      "add.u32 x, %1, 2;\n\tadd.u32 y, %2, 2;\n\tmov.b64 a1, {x, %3};\n\tmov.b64 b1, {y, %3};\n\t"
      "add.u32 x, %1, 4;\n\tadd.u32 y, %2, 4;\n\tmov.b64 a2, {x, %3};\n\tmov.b64 b2, {y, %3};\n\t"
      "add.u32 x, %1, 6;\n\tadd.u32 y, %2, 6;\n\tmov.b64 a3, {x, %3};\n\tmov.b64 b3, {y, %3};\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], a0, b0, %4, p;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], a1, b1, %4, one;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], a2, b2, %4, one;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], a3, b3, %4, one;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(acc)
      : "memory");
}
// Arrive on the mbarrier at this address in both CTAs of the pair.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

// Load 16 consecutive 32-bit columns of this warp's 32 lanes and wait for them.
__device__ __forceinline__ void tmem_ld16_wait(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

}  // namespace qbsa
