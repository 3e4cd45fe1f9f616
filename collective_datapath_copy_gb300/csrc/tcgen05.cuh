// Tensor-core (tcgen05), cluster and TMA helpers of the dense kernels, sm_103a.
#pragma once

#include <stdint.h>

#include "coll.h"
#include "tma.cuh"

namespace coll {

// ------------------------------------------------------------------ clusters

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// Barrier over every thread of the cluster; orders shared-memory accesses between its CTAs.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The address, in the cluster's shared-memory window, of `addr` of this CTA in CTA `rank`.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}

// ------------------------------------------------------------------ barriers by address

// One lane of a converged warp, the same one every time. The compiler knows the branch it guards
// is taken by one lane, which keeps the operands of the instructions below in uniform registers:
// a loop that issues four matrix instructions and a commit took 325 ns under `lane == 0` and
// 177 ns under this.
__device__ __forceinline__ bool elect_one() {
  uint32_t on;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(on));
  return on != 0;
}

__device__ __forceinline__ bool bar_try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// The same without the hardware's suspended wait (up to some 4 us where the phase never ends).
__device__ __forceinline__ bool bar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Every wait is bounded. The slow part of one: false once it has run out of time or another role
// of the CTA has given up; then the roles leave their loops, the CTA drains and `status` says so.
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr uint64_t kDrainNs = 20000000ull;

static __device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, uint32_t *abort_flag,
                                       int32_t *status) {
  volatile uint32_t *flag = abort_flag;
  uint64_t t0 = 0;
  for (uint32_t i = 0;; ++i) {
    if (bar_try_wait(bar, parity)) return true;
    if ((i & 15u) == 15u) {
      if (*flag) return false;
      const uint64_t now = globaltimer();
      if (t0 == 0) t0 = now;
      else if (now - t0 > kWaitNs) break;
    }
  }
  *flag = 1u;
  if (status) *status = COLL_ETIMEDOUT;
  return false;
}

__device__ __forceinline__ bool wait_bar(uint32_t *abort_flag, uint32_t bar, uint32_t parity,
                                         int32_t *status) {
  return bar_try_wait(bar, parity) || wait_long(bar, parity, abort_flag, status);
}

// After an abort: time for the copies and matrix instructions in flight to land.
static __device__ __noinline__ void drain() {
  const uint64_t t0 = globaltimer();
  while (globaltimer() - t0 < kDrainNs) __nanosleep(1000);
}

__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}

// ------------------------------------------------------------------ TMA, 2-D boxes

// One box at element coordinates (x, y) into this CTA's shared memory; completion is counted on
// `bar`. x times the element size is a multiple of 16 bytes.
__device__ __forceinline__ void tma_box(uint32_t sdst, const void *map, int32_t x, int32_t y,
                                        uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(sdst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

// The same for a CTA of a pair: `bar` may be a cluster address in either CTA of the pair.
__device__ __forceinline__ void tma_box_pair(uint32_t sdst, const void *map, int32_t x, int32_t y,
                                             uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile"
      ".mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(sdst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

// ------------------------------------------------------------------ tcgen05

// Shared-memory matrix descriptor, 128-byte swizzle, version 1: the low word holds the address
// and the leading offset, the high word the stride offset (all in 16-byte units).
//   K-major (rows of 64 16-bit elements, 128 bytes): groups of eight rows are `stride` apart.
//   M- or N-major (64 elements of M or N per 128-byte row): groups of eight rows (k) are
//   `stride` apart, the next 64 elements `leading` apart.
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t leading) {
  return ((addr >> 4) & 0x3FFFu) | ((leading >> 4) << 16);
}
__device__ __forceinline__ uint32_t desc_hi(uint32_t stride) {
  return (stride >> 4) | (1u << 14) | (2u << 29);
}

// Instruction descriptor of kind::f16 with binary32 accumulators.
__host__ __device__ inline uint32_t mma_desc(bool bf16, bool a_mn, bool b_mn, uint32_t m,
                                             uint32_t n) {
  const uint32_t t = bf16 ? 1u : 0u;
  return (1u << 4) | (t << 7) | (t << 10) | ((a_mn ? 1u : 0u) << 15) |
         ((b_mn ? 1u : 0u) << 16) | ((n >> 3) << 17) | ((m >> 4) << 24);
}

// Allocate `cols` columns (a power of two from 32) and give up the right to allocate more, which
// another CTA of this SM would wait for otherwise. A whole warp calls these.
template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t *saddr, uint32_t cols) {
  if (CG == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(saddr)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  } else {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(saddr)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
}

template <int CG>
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  if (CG == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
  else
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}

// D (+)= A B^T over 16 of k, with each descriptor given as two words. One thread issues it.
template <int CG>
__device__ __forceinline__ void mma_f16(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo,
                                        uint32_t b_hi, uint32_t idesc, uint32_t add) {
  if (CG == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\tsetp.ne.u32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(add)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\tsetp.ne.u32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(add)
        : "memory");
}

// Arrive on `bar` (the same offset in every CTA of `mask` for a pair) once the matrix
// instructions issued so far by this thread have finished.
template <int CG>
__device__ __forceinline__ void mma_commit(uint32_t bar, uint16_t mask) {
  if (CG == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster"
        ".b64 [%0], %1;" ::"r"(bar),
        "h"(mask)
        : "memory");
  else
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
        : "memory");
}

__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// 32 columns of this warp's 32 lanes: v[c] of lane l is column c of row l.
__device__ __forceinline__ void tmem_load32(uint32_t addr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

}  // namespace coll
