// Device-side helpers of the tensor-core products: tensor-map copies, cluster
// barriers and the tcgen05 instructions for pairs of CTAs, as inline PTX, and
// the host's tensor-map encoder.  sm_103a only.
//
// A pair works on one tile: each CTA holds half of the A rows and half of the
// B rows in its shared memory, the even ("leading") CTA's one thread issues
// the products for both, and each CTA's tensor memory receives its own 128
// rows of the result.
#pragma once

#include <cuda.h>

#include "ep_device.cuh"

namespace ep {

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// All threads of the cluster; memory operations before it are visible after.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The shared::cluster address, in CTA `rank`, of this CTA's shared address.
__device__ __forceinline__ uint32_t map_shared(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

// An arrival at another CTA's barrier that does not order this thread's memory
// operations (a release to the cluster first waits for all its stores to
// global memory).
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// For shared memory that this CTA's products read: its writes were handed to
// the asynchronous proxy by fence_proxy_async_smem, so the arrival needs no
// more than CTA scope (at cluster scope it costs about 2 us with the wait).
__device__ __forceinline__ void mbar_arrive_cluster_local(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

__device__ __forceinline__ void fence_cluster() { asm volatile("fence.acq_rel.cluster;" ::: "memory"); }

__device__ __forceinline__ void store_cluster(uint32_t cluster_addr, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(cluster_addr), "f"(v.x), "f"(v.y), "f"(v.z),
               "f"(v.w)
               : "memory");
}

// Done when it returns: whoever is told of it afterwards sees the new value.
__device__ __forceinline__ void atom_max_cluster(uint32_t cluster_addr, int v) {
  int old;
  asm volatile("atom.acq_rel.cluster.shared::cluster.max.s32 %0, [%1], %2;" : "=r"(old) : "r"(cluster_addr), "r"(v) : "memory");
}

__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t *bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return done != 0;
}

// As mbar_wait_bounded, but the timer (slow to read, where these waits are
// taken once a step) is looked at after every 1024th try only.  kCluster:
// what the other CTA of a pair wrote before it arrived is visible after.
template <bool kCluster>
__device__ __forceinline__ bool mbar_wait_tries(uint64_t *bar, uint32_t parity) {
  uint64_t t0 = 0;
  for (uint32_t i = 1; !(kCluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)); ++i) {
    if (i % 1024 == 0) {
      const uint64_t now = global_timer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > kWaitLimitNs) return false;
    }
  }
  return true;
}

__device__ __forceinline__ bool mbar_wait_pair(uint64_t *bar, uint32_t parity) {
  return mbar_wait_tries<false>(bar, parity);
}

__device__ __forceinline__ bool mbar_wait_cluster(uint64_t *bar, uint32_t parity) {
  return mbar_wait_tries<true>(bar, parity);
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// Tile copies to this CTA's shared memory that complete on the barrier at the
// shared::cluster address `bar` (this CTA's or its pair's).  x must keep the
// source 16-byte aligned; coordinates past an end read zeros.
__device__ __forceinline__ void tile_load_2d(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void tile_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void tile_load_4d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w,
                                             uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

// A tile from shared memory (in the map's swizzle); what lies past an end is
// not written.  Coordinates must not be negative.
__device__ __forceinline__ void tile_store_3d(const CUtensorMap *map, uint32_t src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(x),
               "r"(y), "r"(z), "r"(src)
               : "memory");
}

// 16 bytes to shared memory, zeros unless `some` (src is then not read).
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool some) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(some ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ------------------------------------------------------------------ tcgen05

// Tensor memory for the pair (a whole warp of each CTA calls it); the column
// address is written to *dst.
__device__ __forceinline__ void tmem_alloc_pair(uint32_t *dst, uint32_t columns) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst)), "r"(columns)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}

__device__ __forceinline__ void tmem_free_pair(uint32_t addr, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns));
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// One thread of a converged warp.  The loops that issue copies and products
// run on the whole warp, so what they compute stays in uniform registers, and
// only the instruction itself is left to this thread.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// d (+)= a b^T over 16 elements of the inner dimension, bf16 in, fp32 sums.
// The operands' descriptors as a low word (address, block distance) and the
// high word they share.
__device__ __forceinline__ void mma_pair(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)add), "n"(0x40004040)
      : "memory");
}

// Arrives on the barrier at this offset in the CTAs of `mask` (both of the
// pair) once the products issued so far are done.
__device__ __forceinline__ void commit_pair(uint64_t *bar, uint32_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_addr(bar)),
      "h"((uint16_t)mask)
      : "memory");
}

// The same for a CTA by itself (128 rows of A).

__device__ __forceinline__ void tile_load_one(uint32_t dst, const CUtensorMap *map, int x, int y, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
      : "memory");
}

__device__ __forceinline__ void tmem_alloc_one(uint32_t *dst, uint32_t columns) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst)), "r"(columns)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}

__device__ __forceinline__ void tmem_free_one(uint32_t addr, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns));
}

__device__ __forceinline__ void mma_one(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)add), "n"(0x40004040)
      : "memory");
}

__device__ __forceinline__ void commit_one(uint64_t *bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}

// 32 columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_load32(uint32_t addr, float (&v)[32]) {
  uint32_t *r = reinterpret_cast<uint32_t *>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// Low words of operand descriptors, 128-byte swizzle (high word: groups of 8
// rows 1024 bytes apart, version, swizzle).  inner_desc: inner dimension
// contiguous, rows of 128 bytes.  outer_desc: outer dimension contiguous,
// blocks of 64 outer elements (128 bytes), `block` bytes apart, each one row
// per inner element.  A shared address carries the CTA's rank in the cluster
// above its low 18 bits, which must not reach the block distance.
__device__ __forceinline__ uint32_t inner_desc(uint32_t addr) { return ((addr & 0x3ffffu) >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t outer_desc(uint32_t addr, uint32_t block) {
  return ((addr & 0x3ffffu) >> 4) | ((block >> 4) << 16);
}

// Instruction descriptor: bf16 x bf16 -> fp32, M = 256 over the pair, N
// columns; bit 15 / 16: A / B with the outer dimension contiguous.
__host__ __device__ constexpr uint32_t mma_desc(int n, bool a_outer, bool b_outer) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((a_outer ? 1u : 0u) << 15) | ((b_outer ? 1u : 0u) << 16) |
         ((uint32_t)(n >> 3) << 17) | (16u << 24);
}

// The same for M = 128 on one CTA, inner dimensions contiguous.
__host__ __device__ constexpr uint32_t mma_desc_one(int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (8u << 24);
}

// --------------------------------------------------------------------- host

// A tensor map of bf16 elements, innermost dimension first (contiguous; the
// others' strides in bytes, multiples of 16), with the 128-byte swizzle.
ep_status_t encode_map(CUtensorMap *map, const void *base, int rank, const uint64_t *dims, const uint64_t *strides,
                       const uint32_t *box);

}  // namespace ep
