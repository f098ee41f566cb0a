// Tensor memory, 5th generation tensor core instructions, tiled TMA loads and
// cluster barriers for sm_103a.  Inline PTX written for this library.
//
// kCtas: 1, or 2 where the blocks of a cluster of two work on one tile: a
// matrix instruction of cta_group::2, issued by the cluster's first block,
// reads both blocks' shared memory and writes both blocks' tensor memory.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "device.cuh"

namespace grs {

// One thread of a whole warp, always the same.  What it runs stays in code of
// the whole warp, whose addresses and counters the compiler then keeps in the
// registers that matrix and TMA instructions take them from.
__device__ __forceinline__ bool elected() {
  uint32_t is;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(is));
  return is != 0;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The address, in block `rank` of the cluster, of what lies at `addr` in this one.
__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

// Arrivals at a barrier of the cluster's other block.  What they announce is
// tensor memory that was read or a copy under way, which have orders of their
// own; cluster scope would make the thread wait for all its memory accesses
// (measured: a third of the products' rate).  remote_release is for plain writes.
__device__ __forceinline__ void remote_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void remote_release(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void remote_arrive_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// Writes of this thread to shared memory, visible to TMA and matrix instructions.
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ------------------------------------------------- blocks not yet launched
// Asks for the place of a cluster of this grid that has not begun, which then
// never will; the answer (16 bytes, aligned) comes to every block of the
// cluster and is counted by its barrier.  Not to be asked again after a no.
template <int kCtas>
__device__ __forceinline__ void ask_cluster(void* answer, uint64_t* bar) {
  if constexpr (kCtas == 1)
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(smem_addr(answer)),
                 "r"(smem_addr(bar))
                 : "memory");
  else
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.multicast::cluster::all.b128 [%0], [%1];" ::"r"(
            smem_addr(answer)),
        "r"(smem_addr(bar))
        : "memory");
}
// The first block of the cluster that the answer gives, -1 for none.
__device__ __forceinline__ int64_t cluster_given(const void* answer) {
  uint32_t yes, x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\tld.shared.b128 r, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "selp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, _, _, _}, r;\n\t}"
      : "=r"(yes), "=r"(x)
      : "r"(smem_addr(answer))
      : "memory");
  return yes ? int64_t(x) : -1;
}

// ------------------------------------------------------------- tiled TMA
__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}

// Boxes of a 2- or 3-dimensional tensor to shared memory; `bar` may be the
// cluster's first block's (kCtas 2).
template <int kCtas>
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, uint32_t bar) {
  if constexpr (kCtas == 1)
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
                 "l"(map), "r"(x), "r"(y), "r"(bar)
                 : "memory");
  else
    asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
                     dst),
                 "l"(map), "r"(x), "r"(y), "r"(bar)
                 : "memory");
}
template <int kCtas>
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z, uint32_t bar) {
  if constexpr (kCtas == 1)
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
                 "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
                 : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// A box of shared memory to (x, y, z) of a tensor, cut off at its extents; the
// thread that sends it waits: until what it sent has been read, or written.
__device__ __forceinline__ void tma_store(const CUtensorMap* map, uint32_t from, int32_t x, int32_t y, int32_t z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(x), "r"(y), "r"(z), "r"(from)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// ---------------------------------------------------------- tensor memory
// Columns [address, + n) of 128 lanes of 32 bits; one warp of each block.
template <int kCtas>
__device__ __forceinline__ void tmem_alloc(uint32_t* where, uint32_t columns) {
  if constexpr (kCtas == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(where)), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(where)), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int kCtas>
__device__ __forceinline__ void tmem_free(uint32_t address, uint32_t columns) {
  if constexpr (kCtas == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(address), "r"(columns) : "memory");
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(address), "r"(columns) : "memory");
}

__device__ __forceinline__ void tmem_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 columns of the warp's own 32 lanes (those of its number modulo 4), a lane a thread.
__device__ __forceinline__ void tmem_load32(uint32_t address, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, "
      "%20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]),
        "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]),
        "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]),
        "=r"(v[31])
      : "r"(address));
}
__device__ __forceinline__ void tmem_load8(uint32_t address, uint32_t (&v)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "r"(address));
}
// 32 columns of 16 lanes: as a matrix instruction's result, v[4 i ..] the eight
// columns from 8 i on: of lane t / 4 those from 2 (t % 4) on, two, and the same of
// lane t / 4 + 8, for thread t.
__device__ __forceinline__ void tmem_load_fragments(uint32_t address, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]),
        "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(address));
}
// Four 8 x 8 matrices of 16-bit numbers to shared memory, transposed: thread t
// has two neighbours of row t / 4 of each, and the address of row t % 8 of
// matrix t / 8 as it is stored.
__device__ __forceinline__ void store_transposed(uint32_t address, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(address), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void tmem_wait_load() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// -------------------------------------------------------- matrix product
// Operands in shared memory as TMA lays them out with the 128-byte swizzle:
// rows of 64 bf16 numbers, eight rows (1024 bytes) a swizzled group.  Along a
// row lies either k (kAlongK: rows are the other index) or the other index
// (rows are k; the next 64 of it lie `next64` bytes on).
// The descriptor's lower word has the address, which moves; its upper word stays.
template <bool kAlongK>
__device__ __forceinline__ uint32_t operand(uint32_t addr, uint32_t next64) {
  return (addr & 0x3FFFF) >> 4 | (kAlongK ? 1u : next64 >> 4) << 16;
}
constexpr uint32_t OPERAND_UPPER = 1024 >> 4 | 1u << 14 | 2u << 29;
// Bytes from one step of 16 along k to the next, in units of the descriptor's address.
template <bool kAlongK>
constexpr uint32_t operand_step = (kAlongK ? 32 : 16 * 128) >> 4;

// bf16 x bf16 to fp32, m x n.
__device__ __forceinline__ constexpr uint32_t product_desc(bool a_along_k, bool b_along_k, uint32_t m, uint32_t n) {
  return 1u << 4 | 1u << 7 | 1u << 10 | (a_along_k ? 0u : 1u << 15) | (b_along_k ? 0u : 1u << 16) | (n >> 3) << 17 | (m >> 4) << 24;
}

// d = a b, or d + a b; a and b: lower words of operands.
template <int kCtas>
__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint32_t b, uint32_t desc, bool add) {
  if constexpr (kCtas == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.u32 p, %4, 0;\n\tmov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(desc), "r"(uint32_t(add)), "r"(OPERAND_UPPER)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.u32 p, %4, 0;\n\tmov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(desc), "r"(uint32_t(add)), "r"(OPERAND_UPPER)
        : "memory");
}

// Arrives at `bar` (of both blocks, kCtas 2) when this thread's matrix instructions so far are done.
template <int kCtas>
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  if constexpr (kCtas == 1)
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_addr(bar)),
                 "h"(uint16_t(3))
                 : "memory");
}

}  // namespace grs
