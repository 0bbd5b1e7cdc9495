// tc_pair.cuh -- tcgen05 on a pair of CTAs (cta_group::2): the two CTAs of a
// cluster share one product.  With M = 128 each CTA holds 64 rows of A and half
// of B's N rows in its own shared memory at the same offsets, one thread of the
// even CTA issues, and each CTA's tensor memory receives its 64 rows: lanes 0-63
// columns [0, N/2), lanes 64-127 (the same rows) columns [N/2, N); with M = 256 each holds
// 128 rows of A, and its tensor memory receives them as a CTA's own product would.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "pskv_internal.cuh"
#include "tc_common.cuh"

namespace pskv {
namespace tc2 {

// Operations of one thread take `lead` and are predicated on it: the warp that issues them
// stays together, and addresses and descriptors stay in uniform registers (inside a branch of one
// thread the same instructions ran several times slower).

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// The same shared-memory offset in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_to(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}

// Handing over to the warp of the even CTA that issues the products, by arrivals on its barriers:
// - tensor memory (scores read, P written): each tcgen05 access is waited for and fenced
//   (tcgen05.fence::before_thread_sync), the other side fences behind its wait; only the order of
//   execution crosses, so the arrivals are relaxed.
// - shared memory (P, zeroed rows: written, made visible to the tensor core by
//   fence.proxy.async, and read by a product that the other CTA issues): a release and an
//   acquire at cluster scope.  The fences are those restricted to shared memory: a
//   release of all memory waits for a barrier of ~700 cycles, every tile (8 rows of 10,602 keys
//   under 128 heads: 41.3 us against 37.6).

// Arrive on a barrier of any CTA of the cluster, handing over nothing but the order.
__device__ __forceinline__ void arrive_pair(uint32_t bar, bool lead) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n\t}" ::"r"(bar),
      "r"((uint32_t)lead)
      : "memory");
}

// The same behind what this warp read or wrote in its own CTA's shared memory (all lanes
// call, converged).
__device__ __forceinline__ void arrive_pair_release(uint32_t bar, bool lead) {
  asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
  arrive_pair(bar, lead);
}

// tc::all_wait for arrivals of the other CTA's threads and copies.
__device__ __forceinline__ bool all_wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag,
                                         int32_t *status) {
  auto arrived = [&] {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
  };
  for (uint32_t i = 0; i < kWaitPolls; ++i) {
    if (__all_sync(0xffffffffu, arrived())) {
      asm volatile("fence.acquire.sync_restrict::shared::cluster.cluster;" ::: "memory");
      return true;
    }
    if ((i & 15u) == 15u && __any_sync(0xffffffffu, *abort_flag != 0)) return false;
  }
  *abort_flag = 1;
  raise_fault(status, PSKV_FAULT_WAIT_TIMEOUT);
  return false;
}

// A value that is the same in every lane, known as such to the compiler.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// D[tmem] (+)= A * B over the pair.  The whole warp calls; the thread with `lead` (one of the
// even CTA's) issues.  Called so, in code that all lanes run alike, the descriptors stay in
// uniform registers.
__device__ __forceinline__ void mma(uint32_t tmem_d, uint64_t a, uint64_t b, uint32_t idesc,
                                    bool accumulate, bool lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"((uint32_t)lead));
}

// The same with A (each CTA's own rows, bf16 pairs per 32-bit column) read from tensor memory.
__device__ __forceinline__ void mma_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t b,
                                       uint32_t idesc, bool accumulate, bool lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"((uint32_t)lead));
}

// Arrive on `bar` of both CTAs once every tcgen05 operation the leading thread issued so far is complete.
__device__ __forceinline__ void commit_both(uint64_t *bar, bool lead) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;\n\t}" ::"r"(smem_u32(bar)),
      "h"((uint16_t)3), "r"((uint32_t)lead)
      : "memory");
}

// Tensor-memory allocation over the pair (one warp of each CTA), address written to *slot.
__device__ __forceinline__ void alloc(uint32_t *slot, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(slot)),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void dealloc(uint32_t tmem, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols)
               : "memory");
}

// The leading thread arrives and expects `bytes` more.
__device__ __forceinline__ void expect_tx(uint64_t *bar, uint32_t bytes, bool lead) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t.reg .b64 st;\n\tsetp.ne.b32 q, %2, 0;\n\t"
      "@q mbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n\t}" ::"r"(smem_u32(bar)),
      "r"(bytes), "r"((uint32_t)lead)
      : "memory");
}

// 3-D tensor copy global -> this CTA's shared memory, completion counted on a
// barrier of either CTA of the pair, by the leading thread.  x * 2 bytes is a multiple of 16.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y,
                                            int z, uint32_t bar, bool lead) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %6, 0;\n\t"
      "@q cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar), "r"((uint32_t)lead)
      : "memory");
}

// The same for a 4-D map.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int x, int y,
                                            int z, int w, uint32_t bar, bool lead) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %7, 0;\n\t"
      "@q cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar),
      "r"((uint32_t)lead)
      : "memory");
}

// Fetch a tensor map's descriptor ahead of its first use.
__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// Rows of `cols` bf16 as a 3-D tensor of 64-column slabs (64, rows, cols / 64): a box
// of box_rows rows and box_slabs slabs lands as that many 128-byte swizzled slabs.
inline bool make_slab_map(CUtensorMap *m, const void *base, long long rows, int cols, int box_rows,
                          int box_slabs) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tc::encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)(cols / 64)};
  const cuuint64_t strides[2] = {(cuuint64_t)cols * 2, 128};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, (cuuint32_t)box_slabs};
  const cuuint32_t elem[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box,
             elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The first 256 * blocks columns of the same rows as (64, rows, 4 slabs, blocks): a box of
// box_slabs neighbouring slabs of box_blocks blocks lands block by block.
inline bool make_block_map(CUtensorMap *m, const void *base, long long rows, int cols, int blocks,
                           int box_rows, int box_slabs, int box_blocks) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tc::encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[4] = {64, (cuuint64_t)rows, 4, (cuuint64_t)blocks};
  const cuuint64_t strides[3] = {(cuuint64_t)cols * 2, 128, 512};
  const cuuint32_t box[4] = {64, (cuuint32_t)box_rows, (cuuint32_t)box_slabs,
                             (cuuint32_t)box_blocks};
  const cuuint32_t elem[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box,
             elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace tc2
}  // namespace pskv
