// Steps of a tensor-core pipeline that a whole warp walks together and one lane acts in: waits
// and predicated instructions without branches.  A lane's branch around them costs more than they
// do: with it a block of the 8-bit products took 1000 cycles, twice its multiplication.
#pragma once

#include "gemm.cuh"

namespace moe {

// Wait of a converged warp for a barrier's phase, at most WAIT_LIMIT_CYCLES: then, or once another
// role has given up, it raises the block's abort flag (with MOE_ERR_TIMEOUT in the status) and goes on.
// What follows stays in bounds whether the data came or not; roles look at the flag between tiles.
__device__ __forceinline__ void pipe_wait(uint64_t* bar, uint32_t parity, int* abort_flag, int32_t* status) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u64 t0, t1;\n\t.reg .u32 a;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%0], %1;\n\t"
      "@p bra DONE;\n\t"
      "mov.u64 t0, %%clock64;\n\t"
      "AGAIN:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%0], %1;\n\t"
      "@p bra DONE;\n\t"
      "ld.volatile.shared.u32 a, [%2];\n\t"
      "setp.ne.u32 q, a, 0;\n\t"
      "@q bra DONE;\n\t"
      "mov.u64 t1, %%clock64;\n\t"
      "sub.u64 t1, t1, t0;\n\t"
      "setp.lt.u64 q, t1, %5;\n\t"
      "@q bra AGAIN;\n\t"
      "mov.u32 a, 1;\n\t"
      "st.volatile.shared.u32 [%2], a;\n\t"
      "setp.ne.u64 q, %3, 0;\n\t"
      "@q atom.global.cas.b32 a, [%3], 0, %4;\n\t"
      "DONE:\n\t}" ::"r"(smem_u32(bar)),
      "r"(parity), "r"(smem_u32(abort_flag)), "l"(reinterpret_cast<uint64_t>(status)), "r"(static_cast<int>(MOE_ERR_TIMEOUT)),
      "l"(WAIT_LIMIT_CYCLES)
      : "memory");
}

// Both of two barriers, asked together: their latencies overlap.
__device__ __forceinline__ void pipe_wait_two(uint64_t* bar0, uint32_t parity0, uint64_t* bar1, uint32_t parity1, int* abort_flag,
                                              int32_t* status) {
  uint32_t both;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 q, [%3], %4;\n\t"
      "and.pred p, p, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(both)
      : "r"(smem_u32(bar0)), "r"(parity0), "r"(smem_u32(bar1)), "r"(parity1)
      : "memory");
  if (__all_sync(0xffffffffu, both)) return;
  pipe_wait(bar0, parity0, abort_flag, status);
  pipe_wait(bar1, parity1, abort_flag, status);
}

// The lane with `act` not 0 does it.
__device__ __forceinline__ void pipe_arrive(uint64_t* bar, uint32_t act) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %1, 0;\n\t@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(smem_u32(bar)),
               "r"(act)
               : "memory");
}
__device__ __forceinline__ void pipe_arrive_cluster(uint32_t cluster_addr, uint32_t act) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %1, 0;\n\t@p mbarrier.arrive.shared::cluster.b64 _, [%0];\n\t}" ::"r"(cluster_addr),
               "r"(act)
               : "memory");
}
__device__ __forceinline__ void pipe_expect(uint64_t* bar, uint32_t bytes, uint32_t act) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t@p mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(smem_u32(bar)),
      "r"(bytes), "r"(act)
      : "memory");
}
__device__ __forceinline__ void pipe_load_2d(void* dst, const void* tmap, uint64_t* bar, int32_t x, int32_t y, uint32_t act) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "@p cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];\n\t}" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(act)
      : "memory");
}
__device__ __forceinline__ void pipe_load_2d_pair(void* dst, const void* tmap, uint32_t mbar_cluster, int32_t x, int32_t y, uint32_t act) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "@p cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];\n\t}" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(mbar_cluster), "r"(x), "r"(y), "r"(act)
      : "memory");
}
__device__ __forceinline__ void pipe_commit(uint64_t* bar, uint32_t act) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %1, 0;\n\t"
      "@p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(act)
      : "memory");
}
__device__ __forceinline__ void pipe_commit_pair_mc(uint64_t* bar, uint16_t mask, uint32_t act) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t"
      "@p tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(smem_u32(bar)),
      "h"(mask), "r"(act)
      : "memory");
}
// One K = 32 step of E4M3 operands (kind::f8f6f4), fp32 sums.
__device__ __forceinline__ void pipe_mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate,
                                            uint32_t act) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(act)
      : "memory");
}
// One K = 16 step of 16-bit operands across a CTA pair.
__device__ __forceinline__ void pipe_mma_f16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate,
                                                  uint32_t act) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(act)
      : "memory");
}

}  // namespace moe
