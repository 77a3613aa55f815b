// Inline-PTX wrappers beside smla_sm100.cuh's: batched TMA tile loads, 8-bit
// MMAs with both operands in shared memory, MMAs of a CTA pair, packed fp32
// arithmetic, and a wait that is bounded in time.
#pragma once

#include "smla_sm100.cuh"

namespace smla {
namespace sm100 {

// 3-D tiled TMA load of the box at (x, y, z).
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* map, int32_t x, int32_t y,
                                            int32_t z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];"
      :: "r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void prefetch_tensormap(const void* map) {
  asm volatile("prefetch.tensormap [%0];" :: "l"(map) : "memory");
}

// D[tmem] (+)= A[smem] * B[smem]^T, e4m3 operands, fp32 accumulation, K = 32.
// Its instruction descriptor has the fields of idesc_f16_f32 (type code 0 is
// e4m3 in this kind).
__device__ __forceinline__ void mma_ss_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
      :: "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}

// ------------------------------------------------------------- CTA pairs
// Tensor memory of both CTAs of a pair (a warp of each takes part).
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
               :: "r"(smem_u32(dst_smem)), "r"(ncols) : "memory");
}
__device__ __forceinline__ void tmem_relinquish_pair() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(taddr), "r"(ncols)
               : "memory");
}

// D (+)= A * B^T over a pair's shared and tensor memories, fp16 operands,
// issued by its first CTA: each CTA holds half of A's rows and half of B's at
// the same offsets.  With M = 128 a CTA's 64 rows of D lie in its lanes 0..63
// (the first half of the columns) and 64..127 (the second).
__device__ __forceinline__ void mma_ss_f16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                                uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      :: "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}

// The same on e4m3 operands (K = 32), and on bf16 ones by idesc_bf16_f32.
__device__ __forceinline__ void mma_ss_f8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                               uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
      :: "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}
__host__ __device__ constexpr uint32_t idesc_bf16_f32(int M, int N) {
  return idesc_f16_f32(M, N, false, false) | (1u << 7) | (1u << 10);
}

// Arrive on the barrier at `bar`'s offset in both CTAs when every MMA this
// thread issued so far has completed.
__device__ __forceinline__ void mma_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
      :: "r"(smem_u32(bar)), "h"(uint16_t(3)) : "memory");
}

// Arrive on a barrier of a CTA of the cluster (an address from map_to_cta).  The
// release is the CTA's, so by the letter of the memory model it orders nothing
// for a thread of another CTA.  It is for two hand-overs to the thread that
// issues a pair's MMAs, which itself loads nothing of what it is told about:
//   * operands that this CTA's threads wrote to their own shared memory.  The
//     tensor cores read this CTA's half of them from that memory, the one place
//     where they are; a wider release would have no other copy to bring up to
//     date.  Every writing lane runs fence.proxy.async behind its stores and the
//     warp meets before one lane arrives, so at the arrival the stores are
//     done, as seen by that proxy.  (Bytes that TMA or cp.async brought: the
//     arriving warp has waited on the barrier of their completion.)
//   * tensor memory that this CTA's threads have read: the values are in
//     registers (tcgen05.wait::ld) and tcgen05.fence::before_thread_sync stands
//     before the arrival, after_thread_sync behind the issuing thread's wait.
// At the cluster's scope a release waits for memory accesses in flight on the SM:
// the tree decode's batch takes 2.96 ms instead of 2.07 when the writing warps do
// that, 2.38 when a warp without accesses of its own does it for them (for V and
// P together, 2.53 for each), 2.13 for K alone; 4001 rows through 4096 x 16384
// take 574 us instead of 273.
__device__ __forceinline__ void mbar_arrive_at(uint32_t addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" :: "r"(addr) : "memory");
}

// Two fp32 at once: a * b + c, a + b and a * b, each rounded once.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(lo), "r"(hi));
  return v;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ uint64_t timer_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

// Every wait is bounded in time; one that gives up raises the CTA's abort
// flag, so that its other roles stop waiting too, and `*error` gets `bit`.
constexpr uint64_t kWaitLimitNs = 2000000000ull;

__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity, volatile int* abort,
                                             unsigned* error, unsigned bit) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*abort) return false;
    if (timer_ns() - t0 > kWaitLimitNs) {
      atomicOr(error, bit);
      *abort = 1;
      return false;
    }
  }
  return true;
}

}  // namespace sm100
}  // namespace smla
