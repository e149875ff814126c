// Asynchronous copies into a thread's own shared memory and the exchange of values between the blocks
// of a cluster, for the elementwise scan.
#pragma once

#include "sm100.cuh"

namespace gla {
namespace cluster {

// BYTES (4 or 8) from global to shared memory; zeros when `in` is false (src is then not read).
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool in) {
  const int n = in ? BYTES : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(n) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

__device__ __forceinline__ uint32_t block_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// The address, in the shared memory of block `rank` of the cluster, of this block's address `a`.
__device__ __forceinline__ uint32_t peer(uint32_t a, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}
// Store four floats in a peer's shared memory (16-byte aligned); they count 16 bytes on the peer's mbarrier when they
// arrive.
__device__ __forceinline__ void store_async(uint32_t at, float x, float y, float z, float w, uint32_t bar) {
  asm volatile(
      "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(at),
      "r"(__float_as_uint(x)), "r"(__float_as_uint(y)), "r"(__float_as_uint(z)), "r"(__float_as_uint(w)), "r"(bar)
      : "memory");
}
// Wait (about a second at most, then the latch is set and false returned) for a phase whose data
// comes from other blocks of the cluster.
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, unsigned int* latch) {
  const uint64_t t0 = sm100::globaltimer_ns();
  while (true) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
    if (sm100::globaltimer_ns() - t0 > sm100::kWaitLimitNs) {
      if (latch) atomicCAS(latch, 0u, sm100::kErrTimeout);
      return false;
    }
  }
}

}  // namespace cluster
}  // namespace gla
