// sv_tcgen05.cuh — the tensor-core and tensor-copy primitives of the key-value kernels:
// tensor memory, matrix instructions with their shared-memory descriptors, tiled copies.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "sv_device.cuh"

namespace sv {

// ---- tensor memory --------------------------------------------------------------------------
// One warp allocates (and later frees) `cols` columns, a power of two >= 32; the base address
// lands in shared memory.
__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(dst)),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols)
               : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// Sixteen consecutive columns of the warp's 32 lanes: v[c] of lane l is column c of lane l.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
        "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
        "=f"(v[14]), "=f"(v[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const float (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"f"(v[0]),
      "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]),
      "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]),
      "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// ---- matrix instructions --------------------------------------------------------------------
// A shared-memory operand descriptor. K-major with 128-byte swizzle: rows of 64 elements, sbo =
// bytes between groups of 8 rows (lbo unused). MN-major: lbo = bytes between blocks of one
// swizzle width along the row index, sbo = bytes between groups of 8 along the contraction.
constexpr uint32_t kSwizzle128 = 2, kSwizzle32 = 6;
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo,
                                              uint32_t swizzle) {
  return (uint64_t)((addr & 0x3ffffu) >> 4) | (uint64_t)(lbo >> 4) << 16 |
         (uint64_t)(sbo >> 4) << 32 | 1ull << 46 | (uint64_t)swizzle << 61;
}
// The instruction descriptor of kind::f16: fp32 accumulator, both operands bf16 or both fp16.
__device__ __forceinline__ uint32_t mma_desc(bool bf16, bool a_mn, bool b_mn, int M, int N) {
  return 1u << 4 | (bf16 ? 1u << 7 | 1u << 10 : 0u) | (a_mn ? 1u << 15 : 0u) |
         (b_mn ? 1u << 16 : 0u) | (uint32_t)(N >> 3) << 17 | (uint32_t)(M >> 4) << 24;
}
// D[tmem] (+)= A * B, 16 deep; issued by one thread.
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        bool accumulate) {
  asm volatile(
      "{ .reg .pred p;\n"
      "  setp.ne.b32 p, %4, 0;\n"
      "  tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
// Arrive on `bar` once every matrix instruction this thread issued so far has finished.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   smem_u32(bar))
               : "memory");
}

// ---- tiled copies ---------------------------------------------------------------------------
__device__ __forceinline__ void tile_g2s(void* dst, const CUtensorMap* map, uint64_t* bar, int x,
                                         int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
__device__ __forceinline__ void fence_proxy_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// ---- waits ------------------------------------------------------------------------------------
constexpr uint64_t kTileWaitNs = 2000000000ull;  // 2 s: far past any legitimate wait

// What the waits of a CTA share (in shared memory): whether it has given up, and a wait's limit.
struct Waits {
  int dead;
  uint64_t limit_ns;
};

// Wait for a phase of an mbarrier unless the CTA has given up; a wait that runs out makes the CTA
// give up. After that no wait blocks, every role leaves its loop and every CTA barrier is met; what
// the CTA owes is then written as NaN. (A wait that fails has seen or set `dead`.)
static __device__ __noinline__ bool wait_longer(uint64_t* bar, uint32_t parity,
                                                volatile Waits* w) {
  const uint64_t t0 = globaltimer_ns(), limit = w->limit_ns;
  for (;;) {
    if (mbar_try_wait(bar, parity)) return true;
    if (w->dead) return false;
    if (globaltimer_ns() - t0 > limit) {
      w->dead = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, volatile Waits* w) {
  return mbar_try_wait(bar, parity) || wait_longer(bar, parity, w);
}

}  // namespace sv
