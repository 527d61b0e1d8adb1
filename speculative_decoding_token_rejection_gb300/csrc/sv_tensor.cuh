// sv_tensor.cuh -- the tensor cores' own memory and products (tcgen05), and waits
// with a limit.
#pragma once

#include <cstdint>

#include "sv_device.cuh"

namespace sv {

// Columns of tensor memory (a power of two, 32 at least) for a CTA, by a whole warp, and the end of asking.
__device__ __forceinline__ void tmem_get(uint32_t *dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst)), "r"(cols)
               : "memory");
}
__device__ __forceinline__ void tmem_no_more() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_alloc(uint32_t *dst, uint32_t cols) {
  tmem_get(dst, cols);
  tmem_no_more();
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// D (tensor memory) = A B (+ D), both operands in shared memory.
template <bool ADD>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "n"(ADD ? 1 : 0)
      : "memory");
}
// The same with A in tensor memory.
template <bool ADD>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "n"(ADD ? 1 : 0)
      : "memory");
}
// One lane of a converged warp.
__device__ __forceinline__ bool elected() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// Arrives on `bar` once every product issued so far by this thread is done.
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// Waits for every load so far; the registers go through, so no use of them moves ahead of the wait.
__device__ __forceinline__ void tmem_wait_load(uint32_t r[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory operand with rows of 128 bytes (64 f16), 8-row groups of 1 KB,
// 16-byte columns exchanged within a group (column ^ row % 8).  `next64`:
// bytes from 64 elements to the next 64 where those run along the operand's
// outer dimension.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t next64) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFF) | static_cast<uint64_t>((next64 >> 4) & 0x3FFF) << 16 |
         static_cast<uint64_t>(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
// f16 operands, fp32 sums, m x n; an operand's outer dimension contiguous or its inner one.
__host__ __device__ constexpr uint32_t product(int n, bool b_outer_contiguous, int m = 128, bool a_outer_contiguous = false) {
  return 1u << 4 | (a_outer_contiguous ? 1u << 15 : 0u) | (b_outer_contiguous ? 1u << 16 : 0u) |
         static_cast<uint32_t>(n / 8) << 17 | static_cast<uint32_t>(m / 16) << 24;
}

__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
// A CTA whose waits ran out gives up: no wait begins anew, rows that are not
// done become NaN, and the status word says so at the end.  C has a word `abort`
// in shared memory.
template <typename C>
__device__ __forceinline__ void give_up(C &c) {
  *const_cast<volatile uint32_t *>(&c.abort) = 1;
  __threadfence_block();
}
template <typename C>
__device__ __forceinline__ bool gave_up(const C &c) {
  return *const_cast<const volatile uint32_t *>(&c.abort) != 0;
}
// Waits for phase `parity` of a barrier; false when the CTA gives up (a wait
// of two seconds, `expire`, or another thread that did).
constexpr uint32_t kWaitPolls = 1u << 24;
constexpr uint64_t kWaitNs = 2000000000ull;
template <typename C>
__device__ __forceinline__ bool wait(C &c, uint64_t *bar, uint32_t parity, bool expire = false) {
  if (!expire) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t began = now_ns();
    for (uint32_t it = 0; it < kWaitPolls; ++it) {
      if (mbar_try_wait(bar, parity)) return true;
      if (gave_up(c)) return false;
      if ((it & 15u) == 15u && now_ns() - began > kWaitNs) break;
    }
  }
  give_up(c);
  return false;
}
// The same for all lanes of a warp together.
template <typename C>
__device__ __forceinline__ bool wait_warp(C &c, uint64_t *bar, uint32_t parity, bool expire = false) {
  return __all_sync(0xFFFFFFFFu, wait(c, bar, parity, expire));
}
// Waits for what is in flight, also in a CTA that has given up: shared and
// tensor memory must not go before it.
template <typename C>
__device__ __forceinline__ void settle(C &c, uint64_t *bar, uint32_t parity) {
  const uint64_t began = now_ns();
  while (!mbar_try_wait(bar, parity))
    if (now_ns() - began > kWaitNs) {
      give_up(c);
      return;
    }
}

}  // namespace sv
