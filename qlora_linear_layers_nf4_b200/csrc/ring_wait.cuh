// mbarrier waits (bounded, as tc::mbar_wait) and the elected lane of the expert kernels.
#pragma once

#include "tc_common.cuh"

namespace nf4 {
namespace expert {

// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(p));
  return p != 0;
}

// The first 1024-byte boundary of dynamic shared memory.  An offset added to the array
// keeps its accesses shared-memory instructions; rounding the pointer as an integer
// would make them generic ones, with 64-bit addresses.
__device__ __forceinline__ uint8_t* align_1024(uint8_t* smem_raw) {
  return smem_raw + ((0u - tc::smem_u32(smem_raw)) & 1023u);
}

// A try_wait that may suspend the thread for up to `hint_ns` before it answers:
// waiting warps then take few issue slots from the working ones.
__device__ __forceinline__ bool try_wait_hint(uint64_t* bar, uint32_t parity, uint32_t hint_ns) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(tc::smem_u32(bar)), "r"(parity), "r"(hint_ns)
      : "memory");
  return ok != 0;
}

// SLEEP: nanoseconds between polls of a wait that is long by nature.
template <int SLEEP = 0>
__device__ __forceinline__ bool ring_wait(uint64_t* bar, uint32_t parity, volatile uint32_t* abort_flag,
                                          uint32_t* status) {
  if (tc::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = tc::globaltimer();
  uint32_t polls = 0;
  while (true) {
    if (try_wait_hint(bar, parity, 2000u)) return true;
    if (SLEEP) __nanosleep(SLEEP);
    if ((++polls & 63u) == 0) {
      if (*abort_flag) return false;
      if (tc::globaltimer() - t0 > tc::kWaitLimitNs) {
        *abort_flag = 1u;
        report(status, NF4_ERR_TIMEOUT);
        return false;
      }
    }
  }
}

// The wait of a whole warp: one lane polls.
template <int SLEEP = 0>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile uint32_t* abort_flag,
                                          uint32_t* status) {
  bool ok = true;
  if ((threadIdx.x & 31) == 0) ok = ring_wait<SLEEP>(bar, parity, abort_flag, status);
  return __shfl_sync(0xffffffffu, int(ok), 0) != 0;
}

}  // namespace expert
}  // namespace nf4
