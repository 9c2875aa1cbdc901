// What the pair GEMMs (expert, gated) share: loads and arrivals of a CTA on barriers of
// the pair's leader.
#pragma once

#include "tc_common.cuh"

namespace nf4 {
namespace expert {

using tc::smem_u32;

// 3-D tiled load into this CTA whose bytes complete on the leader's barrier.
__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* map, uint32_t bar_cluster_addr,
                                                 int32_t x, int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster_addr), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Arrive on a barrier of the pair's leader, releasing at cluster scope: the waiter
// may be in the other CTA.  What the arrival announces are operand tiles in this
// CTA's shared memory, which fence.proxy.async has handed to the async proxy, or
// accumulators whose reads tcgen05.wait has completed.  So the release is restricted
// to this CTA's shared memory; a full one waits for every store in flight, the
// epilogue's output included (y of 8192 rows on 8 experts of 11008 x 4096: 894 us
// against 715).
__device__ __forceinline__ void arrive_leader(uint32_t cluster_addr) {
  asm volatile(
      "fence.release.sync_restrict::shared::cta.cluster;\n\t"
      "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
      : "memory");
}

}  // namespace expert
}  // namespace nf4
