// attend.cuh -- what the attention kernels share beyond the schedule: the
// page tensor maps, the 4-D copy, and the entry points of each kernel.
#pragma once
#include <cuda_fp16.h>

#include "schedule.cuh"

namespace nvfp4 {
namespace attn {

// Tensor map of the cache's key or value pages, dimensions (element, slot,
// head, page), for boxes of `inner` elements (64 or 128 bytes, swizzled to
// that width) by `rows` slots.
bool page_map(CUtensorMap* map, const Cache& c, bool values, int inner, int rows);

// Tensor map of the queries, dimensions (element, head, token), for boxes of 64
// elements by one group of heads by `tokens` tokens.
bool query_map(CUtensorMap* map, const Attend& a, int tokens);

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int32_t c0, int32_t c1, int32_t c2, int32_t c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(c0), "r"(c1), "r"(c2),
      "r"(c3)
      : "memory");
}

// rows: query rows of one key/value head in the longest sequence, at most 64.
int run_attend_warp(int rows, const Attend& p, const Device& d, cudaStream_t stream);
int64_t attend_warp_workspace(int head_dim, const Device& d);

// rows: as above, any number.
int run_attend_tc(int64_t rows, const Attend& p, const Device& d, cudaStream_t stream);
int64_t attend_tc_workspace(int head_dim, const Device& d);

}  // namespace attn
}  // namespace nvfp4
