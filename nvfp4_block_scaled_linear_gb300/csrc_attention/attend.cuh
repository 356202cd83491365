// attend.cuh -- what the attention kernels share beyond the schedule: the
// page tensor maps, the 4-D copy, and the entry points of each kernel.
#pragma once
#include <cuda_fp16.h>

#include "schedule.cuh"

namespace nvfp4 {
namespace attn {

// Wait for the phase with the given parity; given up after 2^31 clock ticks
// (about a second), or at once when another wait of the block was, with
// `abort_flag` set and false returned.  Little code, since it is inlined in
// every role of kernels that have to stay within the instruction cache.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint32_t t0 = static_cast<uint32_t>(clock());
#pragma unroll 1
  while (!mbar_try_wait(bar, parity)) {
    if (*abort_flag || static_cast<uint32_t>(clock()) - t0 > 0x7FFFFFFFu) {
      *abort_flag = 1;
      return false;
    }
  }
  return true;
}

// Tensor map of the cache's key or value pages, dimensions (element of a
// chunk, slot, chunk, head, page), for boxes of `rows` slots by `chunks` chunks
// of `inner` elements (64 or 128 bytes, swizzled to that width): chunk after
// chunk in shared memory, each `rows` rows of that width.
bool page_map(CUtensorMap* map, const Cache& c, bool values, int inner, int rows, int chunks);

// Tensor map of the queries, dimensions (element, head, token), for boxes of 64
// elements by one group of heads by `tokens` tokens.
bool query_map(CUtensorMap* map, const Attend& a, int tokens);

// kCluster = 2: into both CTAs of the pair, each told on its own barrier.
template <int kCluster = 1>
__device__ __forceinline__ void tma_load_page(void* dst, const CUtensorMap* map, uint64_t* bar,
                                              int32_t chunk, int32_t slot, int32_t head,
                                              int32_t page) {
  if (kCluster == 1)
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(0), "r"(slot), "r"(chunk),
        "r"(head), "r"(page)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".multicast::cluster [%0], [%1, {%3, %4, %5, %6, %7}], [%2], %8;" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(0), "r"(slot), "r"(chunk),
        "r"(head), "r"(page), "h"(static_cast<uint16_t>((1 << kCluster) - 1))
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
