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
// elements by one group of heads by `box` tokens.
bool query_map(CUtensorMap* map, const Heads& q, int dim, int heads, int tokens, int group, int box);

// Shared-memory matrix descriptors, 128-byte swizzled rows, 8-row groups 1024
// bytes apart: the high word is the same for all, the low word the start
// address (in 16 bytes) and, for the MN-major V (d contiguous), the distance
// of the next 64 columns.  Advancing along k adds to the low word.
constexpr uint32_t kDescHi = (1024u >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) {
  return (addr >> 4 & 0x3FFFu) | (lbo >> 4) << 16;   // (the CTA's number is above)
}
__device__ __forceinline__ void umma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t id,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tmov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(id), "r"(accumulate), "r"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t id,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tmov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "r"(b_lo), "r"(id), "r"(accumulate), "r"(kDescHi)
      : "memory");
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mov.b64 z, {%6, %7};\n\tfma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int32_t c0, int32_t c1, int32_t c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

__device__ __forceinline__ void tma_load_page(void* dst, const CUtensorMap* map, uint64_t* bar,
                                              int32_t chunk, int32_t slot, int32_t head,
                                              int32_t page) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(0), "r"(slot), "r"(chunk),
      "r"(head), "r"(page)
      : "memory");
}

// rows: query rows of one key/value head in the longest sequence, at most 32.
int run_attend_warp(int rows, const Attend& p, const Device& d, cudaStream_t stream);
int64_t attend_warp_workspace(int head_dim, const Device& d);

// rows: as above, any number.
int run_attend_tc(int64_t rows, const Attend& p, const Device& d, cudaStream_t stream);
int64_t attend_tc_workspace(int head_dim, const Device& d);

}  // namespace attn
}  // namespace nvfp4
