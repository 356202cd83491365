// common.cuh -- what the attention block's kernels share: the parameter
// structures, the checked reads of lengths and page numbers, and the launch
// helpers of their host side.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "../../include/nvfp4_attention.h"
#include "../csrc/ptx.cuh"

namespace nvfp4 {
namespace attn {

// Rows of heads: element (token, head, i) at data[token * ts + head * hs + i].
struct Heads {
  __nv_bfloat16* data;
  int64_t ts, hs;
};

struct Cache {
  void* k;
  void* v;
  const float* k_scale;
  const float* v_scale;
  int64_t pages;
  int64_t ks[3], vs[3];   // page, slot and head strides in elements
  int page_size, heads, dim;
  int e4m3;
};

struct Seqs {
  const int32_t* table;
  const int32_t* kv_lens;
  const int32_t* q_starts;
  int count, width;
  int tokens;
  int64_t max_kv;          // width * page_size
};

struct SeqInfo {
  int q0, q_len, kv_len;
};

// The lengths of sequence s, or an empty sequence (and the error bit) where
// they do not lie within the token dimension or the block table.
__device__ __forceinline__ SeqInfo load_seq(const Seqs& q, int s, unsigned int* err) {
  const int a = q.q_starts[s], b = q.q_starts[s + 1], n = q.kv_lens[s];
  if (a < 0 || b < a || b > q.tokens || n < 0 || n > q.max_kv) {
    atomicOr(err, NVFP4_ATTENTION_BAD_INDEX);
    return SeqInfo{0, 0, 0};
  }
  return SeqInfo{a, b - a, n};
}

// Page number of a block-table entry; `pages` (one past the last page, which
// no access is made to) and the error bit where it is out of range.
__device__ __forceinline__ int64_t checked_page(int32_t page, int64_t pages, unsigned int* err) {
  if (page < 0 || page >= pages) {
    atomicOr(err, NVFP4_ATTENTION_BAD_INDEX);
    return pages;
  }
  return page;
}

__device__ __forceinline__ float e4m3_to_f32(uint8_t v) {
  __nv_fp8_e4m3 x;
  x.__x = v;
  return static_cast<float>(x);
}

// Two e4m3 codes (low half of v) as f16x2: exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v) {
  uint32_t d;
  asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}"
      : "=r"(d)
      : "r"(v));
  return d;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// ---------------------------------------------------------------- host side
constexpr int kMaxDevices = 64;

struct Device {
  int id = 0;
  int num_sms = 0;
  unsigned int* err = nullptr;
};

// The current device's set-up (NVFP4_ERR_DEVICE where it is not sm_103).
int device(Device* out);

// Launch, in clusters of `cluster` CTAs, with programmatic stream
// serialization: every kernel here calls griddep_wait() before its first access
// to memory.
template <typename... P, typename... A>
int launch_clusters(int cluster, void (*kernel)(P...), dim3 grid, dim3 block, size_t smem,
                    cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kernel, P(args)...) != cudaSuccess) {
    cudaGetLastError();
    return NVFP4_ERR_LAUNCH;
  }
  return NVFP4_OK;
}

template <typename... P, typename... A>
int launch(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
           const A&... args) {
  return launch_clusters(1, kernel, grid, block, smem, stream, args...);
}

// Let `kernel` use `bytes` of dynamic shared memory, once per device.
template <typename Kernel>
int allow_smem(Kernel kernel, int bytes, const Device& d, std::atomic<bool> (&ready)[kMaxDevices]) {
  if (ready[d.id].load(std::memory_order_acquire)) return NVFP4_OK;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) !=
      cudaSuccess) {
    cudaGetLastError();
    return NVFP4_ERR_LAUNCH;
  }
  ready[d.id].store(true, std::memory_order_release);
  return NVFP4_OK;
}

struct NormRope {
  Heads q, k, v, q_out, k_out;
  const __nv_bfloat16* q_weight;
  const __nv_bfloat16* k_weight;
  const float* cos_sin;
  const int64_t* positions;
  const int64_t* slots;      // with a cache
  Cache cache;
  int64_t tokens, max_position;
  int q_heads, kv_heads, dim, rot;
  int store;                 // key and value rows go to the cache
  float eps;
  unsigned int* err;
};
int run_norm_rope(const NormRope& p, const Device& d, cudaStream_t stream);

struct Attend {
  Heads q, out;
  Cache cache;
  Seqs seqs;
  int q_heads, group;        // group: query heads of one key/value head
  int max_q_len;
  float scale;
  float* lse;                // [tokens, q_heads] or null
  void* workspace;
  unsigned int* err;
};
int run_attend(const Attend& p, const Device& d, cudaStream_t stream);
int64_t attend_workspace(int head_dim, const Device& d);

struct Mass {
  Heads q;
  Cache cache;
  Seqs seqs;
  int q_heads, group, max_q_len;
  float scale;
  const float* lse;
  const float* mass;         // or null
  float* out;
  int64_t room;
  unsigned int* err;
};
int run_mass(const Mass& p, const Device& d, cudaStream_t stream);
int run_mass_tc(const Mass& p, const Device& d, cudaStream_t stream);

struct Evict {
  Cache from, to;
  const int32_t* table;
  const int32_t* kv_lens;
  const int32_t* to_table;
  int count, width, to_width;
  const float* mass;
  int64_t room;
  int keep, recent;
  int32_t* index;
  float* new_mass;
  int32_t* new_lens;
  unsigned int* err;
};
int run_evict(const Evict& p, const Device& d, cudaStream_t stream);

}  // namespace attn
}  // namespace nvfp4
