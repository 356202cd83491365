// attend.cu -- attention of new tokens over the paged cache, one warp per
// token and query head: the plain order of the formula with a running
// maximum and sum, every key row read from the cache as it is needed.
#include <algorithm>
#include <cstring>
#include <mutex>

#include <cudaTypedefs.h>

#include "attend.cuh"

namespace nvfp4 {
namespace attn {
namespace {

constexpr int kThreads = 128;

// Element i of a cache row.
__device__ __forceinline__ float cache_at(const void* base, int64_t off, int e4m3) {
  return e4m3 ? e4m3_to_f32(static_cast<const uint8_t*>(base)[off])
              : __bfloat162float(static_cast<const __nv_bfloat16*>(base)[off]);
}

template <int kDim>
__global__ void __launch_bounds__(kThreads) attend_kernel(const Attend p) {
  constexpr int kPer = kDim / 32;
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t(blockIdx.x) * kThreads + threadIdx.x) >> 5;
  const int t = static_cast<int>(w / p.q_heads), h = static_cast<int>(w % p.q_heads);
  if (t >= p.seqs.tokens) return;
  // the sequence that holds token t
  int s = -1;
  SeqInfo si{0, 0, 0};
  for (int i = 0; i < p.seqs.count; ++i) {
    si = load_seq(p.seqs, i, p.err);
    if (t >= si.q0 && t < si.q0 + si.q_len) {
      s = i;
      break;
    }
  }
  if (s < 0) return;
  const int kvh = h / p.group;
  const int seen = min(si.kv_len, si.kv_len - si.q_len + (t - si.q0) + 1);
  const float ks = p.cache.k_scale ? p.cache.k_scale[kvh] : 1.f;
  const float vs = p.cache.v_scale ? p.cache.v_scale[kvh] : 1.f;
  float q[kPer], o[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    q[i] = __bfloat162float(p.q.data[t * p.q.ts + h * p.q.hs + i * 32 + lane]) * p.scale * ks;
    o[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < seen; ++j) {
    const int64_t page = checked_page(
        p.seqs.table[int64_t(s) * p.seqs.width + j / p.cache.page_size], p.cache.pages, p.err);
    if (page == p.cache.pages) continue;
    const int in = j % p.cache.page_size;
    const int64_t ko = page * p.cache.ks[0] + in * p.cache.ks[1] + kvh * p.cache.ks[2] + lane;
    const int64_t vo = page * p.cache.vs[0] + in * p.cache.vs[1] + kvh * p.cache.vs[2] + lane;
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) x = fmaf(q[i], cache_at(p.cache.k, ko + i * 32, p.cache.e4m3), x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    const float top = fmaxf(m, x);
    const float a = m == top ? 1.f : expf(m - top), e = expf(x - top);
    l = l * a + e;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      o[i] = o[i] * a + e * cache_at(p.cache.v, vo + i * 32, p.cache.e4m3);
    m = top;
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    p.out.data[t * p.out.ts + h * p.out.hs + i * 32 + lane] =
        __float2bfloat16_rn(seen > 0 ? o[i] * vs / l : 0.f);
  if (p.lse && lane == 0)
    p.lse[int64_t(t) * p.q_heads + h] = seen > 0 ? m + logf(l) : -INFINITY;
}

}  // namespace

int64_t attend_workspace(int head_dim, const Device& d) {
  return attend_warp_workspace(head_dim, d);
}

// Encoding a tensor map costs microseconds of host time, so encoded maps are
// kept in a small direct-mapped cache.  The key holds every encoding input,
// so a hit is always valid.
bool page_map(CUtensorMap* map, const Cache& c, bool values, int inner, int rows) {
  struct Key {
    const void* base;
    int64_t pages, stride[3];
    int page_size, heads, dim, e4m3, inner, rows;
  };
  struct Slot {
    Key key;
    CUtensorMap map;
  };
  static Slot slots[64];
  static std::mutex mutex;
  static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  const int64_t* st = values ? c.vs : c.ks;
  Key key;
  std::memset(&key, 0, sizeof(key));
  key.base = values ? c.v : c.k;
  key.pages = c.pages;
  for (int i = 0; i < 3; ++i) key.stride[i] = st[i];
  key.page_size = c.page_size, key.heads = c.heads, key.dim = c.dim, key.e4m3 = c.e4m3;
  key.inner = inner, key.rows = rows;
  uint64_t h = reinterpret_cast<uintptr_t>(key.base) >> 4;
  h ^= uint64_t(c.pages) * 0x9E3779B97F4A7C15ull ^ uint64_t(inner) << 9 ^ uint64_t(rows) << 17;
  h ^= h >> 29;
  std::lock_guard<std::mutex> lock(mutex);
  Slot& slot = slots[h % 64];
  if (std::memcmp(&slot.key, &key, sizeof(key)) != 0) {
    if (!encode) {
      void* fn = nullptr;
      cudaDriverEntryPointQueryResult q;
      if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                           &q) != cudaSuccess ||
          q != cudaDriverEntryPointSuccess || !fn) {
        cudaGetLastError();
        return false;
      }
      encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }
    const int size = c.e4m3 ? 1 : 2;
    const cuuint64_t dims[4] = {cuuint64_t(c.dim), cuuint64_t(c.page_size), cuuint64_t(c.heads),
                                cuuint64_t(c.pages)};
    const cuuint64_t strides[3] = {cuuint64_t(st[1] * size), cuuint64_t(st[2] * size),
                                   cuuint64_t(st[0] * size)};
    const cuuint32_t box[4] = {cuuint32_t(inner), cuuint32_t(rows), 1, 1};
    const cuuint32_t unit[4] = {1, 1, 1, 1};
    CUtensorMap fresh;
    if (encode(&fresh, c.e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
               const_cast<void*>(key.base), dims, strides, box, unit,
               CU_TENSOR_MAP_INTERLEAVE_NONE,
               inner * size == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return false;
    slot.key = key;
    slot.map = fresh;
  }
  *map = slot.map;
  return true;
}

int run_attend(const Attend& p, const Device& d, cudaStream_t stream) {
  const int64_t rows = int64_t(std::max(1, p.max_q_len)) * p.group;
  if (rows <= 64) return run_attend_warp(static_cast<int>(rows), p, d, stream);
  const int64_t blocks = (int64_t(p.seqs.tokens) * p.q_heads * 32 + kThreads - 1) / kThreads;
  if (blocks > INT32_MAX) return NVFP4_ERR_SHAPE;
  auto* kernel = p.cache.dim == 256   ? attend_kernel<256>
                 : p.cache.dim == 128 ? attend_kernel<128>
                                      : attend_kernel<64>;
  return launch(kernel, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, stream, p);
}

}  // namespace attn
}  // namespace nvfp4
