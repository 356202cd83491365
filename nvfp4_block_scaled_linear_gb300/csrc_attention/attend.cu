// attend.cu -- the choice of the attention kernel, and the tensor maps.
#include <algorithm>
#include <cstring>
#include <mutex>

#include <cudaTypedefs.h>

#include "attend.cuh"

namespace nvfp4 {
namespace attn {
namespace {

// Encoding a tensor map costs microseconds of host time, so encoded maps are
// kept in a small direct-mapped cache.  The key holds every encoding input,
// so a hit is always valid.
struct MapKey {
  const void* base;
  uint64_t dims[5], strides[4];
  uint32_t box[5];
  int32_t rank, bytes, zero; // bytes of an element
};
struct MapSlot {
  MapKey key;
  CUtensorMap map;
};
constexpr int kMapSlots = 256;
MapSlot g_maps[kMapSlots];
std::mutex g_map_mutex;
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

bool encode(CUtensorMap* map, const MapKey& key) {
  uint64_t h = 0;
  const unsigned char* bytes = reinterpret_cast<const unsigned char*>(&key);
  for (size_t i = 0; i + 8 <= sizeof(key); i += 8) {
    uint64_t w;
    std::memcpy(&w, bytes + i, 8);
    h = (h ^ w) * 0x9E3779B97F4A7C15ull;
    h ^= h >> 29;
  }
  std::lock_guard<std::mutex> lock(g_map_mutex);
  MapSlot& slot = g_maps[h % kMapSlots];
  if (slot.key.rank == 0 || std::memcmp(&slot.key, &key, sizeof(key)) != 0) {
    if (!g_encode) {
      void* fn = nullptr;
      cudaDriverEntryPointQueryResult q;
      if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                           &q) != cudaSuccess ||
          q != cudaDriverEntryPointSuccess || !fn) {
        cudaGetLastError();
        return false;
      }
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }
    cuuint64_t dims[5], strides[4];
    cuuint32_t box[5];
    const cuuint32_t unit[5] = {1, 1, 1, 1, 1};
    for (int i = 0; i < 5; ++i) dims[i] = key.dims[i], box[i] = key.box[i];
    for (int i = 0; i < 4; ++i) strides[i] = key.strides[i];
    CUtensorMap fresh;
    if (g_encode(&fresh,
                 key.bytes == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                 key.rank, const_cast<void*>(key.base), dims, strides, box, unit,
                 CU_TENSOR_MAP_INTERLEAVE_NONE,
                 key.box[0] * key.bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                               : CU_TENSOR_MAP_SWIZZLE_64B,
                 CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                 CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return false;
    slot.key = key;
    slot.map = fresh;
  }
  *map = slot.map;
  return true;
}

}  // namespace

bool page_map(CUtensorMap* map, const Cache& c, bool values, int inner, int rows, int chunks) {
  const int64_t* st = values ? c.vs : c.ks;
  const int size = c.e4m3 ? 1 : 2;
  MapKey key;
  std::memset(&key, 0, sizeof(key));
  key.base = values ? c.v : c.k;
  key.rank = 5;
  key.bytes = size;
  key.dims[0] = inner, key.dims[1] = c.page_size, key.dims[2] = c.dim / inner;
  key.dims[3] = c.heads, key.dims[4] = c.pages;
  key.strides[0] = st[1] * size, key.strides[1] = inner * size;
  key.strides[2] = st[2] * size, key.strides[3] = st[0] * size;
  key.box[0] = inner, key.box[1] = rows, key.box[2] = chunks, key.box[3] = 1, key.box[4] = 1;
  return encode(map, key);
}

bool query_map(CUtensorMap* map, const Heads& q, int dim, int heads, int tokens, int group, int box) {
  MapKey key;
  std::memset(&key, 0, sizeof(key));
  key.base = q.data;
  key.rank = 3;
  key.bytes = 2;
  key.dims[0] = dim, key.dims[1] = heads, key.dims[2] = tokens;
  key.strides[0] = q.hs * 2, key.strides[1] = q.ts * 2;
  key.box[0] = 64, key.box[1] = group, key.box[2] = box;
  return encode(map, key);
}

int64_t attend_workspace(int head_dim, const Device& d) {
  return std::max(attend_warp_workspace(head_dim, d), attend_tc_workspace(head_dim, d));
}

bool countable(const Seqs& s, int heads, const Plan& p) {
  const double items = double(heads) * (double(s.tokens) / p.tile_tokens + s.count);
  return items * (double(s.max_kv >> p.unit_shift) + 1 + p.extra) < 4294967296.0;
}

int run_attend(const Attend& p, const Device& d, cudaStream_t stream) {
  const int64_t rows = int64_t(std::max(1, p.max_q_len)) * p.group;
  // The warp MMA costs some 34 cycles for each 16 x 8 x 16 on an SM quarter, so
  // its time grows with every 16 rows where that of the tcgen05 kernel stands
  // still.  Over 32771 keys of 256: 5 tokens x 6 heads (30 rows) 39 us against 52,
  // 7 tokens (42 rows) 68 against 52; over e4m3 pages, which the tcgen05 kernel
  // has to widen in shared memory, 42 against 64 and 78 against 65.
  return rows <= 32 ? run_attend_warp(static_cast<int>(rows), p, d, stream)
                    : run_attend_tc(rows, p, d, stream);
}

}  // namespace attn
}  // namespace nvfp4
