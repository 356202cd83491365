// attend.cu -- the choice of the attention kernel, and the tensor maps.
#include <algorithm>

#include <cudaTypedefs.h>

#include "attend.cuh"

namespace nvfp4 {
namespace attn {
namespace {

using Encode = PFN_cuTensorMapEncodeTiled_v12000;

Encode find_encode() {
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                       &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess) {
    cudaGetLastError();
    return nullptr;
  }
  return reinterpret_cast<Encode>(fn);
}

// A map is encoded anew for each call: a few tenths of a microsecond.
bool encode(CUtensorMap* map, int rank, int bytes, void* base, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box) {
  static const Encode fn = find_encode();
  const cuuint32_t unit[5] = {1, 1, 1, 1, 1};
  return fn && fn(map,
                  bytes == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                  rank, base, dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  box[0] * bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool page_map(CUtensorMap* map, const Cache& c, bool values, int inner, int rows, int chunks) {
  const int64_t* st = values ? c.vs : c.ks;
  const int size = c.e4m3 ? 1 : 2;
  const cuuint64_t dims[5] = {cuuint64_t(inner), cuuint64_t(c.page_size), cuuint64_t(c.dim / inner),
                              cuuint64_t(c.heads), cuuint64_t(c.pages)};
  const cuuint64_t strides[4] = {cuuint64_t(st[1] * size), cuuint64_t(inner * size),
                                 cuuint64_t(st[2] * size), cuuint64_t(st[0] * size)};
  const cuuint32_t box[5] = {cuuint32_t(inner), cuuint32_t(rows), cuuint32_t(chunks), 1, 1};
  return encode(map, 5, size, values ? c.v : c.k, dims, strides, box);
}

bool query_map(CUtensorMap* map, const Heads& q, int dim, int heads, int tokens, int group, int box) {
  const cuuint64_t dims[3] = {cuuint64_t(dim), cuuint64_t(heads), cuuint64_t(tokens)};
  const cuuint64_t strides[2] = {cuuint64_t(q.hs * 2), cuuint64_t(q.ts * 2)};
  const cuuint32_t boxes[3] = {64, cuuint32_t(group), cuuint32_t(box)};
  return encode(map, 3, 2, q.data, dims, strides, boxes);
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
  // still.  Over 32771 keys of 256: 5 tokens x 6 heads (30 rows) 39 us against 50,
  // 7 tokens (42 rows) 68 against 51; over e4m3 pages, which the tcgen05 kernel
  // has to widen in shared memory, 42 against 54 and 78 against 55.
  return rows <= 32 ? run_attend_warp(static_cast<int>(rows), p, d, stream)
                    : run_attend_tc(rows, p, d, stream);
}

}  // namespace attn
}  // namespace nvfp4
