// product.cu -- the tensor maps of the products, and the choice between them.
#include <cudaTypedefs.h>

#include "product.cuh"

namespace nvfp4 {
namespace w4a4 {
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

}  // namespace

// Encoded anew for each call: a few tenths of a microsecond.
bool codes_map(CUtensorMap* map, const uint8_t* codes, int64_t rows, int64_t K, int box) {
  static const Encode fn = find_encode();
  const cuuint64_t dims[2] = {cuuint64_t(K / 2), cuuint64_t(rows)};
  const cuuint64_t strides[1] = {cuuint64_t(K / 2)};
  const cuuint32_t boxes[2] = {128, cuuint32_t(box)}, unit[2] = {1, 1};
  return fn && fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(codes), dims, strides, boxes,
                  unit, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scales as rows of 512 bytes, one for each 128 rows x 64 k; boxes of four (256 k).
bool scales_map(CUtensorMap* map, const uint8_t* scales, int64_t rows, int64_t K) {
  static const Encode fn = find_encode();
  const cuuint64_t dims[2] = {128, cuuint64_t((rows + 127) / 128 * (K / kMmaK))};
  const cuuint64_t strides[1] = {kScaleBlock};
  const cuuint32_t boxes[2] = {128, 4}, unit[2] = {1, 1};
  return fn && fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<uint8_t*>(scales), dims, strides, boxes,
                  unit, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int run_product(const Product& p, const Device& d, cudaStream_t stream) {
  return p.M > 128 ? run_product_many(p, d, stream) : run_product_few(p, d, stream);
}

}  // namespace w4a4
}  // namespace nvfp4
