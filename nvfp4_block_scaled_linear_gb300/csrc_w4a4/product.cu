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
  // Up to 32 tokens: the weights as the MMA's rows.  One token by 5120 rows and 6144 k
  // 6.5 us against 7.2 with the tokens there, by 2048 rows 4.0 against 5.2, gated by 12288
  // and 2048 k 5.9 against 6.5; 24 tokens 6.9 against 7.4, 4.7 against 5.5, 6.4 against 6.5;
  // 32 7.5 against 7.2, 4.9 against 5.5, 6.7 against 6.6, gated by 40960 and 5120 k 26.6
  // against 30.0.
  if (p.M <= 32) return run_product_narrow(p, d, stream);
  // The kernel for few tokens takes up to 128 by 128 weight rows (of a pair 256) a CTA
  // and is the faster one as long as every CTA has an SM; beyond that the pairs' 256 by
  // 256 tiles read half as much.  128 tokens by 5120 rows and 17408 k 14.2 us against
  // 22.7, 384 24.3 against 23.5; 515 33.5 against 27.4; gated 130 by 12288 and 2048 k
  // 7.9 against 8.8, by 34816 and 5120 k 34.0 against 22.0.  Up to 128 tokens always:
  // gated by 34816 and 5120 k 128 20.5 against 22.1, 64 19.8 against 21.7, but by 40960,
  // where its CTAs take two rounds, 32.4 against 29.6 and 31.4 against 29.0.
  const int64_t few = (p.M + 127) / 128 * (p.N / (p.swiglu ? 256 : 128));
  return p.M <= 128 || few <= d.num_sms ? run_product_few(p, d, stream) : run_product_many(p, d, stream);
}

}  // namespace w4a4
}  // namespace nvfp4
