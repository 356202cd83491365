// product.cuh -- what the products of NVFP4 rows and NVFP4 weights share: the
// block-scaled MMA, the copy of scales into TMEM, bulk copies.
#pragma once
#include "common.cuh"

namespace nvfp4 {
namespace w4a4 {

constexpr int kStageK = 256;       // k of one pipeline stage: 128 bytes of codes a row
constexpr int kMmaK = 64;          // k of one MMA: 32 bytes of codes a row
constexpr int kScaleBlock = 512;   // the scales of 128 rows x 64 k

// Instruction descriptor, kind::mxf4nvf4: e2m1 A and B, e4m3 scales, K = 64.
__host__ __device__ constexpr uint32_t idesc_nvfp4(uint32_t m, uint32_t n) {
  return (1u << 7) | (1u << 10) | ((n >> 3) << 17) | ((m >> 4) << 24);
}

// D[tmem] (+)= (A . scales) * (B . scales)^T; A and B from shared memory, K-major
// in 128-byte swizzled rows, the scales from TMEM: row r's four in lane r % 32 of
// every quarter, column r / 32.
__device__ __forceinline__ void umma_nvfp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                           uint32_t a_scales, uint32_t b_scales,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], "
      "[%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(a_scales), "r"(b_scales), "r"(accumulate)
      : "memory");
}

// Descriptor of 32 rows of 16 bytes one after another (no swizzle; 8 rows are
// 128 bytes): a block of scales.
__device__ __forceinline__ uint64_t scale_desc(uint32_t smem_byte_addr) {
  return static_cast<uint64_t>((smem_byte_addr >> 4) & 0x3FFFu) |
         static_cast<uint64_t>(128 >> 4) << 32 | static_cast<uint64_t>(1) << 46;
}

// 512 bytes of scales -> 4 TMEM columns, the same in each quarter of the lanes.
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_addr(dst)),
      "l"(__cvta_generic_to_global(src)), "r"(bytes), "r"(smem_addr(bar))
      : "memory");
}

// Wait for the phase with the given parity; given up after 2^31 clock ticks
// (about a second), or at once when another wait of the block was, with
// `abort_flag` set and false returned.  (The clock register, not the global
// timer: reading that takes longer than a stage.)
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

// One lane of a converged warp.  In a branch on this the compiler knows that one
// thread runs and builds the tensor core's descriptors in uniform registers; in a
// branch on the lane's number each instruction waits for its operands to be moved
// there, some 40 clocks, which 16 of them a stage made twice the products' time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// 16 outputs, rounded to bf16.
__device__ __forceinline__ void store_bf16(__nv_bfloat16* y, const float (&v)[16]) {
#pragma unroll
  for (int k = 0; k < 2; ++k)
    reinterpret_cast<uint4*>(y)[k] =
        make_uint4(f32x2_to_bf16x2(v[8 * k], v[8 * k + 1]), f32x2_to_bf16x2(v[8 * k + 2], v[8 * k + 3]),
                   f32x2_to_bf16x2(v[8 * k + 4], v[8 * k + 5]), f32x2_to_bf16x2(v[8 * k + 6], v[8 * k + 7]));
}

enum { kPlain = 0, kGated = 1, kGatedRows = 2 };

// 16 outputs n .. n + 15 of row m from their sums (of a gated product gate and up),
// scaled, gated and rounded.
template <int kMode, int kParts>
__device__ __forceinline__ void outputs16(const Product& p, int64_t m, int n, float (&v)[kParts][16]) {
  const int n_out = static_cast<int>(kMode == kPlain ? p.N : p.N / 2);
  const float s = segment_scale(p.seg, n);
  if (kMode == kPlain) {
#pragma unroll
    for (int k = 0; k < 16; ++k) v[0][k] *= s;
  } else {
    gated16(v[0], v[kParts - 1], s, segment_scale(p.seg, n + n_out));
  }
  if (kMode == kGatedRows) {
    uint2 codes;
    p.scales[scale_row(m, n_out) + scale_in_row(n >> 4)] = static_cast<uint8_t>(quantize16(v[0], p.out_gs, codes));
    *reinterpret_cast<uint2*>(p.codes + m * (n_out >> 1) + (n >> 1)) = codes;
  } else {
    store_bf16(p.y + m * n_out + n, v[0]);
  }
}

// Tensor map of codes [rows, K/2], boxes of `box` rows by 128 bytes.
bool codes_map(CUtensorMap* map, const uint8_t* codes, int64_t rows, int64_t K, int box);

// Tensor map of blocked scales: row (128-row block) * (K / 64) + k / 64, boxes of 4 rows.
bool scales_map(CUtensorMap* map, const uint8_t* scales, int64_t rows, int64_t K);

// Clusters of `split` CTAs, one on each SM, that the device holds at one time.
int most_clusters(int split, const Device& d);

// Up to 32 tokens: 128 weight rows (gated 128 of each) a CTA, the MMA's rows.
int run_product_narrow(const Product& p, const Device& d, cudaStream_t stream);

// 33 tokens and more: 128 tokens by 128 (gated 64 or 128 of each) weight rows a CTA.
int run_product_few(const Product& p, const Device& d, cudaStream_t stream);

// Many tokens: persistent pairs of CTAs, 256 tokens by 256 weight rows.
int run_product_many(const Product& p, const Device& d, cudaStream_t stream);

}  // namespace w4a4
}  // namespace nvfp4
