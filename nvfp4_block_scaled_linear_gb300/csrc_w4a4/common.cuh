// common.cuh -- what the NVFP4 x NVFP4 kernels share: parameters, the scales'
// order, the quantisation of a block of 16, and the launch helpers.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "../../include/nvfp4_w4a4.h"
#include "../csrc/ptx.cuh"

namespace nvfp4 {
namespace w4a4 {

constexpr int kMaxSegments = 8;

// Bytes of a row's scales in the order of nvfp4_w4a4.h (512-byte blocks of 128 rows
// x 4 scales): where row r's begin, and from there to 16-block b's.
__device__ __forceinline__ int64_t scale_row(int64_t r, int64_t K) {
  return (r >> 7) * (K >> 6) * 512 + ((r & 31) * 16 + (r >> 5 & 3) * 4);
}
__device__ __forceinline__ int64_t scale_in_row(int b) { return (b >> 2) * int64_t(512) + (b & 3); }

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(__float_as_uint(lo)), "r"(__float_as_uint(hi)));
  return r;
}
__device__ __forceinline__ float2 split2(uint64_t v) {
  uint32_t lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(v));
  return make_float2(__uint_as_float(lo), __uint_as_float(hi));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// Eight e2m1 codes, value 2i in the low nibble of byte i.
__device__ __forceinline__ uint32_t to_e2m1x8(const float (&q)[8]) {
  uint32_t d;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(d)
      : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]),
        "f"(q[7]));
  return d;
}

// The e4m3 byte of a non-negative value, saturating, and back.
__device__ __forceinline__ uint32_t to_e4m3(float v) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(0.0f), "f"(v));
  return d & 0xFFu;
}
__device__ __forceinline__ float from_e4m3(uint32_t b) {
  uint32_t h;
  asm("{\n\t.reg .b16 x;\n\tcvt.u16.u32 x, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\t}"
      : "=r"(h)
      : "r"(b));
  float f;
  asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %1;\n\tcvt.f32.f16 %0, x;\n\t}" : "=f"(f) : "r"(h));
  return f;
}

// A block of 16 values, the largest of magnitude `top` (as bits, which order as the
// values do and put infinities and NaN above them), -> 8 code bytes and the scale
// byte, by the steps of nvfp4_w4a4.h.  The quotient of x = RN(v gs) by the scale s is
// correctly rounded without a division for each value: with r = RN(1/s), q0 = RN(x r),
// rem = RN(x - q0 s), q = RN(q0 + rem r) (Markstein's refinement; s has 4 significant
// bits, so r is far from the one case it excepts; checked for every significand in
// tests/test_quantize_division.py); the sixth of the largest likewise.
// A quotient so small that a step underflows is far below the first threshold, of
// e2m1 or of e4m3.
__device__ __forceinline__ uint32_t quantize16(const float (&v)[16], uint32_t top, float gs, uint2& codes) {
  const float m = __fmul_rn(__uint_as_float(top), gs);
  codes = make_uint2(0u, 0u);
  if (!(m < __uint_as_float(0x7F800000u))) return 0x7Fu;      // infinity, NaN
  constexpr float kSixth = 0.16666667163372039794921875f;    // RN(1/6)
  const float sixth = __fmul_rn(m, kSixth);
  const uint32_t byte = to_e4m3(__fmaf_rn(__fmaf_rn(sixth, -6.0f, m), kSixth, sixth));
  if (byte == 0u) return 0u;
  const float s = from_e4m3(byte), r = __frcp_rn(s);
  const uint64_t g2 = pack2(gs, gs), r2 = pack2(r, r), ns2 = pack2(-s, -s);
  uint32_t c[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float q[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t x = mul2(pack2(v[8 * h + 2 * i], v[8 * h + 2 * i + 1]), g2);
      const uint64_t q0 = mul2(x, r2);
      const float2 f = split2(fma2(fma2(q0, ns2, x), r2, q0));
      q[2 * i] = f.x;
      q[2 * i + 1] = f.y;
    }
    c[h] = to_e2m1x8(q);
  }
  codes = make_uint2(c[0], c[1]);
  return byte;
}

__device__ __forceinline__ uint32_t quantize16(const float (&v)[16], float gs, uint2& codes) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return quantize16(v, top, gs, codes);
}

// ---------------------------------------------------------------- host side
constexpr int kMaxDevices = 64;
struct Device {
  int id = 0;
  int num_sms = 0;
  unsigned int* err = nullptr;
};

// The current device's set-up (NVFP4_ERR_DEVICE where it is not sm_103).
int device(Device* out);

// Launch, in clusters of `cluster` CTAs, with programmatic stream serialization.
// A kernel lets the next one start (griddep_launch_dependents) only after its own
// griddep_wait: what runs then is that kernel and no earlier one, so that a product's
// early reads of its weight can meet no writes but the kernel's directly ahead.
template <typename... P, typename... A>
int launch(int cluster, void (*kernel)(P...), dim3 grid, dim3 block, size_t smem,
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

struct Norm {
  const __nv_bfloat16* x;
  const __nv_bfloat16* residual;     // or null
  const __nv_bfloat16* weight;
  __nv_bfloat16* residual_out;       // or null
  __nv_bfloat16* y;                  // or null: codes and scales
  int64_t xs, rs, ros, ys;
  int64_t M, K;
  float eps, gs, width;              // width: K
  uint8_t* codes;
  uint8_t* scales;
};
int run_norm(const Norm& p, const Device& d, cudaStream_t stream);

struct Quantize {
  const __nv_bfloat16* x;
  int64_t xs, M, K;
  float gs;
  uint8_t* codes;
  uint8_t* scales;
};
int run_quantize(const Quantize& p, const Device& d, cudaStream_t stream);
int run_scale_layout(const uint8_t* scale, int64_t N, int64_t K, uint8_t* blocked,
                     unsigned int* refused, const Device& d, cudaStream_t stream);

// Scales of a stacked weight's segments: outputs below end[i] and not below the
// one before take scale[i].
struct Segments {
  int n;
  int end[kMaxSegments];
  float scale[kMaxSegments];
};
__device__ __forceinline__ float segment_scale(const Segments& s, int col) {
  float v = s.scale[0];
#pragma unroll
  for (int i = 1; i < kMaxSegments; ++i)
    if (i < s.n && col >= s.end[i - 1]) v = s.scale[i];
  return v;
}

// silu(g) * u = g / (1 + 2^(-g log2 e)) * u, exponential and reciprocal by the
// hardware's approximations (2^-22 and 2^-23 of the value); the exponent's rounding
// to fp32 is |g| 2^-24 of the exponential more, 2^-18 at g = -80.  From g >= -80 the sum
// and its reciprocal stay in fp32's normal range, and an exponential below it is
// nothing beside 1.
__device__ __forceinline__ float gated(float g, float u) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return g * r * u;
}

// Below, where 1 is nothing beside the exponential: silu(g) = g e^g, in fp32's normal
// range down to about g = -92 and smoothly to zero from there.
constexpr float kSiluTail = -80.f;
__device__ __forceinline__ float gated_tail(float g, float u) { return g * expf(g) * u; }

// g[i] = silu(g[i] sg) * (u[i] su).  One comparison for the sixteen: so low a gate is rare.
__device__ __forceinline__ void gated16(float (&g)[16], const float (&u)[16], float sg, float su) {
  float low = 0.f;
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    g[k] *= sg;
    low = fminf(low, g[k]);
  }
  if (low >= kSiluTail) {
#pragma unroll
    for (int k = 0; k < 16; ++k) g[k] = gated(g[k], u[k] * su);
  } else {
#pragma unroll
    for (int k = 0; k < 16; ++k) g[k] = g[k] < kSiluTail ? gated_tail(g[k], u[k] * su) : gated(g[k], u[k] * su);
  }
}

struct Product {
  const uint8_t* a_codes;
  const uint8_t* a_scales;
  const uint8_t* w_codes;
  const uint8_t* w_scales;
  int64_t M, N, K;
  Segments seg;                      // 1 / (the rows' global scale x the segment's)
  int swiglu;
  __nv_bfloat16* y;                  // or null: codes and scales
  uint8_t* codes;
  uint8_t* scales;
  float out_gs;
  unsigned int* err;
};
int run_product(const Product& p, const Device& d, cudaStream_t stream);

}  // namespace w4a4
}  // namespace nvfp4
