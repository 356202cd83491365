// rows.cu -- the passes over rows: the residual's addition with the RMS norm,
// the quantisation of bf16 rows, and the order of a weight's scales.
//
//   r = bf16(x + residual),  y = r * rsqrt(mean(r^2) + eps) * weight  (fp32)
//
// into bf16 or, block of 16 by block of 16, into NVFP4.  Bound by bytes: each
// element is read once and kept in registers between the sum and the output, a
// block of 16 (and so its scale) in one thread.
//
// Measured, 8192 x 5120: addition and norm into bf16 49.7 us, 6.8 TB/s, into NVFP4
// 43.7 us, 6.3 TB/s; quantisation 17.4 us, 6.2 TB/s (8192 x 17408 56.5 us, 6.5 TB/s);
// one row 2.4, 2.6 and 1.7 us, one trip to memory and the launch.
#include "common.cuh"

namespace nvfp4 {
namespace w4a4 {
namespace {

constexpr int kMaxNormThreads = 512;

__device__ __forceinline__ void unpack16(const uint4 (&w)[2], float (&f)[16]) {
  const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
  for (int i = 0; i < 8; ++i) f[2 * i] = bf16_lo(u[i]), f[2 * i + 1] = bf16_hi(u[i]);
}
// The largest magnitude of 16 bf16 numbers, as bits of fp32.
__device__ __forceinline__ uint32_t largest16(const uint4 (&w)[2]) {
  constexpr uint32_t kMagnitude = 0x7FFF7FFFu;
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    m = max_u16x2(m, max_u16x2(w[i].x & kMagnitude, w[i].y & kMagnitude));
    m = max_u16x2(m, max_u16x2(w[i].z & kMagnitude, w[i].w & kMagnitude));
  }
  return max(m << 16, m & 0xFFFF0000u);
}
__device__ __forceinline__ void pack16(const float (&f)[16], uint4 (&w)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = make_uint4(f32x2_to_bf16x2(f[8 * i], f[8 * i + 1]), f32x2_to_bf16x2(f[8 * i + 2], f[8 * i + 3]),
                      f32x2_to_bf16x2(f[8 * i + 4], f[8 * i + 5]), f32x2_to_bf16x2(f[8 * i + 6], f[8 * i + 7]));
}
__device__ __forceinline__ void load16(const __nv_bfloat16* p, uint4 (&w)[2]) {
  w[0] = reinterpret_cast<const uint4*>(p)[0];
  w[1] = reinterpret_cast<const uint4*>(p)[1];
}
__device__ __forceinline__ void store16(__nv_bfloat16* p, const uint4 (&w)[2]) {
  reinterpret_cast<uint4*>(p)[0] = w[0];
  reinterpret_cast<uint4*>(p)[1] = w[1];
}

// A block of threads per row; a thread has kV blocks of 16 elements, blockDim
// apart.
template <int kV>
__global__ void __launch_bounds__(kMaxNormThreads) norm_kernel(const Norm p) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ float part[kMaxNormThreads / 32];
  const int64_t m = blockIdx.x;
  const int blocks = static_cast<int>(p.K >> 4);
  uint4 x[kV][2], w[kV][2], r[kV][2];
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    const int b = threadIdx.x + v * blockDim.x;
    x[v][0] = x[v][1] = r[v][0] = r[v][1] = w[v][0] = w[v][1] = make_uint4(0, 0, 0, 0);
    if (b < blocks) {
      load16(p.x + m * p.xs + b * 16, x[v]);
      if (p.residual) load16(p.residual + m * p.rs + b * 16, r[v]);
      load16(p.weight + b * 16, w[v]);
    }
  }
  float sum = 0.f;
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    const int b = threadIdx.x + v * blockDim.x;
    float f[16];
    unpack16(x[v], f);
    if (p.residual) {
      float g[16];
      unpack16(r[v], g);
#pragma unroll
      for (int i = 0; i < 16; ++i) f[i] += g[i];
      pack16(f, x[v]);
      unpack16(x[v], f);
    }
    if (p.residual_out && b < blocks) store16(p.residual_out + m * p.ros + b * 16, x[v]);
#pragma unroll
    for (int i = 0; i < 16; ++i) sum = fmaf(f[i], f[i], sum);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
  __syncthreads();
  sum = 0.f;
  for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) sum += part[i];
  const float scale = rsqrtf(__fdiv_rn(sum, p.width) + p.eps);
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    const int b = threadIdx.x + v * blockDim.x;
    if (b >= blocks) continue;
    float f[16], g[16];
    unpack16(x[v], f);
    unpack16(w[v], g);
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i] = f[i] * scale * g[i];
    if (p.y) {
      pack16(f, x[v]);
      store16(p.y + m * p.ys + b * 16, x[v]);
    } else {
      uint2 c;
      p.scales[scale_row(m, p.K) + scale_in_row(b)] = static_cast<uint8_t>(quantize16(f, p.gs, c));
      *reinterpret_cast<uint2*>(p.codes + m * (p.K >> 1) + b * 8) = c;
    }
  }
}

constexpr int kQuantThreads = 256;

// blockDim.y rows to a block of threads; of a row a thread takes every blockDim.x-th
// block of 16, two of them on the way at one time.
__global__ void __launch_bounds__(kQuantThreads) quantize_rows_kernel(const Quantize p) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t m = blockIdx.x * static_cast<int64_t>(blockDim.y) + threadIdx.y;
  if (m >= p.M) return;
  const int blocks = static_cast<int>(p.K >> 4);
  const __nv_bfloat16* x = p.x + m * p.xs;
  uint8_t* codes = p.codes + m * (p.K >> 1);
  uint8_t* scales = p.scales + scale_row(m, p.K);
  for (int b = threadIdx.x; b < blocks; b += 2 * blockDim.x) {
    const int b1 = b + blockDim.x;
    uint4 w[2][2];
    load16(x + b * 16, w[0]);
    if (b1 < blocks) load16(x + b1 * 16, w[1]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = i ? b1 : b;
      if (at >= blocks) break;
      float f[16];
      unpack16(w[i], f);
      uint2 c;
      scales[scale_in_row(at)] = static_cast<uint8_t>(quantize16(f, largest16(w[i]), p.gs, c));
      *reinterpret_cast<uint2*>(codes + at * 8) = c;
    }
  }
}

// A thread per four scales of a row (one word in either order).
__global__ void __launch_bounds__(256)
    scale_layout_kernel(const uint8_t* scale, int64_t N, int64_t K, uint8_t* blocked,
                        unsigned int* refused) {
  // No early start of the kernel behind: a product reads scales before it waits.
  griddep_wait();
  const int64_t words = K >> 6, total = N * words;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
    const int64_t n = i / words, j = i - n * words;
    uint32_t w = *reinterpret_cast<const uint32_t*>(scale + i * 4);
    uint32_t out = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t b = w >> (8 * k) & 0xFFu;
      if (b == 0x7Fu || b > 0x80u) atomicOr(refused, 1u);
      out |= (b == 0x80u ? 0u : b) << (8 * k);
    }
    *reinterpret_cast<uint32_t*>(blocked + scale_row(n, K) + j * 512) = out;
  }
  __threadfence();
}

}  // namespace

int run_norm(const Norm& p, const Device& d, cudaStream_t stream) {
  const int blocks = static_cast<int>(p.K >> 4);
  // Few rows: as many threads as blocks of 16.  Many: two blocks a thread, twice the
  // bytes in flight for the threads that an SM holds.  K = 5120, into NVFP4: one row
  // 2.5 us against 2.9, 8192 rows 53.0 against 44.4 (into bf16 52.1 against 49.7).
  const int most = p.M > 2 * d.num_sms ? 128 : kMaxNormThreads;
  const int v = blocks <= most ? 1 : blocks <= 2 * kMaxNormThreads ? 2 : 4;
  const int threads = ((blocks + v - 1) / v + 31) / 32 * 32;
  const dim3 grid(static_cast<unsigned>(p.M));
  return v == 1   ? launch(1, norm_kernel<1>, grid, dim3(threads), 0, stream, p)
         : v == 2 ? launch(1, norm_kernel<2>, grid, dim3(threads), 0, stream, p)
                  : launch(1, norm_kernel<4>, grid, dim3(threads), 0, stream, p);
}

int run_quantize(const Quantize& p, const Device&, cudaStream_t stream) {
  // a row's blocks in equal shares of at most kQuantThreads threads, two to a thread
  // where there are many
  const int blocks = static_cast<int>(p.K >> 4);
  const int rounds = (blocks + kQuantThreads - 1) / kQuantThreads, shares = blocks >= 64 && rounds == 1 ? 2 : rounds;
  const int x = (blocks + shares - 1) / shares, y = kQuantThreads / x;
  return launch(1, quantize_rows_kernel, dim3(static_cast<unsigned>((p.M + y - 1) / y)), dim3(x, y), 0, stream, p);
}

int run_scale_layout(const uint8_t* scale, int64_t N, int64_t K, uint8_t* blocked,
                     unsigned int* refused, const Device& d, cudaStream_t stream) {
  const int64_t want = (N * (K >> 6) + 255) / 256, most = int64_t(d.num_sms) * 8;
  return launch(1, scale_layout_kernel, dim3(static_cast<unsigned>(want < most ? want : most)), dim3(256),
                0, stream, scale, N, K, blocked, refused);
}

}  // namespace w4a4
}  // namespace nvfp4
