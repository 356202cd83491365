// api.cu -- the C ABI of include/nvfp4_w4a4.h: validation on the host, the
// per-device set-up and the error word.
#include <cfloat>
#include <climits>
#include <cmath>
#include <mutex>

#include "common.cuh"

namespace {

__device__ unsigned int g_w4a4_error;
__device__ unsigned int g_w4a4_error_read;

__global__ void read_w4a4_error_kernel(int clear) {
  g_w4a4_error_read = clear ? atomicExch(&g_w4a4_error, 0u) : atomicOr(&g_w4a4_error, 0u);
}

using nvfp4::w4a4::kMaxDevices;
struct Slot {
  bool ready = false, supported = false;
  nvfp4::w4a4::Device d;
};
Slot g_devices[kMaxDevices];
std::mutex g_device_mutex;

bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool bad_scale(float s) { return !(s > 0.f && s < INFINITY); }

// Largest sizes: offsets stay far inside 64 bits, coordinates inside 32.
constexpr int64_t kMaxRows = int64_t(1) << 30;

int check_sizes(int64_t M, int64_t K, int64_t unit) {
  if (M < 0 || K <= 0) return NVFP4_ERR_INVALID;
  if (K % unit != 0 || M > kMaxRows || K > kMaxRows) return NVFP4_ERR_SHAPE;
  return NVFP4_OK;
}

// bf16 rows; the stride counts only where there is more than one.
int check_matrix(const void* p, int64_t stride, int64_t M, int64_t K) {
  if (!p) return NVFP4_ERR_INVALID;
  if (misaligned(p)) return NVFP4_ERR_MISALIGNED;
  if (M > 1) {
    if (stride < K) return NVFP4_ERR_INVALID;
    if (stride % 8 != 0) return NVFP4_ERR_MISALIGNED;
    if (stride >= (int64_t(1) << 31)) return NVFP4_ERR_SHAPE;
  }
  return NVFP4_OK;
}

int check_rows(const nvfp4_rows* r) {
  if (!r || !r->codes || !r->scales || bad_scale(r->global_scale)) return NVFP4_ERR_INVALID;
  if (misaligned(r->codes) || misaligned(r->scales)) return NVFP4_ERR_MISALIGNED;
  return NVFP4_OK;
}

// Memory that a call touches: `rows` pieces of `width` bytes, `stride` bytes apart.
struct Memory {
  uintptr_t p;
  int64_t rows, width, stride;
};
Memory bytes_of(const void* p, int64_t bytes) { return {reinterpret_cast<uintptr_t>(p), 1, bytes, bytes}; }
Memory matrix_of(const void* p, int64_t stride, int64_t M, int64_t K) {
  if (M == 1 || stride == K) return bytes_of(p, M * K * 2);
  return {reinterpret_cast<uintptr_t>(p), M, K * 2, stride * 2};
}
int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b < 0); }

// Whether a byte is in both, exactly: views of one tensor may lie between one another.
bool overlap(const Memory& a, const Memory& b) {
  const int64_t d = static_cast<int64_t>(b.p - a.p);
  if (d >= (a.rows - 1) * a.stride + a.width || -d >= (b.rows - 1) * b.stride + b.width) return false;
  if (a.rows > b.rows) return overlap(b, a);
  if (a.stride == b.stride) {
    // row i of a meets row j of b where (i - j) strides lie in (d - a.width, d + b.width)
    const int64_t first = floor_div(d - a.width, a.stride) + 1, n = first < 1 - b.rows ? 1 - b.rows : first;
    return n < a.rows && n * a.stride < d + b.width;
  }
  for (int64_t i = 0; i < a.rows; ++i) {
    // the first row of b that ends behind this row's begin
    const int64_t at = i * a.stride - d, first = floor_div(at - b.width, b.stride) + 1, j = first < 0 ? 0 : first;
    if (j < b.rows && j * b.stride < at + a.width) return true;
  }
  return false;
}

// Codes and scales of rows [M, K].
struct RowsMemory {
  Memory codes, scales;
};
RowsMemory memory_of(const uint8_t* codes, const uint8_t* scales, int64_t M, int64_t K) {
  return {bytes_of(codes, M * (K / 2)), bytes_of(scales, nvfp4_w4a4_scale_bytes(M, K))};
}
bool overlap(const RowsMemory& r, const Memory& m) { return overlap(r.codes, m) || overlap(r.scales, m); }
bool overlap(const RowsMemory& r, const RowsMemory& s) { return overlap(r, s.codes) || overlap(r, s.scales); }

}  // namespace

namespace nvfp4 {
namespace w4a4 {

int device(Device* out) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    cudaGetLastError();
    return NVFP4_ERR_DEVICE;
  }
  std::lock_guard<std::mutex> lock(g_device_mutex);
  Slot& s = g_devices[dev];
  if (!s.ready) {
    int major = 0, minor = 0, sms = 0;
    void* err = nullptr;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
      cudaGetLastError();
      return NVFP4_ERR_DEVICE;
    }
    s.supported = major == 10 && minor == 3;
    if (s.supported && cudaGetSymbolAddress(&err, g_w4a4_error) != cudaSuccess) {
      cudaGetLastError();
      return NVFP4_ERR_DEVICE;
    }
    s.d.id = dev;
    s.d.num_sms = sms;
    s.d.err = static_cast<unsigned int*>(err);
    s.ready = true;
  }
  if (!s.supported) return NVFP4_ERR_DEVICE;
  *out = s.d;
  return NVFP4_OK;
}

}  // namespace w4a4
}  // namespace nvfp4

using namespace nvfp4::w4a4;

extern "C" {

int64_t nvfp4_w4a4_scale_bytes(int64_t rows, int64_t K) {
  if (rows < 0 || K <= 0 || K % 256 != 0 || rows > kMaxRows || K > kMaxRows) return 0;
  return (rows + 127) / 128 * 128 * (K / 16);
}

int nvfp4_w4a4_scale_layout(const uint8_t* w_scale, int64_t N, int64_t K, uint8_t* blocked,
                            unsigned int* refused, void* stream) {
  if (N <= 0) return NVFP4_ERR_INVALID;
  if (const int st = check_sizes(N, K, 256)) return st;
  if (N % 128 != 0) return NVFP4_ERR_SHAPE;
  if (!w_scale || !blocked || !refused) return NVFP4_ERR_INVALID;
  if (misaligned(w_scale) || misaligned(blocked) || (reinterpret_cast<uintptr_t>(refused) & 3u))
    return NVFP4_ERR_MISALIGNED;
  const Memory laid = bytes_of(blocked, N * (K / 16)), flag = bytes_of(refused, 4);
  if (overlap(laid, bytes_of(w_scale, N * (K / 16))) || overlap(laid, flag)) return NVFP4_ERR_INVALID;
  Device d;
  if (const int st = device(&d)) return st;
  return run_scale_layout(w_scale, N, K, blocked, refused, d, static_cast<cudaStream_t>(stream));
}

int nvfp4_quantize_rows(const void* x, int64_t row_stride, int64_t M, int64_t K,
                        const nvfp4_rows* out, void* stream) {
  if (const int st = check_sizes(M, K, 256)) return st;
  if (M == 0) return NVFP4_OK;
  if (const int st = check_matrix(x, row_stride, M, K)) return st;
  if (const int st = check_rows(out)) return st;
  const RowsMemory o = memory_of(out->codes, out->scales, M, K);
  if (overlap(o, matrix_of(x, row_stride, M, K)) || overlap(o.codes, o.scales)) return NVFP4_ERR_INVALID;
  Device d;
  if (const int st = device(&d)) return st;
  const Quantize p{static_cast<const __nv_bfloat16*>(x), row_stride, M, K, out->global_scale, out->codes,
                   out->scales};
  return run_quantize(p, d, static_cast<cudaStream_t>(stream));
}

int nvfp4_add_rms_norm(const void* x, int64_t x_stride, const void* residual,
                       int64_t residual_stride, const void* weight, float eps, int64_t M,
                       int64_t K, void* residual_out, int64_t residual_out_stride, void* y,
                       int64_t y_stride, const nvfp4_rows* rows, void* stream) {
  if (const int st = check_sizes(M, K, rows ? 256 : 16)) return st;
  if (K > NVFP4_W4A4_MAX_NORM) return NVFP4_ERR_SHAPE;
  if (!(eps >= 0.f && eps < INFINITY) || !weight) return NVFP4_ERR_INVALID;
  if (misaligned(weight)) return NVFP4_ERR_MISALIGNED;
  if (M == 0) return NVFP4_OK;
  if ((y != nullptr) == (rows != nullptr)) return NVFP4_ERR_INVALID;
  if (const int st = check_matrix(x, x_stride, M, K)) return st;
  if (residual)
    if (const int st = check_matrix(residual, residual_stride, M, K)) return st;
  if (residual_out)
    if (const int st = check_matrix(residual_out, residual_out_stride, M, K)) return st;
  if (const int st = rows ? check_rows(rows) : check_matrix(y, y_stride, M, K)) return st;
  // an output is one of the inputs, or apart from all of them; the outputs are apart
  auto apart = [&](const void* out, int64_t stride) {
    const Memory o = matrix_of(out, stride, M, K);
    auto clear = [&](const void* in, int64_t in_stride) {
      return !in || (in == out && (M == 1 || in_stride == stride)) || !overlap(o, matrix_of(in, in_stride, M, K));
    };
    return clear(x, x_stride) && clear(residual, residual_stride) && !overlap(o, bytes_of(weight, K * 2));
  };
  if (residual_out && !apart(residual_out, residual_out_stride)) return NVFP4_ERR_INVALID;
  if (y) {
    if (!apart(y, y_stride)) return NVFP4_ERR_INVALID;
    if (residual_out && overlap(matrix_of(y, y_stride, M, K), matrix_of(residual_out, residual_out_stride, M, K)))
      return NVFP4_ERR_INVALID;
  } else {
    const RowsMemory o = memory_of(rows->codes, rows->scales, M, K);
    if (overlap(o, matrix_of(x, x_stride, M, K)) || overlap(o, bytes_of(weight, K * 2)) ||
        (residual && overlap(o, matrix_of(residual, residual_stride, M, K))) ||
        (residual_out && overlap(o, matrix_of(residual_out, residual_out_stride, M, K))) ||
        overlap(o.codes, o.scales))
      return NVFP4_ERR_INVALID;
  }
  Device d;
  if (const int st = device(&d)) return st;
  Norm p{};
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.residual = static_cast<const __nv_bfloat16*>(residual);
  p.weight = static_cast<const __nv_bfloat16*>(weight);
  p.residual_out = static_cast<__nv_bfloat16*>(residual_out);
  p.y = static_cast<__nv_bfloat16*>(y);
  p.xs = x_stride;
  p.rs = residual_stride;
  p.ros = residual_out_stride;
  p.ys = y_stride;
  p.M = M;
  p.K = K;
  p.eps = eps;
  p.width = static_cast<float>(K);
  if (rows) {
    p.gs = rows->global_scale;
    p.codes = rows->codes;
    p.scales = rows->scales;
  }
  return run_norm(p, d, static_cast<cudaStream_t>(stream));
}

int nvfp4_linear_w4a4(const nvfp4_rows* a, int64_t M, const nvfp4_weight* w, int32_t swiglu,
                      void* y, const nvfp4_rows* out, void* stream) {
  if (!w || w->N <= 0) return NVFP4_ERR_INVALID;
  if (const int st = check_sizes(M, w->K, 256)) return st;
  if (w->N > kMaxRows || w->N % (out ? 512 : swiglu ? 256 : 128) != 0) return NVFP4_ERR_SHAPE;
  if (out && !swiglu) return NVFP4_ERR_INVALID;
  if (!w->codes || !w->scales) return NVFP4_ERR_INVALID;
  if (misaligned(w->codes) || misaligned(w->scales)) return NVFP4_ERR_MISALIGNED;
  if (w->segments < 1 || w->segments > kMaxSegments) return NVFP4_ERR_INVALID;
  int64_t rows = 0;
  for (int i = 0; i < w->segments; ++i) {
    const int64_t n = w->segment_rows[i];
    if (n <= 0 || n > w->N || bad_scale(w->global_scale[i])) return NVFP4_ERR_INVALID;
    if (n % 16 != 0) return NVFP4_ERR_SHAPE;
    rows += n;
  }
  if (rows != w->N) return NVFP4_ERR_INVALID;
  if (M == 0) return NVFP4_OK;
  if (const int st = check_rows(a)) return st;
  if ((y != nullptr) == (out != nullptr)) return NVFP4_ERR_INVALID;
  if (const int st = out ? check_rows(out) : check_matrix(y, w->N, 1, w->N)) return st;
  Product p{};
  p.a_codes = a->codes;
  p.a_scales = a->scales;
  p.w_codes = w->codes;
  p.w_scales = w->scales;
  p.M = M;
  p.N = w->N;
  p.K = w->K;
  p.seg.n = w->segments;
  rows = 0;
  for (int i = 0; i < w->segments; ++i) {
    rows += w->segment_rows[i];
    p.seg.end[i] = static_cast<int>(rows);
    p.seg.scale[i] = static_cast<float>(1.0 / (double(a->global_scale) * double(w->global_scale[i])));
    // (below fp32's normal range it would be left with fewer bits than a result)
    if (bad_scale(p.seg.scale[i]) || p.seg.scale[i] < FLT_MIN) return NVFP4_ERR_INVALID;
  }
  const RowsMemory in[2] = {memory_of(a->codes, a->scales, M, w->K), memory_of(w->codes, w->scales, w->N, w->K)};
  const int64_t n_out = swiglu ? w->N / 2 : w->N;
  if (out) {
    const RowsMemory o = memory_of(out->codes, out->scales, M, n_out);
    if (overlap(o, in[0]) || overlap(o, in[1]) || overlap(o.codes, o.scales)) return NVFP4_ERR_INVALID;
  } else {
    const Memory o = bytes_of(y, M * n_out * 2);
    if (overlap(in[0], o) || overlap(in[1], o)) return NVFP4_ERR_INVALID;
  }
  Device d;
  if (const int st = device(&d)) return st;
  p.swiglu = swiglu != 0;
  p.y = static_cast<__nv_bfloat16*>(y);
  if (out) {
    p.codes = out->codes;
    p.scales = out->scales;
    p.out_gs = out->global_scale;
  }
  p.err = d.err;
  return run_product(p, d, static_cast<cudaStream_t>(stream));
}

int nvfp4_w4a4_status(unsigned int* bits, int clear) {
  if (!bits) return NVFP4_ERR_INVALID;
  Device d;
  if (const int st = device(&d)) return st;
  if (cudaDeviceSynchronize() != cudaSuccess) {
    cudaGetLastError();
    return NVFP4_ERR_DEVICE;
  }
  read_w4a4_error_kernel<<<1, 1>>>(clear);
  if (cudaGetLastError() != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess ||
      cudaMemcpyFromSymbol(bits, g_w4a4_error_read, sizeof(*bits)) != cudaSuccess) {
    cudaGetLastError();
    return NVFP4_ERR_DEVICE;
  }
  return NVFP4_OK;
}

}  // extern "C"
