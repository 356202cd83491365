// evict.cu -- the keys with the most attention weight kept, their rows moved
// together.  Two launches: one block per sequence and head chooses, then the
// rows are copied.
//
// Choosing: the mass becomes an unsigned integer of the same order (negative
// values inverted, others with the sign bit set; -0 made +0 and NaN the
// largest).  Four passes over the candidates, 8 bits each from the top, count
// the values that agree with the bits found so far and narrow down to the
// value of the last key kept; of the keys that equal it the first ones are
// kept.  A last pass in order writes the kept places.
#include "common.cuh"

namespace nvfp4 {
namespace attn {
namespace {

constexpr int kThreads = 1024;

__device__ __forceinline__ uint32_t ordered(float f) {
  if (isnan(f)) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(f + 0.f);        // -0 + 0 = +0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive prefix sum of v over the block; *total its sum.
__device__ __forceinline__ int block_scan(int v, int* total, int* sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += o;
  }
  __syncthreads();
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  int before = 0, all = 0;
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) before += sums[i];
    all += sums[i];
  }
  *total = all;
  return before + x - v;
}

__global__ void __launch_bounds__(kThreads) choose_kernel(const Evict p) {
  __shared__ int count[256];
  __shared__ int sums[32];
  __shared__ uint32_t sh_prefix;
  __shared__ int sh_left;
  griddep_wait();
  griddep_launch_dependents();
  const int s = blockIdx.x / p.from.heads;
  const int64_t row = blockIdx.x;
  int n = p.kv_lens[s];
  if (n < 0 || n > p.room || n > int64_t(p.width) * p.from.page_size) {
    if (threadIdx.x == 0) atomicOr(p.err, NVFP4_ATTENTION_BAD_INDEX);
    n = 0;
  }
  const int m = min(n, p.keep), newest = min(p.recent, m);
  const int old = n - newest;                 // candidates
  const float* mass = p.mass + row * p.room;
  int32_t* index = p.index + row * p.keep;
  float* new_mass = p.new_mass + row * p.keep;
  if (threadIdx.x == 0) {
    sh_prefix = 0;
    sh_left = m - newest;
    if (blockIdx.x % p.from.heads == 0) p.new_lens[s] = m;
  }
  __syncthreads();
  // the (m - newest)-th largest candidate's bits, and how many of its equals are kept
  for (int shift = 24; shift >= 0 && m > newest; shift -= 8) {
    for (int i = threadIdx.x; i < 256; i += kThreads) count[i] = 0;
    __syncthreads();
    const uint32_t prefix = sh_prefix, mask = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
    for (int j = threadIdx.x; j < old; j += kThreads) {
      const uint32_t u = ordered(mass[j]);
      if ((u & mask) == prefix) atomicAdd(&count[(u >> shift) & 255], 1);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      int left = sh_left, b = 255;
      while (count[b] < left) left -= count[b--];
      sh_left = left;
      sh_prefix = prefix | uint32_t(b) << shift;
    }
    __syncthreads();
  }
  const uint32_t bar = sh_prefix;
  const int equals = sh_left;
  int kept = 0, same = 0;
  if (m > newest) {
    for (int j0 = 0; j0 < old; j0 += kThreads) {
      const int j = j0 + threadIdx.x;
      const float f = j < old ? mass[j] : 0.f;
      const uint32_t u = j < old ? ordered(f) : 0u;
      int total_same, total_kept;
      const int eq = j < old && u == bar;
      const int my_same = same + block_scan(eq, &total_same, sums);
      const int take = j < old && (u > bar || (eq && my_same < equals));
      const int at = kept + block_scan(take, &total_kept, sums);
      if (take) {
        index[at] = j;
        new_mass[at] = f;
      }
      same += total_same;
      kept += total_kept;
    }
  }
  for (int i = threadIdx.x; i < p.keep - (m - newest); i += kThreads) {
    const int at = m - newest + i;
    index[at] = at < m ? old + i : -1;
    new_mass[at] = at < m ? mass[old + i] : 0.f;
  }
}

// One warp copies the key and value rows of one kept place.
__global__ void __launch_bounds__(256) move_kernel(const Evict p) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t(blockIdx.x) * 256 + threadIdx.x) >> 5;
  const int64_t row = w / p.keep;
  const int r = static_cast<int>(w - row * p.keep);
  const int s = static_cast<int>(row / p.from.heads), h = static_cast<int>(row % p.from.heads);
  if (s >= p.count) return;
  const int j = p.index[row * p.keep + r];
  if (j < 0) return;
  const int64_t from = checked_page(p.table[int64_t(s) * p.width + j / p.from.page_size],
                                    p.from.pages, p.err);
  const int64_t to = checked_page(p.to_table[int64_t(s) * p.to_width + r / p.to.page_size],
                                  p.to.pages, p.err);
  if (from == p.from.pages || to == p.to.pages) return;
  const int size = p.from.e4m3 ? 1 : 2;
  const int bytes = p.from.dim * size;
  const int jf = j % p.from.page_size, rt = r % p.to.page_size;
  for (int i = lane * 16; i < 2 * bytes; i += 512) {
    const bool v = i >= bytes;
    const int b = v ? i - bytes : i;
    const int64_t* fs = v ? p.from.vs : p.from.ks;
    const int64_t* ts = v ? p.to.vs : p.to.ks;
    const uint8_t* src = static_cast<const uint8_t*>(v ? p.from.v : p.from.k) +
                         (from * fs[0] + jf * fs[1] + h * fs[2]) * size + b;
    uint8_t* dst = static_cast<uint8_t*>(v ? p.to.v : p.to.k) +
                   (to * ts[0] + rt * ts[1] + h * ts[2]) * size + b;
    *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(src);
  }
}

}  // namespace

int run_evict(const Evict& p, const Device&, cudaStream_t stream) {
  const int64_t rows = int64_t(p.count) * p.from.heads;
  const int64_t blocks = (rows * p.keep + 7) / 8;
  if (rows > INT32_MAX || blocks > INT32_MAX) return NVFP4_ERR_SHAPE;
  if (const int st = launch(choose_kernel, dim3(static_cast<unsigned>(rows)), dim3(kThreads), 0,
                            stream, p))
    return st;
  return launch(move_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream, p);
}

}  // namespace attn
}  // namespace nvfp4
