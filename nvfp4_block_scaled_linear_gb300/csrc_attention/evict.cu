// evict.cu -- the keys with the most attention weight kept, their rows moved
// together.  Two launches: a cluster of CTAs per sequence and head chooses,
// then the rows are copied.
//
// Choosing: the mass becomes an unsigned integer of the same order (negative
// values inverted, others with the sign bit set; -0 made +0 and NaN the
// largest).  Four passes over the candidates, 8 bits each from the top, count
// the values that agree with the bits found so far and narrow down to the
// value of the last key kept; of the keys that equal it the first ones are
// kept.  Each CTA of the cluster holds a slice of the candidates in shared
// memory (read once), the counts of the slices are added over distributed
// shared memory, and every thread then writes the kept places of its own run
// of the slice, in order, behind those of the runs and slices before it.
//
// What bounds it: the copy moves every kept row once in and once out; the
// choice is latency (two cluster barriers a pass), so it is spread over as many
// CTAs as the slices keep busy.
#include <algorithm>

#include "common.cuh"

namespace nvfp4 {
namespace attn {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kSmemKeys = 40 * 1024;          // of a slice held in shared memory
constexpr int kMinSlice = 2048;               // candidates worth a CTA of their own

__device__ __forceinline__ uint32_t ordered(float f) {
  if (isnan(f)) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(f + 0.f);        // -0 + 0 = +0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__global__ void __launch_bounds__(kThreads) choose_kernel(const Evict p, int slice_room) {
  extern __shared__ uint32_t keys[];          // the slice, up to slice_room of it
  __shared__ uint32_t count[256];             // this slice's
  __shared__ uint32_t total[256];             // the cluster's
  __shared__ uint32_t warp_sum[kWarps];
  __shared__ uint32_t mine[2];                // larger than the bar, equal to it
  __shared__ uint32_t sh_prefix, sh_left;
  griddep_wait();
  griddep_launch_dependents();
  uint32_t ctas;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ctas));
  const uint32_t rank = cluster_ctarank();
  const int64_t row = blockIdx.x / ctas;
  const int s = static_cast<int>(row / p.from.heads);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int n = p.kv_lens[s];
  if (n < 0 || n > p.room || n > int64_t(p.width) * p.from.page_size) {
    if (tid == 0) atomicOr(p.err, NVFP4_ATTENTION_BAD_INDEX);
    n = 0;
  }
  const int m = min(n, p.keep), newest = min(p.recent, m);
  const int old = n - newest;                 // candidates
  const float* mass = p.mass + row * p.room;
  int32_t* index = p.index + row * p.keep;
  float* new_mass = p.new_mass + row * p.keep;
  // the slice, in runs of `run` candidates per thread (odd: no bank conflicts)
  const int share = static_cast<int>((old + ctas - 1) / ctas);
  const int run = ((share + kThreads - 1) / kThreads) | 1;
  const int j0 = min(static_cast<int64_t>(old), int64_t(rank) * run * kThreads);
  const int len = static_cast<int>(min(static_cast<int64_t>(old), int64_t(rank + 1) * run * kThreads)) - j0;
  const bool choose = m > newest;             // the same in all CTAs of the cluster
  const bool held = len <= slice_room;
  if (rank == 0 && tid == 0 && row % p.from.heads == 0) p.new_lens[s] = m;
  if (choose && held)
    for (int j = tid; j < len; j += kThreads) keys[j] = ordered(mass[j0 + j]);
  if (tid == 0) sh_prefix = 0, sh_left = m - newest;
  auto key_at = [&](int j) { return held ? keys[j] : ordered(mass[j0 + j]); };
  if (choose) {
    // ---- the last kept candidate's bits, and how many of its equals are kept
#pragma unroll 1
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) count[tid] = 0;
      __syncthreads();
      const uint32_t prefix = sh_prefix, mask = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
      for (int j = tid; j < (len + 31) / 32 * 32; j += kThreads) {
        const uint32_t u = j < len ? key_at(j) : 0u;
        const bool in = j < len && (u & mask) == prefix;
        // equal values (and equal high bytes) are common: one add for a warp's
        const uint32_t bin = in ? (u >> shift) & 255 : 256;
        const unsigned same = __match_any_sync(0xffffffffu, bin);
        if (in && lane == __ffs(same) - 1) atomicAdd(&count[bin], __popc(same));
      }
      cluster_sync();
      if (tid < 256) {
        uint32_t sum = 0;
        const uint32_t at = smem_addr(&count[tid]);
        for (uint32_t r = 0; r < ctas; ++r) sum += ld_cluster_u32(map_to_rank(at, r));
        total[tid] = sum;
      }
      cluster_sync();                         // the counts may be cleared again
      if (warp == 0) {
        // from the top: the bin in which the running count reaches `left`
        const uint32_t left = sh_left;
        uint32_t above = 0;
        for (int b0 = 224; b0 >= 0; b0 -= 32) {
          uint32_t c = total[b0 + 31 - lane];             // lane 0: the largest bin
          uint32_t x = c;
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) {
            const uint32_t o = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += o;
          }
          const unsigned reach = __ballot_sync(0xffffffffu, above + x >= left);
          if (reach) {
            const int i = __ffs(reach) - 1;
            if (lane == i) {
              sh_prefix = prefix | static_cast<uint32_t>(b0 + 31 - i) << shift;
              sh_left = left - (above + x - c);
            }
            break;
          }
          above += __shfl_sync(0xffffffffu, x, 31);
        }
      }
      __syncthreads();
    }
    // ---- each thread's run: how many are larger, how many equal
    const uint32_t bar = sh_prefix, equals = sh_left;
    const int from = min(len, tid * run), to = min(len, from + run);
    uint32_t larger = 0, same = 0;
    for (int j = from; j < to; ++j) {
      const uint32_t u = key_at(j);
      larger += u > bar;
      same += u == bar;
    }
    // exclusive sums over the block (16 bits each would overflow: two rounds)
    uint32_t before[2], all[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t v = k ? same : larger;
      uint32_t x = v;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += o;
      }
      __syncthreads();
      if (lane == 31) warp_sum[warp] = x;
      __syncthreads();
      uint32_t b = 0, a = 0;
      for (int i = 0; i < kWarps; ++i) {
        if (i < warp) b += warp_sum[i];
        a += warp_sum[i];
      }
      before[k] = b + x - v;
      all[k] = a;
    }
    if (tid == 0) mine[0] = all[0], mine[1] = all[1];
    cluster_sync();
    uint32_t larger_before = 0, same_before = 0;
    for (uint32_t r = 0; r < rank; ++r) {
      larger_before += ld_cluster_u32(map_to_rank(smem_addr(&mine[0]), r));
      same_before += ld_cluster_u32(map_to_rank(smem_addr(&mine[1]), r));
    }
    // of the equals before this run, the first `equals` are kept
    uint32_t eq = same_before + before[1];
    uint32_t at = larger_before + before[0] + min(eq, equals);
    for (int j = from; j < to; ++j) {
      const uint32_t u = key_at(j);
      const bool take = u > bar || (u == bar && eq < equals);
      eq += u == bar;
      if (take) {
        index[at] = j0 + j;
        new_mass[at] = mass[j0 + j];
        ++at;
      }
    }
    cluster_sync();                           // no CTA ends while its counts are read
  }
  for (int i = rank * kThreads + tid; i < p.keep - (m - newest); i += ctas * kThreads) {
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

int run_evict(const Evict& p, const Device& d, cudaStream_t stream) {
  const int64_t rows = int64_t(p.count) * p.from.heads;
  const int64_t blocks = (rows * p.keep + 7) / 8;
  // CTAs of a cluster: while there are SMs for them and candidates for each
  int ctas = 1;
  while (ctas < kMaxCluster && rows * ctas < d.num_sms && p.room > int64_t(ctas) * kMinSlice) ctas *= 2;
  if (rows * ctas > INT32_MAX || blocks > INT32_MAX) return NVFP4_ERR_SHAPE;
  // the longest slice there can be, as far as it is held
  const int64_t slice = ((p.room + ctas - 1) / ctas + kThreads) / kThreads * kThreads + kThreads;
  const int held = static_cast<int>(std::min<int64_t>(slice, kSmemKeys));
  static std::atomic<bool> ready[kMaxDevices];
  if (const int st = allow_smem(choose_kernel, kSmemKeys * 4, d, ready)) return st;
  if (const int st = launch_clusters(ctas, choose_kernel, dim3(static_cast<unsigned>(rows * ctas)),
                                     dim3(kThreads), held * 4, stream, p, held))
    return st;
  return launch(move_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream, p);
}

}  // namespace attn
}  // namespace nvfp4
