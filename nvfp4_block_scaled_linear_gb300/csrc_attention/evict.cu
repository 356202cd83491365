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
// choice is latency (a cluster barrier a pass), so it is spread over as many
// CTAs as the slices keep busy.
//
// Measured: of 65543 keys of 4 heads of 256, 8192 kept, 39 us (68 MB in and out,
// 10 us at the copy rate: choosing takes some 24, moving 14); of 16 sequences of
// up to 9001 keys in e4m3 pages, 8 heads of 128, 1000 kept each, 36 us.
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
  __shared__ uint32_t counts[4][256];         // this slice's, pass by pass
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
  // the slice, in runs of `run` candidates per thread (odd: no bank conflicts)
  const int share = static_cast<int>((old + ctas - 1) / ctas);
  const int run = ((share + kThreads - 1) / kThreads) | 1;
  const int j0 = min(static_cast<int64_t>(old), int64_t(rank) * run * kThreads);
  const int len = static_cast<int>(min(static_cast<int64_t>(old), int64_t(rank + 1) * run * kThreads)) - j0;
  const bool choose = m > newest;             // the same in all CTAs of the cluster
  const bool held = len <= slice_room;
  if (rank == 0 && tid == 0 && row % p.from.heads == 0) p.new_lens[s] = m;
  if (choose && held)
#pragma unroll 8
    for (int j = tid; j < len; j += kThreads) keys[j] = ordered(mass[j0 + j]);
  if (tid == 0) sh_prefix = 0, sh_left = m - newest;
  auto key_at = [&](int j) { return held ? keys[j] : ordered(mass[j0 + j]); };
  for (int i = tid; i < 4 * 256; i += kThreads) counts[i >> 8][i & 255] = 0;
  if (choose) {
    // ---- the last kept candidate's bits, and how many of its equals are kept
#pragma unroll 1
    for (int shift = 24; shift >= 0; shift -= 8) {
      __syncthreads();
      uint32_t* count = counts[shift >> 3];
      const uint32_t prefix = sh_prefix, mask = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
#pragma unroll 4
      for (int j = tid; j < (len + 31) / 32 * 32; j += kThreads) {
        const uint32_t u = j < len ? key_at(j) : 0u;
        const uint32_t bin = (u >> shift) & 255;
        unsigned left = __ballot_sync(0xffffffffu, j < len && (u & mask) == prefix);
        // equal values (and equal high bytes) are common: the first lane's bin
        // with one add for all that share it, the rest one by one
        if (left) {
          const int lead = __ffs(left) - 1;
          const unsigned same =
              left & __ballot_sync(0xffffffffu, bin == __shfl_sync(0xffffffffu, bin, lead));
          if (lane == lead) atomicAdd(&count[bin], __popc(same));
          left &= ~same;
        }
        if (left >> lane & 1) atomicAdd(&count[bin], 1u);
      }
      cluster_sync();
      if (tid < 256) {
        uint32_t sum = 0;
        const uint32_t at = smem_addr(&count[tid]);
        for (uint32_t r = 0; r < ctas; ++r) sum += ld_cluster_u32(map_to_rank(at, r));
        total[tid] = sum;
      }
      __syncthreads();
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
    }
    __syncthreads();
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
      if (take) index[at++] = j0 + j;
    }
    cluster_sync();                           // no CTA ends while its counts are read
  }
  for (int i = rank * kThreads + tid; i < p.keep - (m - newest); i += ctas * kThreads) {
    const int at = m - newest + i;
    index[at] = at < m ? old + i : -1;
  }
}

// Sixteen e4m3 codes of scale `from` as codes of scale `to`, one rounding each.
__device__ __forceinline__ uint4 rescale(uint4 v, float from, float to) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t c[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
      c[k] = __nv_cvt_float2_to_fp8x2(
          make_float2(e4m3_to_f32(w[i] >> (16 * k) & 0xFFu) * from / to,
                      e4m3_to_f32(w[i] >> (16 * k + 8) & 0xFFu) * from / to),
          __NV_SATFINITE, __NV_E4M3);
    w[i] = c[0] | c[1] << 16;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A block moves the rows of kPlaces kept places of one sequence and head: a
// thread per place hands on its mass and finds where its rows come from and go
// to, then all threads copy 16 bytes at a time, several on their way each.  Where
// the two caches have different scales for the head, the codes are changed on the
// way, so that a row keeps the values that it stands for.
constexpr int kPlaces = 64;
constexpr int kMoveThreads = 256;

__global__ void __launch_bounds__(kMoveThreads) move_kernel(const Evict p) {
  __shared__ int64_t from[2][kPlaces], to[2][kPlaces];     // bytes; from < 0: nothing
  griddep_wait();
  griddep_launch_dependents();
  const int row = blockIdx.x, tid = threadIdx.x;
  const int s = row / p.from.heads, h = row - s * p.from.heads;
  const int size = p.from.e4m3 ? 1 : 2;
  if (tid < kPlaces) {
    const int r = blockIdx.y * kPlaces + tid;
    const int j = r < p.keep ? p.index[int64_t(row) * p.keep + r] : -1;
    if (r < p.keep)
      p.new_mass[int64_t(row) * p.keep + r] = j >= 0 ? p.mass[row * p.room + j] : 0.f;
    from[0][tid] = -1;
    if (j >= 0) {
      const int jp = j / p.from.page_size, rp = r / p.to.page_size;
      const int64_t a = checked_page(p.table[int64_t(s) * p.width + jp], p.from.pages, p.err);
      const int64_t b = checked_page(p.to_table[int64_t(s) * p.to_width + rp], p.to.pages, p.err);
      if (a != p.from.pages && b != p.to.pages) {
        const int jf = j - jp * p.from.page_size, rt = r - rp * p.to.page_size;
        from[0][tid] = (a * p.from.ks[0] + jf * p.from.ks[1] + h * p.from.ks[2]) * size;
        from[1][tid] = (a * p.from.vs[0] + jf * p.from.vs[1] + h * p.from.vs[2]) * size;
        to[0][tid] = (b * p.to.ks[0] + rt * p.to.ks[1] + h * p.to.ks[2]) * size;
        to[1][tid] = (b * p.to.vs[0] + rt * p.to.vs[1] + h * p.to.vs[2]) * size;
      }
    }
  }
  __syncthreads();
  // 16-byte pieces of a row: a power of two, 4 to 32
  const int shift = 31 - __clz(p.from.dim * size >> 4);
  const int piece = tid & ((1 << shift) - 1), first = tid >> shift, step = kMoveThreads >> shift;
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    const uint8_t* src = static_cast<const uint8_t*>(v ? p.from.v : p.from.k) + piece * 16;
    uint8_t* dst = static_cast<uint8_t*>(v ? p.to.v : p.to.k) + piece * 16;
    const float* from_scale = v ? p.from.v_scale : p.from.k_scale;
    const float* to_scale = v ? p.to.v_scale : p.to.k_scale;
    const float a = from_scale ? from_scale[h] : 1.f, b = to_scale ? to_scale[h] : 1.f;
    if (a != b) {
#pragma unroll 1
      for (int i = first; i < kPlaces; i += step)
        if (from[0][i] >= 0)
          *reinterpret_cast<uint4*>(dst + to[v][i]) =
              rescale(__ldcs(reinterpret_cast<const uint4*>(src + from[v][i])), a, b);
      continue;
    }
#pragma unroll 4
    for (int i = first; i < kPlaces; i += step) {
      if (from[0][i] < 0) continue;
      *reinterpret_cast<uint4*>(dst + to[v][i]) =
          __ldcs(reinterpret_cast<const uint4*>(src + from[v][i]));
    }
  }
}

}  // namespace

int run_evict(const Evict& p, const Device& d, cudaStream_t stream) {
  const int64_t rows = int64_t(p.count) * p.from.heads;
  const int64_t blocks = (int64_t(p.keep) + kPlaces - 1) / kPlaces;
  // CTAs of a cluster: while there are SMs for them and candidates for each
  int ctas = 1;
  while (ctas < kMaxCluster && rows * ctas < d.num_sms && p.room > int64_t(ctas) * kMinSlice) ctas *= 2;
  if (rows * ctas > INT32_MAX || blocks > 65535) return NVFP4_ERR_SHAPE;
  // the longest slice there can be, as far as it is held
  const int64_t slice = ((p.room + ctas - 1) / ctas + kThreads) / kThreads * kThreads + kThreads;
  const int held = static_cast<int>(std::min<int64_t>(slice, kSmemKeys));
  static std::atomic<bool> ready[kMaxDevices];
  if (const int st = allow_smem(choose_kernel, kSmemKeys * 4, d, ready)) return st;
  if (const int st = launch_clusters(ctas, choose_kernel, dim3(static_cast<unsigned>(rows * ctas)),
                                     dim3(kThreads), held * 4, stream, p, held))
    return st;
  return launch(move_kernel, dim3(static_cast<unsigned>(rows), static_cast<unsigned>(blocks)),
                dim3(kMoveThreads), 0, stream, p);
}

}  // namespace attn
}  // namespace nvfp4
