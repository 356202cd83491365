// product_narrow.cu -- up to 32 NVFP4 rows times an NVFP4 weight.
//
//   y[m, n] = scale * sum_k w[n, k] a[m, k]
//
// The weights are the MMA's 128 rows and the tokens its 8 to 32 columns: a product
// then reads the weights once and next to nothing else, 32 clocks for 64 k where the
// other order takes 64, and the tokens' sums take 32 columns of TMEM.  A CTA has 128
// outputs (of a gate/up pair 128 rows of each, in two accumulators: both sums of an
// output are in one lane), the k split over the CTAs of a cluster.
//
// A lane holds an output's sums for every token.  They go through shared memory,
// [CTA][part][token][output], to where 16 outputs of a token are one thread's; the
// outputs are shared out over the cluster in pieces of 16, and a piece's owner adds
// the CTAs' sums in their order: no atomics, the same bits on every run.  The sums
// have shared memory of their own and the cluster's CTAs have met before the first
// product, so that one barrier is between a CTA's last product and the outputs.
//
// Bound by the weights' bytes where there are many, by latency where there are few:
// beyond its bytes a call needs the tokens' copy after the kernel ahead has ended (some
// 1.5 us to the first product), the exchange (1 us) and the outputs (0.7 us).  Measured
// back to back, weights from memory, one token: 34816 x 5120 gated 18.2 us, 5.5 TB/s;
// 5120 x 17408 11.5 us, 4.4 TB/s; 8192 x 5120 7.0 us; 5120 x 6144 6.5 us; 32 tokens 19.5,
// 12.0, 8.0, 7.5.
//
// Warps: 0 copies, 1 MMA, 2 TMEM allocation; all eight the outputs.
#include <algorithm>

#include "product.cuh"

namespace nvfp4 {
namespace w4a4 {
namespace {

constexpr int kThreads = 256;
constexpr int kAllSmem = 226 * 1024, kHalfSmem = 112 * 1024;
constexpr int kMaxStages = 12;
constexpr int kMaxSplit = 8;
constexpr int kTile = 128;                       // outputs of a CTA
constexpr int kPieces = kTile / 16;
constexpr int kWeights = kTile * 128;            // bytes of 128 rows' codes a stage
constexpr uint32_t kCols = 128;                  // TMEM: sums of 32 tokens twice, scales
constexpr uint32_t kColW = 64, kColA = 96;

struct Narrow {
  Product p;
  int cols;          // the tokens rounded up to 8
  int split;         // CTAs of a cluster
  int stages, stage_bytes, smem;
};

// Pieces of an owner, at most, and bytes of the sums that it gathers.
__host__ __device__ constexpr int own_pieces(int split) { return (kPieces + split - 1) / split; }
constexpr int sums_bytes(int parts, int split, int cols) {
  return split * parts * cols * own_pieces(split) * 64;
}

__device__ __forceinline__ void tmem_ld_8cols(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void st_cluster_b32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// kPer: parts of an output (its sum, or gate and up) that a stage brings weights for.
template <int kMode, int kPer>
__global__ void __launch_bounds__(kThreads, 1)
    narrow_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w,
                  const Narrow f) {
  constexpr int kParts = kMode == kPlain ? 1 : 2, kRuns = kParts / kPer;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], done;
  __shared__ int abort_word;
  __shared__ uint32_t tmem_slot;
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  volatile int* abort_flag = &abort_word;
  const Product& p = f.p;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = f.split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int tile = blockIdx.x / f.split;
  const int rows = static_cast<int>(p.M);
  const int steps = static_cast<int>(p.K / kStageK);
  const int s0 = static_cast<int>(int64_t(steps) * rank / f.split);
  const int s1 = static_cast<int>(int64_t(steps) * (rank + 1) / f.split);
  const int n_stages = (s1 - s0) * kRuns;
  auto w_row = [&](int i) { return tile * kTile + i * static_cast<int>(p.N / 2); };
  const int a_off = kPer * kWeights, sw_off = a_off + f.cols * 128;
  const int sa_off = sw_off + kPer * 4 * kScaleBlock;
  float* sums = reinterpret_cast<float*>(smem + f.stages * f.stage_bytes);

  if (threadIdx.x == 0) {
    for (int s = 0; s < f.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&done, 1);
    abort_word = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    tmem_alloc(&tmem_slot, kCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncwarp();
  // (the others of the cluster run, so that sums can be stored with them)
  if (f.split > 1)
    cluster_sync();
  else
    __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = tmem_slot;

  if (warp == 0) {
    // the whole warp walks the stages, an elected lane issues
    // stage g: k step g / kRuns, parts from g % kRuns on
    auto weights = [&](int g, int slot) {
      const int it = s0 + g / kRuns;
      uint8_t* st = smem + slot * f.stage_bytes;
      mbar_arrive_expect_tx(&full[slot], f.stage_bytes);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int w = w_row(g % kRuns + i);
        tma_load_2d(st + i * kWeights, &tm_w, &full[slot], it * 128, w);
        bulk_load(st + sw_off + i * 4 * kScaleBlock,
                  p.w_scales + (int64_t(w / 128) * (p.K / kMmaK) + it * 4) * kScaleBlock, 4 * kScaleBlock,
                  &full[slot]);
      }
    };
    auto tokens = [&](int g, int slot) {
      const int it = s0 + g / kRuns;
      uint8_t* st = smem + slot * f.stage_bytes;
      tma_load_2d(st + a_off, &tm_a, &full[slot], it * 128, 0);
      bulk_load(st + sa_off, p.a_scales + int64_t(it) * 4 * kScaleBlock, 4 * kScaleBlock, &full[slot]);
    };
    // weights do not wait for the kernel ahead in the stream, tokens do
    const int pre = n_stages < f.stages ? n_stages : f.stages;
    if (elect_one()) {
      prefetch_tensormap(&tm_a);
      prefetch_tensormap(&tm_w);
      for (int it = 0; it < pre; ++it) weights(it, it);
    }
    __syncwarp();
    griddep_wait();
    if (elect_one()) {
      griddep_launch_dependents();                               // (after the wait: see launch())
      for (int it = 0; it < pre; ++it) tokens(it, it);
    }
    __syncwarp();
    int issued = pre, slot = pre == f.stages ? 0 : pre;
    uint32_t parity = 0;
    for (int it = pre; it < n_stages; ++it) {
      if (!__all_sync(0xffffffffu, wait(&empty[slot], parity, abort_flag))) break;
      if (elect_one()) {
        weights(it, slot);
        tokens(it, slot);
      }
      __syncwarp();
      ++issued;
      if (++slot == f.stages) slot = 0, parity ^= 1u;
    }
    // nothing is left in flight, whatever became of the others
    for (int it = issued > f.stages ? issued - f.stages : 0; it < issued; ++it) {
      volatile int none = 0;
      if (!wait(&full[it % f.stages], (it / f.stages) & 1, &none)) *abort_flag = 1;
    }
  } else if (warp == 1) {
    // (before any wait with a limit: the kernel ahead may take its time)
    griddep_wait();
    const uint32_t idesc = idesc_nvfp4(128, f.cols);
    int slot = 0;
    uint32_t parity = 0;
    for (int g = 0; g < n_stages; ++g) {
      if (!__all_sync(0xffffffffu, wait(&full[slot], parity, abort_flag))) break;
      tc_fence_after_sync();
      if (elect_one()) {
        const uint32_t st = smem_addr(smem) + slot * f.stage_bytes, d = tmem + 32 * (g % kRuns);
        const uint64_t w = umma_desc_sw128(st), a = umma_desc_sw128(st + a_off);
        const uint64_t sw = scale_desc(st + sw_off), sa = scale_desc(st + sa_off);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
          for (int i = 0; i < kPer; ++i)
            copy_scales(tmem + kColW + 4 * (kPer * j + i), sw + (4 * i + j) * (kScaleBlock >> 4));
          copy_scales(tmem + kColA + 4 * j, sa + j * (kScaleBlock >> 4));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < kPer; ++i)
            umma_nvfp4(d + 32 * i, w + 2 * j + i * (kWeights >> 4), a + 2 * j, idesc,
                       tmem + kColW + 4 * (kPer * j + i), tmem + kColA + 4 * j, (g / kRuns | j) != 0);
        umma_commit(&empty[slot]);
      }
      __syncwarp();
      if (++slot == f.stages) slot = 0, parity ^= 1u;
    }
    if (elect_one()) umma_commit(&done);
    __syncwarp();
    volatile int none = 0;
    if (!wait(&done, 0, &none)) *abort_flag = 1;
  }
  __syncwarp();
  // every product and copy of this CTA is over
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const int own = own_pieces(f.split);
  {
    // two warps for each quarter of the lanes, taking eights of tokens in turn
    const int quarter = warp & 3, piece = quarter * 2 + (lane >> 4);
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t here = smem_addr(sums) + ((rank * kParts * f.cols * own + piece / f.split) * 16 + (lane & 15)) * 4;
    const uint32_t to = f.split > 1 ? map_to_rank(here, piece % f.split) : here;
    for (int c = (warp >> 2) * 8; c < f.cols; c += 16) {
#pragma unroll
      for (int part = 0; part < kParts; ++part) {
        uint32_t v[8];
        __syncwarp();
        tmem_ld_8cols(lanes + 32 * part + c, v);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (c + i < rows) st_cluster_b32(to + (part * f.cols + c + i) * own * 64, v[i]);
      }
    }
  }
  if (f.split > 1)
    cluster_sync();
  else
    __syncthreads();
  const int pieces = (kPieces - rank + f.split - 1) / f.split;      // this CTA's: rank, rank + split, ...
  for (int i = threadIdx.x; i < rows * pieces; i += kThreads) {
    const int row = i / pieces, mine = i - row * pieces;
    float v[kParts][16];
#pragma unroll
    for (int part = 0; part < kParts; ++part) {
#pragma unroll
      for (int k = 0; k < 16; ++k) v[part][k] = 0.f;
      for (int q = 0; q < f.split; ++q) {
        const float4* at = reinterpret_cast<const float4*>(sums + ((q * kParts + part) * f.cols + row) * own * 16 + mine * 16);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float4 x = at[k];
          v[part][4 * k] += x.x, v[part][4 * k + 1] += x.y, v[part][4 * k + 2] += x.z, v[part][4 * k + 3] += x.w;
        }
      }
    }
    outputs16<kMode>(p, row, tile * kTile + (rank + mine * f.split) * 16, v);
  }
  if (*abort_flag && threadIdx.x == 0) atomicOr(p.err, NVFP4_W4A4_TIMEOUT);
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 2) tmem_dealloc(tmem, kCols);
}

template <int kMode, int kPer>
int run(const Narrow& f, const Device& d, cudaStream_t stream) {
  static std::atomic<bool> ready[kMaxDevices];
  if (const int st = allow_smem(narrow_kernel<kMode, kPer>, kAllSmem, d, ready)) return st;
  CUtensorMap tm_a, tm_w;
  if (!codes_map(&tm_a, f.p.a_codes, f.p.M, f.p.K, f.cols) || !codes_map(&tm_w, f.p.w_codes, f.p.N, f.p.K, kTile))
    return NVFP4_ERR_LAUNCH;
  constexpr int kParts = kMode == kPlain ? 1 : 2;
  if (f.stages < 1 || f.split < 1 || f.split > kMaxSplit ||
      f.stages * f.stage_bytes + sums_bytes(kParts, f.split, f.cols) > f.smem - 1024)
    return NVFP4_ERR_LAUNCH;
  return launch(f.split, narrow_kernel<kMode, kPer>, dim3(static_cast<unsigned>(f.p.N / (kTile * kParts)) * f.split),
                dim3(kThreads), f.smem, stream, tm_a, tm_w, f);
}

}  // namespace

int run_product_narrow(const Product& p, const Device& d, cudaStream_t stream) {
  Narrow f{};
  f.p = p;
  f.cols = static_cast<int>((p.M + 7) / 8 * 8);
  const int parts = p.swiglu ? 2 : 1;
  const int64_t steps = p.K / kStageK, tiles = p.N / (kTile * parts);
  // A stage for each of gate and up where there are more tiles than SMs: half of an SM's
  // shared memory then holds four, and two CTAs an SM are one round.  One token through
  // 40960 x 5120 22.7 us against 28.9 (two rounds of CTAs with both in a stage); where a
  // tile has an SM for itself 34816 x 5120 19.0 against 18.2.
  const int per = tiles > d.num_sms ? 1 : parts;
  f.stage_bytes = per * kWeights + f.cols * 128 + 4 * kScaleBlock * (per + 1);
  // Of the splits that the device holds at one time the one with the least time, in ns
  // as measured: 180 a step (gated 310), and where sums are exchanged 900 and 60 a CTA.
  f.split = 1;
  int64_t least = INT64_MAX;
  for (int split = 1; split <= kMaxSplit && split <= steps && split * tiles <= std::max<int64_t>(d.num_sms, tiles);
       ++split) {
    if (split > 1 && tiles > most_clusters(split, d)) continue;
    const int64_t ns = (steps + split - 1) / split * (p.swiglu ? 310 : 180) + (split > 1 ? 900 + split * 60 : 0);
    if (ns < least) least = ns, f.split = split;
  }
  const int sums = sums_bytes(parts, f.split, f.cols);
  // With half of an SM's shared memory the next kernel's CTAs are resident, with their
  // first stages on the way, before this one's end; with all of it the ring is twice as
  // deep.  8192 x 5120, 10 steps: 7.0 us against 7.6; 5120 x 17408, 23 steps, 32 tokens:
  // 13.7 against 12.0.  Half holds two stages of both gate and up, too few: 34816 x 5120 22.5 us
  // against 18.2, 12288 x 2048 6.7 against 5.9.
  const int half = (kHalfSmem - 1024 - sums) / f.stage_bytes;
  f.smem = per == 2 || (steps / f.split > 2 * half && tiles <= d.num_sms) ? kAllSmem : kHalfSmem;
  f.stages = std::min((f.smem - 1024 - sums) / f.stage_bytes, kMaxStages);
  if (!p.swiglu) return run<kPlain, 1>(f, d, stream);
  if (per == 1) return p.codes ? run<kGatedRows, 1>(f, d, stream) : run<kGated, 1>(f, d, stream);
  return p.codes ? run<kGatedRows, 2>(f, d, stream) : run<kGated, 2>(f, d, stream);
}

}  // namespace w4a4
}  // namespace nvfp4
