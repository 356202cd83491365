// product_few.cu -- NVFP4 rows times an NVFP4 weight, 33 rows and more, 128 a CTA.
//
//   y[m, n] = scale * sum_k a[m, k] w[n, k]
//
// One tile of up to 128 tokens (the MMA's 128 rows; those beyond the tokens are
// never read back) by kN weight rows (the MMA's columns), the k split over the
// CTAs of a cluster.  Codes come by TMA, 256 k a stage, the blocks of scales by
// bulk copies; tcgen05 multiplies both as they are, with the scales in TMEM.
// Where there are few tokens the tokens' box is only as high as they are, and
// the MMA's other rows read whatever follows in the stage.
//
// The outputs of a tile are shared out over the cluster in pieces of 16 columns:
// each CTA stores its sums of a piece in its owner's shared memory, and the owner
// adds the CTAs' sums in their order: no atomics, the same bits on every run.
//
// Bound by an SM's port to L2 (64 bytes a clock): 128 tokens need 0.28 us a stage of 256
// k, 18 KB of tokens beside 18 KB of weights; and beyond the stages by the tokens' copy after the kernel ahead has ended, the
// exchange (1.3 us and more with more rows) and the outputs.  Measured back to back,
// weights from memory, 128 tokens: 34816 x 5120 gated 20.5 us, 4.9 TB/s (40960 x 5120,
// 160 tiles on 152 SMs, 32.4); 5120 x 17408 14.2 us; 8192 x 5120 9.4 us; 5120 x 6144 9.0 us.
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

struct Few {
  Product p;
  int a_rows;        // rows of a box of tokens
  int split;         // CTAs of a cluster
  int stages, stage_bytes, smem;
};

__device__ __forceinline__ void st_cluster_f32x4(uint32_t addr, const float* v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3])
               : "memory");
}

// Bytes of the sums that an owner gathers: of every CTA its pieces of the rows.
constexpr int sums_bytes(int n, bool gated, int split, int rows) {
  const int parts = gated ? 2 : 1, pieces = n / parts / 16;
  return split * ((pieces + split - 1) / split) * parts * ((rows + 31) / 32 * 32) * 64;
}

// Where the sums lie in their owner: [CTA][piece of the owner's][four columns][row],
// so that a warp, a row a lane, stores and loads 512 bytes together.
struct Sums {
  int rows;          // of whole warps
  int pieces;        // of one owner, at most
  __device__ __forceinline__ uint32_t at(int cta, int piece, int row) const {
    return static_cast<uint32_t>(((cta * pieces + piece) * 4 * rows + row) * 16);
  }
};

// The sum over the CTAs, in their order, of the 16 columns at `at`.
__device__ __forceinline__ void sum16(const uint8_t* at, int split, int cta_bytes, int four_bytes, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = 0.f;
  for (int q = 0; q < split; ++q) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 f = *reinterpret_cast<const float4*>(at + q * cta_bytes + i * four_bytes);
      v[4 * i] += f.x, v[4 * i + 1] += f.y, v[4 * i + 2] += f.z, v[4 * i + 3] += f.w;
    }
  }
}

template <int kN, int kMode>
__global__ void __launch_bounds__(kThreads, 1)
    few_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w,
               const Few f) {
  constexpr int kParts = kMode == kPlain ? 1 : 2;         // parts of an output: its sum, or gate and up
  constexpr int kOut = kN / kParts;                       // outputs of a row of the tile
  constexpr int kBlocks = kMode == kPlain ? kN / 128 : 2; // blocks of 128 rows' scales
  constexpr int kBox = kN / kBlocks;                      // weight rows of a block
  constexpr uint32_t kCols = kN == 256 ? 512 : 256;       // TMEM: sums, then scales
  constexpr uint32_t kScaleA = kN, kScaleB = kN + 16;     // 4 columns per 64 k and 128 rows
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
  const int m0 = blockIdx.y * 128;
  const int rows = static_cast<int>(p.M - m0 < 128 ? p.M - m0 : 128);
  const int steps = static_cast<int>(p.K / kStageK);
  const int s0 = static_cast<int>(int64_t(steps) * rank / f.split);
  const int s1 = static_cast<int>(int64_t(steps) * (rank + 1) / f.split);
  const int n_steps = s1 - s0;
  // first weight row of block i of the tile (of a gated tile of 64 outputs the first or
  // the second half of 128 rows)
  auto w_row = [&](int i) {
    return kMode == kPlain ? tile * kN + i * kBox : tile * kOut + i * static_cast<int>(p.N / 2);
  };
  const int a_bytes = f.a_rows * 128;
  const int w_off = a_bytes, sa_off = w_off + kN * 128, sb_off = sa_off + 4 * kScaleBlock;

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
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = tmem_slot;

  if (warp == 0) {
    // the whole warp walks the stages, an elected lane issues
    auto weights = [&](int it, int slot) {
      uint8_t* st = smem + slot * f.stage_bytes;
      mbar_arrive_expect_tx(&full[slot], f.stage_bytes);
#pragma unroll
      for (int i = 0; i < kBlocks; ++i) {
        tma_load_2d(st + w_off + i * kBox * 128, &tm_w, &full[slot], (s0 + it) * 128, w_row(i));
        bulk_load(st + sb_off + i * 4 * kScaleBlock,
                  p.w_scales + (int64_t(w_row(i) / 128) * (p.K / kMmaK) + (s0 + it) * 4) * kScaleBlock,
                  4 * kScaleBlock, &full[slot]);
      }
    };
    auto tokens = [&](int it, int slot) {
      uint8_t* st = smem + slot * f.stage_bytes;
      tma_load_2d(st, &tm_a, &full[slot], (s0 + it) * 128, m0);
      bulk_load(st + sa_off,
                p.a_scales + (int64_t(blockIdx.y) * (p.K / kMmaK) + (s0 + it) * 4) * kScaleBlock,
                4 * kScaleBlock, &full[slot]);
    };
    // weights do not wait for the kernel ahead in the stream, tokens do
    const int pre = n_steps < f.stages ? n_steps : f.stages;
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
    for (int it = pre; it < n_steps; ++it) {
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
    // two halves of 128 rows' scales cannot be one operand: an MMA for each
    constexpr int kMmas = kBox == 64 ? 2 : 1;
    constexpr uint32_t idesc = idesc_nvfp4(128, kN / kMmas);
    const uint32_t half = kMmas == 2 && (tile & 1) ? 2 : 0;
    int slot = 0;
    uint32_t parity = 0;
    for (int it = 0; it < n_steps; ++it) {
      if (!__all_sync(0xffffffffu, wait(&full[slot], parity, abort_flag))) break;
      tc_fence_after_sync();
      if (elect_one()) {
        const uint32_t st = smem_addr(smem) + slot * f.stage_bytes;
        const uint64_t a = umma_desc_sw128(st), b = umma_desc_sw128(st + w_off);
        const uint64_t sa = scale_desc(st + sa_off), sb = scale_desc(st + sb_off);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          copy_scales(tmem + kScaleA + 4 * j, sa + j * (kScaleBlock >> 4));
#pragma unroll
          for (int i = 0; i < kBlocks; ++i)
            copy_scales(tmem + kScaleB + 4 * (kBlocks * j + i), sb + (4 * i + j) * (kScaleBlock >> 4));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < kMmas; ++i)
            umma_nvfp4(tmem + kBox * i, a + 2 * j, b + 2 * j + i * (kBox * 128 >> 4), idesc, tmem + kScaleA + 4 * j,
                       tmem + kScaleB + 4 * (kBlocks * j + i) + half, (it | j) != 0);
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
  // every product and copy of the cluster is over
  tc_fence_before_sync();
  if (f.split > 1)
    cluster_sync();
  else
    __syncthreads();
  tc_fence_after_sync();
  constexpr int kPieces = kOut / 16;
  auto out = [&](int row, int piece, float (&v)[kParts][16]) {
    outputs16<kMode>(p, m0 + row, tile * kOut + piece * 16, v);
  };
  // two warps for each quarter of the lanes, taking pieces in turn
  const int quarter = warp & 3, row = quarter * 32 + lane;
  const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
  auto load = [&](int piece, float (&v)[kParts][16]) {
    uint32_t r[kParts][16];
    __syncwarp();
#pragma unroll
    for (int part = 0; part < kParts; ++part) tmem_ld_16cols(lanes + 16 * piece + kOut * part, r[part]);
    tmem_ld_wait();
#pragma unroll
    for (int part = 0; part < kParts; ++part)
#pragma unroll
      for (int i = 0; i < 16; ++i) v[part][i] = __uint_as_float(r[part][i]);
  };
  if (f.split == 1) {
    if (quarter * 32 < rows)
      for (int piece = warp >> 2; piece < kPieces; piece += 2) {
        float v[kParts][16];
        load(piece, v);
        if (row < rows) out(row, piece, v);
      }
  } else {
    Sums sums;
    sums.rows = (rows + 31) & ~31;
    sums.pieces = (kPieces + f.split - 1) / f.split * kParts;
    if (quarter * 32 < rows) {
      const uint32_t here = smem_addr(smem) + sums.at(rank, 0, row);
      for (int q = 0; q < f.split; ++q) {
        const uint32_t to = map_to_rank(here, q);
        int mine = 0;
        for (int piece = q; piece < kPieces; piece += f.split, ++mine) {
          if ((piece & 1) != warp >> 2) continue;
          float v[kParts][16];
          load(piece, v);
          if (row < rows)
#pragma unroll
            for (int part = 0; part < kParts; ++part)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                st_cluster_f32x4(to + ((mine * kParts + part) * 4 + i) * sums.rows * 16, v[part] + 4 * i);
        }
      }
    }
    cluster_sync();
    const int pieces = (kPieces - rank + f.split - 1) / f.split;    // this CTA's: rank, rank + split, ...
    const int cta_bytes = sums.pieces * sums.rows * 64, four_bytes = sums.rows * 16;
    for (int i = threadIdx.x; i < sums.rows * pieces; i += kThreads) {
      const int mine = i / sums.rows, r = i - mine * sums.rows;
      if (r >= rows) continue;
      float v[kParts][16];
#pragma unroll
      for (int part = 0; part < kParts; ++part)
        sum16(smem + sums.at(0, mine * kParts + part, r), f.split, cta_bytes, four_bytes, v[part]);
      out(r, rank + mine * f.split, v);
    }
  }
  if (*abort_flag && threadIdx.x == 0) atomicOr(p.err, NVFP4_W4A4_TIMEOUT);
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 2) tmem_dealloc(tmem, kCols);
}

template <int kN, int kMode>
int run(Few f, const Device& d, cudaStream_t stream) {
  static std::atomic<bool> ready[kMaxDevices];
  if (const int st = allow_smem(few_kernel<kN, kMode>, kAllSmem, d, ready)) return st;
  CUtensorMap tm_a, tm_w;
  if (!codes_map(&tm_a, f.p.a_codes, f.p.M, f.p.K, f.a_rows) ||
      !codes_map(&tm_w, f.p.w_codes, f.p.N, f.p.K, kMode == kPlain || kN == 256 ? 128 : 64))
    return NVFP4_ERR_LAUNCH;
  if (f.stages < 1 || f.split < 1 || f.split > kMaxSplit ||
      (f.split > 1 && sums_bytes(kN, kMode != kPlain, f.split, f.a_rows) > f.smem - 1024))
    return NVFP4_ERR_LAUNCH;
  const unsigned tiles = static_cast<unsigned>(f.p.N / kN);
  return launch(f.split, few_kernel<kN, kMode>,
                dim3(tiles * f.split, static_cast<unsigned>((f.p.M + 127) / 128)), dim3(kThreads),
                f.smem, stream, tm_a, tm_w, f);
}

}  // namespace

// Clusters of `split` CTAs, one on each SM, that the device holds at one time: not
// all of its SMs divide by every size (48 clusters of 3, 144 CTAs on 152 SMs, took
// two rounds, 15 us against 10).  Asked once for each size.
int most_clusters(int split, const Device& d) {
  static std::atomic<bool> ready[kMaxDevices];
  static std::atomic<int> known[kMaxDevices][kMaxSplit + 1];
  int n = known[d.id][split].load(std::memory_order_relaxed);
  if (n > 0) return n;
  if (allow_smem(few_kernel<128, kPlain>, kAllSmem, d, ready) != NVFP4_OK) return 0;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(split);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kAllSmem;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = split;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, few_kernel<128, kPlain>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  known[d.id][split].store(n, std::memory_order_relaxed);
  return n;
}

int run_product_few(const Product& p, const Device& d, cudaStream_t stream) {
  Few f{};
  f.p = p;
  f.a_rows = p.M >= 128 ? 128 : static_cast<int>((p.M + 7) / 8 * 8);
  const int64_t steps = p.K / kStageK, token_tiles = (p.M + 127) / 128;
  // Gated tiles of 64 outputs leave room in TMEM and shared memory for a second CTA, of
  // this kernel or the next: 128 tokens through 12288 x 2048 7.2 us against 7.7 with
  // tiles of 128.  With many tokens and more of them than SMs it is the MMAs' operand
  // reads that count: 128 tokens through 34816 x 5120 21.7 us against 20.5.
  const int n = p.swiglu && f.a_rows > 64 && p.N / 128 * token_tiles > d.num_sms ? 256 : 128;
  f.stage_bytes = f.a_rows * 128 + n * 128 + 4 * kScaleBlock * (p.swiglu ? 3 : 2);
  const int64_t tiles = p.N / n * token_tiles;
  // Of the splits that the device holds at one time the one with the least time, in ns
  // as measured: 280 a step (gated, with twice the MMAs and more scales, 400), and
  // where sums are exchanged 1300, 30 a CTA of the cluster and 3 more for each row.
  // 128 tokens by 2048 rows, 24 steps: one CTA 9.7 us, 3 7.4, 4 7.1, 8 9.6; 64 tokens 9.2,
  // 6.3, 5.8, 6.5; 128 by 1024 rows, 4 steps: one 4.4, 4 5.6.
  f.split = 1;
  int64_t least = INT64_MAX;
  for (int split = 1; split <= kMaxSplit && split <= steps && split * tiles <= std::max<int64_t>(d.num_sms, tiles);
       ++split) {
    if (split > 1 && tiles > most_clusters(split, d)) continue;
    const int64_t ns = (steps + split - 1) / split * (p.swiglu ? 400 : 280) +
                       (split > 1 ? 1300 + split * (30 + 3 * f.a_rows) : 0);
    if (ns < least) least = ns, f.split = split;
  }
  // With half of an SM's shared memory the next kernel's CTAs are resident, with their
  // first stages on the way, before this one's end; with all of it the ring is twice as
  // deep.  64 tokens: 2048 x 6144, 6 steps, 5.9 us against 6.2, 34816 x 5120 gated 19.8
  // against 25.7; 128 tokens by 5120 rows: 8 steps 9.8 against 9.1, 23 16.2 against 14.2.  A
  // gated tile of 128 outputs takes all of TMEM and is alone in any case.
  const int half = (kHalfSmem - 1024) / f.stage_bytes;
  f.smem = n == 256 || (steps / f.split > 2 * half && tiles <= d.num_sms) ? kAllSmem : kHalfSmem;
  // the sums lie where the stages were (an odd split leaves its owners unequal pieces,
  // and their sums more room)
  while (f.split > 1 && sums_bytes(n, p.swiglu, f.split, f.a_rows) > f.smem - 1024) --f.split;
  f.stages = std::min((f.smem - 1024) / f.stage_bytes, kMaxStages);
  if (!p.swiglu) return run<128, kPlain>(f, d, stream);
  if (n == 128) return p.codes ? run<128, kGatedRows>(f, d, stream) : run<128, kGated>(f, d, stream);
  return p.codes ? run<256, kGatedRows>(f, d, stream) : run<256, kGated>(f, d, stream);
}

}  // namespace w4a4
}  // namespace nvfp4
