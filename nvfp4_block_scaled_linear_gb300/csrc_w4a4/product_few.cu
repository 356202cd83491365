// product_few.cu -- NVFP4 rows times an NVFP4 weight, up to 128 rows a CTA.
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
// A CTA leaves its sums in its own shared memory, [token][column], and, after a
// cluster barrier, the threads of the cluster take pieces of 16 outputs each,
// adding the CTAs' sums in their order: no atomics, the same bits on every run.
//
// Warps: 0 copies, 1 MMA, 2 TMEM allocation, 4..7 read the accumulator; all
// eight write the outputs.
#include "product.cuh"

namespace nvfp4 {
namespace w4a4 {
namespace {

constexpr int kThreads = 256;
constexpr int kSmem = 227 * 1024;
constexpr int kMaxStages = 12;
constexpr int kMaxSplit = 8;

enum { kPlain = 0, kGated = 1, kGatedRows = 2 };

struct Few {
  Product p;
  int a_rows;        // rows of a box of tokens
  int split;         // CTAs of a cluster
  int stages, stage_bytes;
};

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// The cluster's sums of 16 columns, in the CTAs' order.
__device__ __forceinline__ void sum16(uint32_t local, int split, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = 0.f;
  for (int q = 0; q < split; ++q) {
    const uint32_t at = map_to_rank(local, q);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 f = ld_cluster_f32x4(at + 16 * i);
      v[4 * i] += f.x, v[4 * i + 1] += f.y, v[4 * i + 2] += f.z, v[4 * i + 3] += f.w;
    }
  }
}

template <int kN, int kMode>
__global__ void __launch_bounds__(kThreads, 1)
    few_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w,
               const Few f) {
  constexpr int kBlocks = kN / 128;                       // blocks of 128 weight rows
  constexpr uint32_t kCols = kN == 256 ? 512 : 256;       // TMEM: sums, then scales
  constexpr uint32_t kScaleA = kN, kScaleB = kN + 16;     // 4 columns per 64 k and 128 rows
  constexpr int kPitch = kN + 4;                          // floats of a row of sums
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
  // first weight row of block i of the tile
  auto w_row = [&](int i) {
    return kMode == kPlain ? tile * kN + i * 128 : tile * 128 + i * static_cast<int>(p.N / 2);
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
  if (threadIdx.x == 0) griddep_launch_dependents();

  if (warp == 0) {
    // the whole warp walks the stages, an elected lane issues
    auto weights = [&](int it, int slot) {
      uint8_t* st = smem + slot * f.stage_bytes;
      mbar_arrive_expect_tx(&full[slot], f.stage_bytes);
#pragma unroll
      for (int i = 0; i < kBlocks; ++i) {
        tma_load_2d(st + w_off + i * 128 * 128, &tm_w, &full[slot], (s0 + it) * 128, w_row(i));
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
    if (elect_one())
      for (int it = 0; it < pre; ++it) tokens(it, it);
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
    constexpr uint32_t idesc = idesc_nvfp4(128, kN);
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
          umma_nvfp4(tmem, a + 2 * j, b + 2 * j, idesc, tmem + kScaleA + 4 * j, tmem + kScaleB + 4 * kBlocks * j,
                     (it | j) != 0);
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
  // the sums go where the stages were, once every product and copy is over
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  float* sums = reinterpret_cast<float*>(smem);
  if (warp >= 4 && (warp - 4) * 32 < rows) {
    const int row = (warp - 4) * 32 + lane;
    for (int c = 0; c < kN; c += 32) {
      uint32_t v[32];
      tmem_ld_32cols(tmem + (static_cast<uint32_t>((warp - 4) * 32) << 16) + c, v);
      tmem_ld_wait();
      if (row < rows)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          reinterpret_cast<uint4*>(sums + row * kPitch + c)[i] =
              make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    }
  }
  if (f.split > 1)
    cluster_sync();
  else
    __syncthreads();

  constexpr int kOut = kMode == kPlain ? kN : 128;        // outputs of a row of the tile
  constexpr int kPieces = kOut / 16;
  const int pieces = (kPieces - rank + f.split - 1) / f.split;      // this CTA's: rank, rank + split, ...
  const int64_t n_out = kMode == kPlain ? p.N : p.N / 2;
  for (int i = threadIdx.x; i < rows * pieces; i += kThreads) {
    const int row = i / pieces, c = (rank + (i - row * pieces) * f.split) * 16;
    const int64_t m = m0 + row, n = int64_t(tile) * kOut + c;
    const uint32_t at = smem_addr(sums + row * kPitch + c);
    float v[16];
    sum16(at, f.split, v);
    const float s = segment_scale(p.seg, static_cast<int>(n));
    if (kMode == kPlain) {
#pragma unroll
      for (int k = 0; k < 16; ++k) v[k] *= s;
    } else {
      float u[16];
      sum16(at + 128 * 4, f.split, u);
      const float su = segment_scale(p.seg, static_cast<int>(n + p.N / 2));
#pragma unroll
      for (int k = 0; k < 16; ++k) v[k] = gated(v[k] * s, u[k] * su);
    }
    if (kMode == kGatedRows) {
      uint2 codes;
      p.scales[scale_at(m, n >> 4, n_out)] = static_cast<uint8_t>(quantize16(v, p.out_gs, codes));
      *reinterpret_cast<uint2*>(p.codes + m * (n_out >> 1) + (n >> 1)) = codes;
    } else {
      uint4* y = reinterpret_cast<uint4*>(p.y + m * n_out + n);
#pragma unroll
      for (int k = 0; k < 2; ++k)
        y[k] = make_uint4(f32x2_to_bf16x2(v[8 * k], v[8 * k + 1]), f32x2_to_bf16x2(v[8 * k + 2], v[8 * k + 3]),
                          f32x2_to_bf16x2(v[8 * k + 4], v[8 * k + 5]),
                          f32x2_to_bf16x2(v[8 * k + 6], v[8 * k + 7]));
    }
  }
  if (*abort_flag && threadIdx.x == 0) atomicOr(p.err, NVFP4_W4A4_TIMEOUT);
  // (peers may still be reading this CTA's sums)
  if (f.split > 1)
    cluster_sync();
  else
    __syncthreads();
  if (warp == 2) tmem_dealloc(tmem, kCols);
}

template <int kN, int kMode>
int run(Few f, const Device& d, cudaStream_t stream) {
  static std::atomic<bool> ready[kMaxDevices];
  if (const int st = allow_smem(few_kernel<kN, kMode>, kSmem - 1024, d, ready)) return st;
  CUtensorMap tm_a, tm_w;
  if (!codes_map(&tm_a, f.p.a_codes, f.p.M, f.p.K, f.a_rows) ||
      !codes_map(&tm_w, f.p.w_codes, f.p.N, f.p.K, 128))
    return NVFP4_ERR_LAUNCH;
  f.stage_bytes = f.a_rows * 128 + kN * 128 + 4 * kScaleBlock * (1 + kN / 128);
  f.stages = (kSmem - 1024 - 1024) / f.stage_bytes;
  if (f.stages > kMaxStages) f.stages = kMaxStages;
  const unsigned tiles = static_cast<unsigned>(f.p.N / (kMode == kPlain ? kN : 256));
  return launch(f.split, few_kernel<kN, kMode>,
                dim3(tiles * f.split, static_cast<unsigned>((f.p.M + 127) / 128)), dim3(kThreads),
                kSmem - 1024, stream, tm_a, tm_w, f);
}

}  // namespace

int run_product_few(const Product& p, const Device& d, cudaStream_t stream) {
  Few f{};
  f.p = p;
  f.a_rows = p.M >= 128 ? 128 : static_cast<int>((p.M + 7) / 8 * 8);
  const int64_t steps = p.K / kStageK, token_tiles = (p.M + 127) / 128;
  const int64_t tiles = p.N / (p.swiglu ? 256 : 128) * token_tiles;
  int64_t split = d.num_sms / tiles;
  split = split < 1 ? 1 : split > kMaxSplit ? kMaxSplit : split;
  f.split = static_cast<int>(split < steps ? split : steps);
  if (!p.swiglu) return run<128, kPlain>(f, d, stream);
  return p.codes ? run<256, kGatedRows>(f, d, stream) : run<256, kGated>(f, d, stream);
}

}  // namespace w4a4
}  // namespace nvfp4
