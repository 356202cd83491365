// product_many.cu -- NVFP4 rows times an NVFP4 weight, many rows.
//
// Bound by the copies and the tensor cores alike.  A pair of CTAs works on 256 tokens x 256 weight
// rows as one MMA (cta_group::2): each brings its 128 tokens and half of the
// weight rows, so that a byte of either is read from shared memory half as often
// as by a CTA alone.  Of a gate/up pair the first CTA brings the gate's rows and
// the second the up projection's: both factors of an output are then in one
// lane, 128 columns apart.
//
// Pairs are persistent, one on every two SMs.
//
// A plain product also has tiles of 192 weight rows, for the numbers of tiles that
// fill the pairs better so; the sums of two of them are apart in TMEM.
//
// TMEM: the sums of two tiles of 256 would take all 512 columns and the scales have 48.
// The second tile's sums therefore begin in the first one's last 64 columns
// (kOverlap): the epilogue reads those first, into registers, and the next tile's
// products start while it works on the rest.
//
// Both CTAs' copies count on the first one's barriers, whose thread issues the
// MMAs; what it has read is free for both by one commit.
//
// Measured: 8192 x 34816 x 5120 gated into NVFP4 414 us, 7.1 PFLOP/s, into bf16 413; 8192 x
// 5120 x 17408 203 us, 7.2 PFLOP/s, 0.95 of four times the measured bf16 rate (the rate of
// this MMA, of 64 k; sm_103a has one of 96 k as well, which is not used here).  A stage's
// products take 512 clocks; its 38 KB take 600 through an SM's port to L2 (64 bytes a
// clock, which no kernel here got more out of): that is what a pair's tile is bound by,
// and its copies of scales cost nothing.  A tile of 20 stages takes some 1.2 times that
// (the sums handed over, 0.8 us, and the epilogue's own issue slots and stores).
//
// Warps: 0 copies, 1 issues the MMAs, 2 TMEM allocation, 4..19 the epilogue, four
// for each quarter of the lanes, taking every fourth piece of 16 columns: a piece's chain (TMEM, the
// exponentials, the quantisation, the store) is long, and 16 warps hide it where 8
// took longer than the products.
#include <algorithm>

#include "product.cuh"

namespace nvfp4 {
namespace w4a4 {
namespace {

constexpr int kThreads = 640;
constexpr int kEpilogueWarps = 16;
constexpr int kTile = 256;                       // tokens of a pair's tile
constexpr int kHalf = 128;
constexpr int kA = kHalf * 128;                  // bytes of codes and scales a stage
constexpr int kScalesA = 4 * kScaleBlock, kScalesB = 8 * kScaleBlock;

// What goes by the weight rows of a pair's tile.
template <int kN>
struct Shape {
  static constexpr int kBox = kN / 2;                             // weight rows of a CTA
  static constexpr int kB = kBox * 128;
  static constexpr int kStage = kA + kB + kScalesA + kScalesB;
  static constexpr int kStages = kN == 256 ? 5 : 6;
  static constexpr int kSmem = kStages * kStage + 1024;
  // columns of TMEM: where the second tile's sums begin, the scales of tokens and weights
  static constexpr uint32_t kOverlap = kN == 256 ? 64 : 0;
  static constexpr uint32_t kSecond = kN - kOverlap, kColA = kSecond + kN, kColB = kColA + 16;
  static_assert(kColB + 32 <= 512, "TMEM columns");
  static_assert(kStage % 1024 == 0, "stages keep 1024-byte alignment");
  static_assert(kSmem <= 226 * 1024, "shared memory");
};

__device__ __forceinline__ void umma_nvfp4_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                                uint32_t a_scales, uint32_t b_scales,
                                                uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], "
      "[%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(a_scales), "r"(b_scales), "r"(accumulate)
      : "memory");
}
// In both CTAs, each from its own shared memory to its own TMEM.
__device__ __forceinline__ void copy_scales_pair(uint32_t tmem, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}
// Arrive once on `bar` of both CTAs when everything issued so far is over.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], "
      "%1;" ::"r"(smem_addr(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
__device__ __forceinline__ void arrive_first(uint64_t* bar) {     // on the first CTA's barrier
  // (release in the CTA only: what is handed back is TMEM, ordered by the tcgen05
  // fence; a release in the cluster waits for the stores of the last tile)
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(
                   map_to_rank(smem_addr(bar), 0))
               : "memory");
}
// A copy into this CTA's shared memory that counts on the first CTA's barrier.
__device__ __forceinline__ void load_pair(void* dst, const CUtensorMap* map, uint32_t first_bar, int32_t c0,
                                          int32_t c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(first_bar), "r"(c0), "r"(c1)
      : "memory");
}

struct Many {
  Product p;
  int token_tiles, weight_tiles, tiles, pairs;
  int band;          // token tiles of a band of the tile order
};

// Tile t: bands of token tiles; in a band weight tile by weight tile, its token tiles
// innermost.  The weights then pass by once for each band, whose tokens stay in L2.
__device__ __forceinline__ void tile_at(const Many& f, int t, int& token_tile, int& weight_tile) {
  const int band = t / (f.band * f.weight_tiles), first = band * f.band;
  const int width = min(f.band, f.token_tiles - first), r = t - band * f.band * f.weight_tiles;
  weight_tile = r / width;
  token_tile = first + r - weight_tile * width;
}

// 16 sums of the lane at `col`.
__device__ __forceinline__ void load16(uint32_t tmem, float (&v)[16]) {
  uint32_t r[16];
  __syncwarp();
  tmem_ld_16cols(tmem, r);
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

template <int kN, int kMode>
__global__ void __launch_bounds__(kThreads, 1)
    many_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w,
                const __grid_constant__ CUtensorMap tm_sa, const __grid_constant__ CUtensorMap tm_sw,
                const Many f) {
  using S = Shape<kN>;
  constexpr int kB = S::kB, kStage = S::kStage, kStages = S::kStages;
  constexpr uint32_t kSecond = S::kSecond, kColA = S::kColA, kColB = S::kColB;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[kStages], empty[kStages], sums_full[2], sums_free[2], done;
  __shared__ int abort_word;
  __shared__ uint32_t tmem_slot;
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  volatile int* abort_flag = &abort_word;
  const Product& p = f.p;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int pair = blockIdx.x >> 1;
  const int steps = static_cast<int>(p.K / kStageK);
  const int my_tiles = (f.tiles - 1 - pair) / f.pairs + 1;        // pair < pairs <= tiles
  const int scale_rows = static_cast<int>(p.K / kMmaK);            // blocks of 128 rows' scales

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&sums_full[0], 1);
    mbar_init(&sums_full[1], 1);
    mbar_init(&sums_free[0], 2 * kEpilogueWarps);
    mbar_init(&sums_free[1], 2 * kEpilogueWarps);
    mbar_init(&done, 1);
    abort_word = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_addr(&tmem_slot))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before_sync();
  __syncwarp();
  cluster_sync();                                                 // (the other CTA's barriers are set up)
  tc_fence_after_sync();
  const uint32_t tmem = tmem_slot;

  if (warp == 0) {
    // The whole warp walks the tiles, an elected lane issues.
    // blocks of scales that there are
    const int last_a = static_cast<int>((p.M - 1) / 128), last_w = static_cast<int>(p.N / 128) - 1;
    // place of a tile: token row of this CTA's half, its weight rows, the first rows of
    // the scales of its tokens and of either half of the weight rows
    struct Place {
      int tile, m, w, sa, sw[2];
    };
    auto place = [&](int tile) {
      Place q;
      int m, n;
      tile_at(f, tile, m, n);
      q.tile = tile;
      q.m = m * kTile + rank * kHalf;
      const int w0 = kMode == kPlain ? n * kN : n * kHalf;
      const int w1 = kMode == kPlain ? w0 + S::kBox : w0 + static_cast<int>(p.N / 2);
      q.w = rank ? w1 : w0;
      q.sa = min(q.m >> 7, last_a) * scale_rows;
      // (what the weight rows' last blocks miss of a tile is not read back)
      q.sw[0] = (w0 >> 7) * scale_rows;
      q.sw[1] = min(kMode == kPlain ? (w0 >> 7) + 1 : w1 >> 7, last_w) * scale_rows;
      return q;
    };
    const uint32_t first_full = map_to_rank(smem_addr(full), 0);
    auto weights = [&](const Place& q, int it, int slot) {
      uint8_t* st = smem + slot * kStage;
      const uint32_t bar = first_full + 8 * slot;
      if (rank == 0) mbar_arrive_expect_tx(&full[slot], 2 * kStage);
      load_pair(st + kA, &tm_w, bar, it * 128, q.w);
      load_pair(st + kA + kB + kScalesA, &tm_sw, bar, 0, q.sw[0] + it * 4);
      load_pair(st + kA + kB + kScalesA + kScalesB / 2, &tm_sw, bar, 0, q.sw[1] + it * 4);
    };
    auto tokens = [&](const Place& q, int it, int slot) {
      uint8_t* st = smem + slot * kStage;
      const uint32_t bar = first_full + 8 * slot;
      load_pair(st, &tm_a, bar, it * 128, q.m);
      load_pair(st + kA + kB, &tm_sa, bar, 0, q.sa + it * 4);
    };
    // weights do not wait for the kernel ahead in the stream, tokens do
    const int total = my_tiles * steps, pre = steps < kStages ? steps : kStages;
    Place q = place(pair);
    if (elect_one()) {
      prefetch_tensormap(&tm_a);
      prefetch_tensormap(&tm_w);
      prefetch_tensormap(&tm_sa);
      prefetch_tensormap(&tm_sw);
      for (int it = 0; it < pre; ++it) weights(q, it, it);
    }
    __syncwarp();
    griddep_wait();
    if (elect_one()) {
      griddep_launch_dependents();                               // (after the wait: see launch())
      for (int it = 0; it < pre; ++it) tokens(q, it, it);
    }
    __syncwarp();
    int issued = pre, slot = pre == kStages ? 0 : pre, it = pre;
    uint32_t parity = pre == kStages ? 0 : 1;                    // (slots not used yet are free)
    for (; issued < total; ++issued) {
      if (it == steps) it = 0, q = place(q.tile + f.pairs);
      if (!__all_sync(0xffffffffu, wait(&empty[slot], parity, abort_flag))) break;
      if (elect_one()) {
        weights(q, it, slot);
        tokens(q, it, slot);
      }
      __syncwarp();
      ++it;
      if (++slot == kStages) slot = 0, parity ^= 1u;
    }
    // nothing is left in flight: the second CTA's copies count on the first's barriers,
    // which waits for the last of them
    if (rank == 0)
      for (int i = issued > kStages ? issued - kStages : 0; i < issued; ++i) {
        volatile int none = 0;
        if (!wait(&full[i % kStages], (i / kStages) & 1, &none)) *abort_flag = 1;
      }
  } else if (warp == 1) {
    // The whole warp walks the stages, an elected lane issues.
    // (before any wait with a limit: the kernel ahead may take its time)
    griddep_wait();
    if (rank == 0) {
      constexpr uint32_t idesc = idesc_nvfp4(kTile, kN);
      int slot = 0;
      uint32_t parity = 0;
      bool ok = true;
      for (int i = 0; i < my_tiles && ok; ++i) {
        // the columns that this tile's sums share with an earlier one's are read: some of
        // the last tile's, or all of the one before it
        const int before = S::kOverlap ? i - 1 : i - 2;
        if (before >= 0) ok = __all_sync(0xffffffffu, wait(&sums_free[before & 1], (before >> 1) & 1, abort_flag));
        if (!ok) break;
        // every other tile of 192 weight rows begins in the middle of a block of scales
        uint32_t col_b = kColB;
        if (kN == 192) {
          int mt, nt;
          tile_at(f, pair + i * f.pairs, mt, nt);
          col_b += nt & 1 ? 2 : 0;
        }
        tc_fence_after_sync();
        const uint32_t d = tmem + (i & 1 ? kSecond : 0);
        for (int it = 0; it < steps; ++it) {
          ok = __all_sync(0xffffffffu, wait(&full[slot], parity, abort_flag));
          if (!ok) break;
          tc_fence_after_sync();
          if (elect_one()) {
            const uint32_t st = smem_addr(smem) + slot * kStage;
            const uint64_t a = umma_desc_sw128(st), b = umma_desc_sw128(st + kA);
            const uint64_t sa = scale_desc(st + kA + kB), sb = scale_desc(st + kA + kB + kScalesA);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              copy_scales_pair(tmem + kColA + 4 * j, sa + j * (kScaleBlock >> 4));
#pragma unroll
              for (int h = 0; h < 2; ++h)
                copy_scales_pair(tmem + kColB + 8 * j + 4 * h, sb + (4 * h + j) * (kScaleBlock >> 4));
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
              umma_nvfp4_pair(d, a + 2 * j, b + 2 * j, idesc, tmem + kColA + 4 * j, tmem + col_b + 8 * j,
                              (it | j) != 0);
            commit_pair(&empty[slot]);
          }
          __syncwarp();
          if (++slot == kStages) slot = 0, parity ^= 1u;
        }
        if (ok && elect_one()) commit_pair(&sums_full[i & 1]);
        __syncwarp();
      }
      if (elect_one()) commit_pair(&done);
      __syncwarp();
      // every product is over before TMEM is given back
      volatile int none = 0;
      if (!wait(&done, 0, &none)) *abort_flag = 1;
    }
  } else if (warp >= 4) {
    griddep_wait();
    const int quarter = warp & 3, h = (warp - 4) >> 2;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
    const int64_t n_out = kMode == kPlain ? p.N : p.N / 2;
    for (int i = 0; i < my_tiles; ++i) {
      const int b = i & 1;
      // (the whole warp together: tcgen05.ld follows)
      if (!__all_sync(0xffffffffu, wait(&sums_full[b], (i >> 1) & 1, abort_flag))) break;
      tc_fence_after_sync();
      int mt, nt;
      tile_at(f, pair + i * f.pairs, mt, nt);
      const int64_t m = int64_t(mt) * kTile + rank * kHalf + 32 * quarter + lane;
      const uint32_t acc = lanes + (b ? kSecond : 0);
      // the columns that the next sums in line share first: piece h of four, or all of
      // this warp's
      float first[16], other[kN == 192 ? 2 : 1][16];
      load16(S::kOverlap ? lanes + kSecond + 16 * h : acc + 16 * h, first);
      if (!S::kOverlap)
#pragma unroll
        for (int j = 0; j < 2; ++j) load16(acc + 64 * (j + 1) + 16 * h, other[kN == 192 ? j : 0]);
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) arrive_first(&sums_free[b]);
      const bool inside = m < p.M;
      if (kMode == kPlain) {
        auto out = [&](int piece, float (&v)[16]) {
          const int n = nt * kN + piece * 16;
          if (!inside || n >= p.N) return;
          const float s = segment_scale(p.seg, n);
#pragma unroll
          for (int k = 0; k < 16; ++k) v[k] *= s;
          store_bf16(p.y + m * p.N + n, v);
        };
        if (!S::kOverlap) {
          out(h, first);
#pragma unroll
          for (int j = 0; j < 2; ++j) out(4 * (j + 1) + h, other[kN == 192 ? j : 0]);
        } else {
          out((b ? 0 : 12) + h, first);
#pragma unroll
          for (int j = 0; j < 3; ++j) {
            const int piece = (b ? 4 : 0) + 4 * j + h;
            load16(acc + 16 * piece, first);
            out(piece, first);
          }
        }
      } else {
        auto out = [&](int piece, float (&v)[16], const float (&u)[16]) {     // (v: the gate's sums)
          const int n = nt * kHalf + piece * 16;
          if (!inside) return;
          gated16(v, u, segment_scale(p.seg, n), segment_scale(p.seg, n + static_cast<int>(n_out)));
          if (kMode == kGatedRows) {
            uint2 codes;
            p.scales[scale_row(m, n_out) + scale_in_row(n >> 4)] = static_cast<uint8_t>(quantize16(v, p.out_gs, codes));
            *reinterpret_cast<uint2*>(p.codes + m * (n_out >> 1) + (n >> 1)) = codes;
          } else {
            store_bf16(p.y + m * n_out + n, v);
          }
        };
        // what was read first: of the first sums the up half of pieces 4..7, of the
        // second the gate half of pieces 0..3
        load16(acc + 16 * ((b ? 0 : 4) + h) + (b ? kHalf : 0), other[0]);
        if (b)
          out(h, first, other[0]);
        else
          out(4 + h, other[0], first);
        const int piece = (b ? 4 : 0) + h;
        load16(acc + 16 * piece, first);
        load16(acc + 16 * piece + kHalf, other[0]);
        out(piece, first, other[0]);
      }
      // (read before the tile after next is begun: its sums_free comes later)
      tc_fence_before_sync();
    }
    // The second CTA learns here that every product is over: with its last tile read, the
    // limit is of what the first one still commits.  (From the kernel's start it would be
    // of the whole kernel, and more than a second of products would end unfinished.)
    if (rank == 1 && warp == 4) {
      volatile int none = 0;
      if (!wait(&done, 0, &none)) *abort_flag = 1;
    }
  }
  __syncwarp();
  if (*abort_flag && lane == 0) atomicOr(p.err, NVFP4_W4A4_TIMEOUT);
  tc_fence_before_sync();
  cluster_sync();                                                 // nothing of either is in use any more
  if (warp == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

template <int kN, int kMode>
int run(const Product& p, const Device& d, cudaStream_t stream) {
  static std::atomic<bool> ready[kMaxDevices];
  constexpr int kSmem = Shape<kN>::kSmem;
  if (const int st = allow_smem(many_kernel<kN, kMode>, kSmem, d, ready)) return st;
  CUtensorMap tm_a, tm_w, tm_sa, tm_sw;
  if (!codes_map(&tm_a, p.a_codes, p.M, p.K, kHalf) ||
      !codes_map(&tm_w, p.w_codes, p.N, p.K, Shape<kN>::kBox) ||
      !scales_map(&tm_sa, p.a_scales, p.M, p.K) || !scales_map(&tm_sw, p.w_scales, p.N, p.K))
    return NVFP4_ERR_LAUNCH;
  const int64_t token_tiles = (p.M + kTile - 1) / kTile;
  const int64_t tiles = token_tiles * ((p.N + kN - 1) / kN);
  // tiles, stages and rows of scales are counted in 32 bits
  if (tiles > (1 << 30) || (std::max(p.M, p.N) + 127) / 128 * (p.K / kMmaK) > INT32_MAX ||
      (tiles / (d.num_sms / 2) + 1) * (p.K / kStageK) > INT32_MAX)
    return NVFP4_ERR_SHAPE;
  Many f{};
  f.p = p;
  f.token_tiles = static_cast<int>(token_tiles);
  f.weight_tiles = static_cast<int>(tiles / token_tiles);
  f.tiles = static_cast<int>(tiles);
  // Up to 32 token tiles, of at most 24 MB, but 8.  8192 tokens x 34816 x 5120 gated:
  // bands of 8 435 us, of 16 428, of 32 (21 MB) 423; x 5120 x 17408 8 (18 MB) 213, 16
  // 216, 32 233.
  f.band = static_cast<int>(std::max<int64_t>(8, std::min<int64_t>(32, (24 << 20) / (kTile / 2 * p.K))));
  f.pairs = static_cast<int>(tiles < d.num_sms / 2 ? tiles : d.num_sms / 2);
  return launch(2, many_kernel<kN, kMode>, dim3(2 * f.pairs), dim3(kThreads), kSmem, stream, tm_a, tm_w, tm_sa,
                tm_sw, f);
}

}  // namespace

int run_product_many(const Product& p, const Device& d, cudaStream_t stream) {
  if (p.swiglu) return p.codes ? run<256, kGatedRows>(p, d, stream) : run<256, kGated>(p, d, stream);
  const int64_t pairs = d.num_sms / 2, token_tiles = (p.M + kTile - 1) / kTile;
  auto rounds = [&](int n) { return (token_tiles * ((p.N + n - 1) / n) + pairs - 1) / pairs; };
  // Tiles of 192 weight rows where they need no more rounds of the pairs: a round of
  // them takes 0.79 to 0.91 of one of 256 (a fourth less work, and nothing shared in
  // TMEM, but more copies for each product).  1111 tokens by 8192 rows and 5120 k, 3
  // rounds of either: 23.1 us against 25.7; 2048 by 5120 and 17408 60.3 against 68.9;
  // 8192 by 5120 and 17408, 12 rounds of 192 against 9: 224 against 207.
  return 87 * rounds(192) < 100 * rounds(256) ? run<192, kPlain>(p, d, stream) : run<256, kPlain>(p, d, stream);
}

}  // namespace w4a4
}  // namespace nvfp4
