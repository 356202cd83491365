// mass_tc.cu -- the attention weight that each cached key receives (mass.cu has
// the formula), for many query rows, on the tcgen05 tensor cores.
//
// A CTA keeps 256 keys of one head in shared memory, two tiles of the MMA's 128
// rows, and all query rows that see any of them pass by as the other operand,
// 128 at a time:  S = K Q^T  puts a key's scores in one TMEM lane, so that one
// thread adds up all that a key receives, in one order, with no exchange.  The
// two tiles share every copy of the queries (one tile alone would want 64 bytes
// a clock of L2 per SM), and each has two score buffers, so that a buffer is
// read out and summed while the products go on in the other.
//
// Queries that a cluster of CTAs shares (run has the rule) are added up by its
// first, over distributed shared memory, in the CTAs' order.
//
// Bound by the products, 2 * 128 * 256 * head_dim flops for 128 query rows;
// the exponentials, 256 for a thread in the same time, run beside them.
//
// Measured at 24 query and 4 key/value heads of 256: 2048 tokens over 16411 keys
// 308 us, 1256 TFLOP/s, 65% of the burst rate of a matrix product.
//
// Warps: 0-3 and 4-7 sum up (tile 0, tile 1); 8 copies K once and then the
// queries; 9 and 11 MMA (tile 0, tile 1); 10 the rows' log-sums.  An e4m3 K
// becomes bf16 (exact) on its way to shared memory, by warps 0-7.
#include <algorithm>

#include "attend.cuh"

namespace nvfp4 {
namespace attn {
namespace {

constexpr int kThreads = 384;
constexpr int kM = 128, kN = 128;
constexpr int kKeys = 2 * kM;
constexpr int kLogs = 3;                      // query tiles whose log-sums are held

template <int kDim>
struct Cfg {
  static constexpr int kChunk = kM * 128;                      // 64 columns of 128 rows
  static constexpr int kTileBytes = kM * kDim * 2;
  static constexpr int kSlotChunks = kDim == 64 ? 1 : 2;       // of a query slot
  static constexpr int kSlotBytes = kSlotChunks * kChunk;
  static constexpr int kPieces = kDim / 64 / kSlotChunks;      // slots of a query tile
  static constexpr int kMaxSlots = 4;
  static constexpr int kBars = 2 * kMaxSlots + 8 + 2 * kLogs + 2;
  static constexpr int kLogOff = (kBars * 8 + 8 + 15) / 16 * 16;
  static constexpr int kFixed = kLogOff + kLogs * kN * 4;
  static constexpr int kBudget = 227 * 1024 - 1024 - kFixed - 2 * kTileBytes;
  static constexpr int kSlots = std::min(kMaxSlots, kBudget / kSlotBytes);
  static constexpr int kSmem = 2 * kTileBytes + kSlots * kSlotBytes + kFixed + 1024;
  static_assert(kSlots > kPieces, "a query tile and the start of the next");
};

struct MassTc {
  Mass a;
  int tile_tokens, box_shift;
};

template <int kDim, bool kE4m3>
__global__ void __launch_bounds__(kThreads, 1)
    mass_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const MassTc p) {
  using C = Cfg<kDim>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* k_sm = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  uint8_t* ring = k_sm + 2 * C::kTileBytes;
  uint8_t* fixed = ring + C::kSlots * C::kSlotBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(fixed);
  uint64_t* empty = full + C::kMaxSlots;
  uint64_t* s_full = empty + C::kMaxSlots;     // [tile][buffer]
  uint64_t* s_free = s_full + 4;
  uint64_t* log_full = s_free + 4;
  uint64_t* log_free = log_full + kLogs;
  uint64_t* k_full = log_free + kLogs;
  uint64_t* mma_done = k_full + 1;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(full + C::kBars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(full + C::kBars) + 1;
  float* logs = reinterpret_cast<float*>(fixed + C::kLogOff);     // [kLogs][kN], -log2 of a row's sum
  const Mass& a = p.a;

  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t ctas;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ctas));
  const int rank = static_cast<int>(cluster_ctarank());
  const int s = blockIdx.z, kvh = blockIdx.y, key0 = static_cast<int>(blockIdx.x / ctas) * kKeys;
  const SeqInfo si = load_seq(a.seqs, s, a.err);
  const int64_t out0 = (int64_t(s) * a.cache.heads + kvh) * a.room;
  const int before = si.kv_len - si.q_len;              // keys before the first new token
  const int tiles = (si.q_len + p.tile_tokens - 1) / p.tile_tokens;
  const int seeing = max(0, key0 - before) / p.tile_tokens;     // first query tile that sees key0
  const int all = key0 < si.kv_len ? max(0, tiles - seeing) : 0;
  // query tiles of this CTA: an equal share of the cluster's
  const int share = (all + static_cast<int>(ctas) - 1) / static_cast<int>(ctas);
  const int first = seeing + rank * share, n = max(0, min(share, all - rank * share));
  if (all == 0) {                                       // no row sees these keys
    const int key = key0 + static_cast<int>(threadIdx.x);
    if (rank == 0 && threadIdx.x < kKeys && key < a.room)
      a.out[out0 + key] = key < si.kv_len && a.mass ? a.mass[out0 + key] : 0.f;
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kSlots; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 2);
    for (int i = 0; i < 4; ++i) mbar_init(&s_full[i], 1), mbar_init(&s_free[i], 4);
    for (int i = 0; i < kLogs; ++i) mbar_init(&log_full[i], 1), mbar_init(&log_free[i], 8);
    mbar_init(k_full, kE4m3 ? 8 : 1);
    mbar_init(mma_done, 2);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  // query rows that no token fills (128 is no multiple of every group): zeros
  const int rows = p.tile_tokens * a.group;
  for (int i = threadIdx.x; i < C::kSlots * C::kSlotChunks * (kN - rows) * 8; i += kThreads) {
    const int chunk = i / ((kN - rows) * 8), r = i % ((kN - rows) * 8);
    *reinterpret_cast<uint4*>(ring + chunk * C::kChunk + (rows + r / 8) * 128 + r % 8 * 16) =
        make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  float received = 0.f;                                 // key0 + threadIdx.x, by this CTA's queries
  if (n == 0) {
  } else if (warp < 8) {
    // --------------------------------------------------------------- sums
    const int x = warp >> 2, quad = warp & 3;
    if constexpr (kE4m3) {
      // 16 codes a thread and pass: 8 (head_dim 128) keys at once for a warp
      constexpr int kPerRow = kDim / 16, kRowsAtOnce = 32 / kPerRow;
      const int col = lane % kPerRow * 16;
#pragma unroll 4
      for (int r = 0; r < 32; r += kRowsAtOnce) {
        const int row = warp * 32 + r + lane / kPerRow;          // of the 256
        const int key = key0 + row;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (key < si.kv_len) {
          const int pg = key / a.cache.page_size;
          const int64_t page =
              checked_page(a.seqs.table[int64_t(s) * a.seqs.width + pg], a.cache.pages, a.err);
          if (page != a.cache.pages)
            v = *reinterpret_cast<const uint4*>(
                static_cast<const uint8_t*>(a.cache.k) + page * a.cache.ks[0] +
                (key - pg * a.cache.page_size) * a.cache.ks[1] + kvh * a.cache.ks[2] + col);
        }
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t f[8];
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t c2 = h ? w[k] >> 16 : w[k] & 0xFFFFu;
            const __half2_raw two = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c2), __NV_E4M3);
            const float2 f2 = __half22float2(__half2(two));
            f[2 * k + h] = f32x2_to_bf16x2(f2.x, f2.y);
          }
        uint8_t* at = k_sm + (row >> 7) * C::kTileBytes + (col >> 6) * C::kChunk + (row & 127) * 128;
        const int c16 = (col & 63) >> 3;
        *reinterpret_cast<uint4*>(at + ((c16 ^ (row & 7)) << 4)) = make_uint4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<uint4*>(at + (((c16 + 1) ^ (row & 7)) << 4)) = make_uint4(f[4], f[5], f[6], f[7]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(k_full);
    }
    const int key = key0 + x * kM + quad * 32 + lane;
    const uint32_t t_s = tmem + (static_cast<uint32_t>(quad * 32) << 16) + x * 2 * kN;
    float c = a.scale * 1.44269504088896f;
    if (kE4m3 && a.cache.k_scale) c *= a.cache.k_scale[kvh];
    const float2 c2 = make_float2(c, c);
    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    for (int i = 0; i < n; ++i) {
      const int b = i & 1, l = i % kLogs;
      const int tok0 = (first + i) * p.tile_tokens;
      wait(&log_full[l], i / kLogs & 1, abort_flag);
      wait(&s_full[2 * x + b], i >> 1 & 1, abort_flag);
      __syncwarp();
      tc_fence_after_sync();
      uint32_t sc[4][32];
#pragma unroll
      for (int k = 0; k < 4; ++k) tmem_ld_32cols(t_s + b * kN + k * 32, sc[k]);
      tmem_ld_wait();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_free[2 * x + b]);
      const float* lg = logs + l * kN;
      // rows that see this key, where not all rows of the tile see all keys
      const int lo = max(0, key - before - tok0) * a.group;
      const int hi = min(p.tile_tokens, si.q_len - tok0) * a.group;
      if (__any_sync(0xffffffffu, lo > 0) || hi < rows) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (k * 32 + j < lo || k * 32 + j >= hi) sc[k][j] = 0xFF800000u;     // weight 0
      } else {
        // rows that hold no token: 0 times a key that is not finite need not be 0
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (rows < (k + 1) * 32) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (k * 32 + j >= rows) sc[k][j] = 0xFF800000u;
          }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float4 g = *reinterpret_cast<const float4*>(lg + k * 32 + j);
          float2 e = fma2(make_float2(__uint_as_float(sc[k][j]), __uint_as_float(sc[k][j + 1])), c2,
                          make_float2(g.x, g.y));
          float2 f = fma2(make_float2(__uint_as_float(sc[k][j + 2]), __uint_as_float(sc[k][j + 3])),
                          c2, make_float2(g.z, g.w));
          e.x = ex2(e.x), e.y = ex2(e.y), f.x = ex2(f.x), f.y = ex2(f.y);
          sum[0] = add2(sum[0], e);
          sum[1] = add2(sum[1], f);
        }
      __syncwarp();
      if (lane == 0) mbar_arrive(&log_free[l]);
    }
    sum[0] = add2(sum[0], sum[1]);
    received = sum[0].x + sum[0].y;
  } else if (warp == 8) {
    // ------------------------------------------------------------- copies
    if (!kE4m3) {
      // K: lane i the copies of rows i << box_shift on
      const int boxes = kKeys >> p.box_shift;
      const int row = lane << p.box_shift, key = key0 + row;
      int page = -1, in_page = 0;
      if (lane < boxes && key < si.kv_len) {
        const int pg = key / a.cache.page_size;
        page = static_cast<int>(
            checked_page(a.seqs.table[int64_t(s) * a.seqs.width + pg], a.cache.pages, a.err));
        in_page = key - pg * a.cache.page_size;
      }
      const int there = __popc(__ballot_sync(0xffffffffu, page >= 0));
      if (lane == 0) mbar_arrive_expect_tx(k_full, (there * (kDim / 64)) << (p.box_shift + 7));
      __syncwarp();
      if (page >= 0)
        for (int ch = 0; ch < kDim / 64; ++ch)
          tma_load_page(k_sm + (row >> 7) * C::kTileBytes + ch * C::kChunk + (row & 127) * 128, &tm_k,
                        k_full, ch, in_page, kvh, page);
      __syncwarp();
    }
    if (lane == 0) {
      int slot = 0, turns = 0;
      uint32_t par = 0;
      bool ok = true;
      for (int i = 0; i < n && ok; ++i) {
        const int token = si.q0 + (first + i) * p.tile_tokens;
        for (int h = 0; h < C::kPieces; ++h) {
          if (turns == C::kSlots)
            ok = wait(&empty[slot], par ^ 1, abort_flag);
          else
            ++turns;
          if (!ok) break;
          mbar_arrive_expect_tx(&full[slot], C::kSlotChunks * rows * 128);
#pragma unroll
          for (int ch = 0; ch < C::kSlotChunks; ++ch)
            tma_load_3d(ring + slot * C::kSlotBytes + ch * C::kChunk, &tm_q, &full[slot],
                        (h * C::kSlotChunks + ch) * 64, kvh * a.group, token);
          if (++slot == C::kSlots) slot = 0, par ^= 1u;
        }
      }
      // every copy has landed before the block may end
      for (int i = 0; i < turns; ++i) {
        volatile int no_abort = 0;
        if (!wait(&full[i], i < slot ? par : par ^ 1, &no_abort)) atomicOr(a.err, NVFP4_ATTENTION_TIMEOUT);
      }
      if (!kE4m3) {
        volatile int no_abort = 0;
        if (!wait(k_full, 0, &no_abort)) atomicOr(a.err, NVFP4_ATTENTION_TIMEOUT);
      }
    }
    __syncwarp();
  } else if (warp == 9 || warp == 11) {
    // ------------------------------- MMA, a warp for each tile: an issue waits for
    // the pipe, so that what one warp spends between its products the other fills
    constexpr uint32_t id = umma_idesc_bf16(kM, kN);
    const int x = warp == 11;
    const uint32_t k_lo = desc_lo(smem_addr(k_sm), 0) + x * (C::kTileBytes >> 4);
    const uint32_t q_lo = desc_lo(smem_addr(ring), 0);
    bool ok = true;
    auto ready = [&](uint64_t* bar, uint32_t parity) {
      ok = ok && __all_sync(0xffffffffu, wait(bar, parity, abort_flag));
    };
    ready(k_full, 0);
    int slot = 0;
    uint32_t par = 0;
    for (int i = 0; i < n && ok; ++i) {
      const int b = i & 1;
      if (i >= 2) ready(&s_free[2 * x + b], (i >> 1 & 1) ^ 1);
#pragma unroll 1
      for (int h = 0; h < C::kPieces; ++h) {
        ready(&full[slot], par);
        if (!ok) break;
        tc_fence_after_sync();
        if (lane == 0) {
          const uint32_t k = k_lo + h * (C::kSlotBytes >> 4);
          const uint32_t q = q_lo + slot * (C::kSlotBytes >> 4);
          const uint32_t t_s = tmem + (2 * x + b) * kN, acc = h != 0;
#pragma unroll
          for (int kk = 0; kk < C::kSlotChunks * 4; ++kk) {
            const uint32_t off = ((kk >> 2) * C::kChunk + (kk & 3) * 32) >> 4;
            umma_ss(t_s, k + off, q + off, id, kk == 0 ? acc : 1u);
          }
          umma_commit(&empty[slot]);
          if (h == C::kPieces - 1) umma_commit(&s_full[2 * x + b]);
        }
        __syncwarp();
        if (++slot == C::kSlots) slot = 0, par ^= 1u;
      }
    }
    if (lane == 0) {
      umma_commit(mma_done);
      volatile int no_abort = 0;
      if (!wait(mma_done, 0, &no_abort)) atomicOr(a.err, NVFP4_ATTENTION_TIMEOUT);
    }
    __syncwarp();
  } else if (warp == 10) {
    // ----------------------------------------------------- the rows' log-sums
    for (int i = 0; i < n; ++i) {
      const int l = i % kLogs;
      if (i >= kLogs) {
        wait(&log_free[l], (i / kLogs & 1) ^ 1, abort_flag);
        __syncwarp();
      }
      const int tok0 = (first + i) * p.tile_tokens;
#pragma unroll
      for (int r = lane; r < kN; r += 32) {
        const int tok = r / a.group, g = r - tok * a.group;
        float v = -INFINITY;                             // rows that hold no token
        if (tok < p.tile_tokens && tok0 + tok < si.q_len) {
          const float lse = a.lse[int64_t(si.q0 + tok0 + tok) * a.q_heads + kvh * a.group + g];
          if (lse != -INFINITY) v = -1.44269504088896f * lse;   // (-inf: it sees no key)
        }
        logs[l * kN + r] = v;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&log_full[l]);
    }
  }
  if (*abort_flag && threadIdx.x == 0) atomicOr(a.err, NVFP4_ATTENTION_TIMEOUT);
  tc_fence_before_sync();
  __syncthreads();
  float* sums = reinterpret_cast<float*>(ring);         // (no copy or product is on its way)
  if (ctas > 1) {
    if (threadIdx.x < kKeys) sums[threadIdx.x] = received;
    cluster_sync();
  }
  const int key = key0 + static_cast<int>(threadIdx.x);
  if (rank == 0 && threadIdx.x < kKeys && key < a.room) {
    for (uint32_t r = 1; r < ctas; ++r)
      received += ld_cluster_f32(map_to_rank(smem_addr(&sums[threadIdx.x]), r));
    a.out[out0 + key] = key < si.kv_len ? (a.mass ? a.mass[out0 + key] : 0.f) + received : 0.f;
  }
  if (ctas > 1) cluster_sync();                         // no CTA ends while its sums are read
  if (warp == 9) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

template <int kDim, bool kE4m3>
int run(const Mass& a, const Device& d, cudaStream_t stream) {
  using C = Cfg<kDim>;
  auto* kernel = mass_tc_kernel<kDim, kE4m3>;
  static std::atomic<bool> ready[kMaxDevices];
  if (const int st = allow_smem(kernel, C::kSmem, d, ready)) return st;
  const int64_t blocks = (a.room + kKeys - 1) / kKeys;
  if (a.cache.heads > 65535 || a.seqs.count > 65535) return NVFP4_ERR_SHAPE;
  MassTc p{a, kM / a.group, 4};
  while (p.box_shift < 7 && a.cache.page_size % (2 << p.box_shift) == 0) ++p.box_shift;
  CUtensorMap tm_q{}, tm_k{};
  if (!query_map(&tm_q, a.q, a.cache.dim, a.q_heads, a.seqs.tokens, a.group, p.tile_tokens) ||
      (!kE4m3 && !page_map(&tm_k, a.cache, false, 64, 1 << p.box_shift, 1)))
    return NVFP4_ERR_LAUNCH;
  // Where the new tokens may be half of all, the CTAs of the first keys would see
  // far more queries than those of the last: a cluster of 4 shares them.  8192
  // keys, 8192 new: 305 us against 582 with one CTA; 4096: 244 against 298; 1024,
  // where each CTA's start counts: 104 against 81.  (The lengths lie on the device:
  // the rule goes by the room for them, so that a prompt in a wider mass tensor
  // takes one CTA.)
  const int ctas = 2 * int64_t(a.max_q_len) >= a.room ? 4 : 1;
  if (blocks > INT32_MAX / ctas) return NVFP4_ERR_SHAPE;
  return launch_clusters(ctas, kernel,
                         dim3(static_cast<unsigned>(blocks * ctas), a.cache.heads, a.seqs.count),
                         dim3(kThreads), C::kSmem, stream, tm_q, tm_k, p);
}

}  // namespace

int run_mass_tc(const Mass& p, const Device& d, cudaStream_t stream) {
  const bool f8 = p.cache.e4m3;
  switch (p.cache.dim) {
    case 64:
      return f8 ? run<64, true>(p, d, stream) : run<64, false>(p, d, stream);
    case 128:
      return f8 ? run<128, true>(p, d, stream) : run<128, false>(p, d, stream);
    default:
      return f8 ? run<256, true>(p, d, stream) : run<256, false>(p, d, stream);
  }
}

}  // namespace attn
}  // namespace nvfp4
