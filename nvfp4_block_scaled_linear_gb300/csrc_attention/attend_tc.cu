// attend_tc.cu -- paged attention for many query rows (prefill chunks, wide
// verify) on the tcgen05 tensor cores.
//
// A tile is 128 query rows (128 / group tokens times the group's heads) in
// the 128 lanes of TMEM; a block is 128 keys.  S = Q K^T lands in one of two
// 128-column buffers, a thread per row turns it into weights P in place (16
// bits, over the first half of the same columns), and O += P V takes P from
// TMEM.  The one issuing thread keeps two blocks of scores ahead of the
// weights:   S0 S1 | PV0 S2 | PV1 S3 | ...
// so that the softmax of one block overlaps the products of the others.
//
// kTiles = 1 (head_dim 256, whose accumulator takes half of TMEM; or few
// rows): the two score buffers hold consecutive blocks of one tile, and two
// warpgroups take them in turn, handing on the running maximum.
// kTiles = 2 (head_dim 64, 128): the buffers hold two tiles on the same
// block, which halves the copies per product.
//
// The accumulator is rescaled only when a row's maximum has grown by more
// than 2^8 since the last time (weights stay below 2^8, and the sums are
// fp32), which after the first blocks is rare.
//
// What bounds it: the products, 4 * 128 * 128 * head_dim flops a block and
// tile, and beside them the shared-memory traffic of their operands (Q and K
// each read per product, V once, plus the copies that bring K and V).
//
// Warps: 0-3 and 4-7 softmax and output; 8 K/V copies; 9 MMA; 10 the check of
// V rows that not every row of the tile sees (or that lie past the length:
// zeroed, as 0 times what a page happens to hold need not be 0); 11 Q copies.
// Over an e4m3 cache warps 12-15 widen K and V to f16 (exact) on their way to
// shared memory and do warp 10's work as they go, and warps 8, 10 and 11 bring
// Q, scaled per row by a power of two (attend_warp.cu says why), in f16.
//
// A V value that is not finite and that only some rows of the tile see would
// reach the others as 0 * NaN: it is replaced by zero before the product and
// added to the rows that see it at the end (`dirty`).
#include <algorithm>
#include <type_traits>

#include "attend.cuh"

namespace nvfp4 {
namespace attn {
namespace {

constexpr int kM = 128;                       // rows of a tile
constexpr int kN = 128;                       // keys of a block (one unit)
constexpr float kSlack = 8.f;                 // growth of log2 of a weight before rescaling
constexpr int kQFactors = 4;                  // items whose row factors are held
constexpr int kDirty = 8;                     // items whose `dirty` note is held: more than the ring's

template <int kDim, bool kE4m3, int kTiles>
struct Cfg {
  static constexpr int kThreads = kE4m3 ? 512 : 384;
  // A slot holds 16 KB: 64 of head_dim of all keys of a K block, or all of
  // head_dim of some keys of a V block (64 columns by 64 columns).  Small
  // slots are refilled as soon as a few MMAs are done with them: at head_dim
  // 256 the ring is little more than one block deep.
  static constexpr int kPieces = kDim / 64;                    // slots of one K (or V) block
  static constexpr int kSlotBytes = kN * 128;
  static constexpr int kVKeys = kN / kPieces;                  // keys of a V slot
  static constexpr int kVChunk = kVKeys * 128;                 // bytes of 64 columns of it
  static constexpr int kQTile = kM * kDim * 2;
  static constexpr int kQBytes = kTiles * kQTile;
  static constexpr int kMaxSlots = 12;
  static constexpr int kBars = 3 * kMaxSlots + 19;
  static constexpr int kBarOff = 0;
  static constexpr int kMaxOff = (kBarOff + kBars * 8 + 8 + kDirty * 4 + 15) / 16 * 16;   // running maxima
  static constexpr int kSumOff = kMaxOff + (kTiles == 1 ? kM * 4 : 0);        // row sums
  static constexpr int kFacOff = kSumOff + (kTiles == 1 ? 2 * kM * 4 : 0);    // Q row factors
  static constexpr int kRowOff = kFacOff + (kE4m3 ? kQFactors * kTiles * kM * 4 : 0);
  static constexpr int kFixed = kRowOff + (kE4m3 ? 2 * kN * 8 : 0);
  static constexpr int kBudget = 227 * 1024 - 1024 - kFixed - kQBytes;
  static constexpr int kSlots = std::min(kMaxSlots, kBudget / kSlotBytes);
  static constexpr int kSmem = kQBytes + kSlots * kSlotBytes + kFixed + 1024;
  static_assert(kSlots >= 2 * kPieces, "K and V of one block have to fit");
  static_assert(kSlots * kSlotBytes >= static_cast<int>(sizeof(RangeSmem)), "scratch of the start");
  // TMEM columns: the accumulators, then the two score buffers
  static constexpr uint32_t kO = 0;
  static constexpr uint32_t kS = kTiles * kDim;
  static_assert(kS + 2 * kN <= 512, "TMEM");
};

// MN-major operand (d contiguous): 64 d per 128-byte row, 8-key groups 1024 B
// apart, the next 64 d `lbo` bytes on.
__device__ __forceinline__ uint64_t umma_desc_mn_sw128(uint32_t addr, uint32_t lbo) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((addr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

template <bool kE4m3>
__device__ __forceinline__ uint32_t idesc(uint32_t n, bool b_mn_major) {
  return (kE4m3 ? umma_idesc_f16(kM, n) : umma_idesc_bf16(kM, n)) | (b_mn_major ? 1u << 16 : 0u);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mov.b64 z, {%6, %7};\n\tfma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

template <int kRegs>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int32_t c0, int32_t c1, int32_t c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v) {
  uint32_t d;
  asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}"
      : "=r"(d)
      : "r"(v));
  return d;
}

// Whether any of a word's two 16-bit values is not finite.
template <bool kE4m3>
__device__ __forceinline__ bool non_finite(uint32_t w) {
  constexpr uint32_t e = kE4m3 ? 0x7C00u : 0x7F80u;
  return (w & e) == e || (w & (e << 16)) == (e << 16);
}
template <bool kE4m3>
__device__ __forceinline__ uint32_t finite_mask(uint32_t w) {
  constexpr uint32_t e = kE4m3 ? 0x7C00u : 0x7F80u;
  return ((w & e) == e ? 0u : 0xFFFFu) | ((w & (e << 16)) == (e << 16) ? 0u : 0xFFFF0000u);
}

struct TcParams {
  Attend a;
  Plan plan;
  Parts parts;
  int tile_tokens;          // tokens of one 128-row tile
  int box_rows;             // slots of one page copy
};

// The blocks of a CTA's range in order, tile by tile where a block serves two.
template <int kTiles>
struct Steps {
  Walk w;
  int b = 0, x = 0;           // block of the item, tile
  int item = 0;               // ordinal of the item in this CTA
  __device__ Steps(const Range& r, const TcParams& p) : w(r, p.a.seqs, p.plan, p.a.err) {}
  __device__ bool more() const { return w.more(); }
  __device__ bool first() const { return b == 0; }
  __device__ bool last() const { return b + 1 == w.count; }
  __device__ void next(const TcParams& p) {
    if (kTiles == 2 && x == 0) {
      x = 1;
      return;
    }
    x = 0;
    if (++b < w.count) return;
    b = 0;
    ++item;
    w.next(p.a.seqs, p.a.cache.heads, p.plan, p.a.err);
  }
};

template <int kDim, bool kE4m3, int kTiles>
__global__ void __launch_bounds__(Cfg<kDim, kE4m3, kTiles>::kThreads, 1)
    attend_tc_kernel(const __grid_constant__ CUtensorMap tm_q,
                     const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const TcParams p) {
  using C = Cfg<kDim, kE4m3, kTiles>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* q_sm = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  uint8_t* ring = q_sm + C::kQBytes;
  uint8_t* fixed = ring + C::kSlots * C::kSlotBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(fixed + C::kBarOff);
  uint64_t* empty = full + C::kMaxSlots;
  uint64_t* checked = empty + C::kMaxSlots;       // slot looked over by warp 10 (bf16)
  uint64_t* s_full = checked + C::kMaxSlots;      // [2] scores in buffer x
  uint64_t* p_full = s_full + 2;                  // [2] weights in buffer x
  uint64_t* pv_done = p_full + 2;                 // [2] product with buffer x's weights
  uint64_t* o_free = pv_done + 2;                 // [2] accumulator read out
  uint64_t* m_ready = o_free + 2;                 // [2][4] running maximum handed on, per warp
  uint64_t* q_full = m_ready + 8;
  uint64_t* q_empty = q_full + 1;
  uint64_t* mma_done = q_empty + 1;               // every product issued has completed
  volatile int* abort_flag = reinterpret_cast<volatile int*>(full + C::kBars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(full + C::kBars) + 1;
  volatile int* dirty = reinterpret_cast<volatile int*>(full + C::kBars) + 2;  // item ordinal + 1
  float* run_max = reinterpret_cast<float*>(fixed + C::kMaxOff);
  float* row_sum = reinterpret_cast<float*>(fixed + C::kSumOff);
  float* q_factor = reinterpret_cast<float*>(fixed + C::kFacOff);
  const Attend& a = p.a;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(&full[i], kE4m3 ? 4 : 1);
      mbar_init(&empty[i], 1);
      mbar_init(&checked[i], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[x], 4);
      mbar_init(&pv_done[x], 1);
      mbar_init(&o_free[x], kTiles == 1 ? 8 : 4);
      for (int i = 0; i < 4; ++i) mbar_init(&m_ready[x * 4 + i], 1);
    }
    mbar_init(q_full, kE4m3 ? 3 : 1);
    mbar_init(q_empty, 1);
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    for (int i = 0; i < kDirty; ++i) dirty[i] = 0;
    fence_mbar_init();
    if (!kE4m3) {
      prefetch_tensormap(&tm_q);
      prefetch_tensormap(&tm_k);
      prefetch_tensormap(&tm_v);
    }
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  griddep_wait();
  griddep_launch_dependents();
  // the range, in scratch that the ring's first copies will overwrite
  const Range range =
      find_range(a.seqs, a.cache.heads, p.plan, static_cast<int>(blockIdx.x),
                 static_cast<int>(gridDim.x), reinterpret_cast<RangeSmem*>(ring), a.err);
  fence_proxy_async_smem();
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  // Keys that every token of the item sees, and that its last one does.
  auto least_of = [&](const Walk& w) {
    return max(0, w.seq.kv_len - w.seq.q_len + w.r.tile * p.plan.tile_tokens + 1);
  };

  if (warp < 8) {
    // ------------------------------------------------------ softmax, output
    if constexpr (kE4m3) regs_inc<168>(); else regs_inc<208>();
    const int x = warp >> 2, quad = warp & 3;
    const int row = quad * 32 + lane;                 // of the tile
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t t_s = lane_base + C::kS + x * kN;
    const uint32_t t_o = lane_base + C::kO + (kTiles == 2 ? x * kDim : 0);
    const int tok = row / a.group, gi = row - tok * a.group;
    int flags = 0;
    int4 note = make_int4(0, 0, 0, 0);
    int step = 0;                                     // of both buffers (kTiles == 1)
    int uses = 0;                                     // of buffer x
    int item = 0;
    for (Walk w(range, a.seqs, p.plan, a.err); w.more();
         w.next(a.seqs, a.cache.heads, p.plan, a.err), ++item) {
      const SeqInfo seq = w.seq;
      const int ti = w.r.tile * p.plan.tile_tokens + (kTiles == 2 ? x * p.tile_tokens : 0) + tok;
      const bool valid = tok < p.tile_tokens && ti < seq.q_len;
      const int lim = valid ? max(0, seq.kv_len - seq.q_len + ti + 1) : 0;
      float c = a.scale * 1.44269504088896f;
      if (kE4m3 && a.cache.k_scale) c *= a.cache.k_scale[w.r.h];
      float m = -INFINITY, l = 0.f;                   // of the blocks that this thread saw
      for (int b = 0; b < w.count; ++b, ++step) {
        if (kTiles == 1 && (step & 1) != x) continue;
        mbar_wait(&s_full[x], uses & 1, abort_flag);
        __syncwarp();
        tc_fence_after_sync();
        if (kE4m3 && (b == 0 || (kTiles == 1 && b == 1)))
          c *= q_factor[(item % kQFactors) * kTiles * kM + (kTiles == 2 ? x * kM : 0) + row];
        uint32_t s[4][32];
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld_32cols(t_s + i * 32, s[i]);
        tmem_ld_wait();
        const int seen = lim - (w.r.unit0 + b) * kN;  // of this block, by this row
        if (__any_sync(0xffffffffu, seen < kN)) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (i * 32 + j >= seen) s[i][j] = 0xFF800000u;
        }
        float t4[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          t4[i] = fmaxf(__uint_as_float(s[i][0]), __uint_as_float(s[i][1]));
#pragma unroll
          for (int j = 2; j < 32; j += 2)
            t4[i] = fmaxf(t4[i], fmaxf(__uint_as_float(s[i][j]), __uint_as_float(s[i][j + 1])));
        }
        const float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])) * c;
        // ---- the maximum the weights are taken against
        float now = top;
        if (b > 0) {
          float prev = m;
          if (kTiles == 1) {
            mbar_wait(&m_ready[(x ^ 1) * 4 + quad], ((step - 1) >> 1) & 1, abort_flag);
            __syncwarp();
            prev = run_max[row];
          }
          now = fmaxf(prev, top);
          if (__any_sync(0xffffffffu, now - prev > kSlack)) {
            // the accumulator, complete up to the block before
            if (kTiles == 1)
              mbar_wait(&pv_done[x ^ 1], ((step - 1) >> 1) & 1, abort_flag);
            else
              mbar_wait(&pv_done[x], (uses - 1) & 1, abort_flag);
            __syncwarp();
            tc_fence_after_sync();
            const float alpha = prev == -INFINITY ? 0.f : ex2(prev - now);
#pragma unroll 1
            for (int i = 0; i < kDim; i += 32) {
              uint32_t o[32];
              tmem_ld_32cols(t_o + i, o);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
              tmem_st_32cols(t_o + i, o);
            }
            tmem_st_wait();
          } else {
            now = prev;
          }
        }
        if (kTiles == 1) {
          run_max[row] = now;
          __syncwarp();
          if (lane == 0) mbar_arrive(&m_ready[x * 4 + quad]);
        }
        const float base = now == -INFINITY ? 0.f : now;
        if (m != now) l *= m == -INFINITY ? 0.f : ex2(m - base);
        m = now;
        // ---- the weights
        const float2 c2 = make_float2(c, c), b2 = make_float2(-base, -base);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          uint32_t w16[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const uint32_t* sj = &s[i + (j >> 4)][2 * (j & 15)];
            float2 e = fma2(make_float2(__uint_as_float(sj[0]), __uint_as_float(sj[1])), c2, b2);
            e.x = ex2(e.x), e.y = ex2(e.y);
            sum[j & 1] = add2(sum[j & 1], e);
            w16[j] = kE4m3 ? f32x2_to_f16x2(e.x, e.y) : f32x2_to_bf16x2(e.x, e.y);
          }
          tmem_st_32cols(t_s + i * 16, w16);
        }
        sum[0] = add2(sum[0], sum[1]);
        l += sum[0].x + sum[0].y;
        tmem_st_wait();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[x]);
        ++uses;
      }
      // ---- the row's sum, and the result
      const bool whole = w.begins() && w.ends();
      const int part = w.begins() ? 1 : 0;
      if (!whole) {
        flags |= part ? kPart1 : kPart0 | (w.ends() ? kPart0Ends : 0);
        if (part) note = make_int4(0, w.r.s, w.r.h, w.r.tile);
      }
      if (kTiles == 1) {
        // the last product with either buffer, whose weights both groups gave
        mbar_wait(&pv_done[(step - 1) & 1], ((step - 1) >> 1) & 1, abort_flag);
        __syncwarp();
        const float now = run_max[row];               // of the last block
        row_sum[x * kM + row] = m == -INFINITY ? l : l * ex2(m - now);
        asm volatile("bar.sync 1, 256;" ::: "memory");
        l = row_sum[row] + row_sum[kM + row];
        m = now;
      } else {
        mbar_wait(&pv_done[x], (uses - 1) & 1, abort_flag);
        __syncwarp();
      }
      tc_fence_after_sync();
      const float vs = kE4m3 && a.cache.v_scale ? a.cache.v_scale[w.r.h] : 1.f;
      const float inv = l == 0.f ? 0.f : vs / l;
      const int64_t token = seq.q0 + ti;
      const int head = w.r.h * a.group + gi;
      const int prow = (kTiles == 2 ? x * kM : 0) + row;
      const int64_t at_part = p.parts.row(blockIdx.x, part, prow);
      if (valid && (kTiles == 2 || x == 0)) {
        const float lse2 = l == 0.f ? -INFINITY : m + log2f(l);
        if (whole && a.lse) a.lse[token * a.q_heads + head] = lse2 * 0.693147180559945f;
        if (!whole) p.parts.lse2[at_part] = lse2;
      }
      const bool fix = dirty[item % kDirty] == item + 1;
      // kTiles == 1: each group writes half of the columns
      constexpr int kCols = kTiles == 1 ? kDim / 2 : kDim;
      const int col0 = kTiles == 1 ? x * kCols : 0;
#pragma unroll 1
      for (int i = col0; i < col0 + kCols; i += 32) {
        uint32_t o[32];
        tmem_ld_32cols(t_o + i, o);
        tmem_ld_wait();
        if (i + 32 == col0 + kCols) {
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&o_free[kTiles == 1 ? 0 : x]);
        }
        if (valid) {
#pragma unroll
        for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * inv);
        if (fix) {
          // values that are not finite, of the keys that not all rows see
          const int from = max(least_of(w), w.r.unit0 * kN);
          const int to = min(lim, (w.r.unit0 + w.count) * kN);
#pragma unroll 1
          for (int key = from; key < to; ++key) {
            const int64_t page = checked_page(
                a.seqs.table[int64_t(w.r.s) * a.seqs.width + key / a.cache.page_size],
                a.cache.pages, a.err);
            if (page == a.cache.pages) continue;
            const int64_t off = page * a.cache.vs[0] + key % a.cache.page_size * a.cache.vs[1] +
                                w.r.h * a.cache.vs[2] + i;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const float v = kE4m3
                                  ? e4m3_to_f32(static_cast<const uint8_t*>(a.cache.v)[off + j])
                                  : __bfloat162float(static_cast<const __nv_bfloat16*>(a.cache.v)[off + j]);
              if (!isfinite(v)) o[j] = __float_as_uint(__uint_as_float(o[j]) + v);
            }
          }
        }
        if (whole) {
          uint4* dst = reinterpret_cast<uint4*>(a.out.data + token * a.out.ts + head * a.out.hs + i);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t y[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              y[k] = f32x2_to_bf16x2(__uint_as_float(o[8 * j + 2 * k]),
                                     __uint_as_float(o[8 * j + 2 * k + 1]));
            dst[j] = make_uint4(y[0], y[1], y[2], y[3]);
          }
        } else {
          uint4* dst = reinterpret_cast<uint4*>(p.parts.out + at_part * kDim + i);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            dst[j] = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
        }
        }
        __syncwarp();
      }
      if (kTiles == 1) asm volatile("bar.sync 1, 256;" ::: "memory");   // row_sum is free again
    }
    if (threadIdx.x == 0) {
      note.x = flags;
      p.parts.note[blockIdx.x] = note;
    }
  } else if (warp < 12) {
    if constexpr (kE4m3) regs_dec<72>(); else regs_dec<80>();
    if (warp == 9) {
      // ------------------------------------------------------------- MMA
      if (lane == 0) {
        const uint32_t id_s = idesc<kE4m3>(kN, false);
        const uint32_t id_o = idesc<kE4m3>(kDim, true);
        const uint32_t q_addr = smem_addr(q_sm), ring_addr = smem_addr(ring);
        uint64_t* v_bar = kE4m3 ? full : checked;
        Steps<kTiles> qk(range, p), pv(range, p);
        int slot_q = 0, slot_v = 0;               // ring positions of the next K and V
        int it = 0;                               // ring position in the order of the copies
        bool ok = true;
        for (int i = 0; ok && (qk.more() || pv.more()); ++i) {
          if (i >= 2) {
            // ---- O += P V
            const int x = i & 1, u = (i - 2) >> 1;
            ok = mbar_wait(&p_full[x], u & 1, abort_flag);
            if (ok && pv.first() && pv.item > 0 && (kTiles == 2 || pv.b == 0))
              ok = mbar_wait(&o_free[kTiles == 1 ? 0 : x], (pv.item - 1) & 1, abort_flag);
            if (pv.x == 0) {
              slot_v = it;
              it += C::kPieces;
            }
            const uint32_t t_o = tmem + C::kO + (kTiles == 2 ? x * kDim : 0);
            for (int h = 0; h < C::kPieces && ok; ++h) {
              const int s = (slot_v + h) % C::kSlots;
              ok = mbar_wait(&v_bar[s], ((slot_v + h) / C::kSlots) & 1, abort_flag);
              if (!ok) break;
              tc_fence_after_sync();
              const uint32_t v = ring_addr + s * C::kSlotBytes;
              const uint32_t t_p = tmem + C::kS + x * kN + h * (C::kVKeys / 2);
#pragma unroll
              for (int kk = 0; kk < C::kVKeys / 16; ++kk)
                umma_f16_tmem_a(t_o, t_p + kk * 8, umma_desc_mn_sw128(v + kk * 2048, C::kVChunk),
                                id_o, !(pv.first() && (h | kk) == 0));
              if (kTiles == 1 || x == 1) umma_commit(&empty[s]);
            }
            if (!ok) break;
            umma_commit(&pv_done[x]);
            pv.next(p);
          }
          if (qk.more()) {
            // ---- S = Q K^T
            const int x = i & 1;
            if (qk.first() && qk.x == 0) ok = mbar_wait(q_full, qk.item & 1, abort_flag);
            if (qk.x == 0) {
              slot_q = it;
              it += C::kPieces;
            }
            for (int h = 0; h < C::kPieces && ok; ++h) {
              const int s = (slot_q + h) % C::kSlots;
              ok = mbar_wait(&full[s], ((slot_q + h) / C::kSlots) & 1, abort_flag);
              if (!ok) break;
              tc_fence_after_sync();
              const uint32_t k = ring_addr + s * C::kSlotBytes;
              const uint32_t q = q_addr + (kTiles == 2 ? x * C::kQTile : 0) + h * C::kSlotBytes;
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                umma_bf16(tmem + C::kS + x * kN, umma_desc_sw128(q + kk * 32),
                          umma_desc_sw128(k + kk * 32), id_s, (h | kk) != 0);
              if (kTiles == 1 || x == 1) umma_commit(&empty[s]);
            }
            if (!ok) break;
            umma_commit(&s_full[x]);
            if (qk.last() && qk.x == kTiles - 1) umma_commit(q_empty);
            qk.next(p);
          }
        }
        // nothing may be in flight when TMEM is released
        umma_commit(mma_done);
        volatile int no_abort = 0;
        if (!mbar_wait(mma_done, 0, &no_abort)) atomicOr(a.err, NVFP4_ATTENTION_TIMEOUT);
      }
      __syncwarp();
    } else if (warp == 8 && !kE4m3) {
      // ------------------------------------------------------ K, V copies
      Steps<1> kc(range, p), vc(range, p);        // block by block for either kTiles
      int it = 0;
      bool ok = true;
      // A block's pages: lane i holds that of rows i * box_rows on, read one
      // block ahead of its use and kept for the V of the same keys.
      struct Pages {
        int key, entry, page, in_page;
      };
      const int k_boxes = kN / p.box_rows;
      const int v_rows = min(p.box_rows, C::kVKeys), v_boxes = C::kVKeys / v_rows;
      auto look_up = [&](const Steps<1>& st) {
        Pages g{-1, 0, -1, 0};
        if (!st.more()) return g;
        const int key = (st.w.r.unit0 + st.b) * kN + lane * p.box_rows;
        if (lane < k_boxes && key < st.w.seq.kv_len) {
          g.key = key;
          g.entry = a.seqs.table[int64_t(st.w.r.s) * a.seqs.width + key / a.cache.page_size];
        }
        return g;
      };
      auto next_slot = [&](uint32_t bytes) {
        const int s = it % C::kSlots;
        if (it >= C::kSlots)
          ok = __all_sync(0xffffffffu, mbar_wait(&empty[s], ((it / C::kSlots) & 1) ^ 1, abort_flag));
        if (ok && lane == 0) mbar_arrive_expect_tx(&full[s], bytes);
        return s;
      };
      // One lane issues: a copy's operands are warp-uniform registers, and
      // copies from several lanes took some 250 cycles each.
      auto copy_k = [&](const Walk& w, const Pages& g) {
        const int n = __popc(__ballot_sync(0xffffffffu, g.page >= 0));
        for (int h = 0; h < C::kPieces; ++h, ++it) {
          const int s = next_slot(n * p.box_rows * 128);
          if (!ok) return;
          for (int i = 0; i < k_boxes; ++i) {
            const int page = __shfl_sync(0xffffffffu, g.page, i);
            const int in_page = __shfl_sync(0xffffffffu, g.in_page, i);
            if (lane == 0 && page >= 0)
              tma_load_page(ring + s * C::kSlotBytes + i * p.box_rows * 128, &tm_k, &full[s], h,
                            in_page, w.r.h, page);
          }
        }
      };
      auto copy_v = [&](const Walk& w, const Pages& g) {
        const int v_chunks = v_boxes == 1 ? C::kPieces : 1;         // of one copy
        for (int h = 0; h < C::kPieces; ++h, ++it) {
          int n = 0;
          for (int i = 0; i < v_boxes; ++i)
            n += __shfl_sync(0xffffffffu, g.page, (h * C::kVKeys + i * v_rows) / p.box_rows) >= 0;
          const int s = next_slot(n * C::kPieces * v_rows * 128);
          if (!ok) return;
          for (int i = 0; i < v_boxes; ++i) {
            const int row = h * C::kVKeys + i * v_rows;             // of the block
            const int from = row / p.box_rows;
            const int page = __shfl_sync(0xffffffffu, g.page, from);
            const int in_page = __shfl_sync(0xffffffffu, g.in_page, from) + row - from * p.box_rows;
            if (lane == 0 && page >= 0)
              for (int ch = 0; ch < C::kPieces; ch += v_chunks)
                tma_load_page(ring + s * C::kSlotBytes + ch * C::kVChunk + i * v_rows * 128, &tm_v,
                              &full[s], ch, in_page, w.r.h, page);
          }
        }
      };
      // in the order of the products: with one tile V0 after K1, with two after K0
      constexpr int kAhead = kTiles == 1 ? 2 : 1;
      Pages ahead = look_up(kc), held[kAhead];
      for (int i = 0; ok && (kc.more() || vc.more()); ++i) {
        Pages now = ahead;
        if (now.key >= 0) {
          now.page = static_cast<int>(checked_page(now.entry, a.cache.pages, a.err));
          now.in_page = now.key % a.cache.page_size;
        }
        const Walk kw = kc.w;
        const bool k_left = kc.more();
        if (k_left) {
          kc.next(p);
          ahead = look_up(kc);
        }
        if (i >= kAhead) {
          copy_v(vc.w, held[0]);
          vc.next(p);
        }
        if (ok && k_left) copy_k(kw, now);
        if (kAhead == 2) held[0] = held[kAhead - 1];
        held[kAhead - 1] = now;
      }
      for (int i = max(0, it - C::kSlots); i < it; ++i) {
        volatile int no_abort = 0;
        if (!mbar_wait(&full[i % C::kSlots], (i / C::kSlots) & 1, &no_abort))
          atomicOr(a.err, NVFP4_ATTENTION_TIMEOUT);
      }
    } else if (warp == 10 && !kE4m3) {
      // ---------------------------------------------- V rows not all rows see
      Steps<1> kc(range, p), vc(range, p);
      int it = 0;
      constexpr int kAhead = kTiles == 1 ? 2 : 1;
      for (int i = 0; kc.more() || vc.more(); ++i) {
        if (i >= kAhead) {
          const Walk& w = vc.w;
          const int seen = tile_keys(w.seq, w.r.tile, p.plan);
          const int least = least_of(w);
          for (int h = 0; h < C::kPieces; ++h, ++it) {
            const int key0 = (w.r.unit0 + vc.b) * kN + h * C::kVKeys;
            const int s = it % C::kSlots;
            mbar_wait(&full[s], (it / C::kSlots) & 1, abort_flag);
            __syncwarp();
            if (key0 + C::kVKeys > least) {
              // 16-byte pieces of the rows from `lo` on: the first `look` of them
              // are looked at, the others zeroed
              constexpr int kPer = C::kPieces * 8;
              const int lo = max(0, least - key0);
              const int look = (min(max(seen - key0, lo), C::kVKeys) - lo) * kPer;
              uint8_t* slot = ring + s * C::kSlotBytes;
              auto at = [&](int j) {
                return reinterpret_cast<uint4*>(slot + (j % kPer >> 3) * C::kVChunk +
                                                (lo + j / kPer) * 128 + (j & 7) * 16);
              };
              bool bad = false;
#pragma unroll 4
              for (int j = lane; j < look; j += 32) {
                uint4 v = *at(j);
                if (non_finite<kE4m3>(v.x) || non_finite<kE4m3>(v.y) || non_finite<kE4m3>(v.z) ||
                    non_finite<kE4m3>(v.w)) {
                  bad = true;
                  v.x &= finite_mask<kE4m3>(v.x), v.y &= finite_mask<kE4m3>(v.y);
                  v.z &= finite_mask<kE4m3>(v.z), v.w &= finite_mask<kE4m3>(v.w);
                  *at(j) = v;
                }
              }
#pragma unroll 4
              for (int j = look + lane; j < (C::kVKeys - lo) * kPer; j += 32)
                *at(j) = make_uint4(0, 0, 0, 0);
              if (bad) dirty[vc.item % kDirty] = vc.item + 1;
              fence_proxy_async_smem();
              __syncwarp();
            }
            if (lane == 0) mbar_arrive(&checked[s]);
          }
          vc.next(p);
        }
        if (kc.more()) {
          // nothing to check in K, but a phase of `checked` goes with every
          // turn of the slot, and follows the turn's copy
          for (int h = 0; h < C::kPieces; ++h, ++it) {
            const int s = it % C::kSlots;
            mbar_wait(&full[s], (it / C::kSlots) & 1, abort_flag);
            __syncwarp();
            if (lane == 0) mbar_arrive(&checked[s]);
          }
          kc.next(p);
        }
      }
    } else if (!kE4m3) {
      // --------------------------------------------------------- Q copies
      if (lane == 0) {
        int item = 0;
        const int rows = p.tile_tokens * a.group;
        for (Walk w(range, a.seqs, p.plan, a.err); w.more();
             w.next(a.seqs, a.cache.heads, p.plan, a.err), ++item) {
          if (item > 0 && !mbar_wait(q_empty, (item - 1) & 1, abort_flag)) break;
          mbar_arrive_expect_tx(q_full, kTiles * (kDim / 64) * rows * 128);
          const int t0 = w.seq.q0 + w.r.tile * p.plan.tile_tokens;
#pragma unroll
          for (int x = 0; x < kTiles; ++x)
#pragma unroll
            for (int ch = 0; ch < kDim / 64; ++ch)
              tma_load_3d(q_sm + x * C::kQTile + ch * kM * 128, &tm_q, q_full, ch * 64,
                          w.r.h * a.group, t0 + x * p.tile_tokens);
        }
        if (item > 0) {
          volatile int no_abort = 0;
          if (!mbar_wait(q_full, (item - 1) & 1, &no_abort)) atomicOr(a.err, NVFP4_ATTENTION_TIMEOUT);
        }
      }
      __syncwarp();
    } else {
      // ---------------------------------- Q rows scaled to f16 (warps 8, 10, 11)
      const int part = warp == 8 ? 0 : warp - 9;
      constexpr int kWords = kDim / 64;             // 32-bit words per lane
      int item = 0;
      for (Walk w(range, a.seqs, p.plan, a.err); w.more();
           w.next(a.seqs, a.cache.heads, p.plan, a.err), ++item) {
        if (item > 0) {
          mbar_wait(q_empty, (item - 1) & 1, abort_flag);
          __syncwarp();
        }
        constexpr int kAtOnce = 4;
        for (int r0 = part * kAtOnce; r0 < kTiles * kM; r0 += 3 * kAtOnce) {
          uint32_t v[kAtOnce][kWords];
#pragma unroll
          for (int i = 0; i < kAtOnce; ++i) {
            const int r = r0 + i, x = r / kM, rr = r % kM;
            const int tok = rr / a.group, gi = rr - tok * a.group;
            const int ti = w.r.tile * p.plan.tile_tokens + x * p.tile_tokens + tok;
            const bool valid = tok < p.tile_tokens && ti < w.seq.q_len;
            const uint32_t* src = reinterpret_cast<const uint32_t*>(
                a.q.data + int64_t(w.seq.q0 + ti) * a.q.ts + int64_t(w.r.h * a.group + gi) * a.q.hs);
#pragma unroll
            for (int k = 0; k < kWords; ++k) v[i][k] = valid ? src[k * 32 + lane] : 0u;
          }
#pragma unroll
          for (int i = 0; i < kAtOnce; ++i) {
            const int r = r0 + i, x = r / kM, rr = r % kM;
            float top = 0.f;
#pragma unroll
            for (int k = 0; k < kWords; ++k)
              top = fmaxf(top, fmaxf(fabsf(bf16_lo(v[i][k])), fabsf(bf16_hi(v[i][k]))));
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            int e = 141 - static_cast<int>(__float_as_uint(top) >> 23);
            e = top == 0.f || top > 3.4e38f ? 0 : min(e, 100);
            const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
            if (lane == 0)
              q_factor[(item % kQFactors) * kTiles * kM + r] =
                  __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
            for (int k = 0; k < kWords; ++k) {
              // elements 64 k + 2 lane and the next: chunk k, byte 4 lane of the row
              const uint32_t f = f32x2_to_f16x2(bf16_lo(v[i][k]) * up, bf16_hi(v[i][k]) * up);
              *reinterpret_cast<uint32_t*>(q_sm + x * C::kQTile + k * kM * 128 + rr * 128 +
                                           (((lane >> 2) ^ (rr & 7)) << 4) + (lane & 3) * 4) = f;
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
      }
    }
  } else {
    // ------------------------------------------ K, V codes widened to f16
    if constexpr (kE4m3) {
      regs_dec<96>();
      const int tid = threadIdx.x - 384;            // 0..127
      constexpr int kPasses = 4;                    // 16 codes a thread each
      int64_t* row_at = reinterpret_cast<int64_t*>(fixed + C::kRowOff);   // [2][128], then V's
      Steps<1> kc(range, p), vc(range, p);
      int it = 0;
      constexpr int kAhead = kTiles == 1 ? 2 : 1;
      auto fill = [&](auto values, const Steps<1>& st, const int64_t* rows, const uint8_t* base) {
        constexpr bool kV = decltype(values)::value;
        constexpr int kPerRow = kV ? kDim / 16 : 4;          // threads of a row
        constexpr int kRowsAtOnce = 128 / kPerRow;
        const int my_row = tid / kPerRow, my_col = (tid % kPerRow) * 16;
        const Walk& w = st.w;
        const int seen = tile_keys(w.seq, w.r.tile, p.plan);
        const int least = least_of(w);
        for (int h = 0; h < C::kPieces; ++h, ++it) {
          const int s = it % C::kSlots;
          uint4 v[kPasses];
#pragma unroll
          for (int i = 0; i < kPasses; ++i) {
            const int64_t at = rows[(kV ? h * C::kVKeys : 0) + i * kRowsAtOnce + my_row];
            v[i] = make_uint4(0, 0, 0, 0);
            if (at >= 0)                                      // else: a row past the length
              v[i] = *reinterpret_cast<const uint4*>(base + at + (kV ? 0 : h * 64) + my_col);
          }
          if (it >= C::kSlots) {
            mbar_wait(&empty[s], ((it / C::kSlots) & 1) ^ 1, abort_flag);
            __syncwarp();
          }
          const int key0 = (w.r.unit0 + st.b) * kN + (kV ? h * C::kVKeys : 0);
          const bool check = kV && key0 + C::kVKeys > least;
          bool bad = false;
#pragma unroll
          for (int i = 0; i < kPasses; ++i) {
            const int r = i * kRowsAtOnce + my_row;
            const uint32_t cw[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            uint32_t f[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              f[2 * k] = e4m3x2_to_f16x2(cw[k] & 0xFFFFu);
              f[2 * k + 1] = e4m3x2_to_f16x2(cw[k] >> 16);
            }
            if (check) {
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                if (key0 + r >= seen) f[k] = 0;
                if (key0 + r >= least && non_finite<true>(f[k])) {
                  bad = true;
                  f[k] &= finite_mask<true>(f[k]);
                }
              }
            }
            // 16 codes: two 16-byte pieces of the 128-byte row
            uint8_t* row = ring + s * C::kSlotBytes + (kV ? (my_col >> 6) * C::kVChunk : 0) + r * 128;
            const int c16 = (my_col & 63) >> 3;
            *reinterpret_cast<uint4*>(row + ((c16 ^ (r & 7)) << 4)) = make_uint4(f[0], f[1], f[2], f[3]);
            *reinterpret_cast<uint4*>(row + (((c16 + 1) ^ (r & 7)) << 4)) =
                make_uint4(f[4], f[5], f[6], f[7]);
          }
          if (bad) dirty[st.item % kDirty] = st.item + 1;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[s]);
        }
      };
      // row offsets of a block, by one thread per row
      auto lookup = [&](const Steps<1>& st, const int64_t (&strides)[3], int64_t* rows) {
        const Walk& w = st.w;
        const int key = (w.r.unit0 + st.b) * kN + tid;
        int64_t at = -1;
        if (key < w.seq.kv_len) {
          const int64_t page = checked_page(
              a.seqs.table[int64_t(w.r.s) * a.seqs.width + key / a.cache.page_size], a.cache.pages,
              a.err);
          if (page != a.cache.pages)
            at = page * strides[0] + key % a.cache.page_size * strides[1] + w.r.h * strides[2];
        }
        asm volatile("bar.sync 2, 128;" ::: "memory");    // the rows before are read
        rows[tid] = at;
        asm volatile("bar.sync 2, 128;" ::: "memory");
      };
      for (int i = 0; kc.more() || vc.more(); ++i) {
        if (i >= kAhead) {
          lookup(vc, a.cache.vs, row_at + kN);
          fill(std::true_type{}, vc, row_at + kN, static_cast<const uint8_t*>(a.cache.v));
          vc.next(p);
        }
        if (kc.more()) {
          lookup(kc, a.cache.ks, row_at);
          fill(std::false_type{}, kc, row_at, static_cast<const uint8_t*>(a.cache.k));
          kc.next(p);
        }
      }
    }
  }
  if (*abort_flag && threadIdx.x == 0) atomicOr(a.err, NVFP4_ATTENTION_TIMEOUT);
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

template <int kDim, bool kE4m3, int kTiles>
int run(const Attend& a, const Device& d, cudaStream_t stream) {
  using C = Cfg<kDim, kE4m3, kTiles>;
  auto* kernel = attend_tc_kernel<kDim, kE4m3, kTiles>;
  static std::atomic<bool> ready[kMaxDevices];
  if (!ready[d.id].load(std::memory_order_acquire)) {
    // the warpgroups' shares (setmaxnreg) have to come out of what the block
    // is launched with
    cudaFuncAttributes attr;
    if (cudaFuncGetAttributes(&attr, kernel) != cudaSuccess) {
      cudaGetLastError();
      return NVFP4_ERR_LAUNCH;
    }
    constexpr int need = kE4m3 ? 256 * 168 + 128 * 72 + 128 * 96 : 256 * 208 + 128 * 80;
    if (attr.numRegs * C::kThreads < need) return NVFP4_ERR_LAUNCH;
  }
  if (const int st = allow_smem(kernel, C::kSmem, d, ready)) return st;
  TcParams p{a, {}, Parts(a.workspace, d.num_sms, kM, kTiles, kDim), kM / a.group, 0};
  p.plan = Plan{kTiles * p.tile_tokens, kN, 1};
  p.box_rows = 16;
  while (p.box_rows < kN && a.cache.page_size % (2 * p.box_rows) == 0) p.box_rows *= 2;
  CUtensorMap tm_q{}, tm_k{}, tm_v{};
  if (!kE4m3 && (!query_map(&tm_q, a, p.tile_tokens) ||
                 !page_map(&tm_k, a.cache, false, 64, p.box_rows, 1) ||
                 !page_map(&tm_v, a.cache, true, 64, std::min(p.box_rows, C::kVKeys),
                           p.box_rows >= C::kVKeys ? C::kPieces : 1)))
    return NVFP4_ERR_LAUNCH;
  if (const int st = launch(kernel, dim3(d.num_sms), dim3(C::kThreads), C::kSmem, stream, tm_q,
                            tm_k, tm_v, p))
    return st;
  return run_join(a, p.parts, p.plan, d.num_sms, stream);
}

template <int kDim, bool kE4m3>
int run_tiles(bool two, const Attend& a, const Device& d, cudaStream_t stream) {
  if constexpr (kDim < 256) {
    if (two) return run<kDim, kE4m3, 2>(a, d, stream);
  }
  return run<kDim, kE4m3, 1>(a, d, stream);
}

}  // namespace

int64_t attend_tc_workspace(int head_dim, const Device& d) {
  return Parts::bytes(d.num_sms, head_dim == 256 ? kM : 2 * kM, head_dim);
}

int run_attend_tc(int64_t rows, const Attend& a, const Device& d, cudaStream_t stream) {
  const bool two = rows > kM, f8 = a.cache.e4m3;
  switch (a.cache.dim) {
    case 64:
      return f8 ? run_tiles<64, true>(two, a, d, stream) : run_tiles<64, false>(two, a, d, stream);
    case 128:
      return f8 ? run_tiles<128, true>(two, a, d, stream) : run_tiles<128, false>(two, a, d, stream);
    default:
      return f8 ? run_tiles<256, true>(two, a, d, stream) : run_tiles<256, false>(two, a, d, stream);
  }
}

}  // namespace attn
}  // namespace nvfp4
