// attend_warp.cu -- paged attention for few query rows (decode, verify).
//
// The rows of one key/value head (its group's query heads times a few tokens)
// fill at most two 16-row tiles of the warp MMA, so the work is reading the
// cache once: bound by bytes.  The design is about keeping the memory busy:
// one CTA per SM (two where rows are short) takes an equal share of all keys
// (schedule.cuh) and one producer warp keeps a ring of 64-key tiles in flight
// through TMA, about 200 KB per SM, ahead of eight consumer warps.
//
// A block of 128 keys: warp w multiplies Q by its 16 keys' K (all of head_dim
// in registers' accumulators), the warps agree on the rows' new maximum
// through shared memory, write their weights there, and then each warp takes
// its own eighth of head_dim for P V over all 128 keys.  So every K and V
// element is read from shared memory once, the accumulator is rows x dim/8
// per warp, and nothing has to be merged between warps at the end but the row
// sums.  Two block barriers per 128 keys.
//
// Over an e4m3 cache the MMA is f16, in which every e4m3 value is exact: the
// codes are widened in registers, each query row is scaled by a power of two
// that puts its largest value near 2^14 (exact for values within 2^28 of it,
// and an absolute error below 2^-39 of it for smaller ones), and the scales of
// row and head are applied to the scores in fp32.  The k index inside an MMA
// is permuted so that a lane's codes are 16 consecutive bytes.
//
// The weights are rounded to the MMA's 16 bits (bf16, f16 over e4m3 pages)
// before P V, relative error 2^-8 or 2^-11 at most, no more than that of the bf16
// result; the row sums add the unrounded weights in fp32.  f16 has no weight below
// 2^-25, so there the row's largest is 2^kLift and not 1: relative error 2^-11 down
// to 2^-29 of the largest, nothing lost above 2^-40.  With the largest at 1 a tail of
// n keys near 2^-26 was lost from P V and not from the sum, up to n 2^-25 of the
// output.
//
// Measured with the join at 24 query and 4 key/value heads of 256: 32 ragged
// sequences of one token (451 MB of cache) 77.5 us, 5.83 TB/s, 87% of the copy
// rate; one token over 4099 keys 14.2 us, of which reading 16.8 MB is 2.5: the
// rest is the search for the range, one block's latency and the join.
#include <algorithm>

#include "attend.cuh"

namespace nvfp4 {
namespace attn {
namespace {

constexpr int kWarps = 8;
constexpr int kConsumers = kWarps * 32;
constexpr int kThreads = kConsumers + 32;
constexpr int kUnitShift = 4;
constexpr int kUnit = 1 << kUnitShift;        // keys of one warp in a block
constexpr int kSlotKeys = 64;
// Units that an item's beginning costs.  The 32 sequences measured 83 us at 2, 81
// at 4, 77.6 at 8 and 77.7 at 16; one token over 4099 keys 13.8, 15.5, 13.9 and
// 13.5.
constexpr int kExtra = 8;
constexpr int kPPitch = 128 * 2 + 16;         // bytes of a row of weights
// log2 of a row's largest weight (f16 ends at 2^16).
template <bool kE4m3>
constexpr float kLift = kE4m3 ? 15.f : 0.f;

template <int kDim, bool kE4m3, int kR>
struct Cfg {
  static constexpr int kEsz = kE4m3 ? 1 : 2;
  static constexpr int kRowBytes = kDim * kEsz;
  static constexpr int kChunkBytes = kRowBytes < 128 ? kRowBytes : 128;
  static constexpr int kChunks = kRowBytes / kChunkBytes;
  // a unit: chunk after chunk, each 16 rows of kChunkBytes
  static constexpr int kUnitBytes = kUnit * kRowBytes;
  static constexpr int kUnitChunk = kUnit * kChunkBytes;
  static constexpr int kSlotBytes = kSlotKeys * kRowBytes;
  static constexpr int kRows = 16 * kR;
  static constexpr int kQPitch = kDim * 2 + 16;
  // Two CTAs per SM where a block's copy is too short to hide one block's
  // two barriers behind the next block's.
  static constexpr int kCtas = kRowBytes <= 128 && kR == 1 ? 2 : 1;
  static constexpr int kQOff = 0;
  static constexpr int kPOff = kQOff + kRows * kQPitch;
  static constexpr int kRedOff = kPOff + kRows * kPPitch;
  static constexpr int kLimOff = kRedOff + kRows * kWarps * 4;
  static constexpr int kFacOff = kLimOff + kRows * 4;
  static constexpr int kBarOff = (kFacOff + kRows * 4 + 15) / 16 * 16;
  static constexpr int kMaxSlots = 12;
  static constexpr int kRangeOff = kBarOff + 2 * kMaxSlots * 8 + 16;
  static constexpr int kFixed = kRangeOff + static_cast<int>(sizeof(RangeSmem)) + 1024;
  static constexpr int kBudget = kCtas == 2 ? 112 * 1024 : 227 * 1024;
  static constexpr int kSlots = std::min(kMaxSlots, (kBudget - kFixed) / kSlotBytes);
  static constexpr int kSmem = kSlots * kSlotBytes + kFixed;
  static_assert(kSlots >= 4, "K and V of one block have to fit");
};

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x2_t(uint32_t addr, uint32_t& r0, uint32_t& r1) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];"
               : "=r"(r0), "=r"(r1)
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ void consumer_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory");
}

template <bool kE4m3>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  if (kE4m3)
    mma_f16_16816(d, a[0], a[1], a[2], a[3], b0, b1);
  else
    mma_bf16_16816(d, a[0], a[1], a[2], a[3], b0, b1);
}

template <bool kE4m3>
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  return kE4m3 ? f32x2_to_f16x2(lo, hi) : f32x2_to_bf16x2(lo, hi);
}

// One half of an operand register as fp32, and whether it is not finite.
template <bool kE4m3>
__device__ __forceinline__ float half_value(uint32_t w, int hi) {
  const uint32_t v = hi ? w >> 16 : w & 0xFFFFu;
  return kE4m3 ? __half2float(__ushort_as_half(static_cast<unsigned short>(v)))
               : __uint_as_float(v << 16);
}
template <bool kE4m3>
__device__ __forceinline__ uint32_t non_finite_mask(uint32_t w) {
  constexpr uint32_t e = kE4m3 ? 0x7C00u : 0x7F80u;
  return ((w & e) == e ? 0xFFFFu : 0u) | ((w & (e << 16)) == (e << 16) ? 0xFFFF0000u : 0u);
}

template <int kDim, bool kE4m3, int kR>
__global__ void __launch_bounds__(kThreads, Cfg<kDim, kE4m3, kR>::kCtas)
    attend_warp_kernel(const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const Attend p, const Plan plan,
                       const Parts parts) {
  using C = Cfg<kDim, kE4m3, kR>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  uint8_t* fixed = smem + C::kSlots * C::kSlotBytes;
  float* red = reinterpret_cast<float*>(fixed + C::kRedOff);          // [rows][warps]
  int* limit = reinterpret_cast<int*>(fixed + C::kLimOff);            // keys a row sees
  float* factor = reinterpret_cast<float*>(fixed + C::kFacOff);       // of a row's scores
  uint64_t* full = reinterpret_cast<uint64_t*>(fixed + C::kBarOff);
  uint64_t* empty = full + C::kMaxSlots;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(empty + C::kMaxSlots);
  RangeSmem* range_sm = reinterpret_cast<RangeSmem*>(fixed + C::kRangeOff);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kWarps);
    }
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
  }
  griddep_wait();
  griddep_launch_dependents();
  const Range range = find_range(p.seqs, p.cache.heads, plan, blockIdx.x,
                                 gridDim.x, range_sm, p.err);
  Walk w(range, p.seqs, p.cache.heads, plan, p.err);

  if (warp == kWarps) {
    // ------------------------------------------------------------ producer
    int it = 0;                                   // slots filled so far
    bool ok = true;
    for (; w.more() && ok; w.next(p.seqs, p.cache.heads, plan, p.err)) {
      for (int u0 = 0; u0 < w.count && ok; u0 += kWarps) {
        const int n = min(kWarps, w.count - u0);  // units of this block
        const int u = lane & 7;
        const int key = (w.unit0 + u0 + u) * kUnit;
        int page = 0, in_page = 0;
        if (u < n) {
          // the last unit of a sequence may start past its length when it
          // holds no key at all: no page is looked up then
          page = static_cast<int>(p.cache.pages);
          if (key < w.seq.kv_len)
            page = static_cast<int>(checked_page(
                p.seqs.table[int64_t(w.r.s) * p.seqs.width + key / p.cache.page_size],
                p.cache.pages, p.err));
          in_page = key % p.cache.page_size;
        }
        const int slots = (n + 3) / 4;
        for (int i = 0; i < 2 * slots && ok; ++i, ++it) {
          const bool is_v = i >= slots;
          const int half = is_v ? i - slots : i;
          const int units = min(4, n - half * 4);
          const int slot = it % C::kSlots;
          if (it >= C::kSlots)
            ok = __all_sync(0xffffffffu,
                            wait(&empty[slot], ((it / C::kSlots) & 1) ^ 1, abort_flag));
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&full[slot], units * kUnit * C::kRowBytes);
          // one lane issues: a copy's operands are warp-uniform registers, and
          // copies from several lanes took some 250 cycles each
#pragma unroll 1
          for (int lu = 0; lu < units; ++lu) {
            const int pg = __shfl_sync(0xffffffffu, page, half * 4 + lu);
            const int ip = __shfl_sync(0xffffffffu, in_page, half * 4 + lu);
            if (lane == 0)
              tma_load_page(smem + slot * C::kSlotBytes + lu * C::kUnitBytes, is_v ? &tm_v : &tm_k,
                            &full[slot], 0, ip, w.r.h, pg);
          }
        }
      }
    }
    // every copy has landed before the block may end
    for (int i = max(0, it - C::kSlots); i < it; ++i) {
      volatile int no_abort = 0;
      if (!wait(&full[i % C::kSlots], (i / C::kSlots) & 1, &no_abort))
        atomicOr(p.err, NVFP4_ATTENTION_TIMEOUT);
    }
  } else {
    // ----------------------------------------------------------- consumers
    constexpr int kSteps = kDim / 16;             // k steps of Q K^T
    constexpr int kNt = kDim / 64;                // 8-column tiles of this warp's slice of V
    const int g = lane >> 2, t = lane & 3;
    const uint32_t q_addr = smem_addr(fixed + C::kQOff);
    const uint32_t p_addr = smem_addr(fixed + C::kPOff);
    const uint32_t ring = smem_addr(smem);
    const int rows_used = plan.tile_tokens * p.group;
    int flags = 0;
    int4 note = make_int4(0, 0, 0, 0);
    int it = 0;
    for (; w.more(); w.next(p.seqs, p.cache.heads, plan, p.err)) {
      const SeqInfo seq = w.seq;
      const int tok0 = w.r.tile * plan.tile_tokens;
      // ---- the item's queries, limits and factors to shared memory
      const float head_scale =
          p.scale * 1.44269504088896f * (kE4m3 && p.cache.k_scale ? p.cache.k_scale[w.r.h] : 1.f);
#pragma unroll
      for (int i = 0; i < C::kRows / kWarps; ++i) {
        const int r = warp * (C::kRows / kWarps) + i;
        const int tok = r / p.group, gi = r - tok * p.group;
        const bool valid = r < rows_used && tok0 + tok < seq.q_len;
        constexpr int kWords = kDim / 64;         // 32-bit words per lane
        const uint32_t* src = reinterpret_cast<const uint32_t*>(
            p.q.data + int64_t(seq.q0 + tok0 + tok) * p.q.ts +
            int64_t(w.r.h * p.group + gi) * p.q.hs);
        uint32_t x[kWords];
#pragma unroll
        for (int k = 0; k < kWords; ++k) x[k] = valid ? src[k * 32 + lane] : 0u;
        float f = head_scale;
        if (kE4m3) {
          float top = 0.f;
#pragma unroll
          for (int k = 0; k < kWords; ++k)
            top = fmaxf(top, fmaxf(fabsf(bf16_lo(x[k])), fabsf(bf16_hi(x[k]))));
#pragma unroll
          for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
          // 2^s, s = 14 - exponent of the row's largest value, within 2^+-100
          int s = 141 - static_cast<int>(__float_as_uint(top) >> 23);
          s = top == 0.f || top > 3.4e38f ? 0 : min(s, 100);
          const float up = __uint_as_float(static_cast<uint32_t>(127 + s) << 23);
          f *= __uint_as_float(static_cast<uint32_t>(127 - s) << 23);
#pragma unroll
          for (int k = 0; k < kWords; ++k)
            x[k] = f32x2_to_f16x2(bf16_lo(x[k]) * up, bf16_hi(x[k]) * up);
        }
        uint32_t* dst = reinterpret_cast<uint32_t*>(fixed + C::kQOff + r * C::kQPitch);
#pragma unroll
        for (int k = 0; k < kWords; ++k) dst[k * 32 + lane] = x[k];
        if (lane == 0) {
          factor[r] = f;
          limit[r] = valid ? max(0, seq.kv_len - seq.q_len + tok0 + tok + 1) : 0;
        }
      }
      consumer_sync();
      // A fragments of Q: f16 in the permuted order of the codes
      auto q_frag = [&](int rt, int ks, uint32_t (&a)[4]) {
        if (kE4m3) {
          // step ks covers, for lane t, the four codes at this offset
          const int d0 = C::kChunkBytes == 128
                             ? (ks >> 3) * 128 + 16 * (2 * t + (ks >> 2 & 1)) + 4 * (ks & 3)
                             : 16 * t + 4 * ks;
          const uint2 lo = lds64(q_addr + (rt * 16 + g) * C::kQPitch + d0 * 2);
          const uint2 hi = lds64(q_addr + (rt * 16 + g + 8) * C::kQPitch + d0 * 2);
          a[0] = lo.x, a[1] = hi.x, a[2] = lo.y, a[3] = hi.y;
        } else {
          ldsm_x4(q_addr + (rt * 16 + (lane & 15)) * C::kQPitch + ks * 32 + (lane >> 4) * 16, a);
        }
      };
      uint32_t qf[kR == 1 ? kSteps : 1][4];
      if (kR == 1) {
#pragma unroll
        for (int ks = 0; ks < kSteps; ++ks) q_frag(0, ks, qf[kR == 1 ? ks : 0]);
      }
      int lim[kR][2];
      float fac[kR][2], m[kR][2], l[kR][2], o[kR][kNt][4];
      int least = INT32_MAX;                      // keys that every used row sees
#pragma unroll
      for (int rt = 0; rt < kR; ++rt) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          lim[rt][i] = limit[rt * 16 + g + 8 * i];
          fac[rt][i] = factor[rt * 16 + g + 8 * i];
          m[rt][i] = -INFINITY;
          l[rt][i] = 0.f;
        }
#pragma unroll
        for (int n = 0; n < kNt; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[rt][n][i] = 0.f;
      }
      least = max(0, seq.kv_len - seq.q_len + tok0 + 1);
      const int seen = tile_keys(seq, w.r.tile, plan);

      for (int u0 = 0; u0 < w.count; u0 += kWarps) {
        const int n = min(kWarps, w.count - u0);
        const int slots = (n + 3) / 4;
        const int key0 = (w.unit0 + u0) * kUnit;
        // ---- scores of this warp's 16 keys
        float s[kR][2][4];
#pragma unroll
        for (int rt = 0; rt < kR; ++rt)
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[rt][j][i] = 0.f;
        if (warp < n) {
          const int si = it + (warp >> 2);
          wait(&full[si % C::kSlots], (si / C::kSlots) & 1, abort_flag);
          __syncwarp();
          const uint32_t base = ring + (si % C::kSlots) * C::kSlotBytes +
                                (warp & 3) * C::kUnitBytes;
          if (kE4m3) {
#pragma unroll
            for (int cc = 0; cc < kDim / 64; ++cc) {
              uint4 kc[2];
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const int row = j * 8 + g;
                if (C::kChunkBytes == 128)
                  kc[j] = lds128(base + (cc >> 1) * C::kUnitChunk + row * 128 +
                                 (((2 * t + (cc & 1)) ^ g) << 4));
                else
                  kc[j] = lds128(base + row * 64 + ((t ^ (row >> 1 & 3)) << 4));
              }
#pragma unroll
              for (int st = 0; st < 4; ++st) {
                uint32_t b[2][2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  const uint32_t c4 = st == 0 ? kc[j].x : st == 1 ? kc[j].y : st == 2 ? kc[j].z : kc[j].w;
                  b[j][0] = e4m3x2_to_f16x2(c4 & 0xFFFFu);
                  b[j][1] = e4m3x2_to_f16x2(c4 >> 16);
                }
#pragma unroll
                for (int rt = 0; rt < kR; ++rt) {
                  uint32_t a[4];
                  if (kR == 1) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) a[i] = qf[kR == 1 ? cc * 4 + st : 0][i];
                  } else {
                    q_frag(rt, cc * 4 + st, a);
                  }
                  mma<kE4m3>(s[rt][0], a, b[0][0], b[0][1]);
                  mma<kE4m3>(s[rt][1], a, b[1][0], b[1][1]);
                }
              }
            }
          } else {
            const int mi = lane >> 3, r8 = lane & 7;
            const uint32_t row = base + ((mi >> 1) * 8 + r8) * 128;
#pragma unroll
            for (int ks = 0; ks < kSteps; ++ks) {
              uint32_t b[4];
              const int c16 = ks * 2 + (mi & 1);
              ldsm_x4(row + (c16 >> 3) * C::kUnitChunk + (((c16 & 7) ^ r8) << 4), b);
#pragma unroll
              for (int rt = 0; rt < kR; ++rt) {
                uint32_t a[4];
                if (kR == 1) {
#pragma unroll
                  for (int i = 0; i < 4; ++i) a[i] = qf[kR == 1 ? ks : 0][i];
                } else {
                  q_frag(rt, ks, a);
                }
                mma<kE4m3>(s[rt][0], a, b[0], b[1]);
                mma<kE4m3>(s[rt][1], a, b[2], b[3]);
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0)
#pragma unroll 1
          for (int i = 0; i < slots; ++i) mbar_arrive(&empty[(it + i) % C::kSlots]);
        // ---- scale, mask, and the rows' maxima over this warp's keys
        const int kb = key0 + warp * kUnit + 2 * t;      // keys kb, kb + 1, kb + 8, kb + 9
#pragma unroll
        for (int rt = 0; rt < kR; ++rt) {
          float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int key = kb + j * 8 + (i & 1);
              const bool sees = warp < n && key < lim[rt][i >> 1];
              s[rt][j][i] = sees ? s[rt][j][i] * fac[rt][i >> 1] : -INFINITY;
              top[i >> 1] = fmaxf(top[i >> 1], s[rt][j][i]);
            }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
            top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
            if (t == 0) red[(rt * 16 + g + 8 * i) * kWarps + warp] = top[i];
          }
        }
        consumer_sync();
        // ---- the new maximum, the weights, and the accumulators' rescaling
#pragma unroll
        for (int rt = 0; rt < kR; ++rt) {
          float base[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float4* rr =
                reinterpret_cast<const float4*>(red + (rt * 16 + g + 8 * i) * kWarps);
            const float4 a = rr[0], b = rr[1];
            const float now = fmaxf(fmaxf(fmaxf(a.x, a.y), fmaxf(a.z, a.w)),
                                    fmaxf(fmaxf(b.x, b.y), fmaxf(b.z, b.w)));
            const float top = fmaxf(m[rt][i], now);
            base[i] = top == -INFINITY ? 0.f : top;
            const float alpha = exp2f(m[rt][i] - base[i]);      // 0 from -inf
            base[i] -= kLift<kE4m3>;
            m[rt][i] = top;
            l[rt][i] *= alpha;
#pragma unroll
            for (int nt = 0; nt < kNt; ++nt) {
              o[rt][nt][2 * i] *= alpha;
              o[rt][nt][2 * i + 1] *= alpha;
            }
          }
          if (warp < n) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const float e0 = exp2f(s[rt][j][2 * i] - base[i]);
                const float e1 = exp2f(s[rt][j][2 * i + 1] - base[i]);
                l[rt][i] += e0 + e1;
                asm volatile("st.shared.u32 [%0], %1;" ::"r"(
                                 p_addr + (rt * 16 + g + 8 * i) * kPPitch +
                                 (warp * kUnit + j * 8 + 2 * t) * 2),
                             "r"(pack<kE4m3>(e0, e1))
                             : "memory");
              }
          }
        }
        consumer_sync();
        // ---- P V for this warp's columns
#pragma unroll 1
        for (int half = 0; half < slots; ++half) {
          const int si = it + slots + half;
          wait(&full[si % C::kSlots], (si / C::kSlots) & 1, abort_flag);
          __syncwarp();
          const uint32_t base = ring + (si % C::kSlots) * C::kSlotBytes;
#pragma unroll 1
          for (int lu = 0; lu < 4; ++lu) {              // (not unrolled: code size)
            const int u = half * 4 + lu;
            if (u >= n) break;
            uint32_t b[kNt][2];
            const uint32_t unit = base + lu * C::kUnitBytes;
            if (kE4m3) {
              // columns 8 kNt warp + kNt g + i of keys 2t, 2t+1, 2t+8, 2t+9
              uint32_t c4[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int row = 2 * t + (i & 1) + 8 * (i >> 1);
                const int byte = warp * (8 * kNt) + kNt * g;
                uint32_t a;
                if (C::kChunkBytes == 128)
                  a = unit + (byte >> 7) * C::kUnitChunk + row * 128 +
                      ((((byte >> 4) & 7) ^ (row & 7)) << 4) + (byte & 15);
                else
                  a = unit + row * 64 + (((byte >> 4) ^ (row >> 1 & 3)) << 4) + (byte & 15);
                c4[i] = kNt == 4 ? lds32(a) : kNt == 2 ? lds16(a) : lds8(a);
              }
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t x = prmt(c4[2 * h], c4[2 * h + 1], 0x5140);
                const uint32_t y = prmt(c4[2 * h], c4[2 * h + 1], 0x7362);
                b[0][h] = e4m3x2_to_f16x2(x & 0xFFFFu);
                if (kNt > 1) b[1 % kNt][h] = e4m3x2_to_f16x2(x >> 16);
                if (kNt > 2) {
                  b[2 % kNt][h] = e4m3x2_to_f16x2(y & 0xFFFFu);
                  b[3 % kNt][h] = e4m3x2_to_f16x2(y >> 16);
                }
              }
            } else {
              const int mi = lane >> 3, r8 = lane & 7;
              const uint32_t row = unit + ((mi & 1) * 8 + r8) * 128;
              if (kNt == 1) {
                ldsm_x2_t(row + ((warp ^ r8) << 4), b[0][0], b[0][1]);
              } else {
#pragma unroll
                for (int i = 0; i < kNt / 2; ++i) {
                  const int c16 = warp * kNt + 2 * i + (mi >> 1);
                  uint32_t r4[4];
                  ldsm_x4_t(row + (c16 >> 3) * C::kUnitChunk + (((c16 & 7) ^ r8) << 4), r4);
                  b[2 * i][0] = r4[0], b[2 * i][1] = r4[1];
                  b[(2 * i + 1) % kNt][0] = r4[2], b[(2 * i + 1) % kNt][1] = r4[3];
                }
              }
            }
            const int k0 = key0 + u * kUnit;
            if (k0 + kUnit > seen) {
              // keys that no row sees: whatever the page holds there
              const int k = k0 + 2 * t;
              const uint32_t m0 = (k < seen ? 0xFFFFu : 0u) | (k + 1 < seen ? 0xFFFF0000u : 0u);
              const uint32_t m1 = (k + 8 < seen ? 0xFFFFu : 0u) | (k + 9 < seen ? 0xFFFF0000u : 0u);
#pragma unroll
              for (int nt = 0; nt < kNt; ++nt) b[nt][0] &= m0, b[nt][1] &= m1;
            }
            if (k0 + kUnit > least) {
              // keys that some rows see and others do not: 0 times a value
              // that is not finite must not reach the others
              uint32_t bad = 0;
#pragma unroll
              for (int nt = 0; nt < kNt; ++nt)
                bad |= non_finite_mask<kE4m3>(b[nt][0]) | non_finite_mask<kE4m3>(b[nt][1]);
              if (__any_sync(0xffffffffu, bad != 0)) {
#pragma unroll 1
                for (int k = 0; k < kUnit; ++k) {
#pragma unroll
                  for (int nt = 0; nt < kNt; ++nt) {
                    const uint32_t mine = k < 8 ? b[nt][0] : b[nt][1];
                    const int from = (k & 7) >> 1;
                    const uint32_t w0 = __shfl_sync(0xffffffffu, mine, 8 * t + from);
                    const uint32_t w1 = __shfl_sync(0xffffffffu, mine, 8 * t + 4 + from);
                    const uint32_t half = k & 1 ? 0xFFFF0000u : 0xFFFFu;
                    const bool bad0 = non_finite_mask<kE4m3>(w0) & half;
                    const bool bad1 = non_finite_mask<kE4m3>(w1) & half;
#pragma unroll
                    for (int rt = 0; rt < kR; ++rt)
#pragma unroll
                      for (int i = 0; i < 2; ++i) {
                        if (k0 + k >= lim[rt][i]) continue;
                        const float pw = half_value<kE4m3>(
                            lds16(p_addr + (rt * 16 + g + 8 * i) * kPPitch + (u * kUnit + k) * 2), 0);
                        if (bad0) o[rt][nt][2 * i] += pw * half_value<kE4m3>(w0, k & 1);
                        if (bad1) o[rt][nt][2 * i + 1] += pw * half_value<kE4m3>(w1, k & 1);
                      }
                  }
                }
#pragma unroll
                for (int nt = 0; nt < kNt; ++nt) {
                  b[nt][0] &= ~non_finite_mask<kE4m3>(b[nt][0]);
                  b[nt][1] &= ~non_finite_mask<kE4m3>(b[nt][1]);
                }
              }
            }
#pragma unroll
            for (int rt = 0; rt < kR; ++rt) {
              uint32_t a[4];
              ldsm_x4(p_addr + (rt * 16 + (lane & 15)) * kPPitch + u * 32 + (lane >> 4) * 16, a);
#pragma unroll
              for (int nt = 0; nt < kNt; ++nt) mma<kE4m3>(o[rt][nt], a, b[nt][0], b[nt][1]);
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&empty[si % C::kSlots]);
        }
        it += 2 * slots;
      }

      // ---- the rows' sums, and the result
#pragma unroll
      for (int rt = 0; rt < kR; ++rt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          l[rt][i] += __shfl_xor_sync(0xffffffffu, l[rt][i], 1);
          l[rt][i] += __shfl_xor_sync(0xffffffffu, l[rt][i], 2);
          if (t == 0) red[(rt * 16 + g + 8 * i) * kWarps + warp] = l[rt][i];
        }
      consumer_sync();
      const bool whole = w.begins() && w.ends();
      const int part = w.begins() ? 1 : 0;
      if (!whole) {
        flags |= part ? kPart1 : kPart0 | (w.ends() ? kPart0Ends : 0);
        if (part) note = make_int4(0, w.r.s, w.r.h, w.r.tile);
      }
      const float vs = kE4m3 && p.cache.v_scale ? p.cache.v_scale[w.r.h] : 1.f;
#pragma unroll
      for (int rt = 0; rt < kR; ++rt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = rt * 16 + g + 8 * i;
          const float4* rr = reinterpret_cast<const float4*>(red + r * kWarps);
          const float4 a = rr[0], b = rr[1];
          const float sum = ((a.x + a.y) + (a.z + a.w)) + ((b.x + b.y) + (b.z + b.w));
          const float inv = sum == 0.f ? 0.f : vs / sum;
          const int tok = r / p.group, gi = r - tok * p.group;
          if (r >= rows_used || tok0 + tok >= seq.q_len) continue;
          const int64_t token = seq.q0 + tok0 + tok;
          const int head = w.r.h * p.group + gi;
          const float lse2 = sum == 0.f ? -INFINITY : m[rt][i] + (log2f(sum) - kLift<kE4m3>);
          if (warp == 0 && t == 0) {
            if (whole && p.lse) p.lse[token * p.q_heads + head] = lse2 * 0.693147180559945f;
            if (!whole) parts.lse2[parts.row(blockIdx.x, part, r)] = lse2;
          }
          __nv_bfloat16* dst = p.out.data + token * p.out.ts + int64_t(head) * p.out.hs;
          float* dst_part = parts.out + parts.row(blockIdx.x, part, r) * kDim;
          if (kE4m3) {
            // columns kNt (2t) .. kNt (2t + 2) - 1 of the warp's slice
            float y[2 * kNt];
#pragma unroll
            for (int nt = 0; nt < kNt; ++nt) {
              y[nt] = o[rt][nt][2 * i] * inv;
              y[kNt + nt] = o[rt][nt][2 * i + 1] * inv;
            }
            const int col = warp * 8 * kNt + kNt * 2 * t;
#pragma unroll
            for (int c = 0; c < 2 * kNt; c += 2) {
              if (whole)
                *reinterpret_cast<uint32_t*>(dst + col + c) = f32x2_to_bf16x2(y[c], y[c + 1]);
              else
                *reinterpret_cast<float2*>(dst_part + col + c) = make_float2(y[c], y[c + 1]);
            }
          } else {
#pragma unroll
            for (int nt = 0; nt < kNt; ++nt) {
              const int col = warp * 8 * kNt + nt * 8 + 2 * t;
              const float y0 = o[rt][nt][2 * i] * inv, y1 = o[rt][nt][2 * i + 1] * inv;
              if (whole)
                *reinterpret_cast<uint32_t*>(dst + col) = f32x2_to_bf16x2(y0, y1);
              else
                *reinterpret_cast<float2*>(dst_part + col) = make_float2(y0, y1);
            }
          }
        }
      consumer_sync();                            // red, Q and the limits are free again
    }
    if (threadIdx.x == 0) {
      note.x = flags;
      parts.note[blockIdx.x] = note;
    }
  }
  __syncthreads();
  if (*abort_flag && threadIdx.x == 0) atomicOr(p.err, NVFP4_ATTENTION_TIMEOUT);
}

template <int kDim, bool kE4m3, int kR>
int run(const Attend& p, const Device& d, cudaStream_t stream) {
  using C = Cfg<kDim, kE4m3, kR>;
  auto* kernel = attend_warp_kernel<kDim, kE4m3, kR>;
  static std::atomic<bool> ready[kMaxDevices];
  if (const int st = allow_smem(kernel, C::kSmem, d, ready)) return st;
  CUtensorMap tm_k, tm_v;
  constexpr int inner = C::kChunkBytes / C::kEsz;
  if (!page_map(&tm_k, p.cache, false, inner, kUnit, C::kChunks) ||
      !page_map(&tm_v, p.cache, true, inner, kUnit, C::kChunks))
    return NVFP4_ERR_LAUNCH;
  const Plan plan{std::max(1, C::kRows / p.group), kUnitShift, 4, kExtra};
  if (!countable(p.seqs, p.cache.heads, plan)) return NVFP4_ERR_SHAPE;
  const int ctas = d.num_sms * C::kCtas;
  const Parts parts(p.workspace, ctas, C::kRows, 1, kDim);
  if (const int st = launch(kernel, dim3(ctas), dim3(kThreads), C::kSmem, stream, tm_k, tm_v, p,
                            plan, parts))
    return st;
  return run_join(false, p, parts, plan, ctas, d.id, stream);
}

template <int kDim, bool kE4m3>
int run_rows(int rows, const Attend& p, const Device& d, cudaStream_t stream) {
  return rows <= 16 ? run<kDim, kE4m3, 1>(p, d, stream) : run<kDim, kE4m3, 2>(p, d, stream);
}

}  // namespace

int64_t attend_warp_workspace(int head_dim, const Device& d) {
  return std::max(Parts::bytes(2 * d.num_sms, 16, head_dim), Parts::bytes(d.num_sms, 32, head_dim));
}

int run_attend_warp(int rows, const Attend& p, const Device& d, cudaStream_t stream) {
  const bool f8 = p.cache.e4m3;
  switch (p.cache.dim) {
    case 64:
      return f8 ? run_rows<64, true>(rows, p, d, stream) : run_rows<64, false>(rows, p, d, stream);
    case 128:
      return f8 ? run_rows<128, true>(rows, p, d, stream) : run_rows<128, false>(rows, p, d, stream);
    default:
      return f8 ? run_rows<256, true>(rows, p, d, stream) : run_rows<256, false>(rows, p, d, stream);
  }
}

}  // namespace attn
}  // namespace nvfp4
