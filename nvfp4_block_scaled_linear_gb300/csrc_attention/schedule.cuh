// schedule.cuh -- how the attention kernels share out their work.
//
// An item is one tile of query rows (a few tokens of one sequence, times the
// query heads of one key/value head); its work is the units of `unit` keys
// that its last token sees, one at least.  Items are ordered by sequence,
// head and tile, and the units of all items, end to end, are cut into equal
// ranges, one per CTA: long sequences are split over many CTAs, short ones
// share one, and causal tiles of different length balance.  A range that
// begins or ends inside an item leaves a partial result for the join kernel.
// The lengths live on the device, so each CTA finds its own range.
#pragma once
#include "common.cuh"

namespace nvfp4 {
namespace attn {

constexpr int kMaxBatches = 256;            // of 32 sequences

struct Plan {
  int tile_tokens;                          // tokens of one tile
  int unit_shift;                           // log2 of the keys of one unit
  int min_units;                            // least units worth a CTA of its own
};

__device__ __forceinline__ int tiles_of(const SeqInfo& s, const Plan& p) {
  return (s.q_len + p.tile_tokens - 1) / p.tile_tokens;
}

// Keys that the last token of a tile sees.
__device__ __forceinline__ int tile_keys(const SeqInfo& s, int tile, const Plan& p) {
  const int last = min(s.q_len, (tile + 1) * p.tile_tokens);
  return max(0, s.kv_len - s.q_len + last);
}

__device__ __forceinline__ int tile_units(const SeqInfo& s, int tile, const Plan& p) {
  return max(1, (tile_keys(s, tile, p) + (1 << p.unit_shift) - 1) >> p.unit_shift);
}

// Units of one head of each lane's sequence, all lanes of the warp together.
__device__ __forceinline__ int64_t seq_units(const SeqInfo& s, const Plan& p) {
  const int lane = threadIdx.x & 31, n = tiles_of(s, p);
  int64_t u = n == 1 ? tile_units(s, 0, p) : 0;
  unsigned many = __ballot_sync(0xffffffffu, n > 1);
  while (many) {
    const int src = __ffs(many) - 1;
    many &= many - 1;
    const SeqInfo o{__shfl_sync(0xffffffffu, s.q0, src), __shfl_sync(0xffffffffu, s.q_len, src),
                    __shfl_sync(0xffffffffu, s.kv_len, src)};
    int64_t sum = 0;
    const int tiles = tiles_of(o, p);
#pragma unroll 1
    for (int i = lane; i < tiles; i += 32) sum += tile_units(o, i, p);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == src) u = sum;
  }
  return u;
}

__device__ __forceinline__ int64_t warp_inclusive(int64_t v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// Where a CTA's range begins, and how many units it holds.
struct Range {
  int64_t left;
  int s, h, tile, unit0;
};

struct RangeSmem {
  int64_t batch[kMaxBatches];
  Range range;
};

// The range of CTA `cta` of `ctas`, found by all threads of the block.
__device__ inline Range find_range(const Seqs& q, int heads, const Plan& p, uint32_t cta, uint32_t ctas,
                                   RangeSmem* sm, unsigned int* err) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int warps = blockDim.x >> 5, batches = (q.count + 31) / 32;
  auto lane_seq = [&](int b) {
    const int s = b * 32 + lane;
    return s < q.count ? load_seq(q, s, err) : SeqInfo{0, 0, 0};
  };
#pragma unroll 1
  for (int b = warp; b < batches; b += warps) {
    const int64_t sum = warp_inclusive(seq_units(lane_seq(b), p));
    if (lane == 31) sm->batch[b] = sum * heads;
  }
  __syncthreads();
  if (warp == 0) {
    int64_t total = 0;
#pragma unroll 1
    for (int b = lane; b < batches; b += 32) total += sm->batch[b];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
    // the units in equal shares, over no more CTAs than min_units leaves work for
    const uint32_t used = total >= int64_t(ctas) * p.min_units
                              ? ctas
                              : max(1u, static_cast<uint32_t>(total) / p.min_units);
    const int64_t share = total >> 32 ? total / used : static_cast<uint32_t>(total) / used;
    const int64_t extra = total - share * used;         // of them take one more
    const int64_t begin = share * cta + min(int64_t(cta), extra);
    const int64_t end = begin + (cta < used ? share + (cta < extra) : 0);
    Range r{end - begin, 0, 0, 0, 0};
    if (r.left > 0) {
      int64_t at = begin;
      int b = 0;
#pragma unroll 1
      while (at >= sm->batch[b]) at -= sm->batch[b++];
      const SeqInfo mine = lane_seq(b);
      const int64_t one = seq_units(mine, p);
      const int64_t upto = warp_inclusive(one) * heads;
      const int src = __ffs(__ballot_sync(0xffffffffu, upto > at)) - 1;
      at -= __shfl_sync(0xffffffffu, upto - one * heads, src);
      const int64_t per_head = __shfl_sync(0xffffffffu, one, src);
      const SeqInfo o{__shfl_sync(0xffffffffu, mine.q0, src),
                      __shfl_sync(0xffffffffu, mine.q_len, src),
                      __shfl_sync(0xffffffffu, mine.kv_len, src)};
      r.s = b * 32 + src;
#pragma unroll 1
      for (; at >= per_head; at -= per_head) ++r.h;
      const int tiles = tiles_of(o, p);
#pragma unroll 1
      for (int t0 = 0;; t0 += 32) {
        const int u = t0 + lane < tiles ? tile_units(o, t0 + lane, p) : 0;
        const int64_t sum = warp_inclusive(u);
        const unsigned past = __ballot_sync(0xffffffffu, sum > at);
        if (past) {
          const int i = __ffs(past) - 1;
          r.tile = t0 + i;
          r.unit0 = static_cast<int>(at - __shfl_sync(0xffffffffu, sum - u, i));
          break;
        }
        at -= __shfl_sync(0xffffffffu, sum, 31);
      }
    }
    if (lane == 0) sm->range = r;
  }
  __syncthreads();
  return sm->range;
}

// Walks a range item by item.
struct Walk {
  Range r;
  SeqInfo seq;
  int units;          // of the item
  int count;          // of them in this range, from r.unit0

  __device__ Walk(const Range& range, const Seqs& q, const Plan& p, unsigned int* err) : r(range) {
    if (r.left > 0) {
      seq = load_seq(q, r.s, err);
      item(p);
    }
  }
  __device__ bool more() const { return r.left > 0; }
  __device__ bool begins() const { return r.unit0 == 0; }
  __device__ bool ends() const { return r.unit0 + count == units; }
  __device__ void item(const Plan& p) {
    units = tile_units(seq, r.tile, p);
    count = static_cast<int>(min(int64_t(units - r.unit0), r.left));
  }
  __device__ void next(const Seqs& q, int heads, const Plan& p, unsigned int* err) {
    r.left -= count;
    r.unit0 = 0;
    if (r.left <= 0) return;
    if (++r.tile == tiles_of(seq, p)) {
      r.tile = 0;
      if (++r.h == heads) {
        r.h = 0;
        do {
          if (++r.s >= q.count) {          // lengths that changed under the call
            r.left = 0;
            return;
          }
          seq = load_seq(q, r.s, err);
        } while (seq.q_len == 0);
      }
    }
    item(p);
  }
};

// What a CTA's range leaves for the join kernel.  Part 0 holds the item that
// began in an earlier CTA, part 1 the item that begins in this one and goes
// on in the next.
enum : int { kPart0 = 1, kPart0Ends = 2, kPart1 = 4 };

// The workspace: one note per CTA, then the parts' rows: log2 of the sum and
// the normalised output, fp32 (32-byte aligned where the workspace is).
struct Parts {
  int4* note;             // {flags, s, h, tile} of part 1's item
  float* lse2;            // [ctas][2][rows]
  float* out;             // [ctas][2][rows][dim]
  int tile_rows, rows;    // of one MMA tile (whole tokens from its first row on), of all
  int dim;

  Parts(void* base, int ctas, int tile_rows_, int tiles, int dim_)
      : note(static_cast<int4*>(base)),
        lse2(reinterpret_cast<float*>(note + (ctas + 1) / 2 * 2)),
        out(lse2 + (int64_t(ctas) * 2 * tile_rows_ * tiles + 7) / 8 * 8),
        tile_rows(tile_rows_),
        rows(tile_rows_ * tiles),
        dim(dim_) {}
  __device__ int64_t row(int cta, int part, int r) const {
    return (int64_t(cta) * 2 + part) * rows + r;
  }
  static int64_t bytes(int ctas, int rows, int dim) {
    return int64_t(ctas) * (16 + 2 * int64_t(rows) * (dim + 1) * 4) + 64;
  }
};

int run_join(const Attend& p, const Parts& parts, const Plan& plan, int ctas, cudaStream_t stream);

}  // namespace attn
}  // namespace nvfp4
