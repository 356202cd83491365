// schedule.cuh -- how the attention kernels share out their work.
//
// An item is one tile of query rows (a few tokens of one sequence, times the
// query heads of one key/value head); its work is the units of `unit` keys
// that its last token sees, one at least.  Items are ordered by sequence,
// head and tile, and the units of all items, end to end, are cut into equal
// ranges, one per CTA: long sequences are split over many CTAs, short ones
// share one, and causal tiles of different length balance.  An item counts
// `extra` units more than it has, ahead of its first, for what it costs to
// begin and to end one.  A range that begins or ends inside an item leaves a
// partial result for the join kernel.  The lengths live on the device, so each
// CTA finds its own range.
#pragma once
#include "common.cuh"

namespace nvfp4 {
namespace attn {

constexpr int kMaxBatches = 256;            // of 32 sequences

struct Plan {
  int tile_tokens;                          // tokens of one tile
  int unit_shift;                           // log2 of the keys of one unit
  int min_units;                            // least units worth a CTA of its own
  int extra;                                // units that beginning an item costs
};

__device__ __forceinline__ int tiles_of(const SeqInfo& s, const Plan& p) {
  return (s.q_len + p.tile_tokens - 1) / p.tile_tokens;
}

// Whether the units of any batch of these sizes can be counted in 32 bits.
bool countable(const Seqs& s, int heads, const Plan& p);

// Keys that the last token of a tile sees.
__device__ __forceinline__ int tile_keys(const SeqInfo& s, int tile, const Plan& p) {
  const int last = min(s.q_len, (tile + 1) * p.tile_tokens);
  return max(0, s.kv_len - s.q_len + last);
}

// Units of an item (it counts p.extra more).
__device__ __forceinline__ int tile_units(const SeqInfo& s, int tile, const Plan& p) {
  return max(1, (tile_keys(s, tile, p) + (1 << p.unit_shift) - 1) >> p.unit_shift);
}

// Sum of the lanes before and with this one.
__device__ __forceinline__ uint32_t warp_inclusive(uint32_t v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// Where a CTA's range begins, and how many units it holds.
struct Range {
  uint32_t left;           // counted units
  int s, h, tile, at;      // `at`: counted units of the item before the range
};

struct RangeSmem {
  uint32_t batch[kMaxBatches];              // units of 32 sequences
  Range range;
};

// The range of CTA `cta` of `ctas`, found by all threads of the block: each
// warp sums up batches of 32 sequences, and the warp whose batch holds the
// range's first unit finds its place in it.  Everything is in two passes over
// the same code, since what runs once per launch costs as much in instruction
// fetches as in instructions.  Where q_starts descends anywhere, sequences may
// overlap and have more tokens in all than the units' count allows for
// (countable), so that no CTA gets a range.
__device__ inline Range find_range(const Seqs& q, int heads, const Plan& p, uint32_t cta,
                                   uint32_t ctas, RangeSmem* sm, unsigned int* err) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int warps = blockDim.x >> 5;
  int batches = (q.count + 31) / 32;
  uint32_t begin = 0;
  bool descends = false;
  SeqInfo mine{0, 0, 0};
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    uint32_t before = 0;                    // units of the batches before b
#pragma unroll 1
    for (int b = 0; b < batches; ++b) {
      if (pass == 1) {
        const uint32_t here = sm->batch[b];
        if (begin - before >= here) {       // (also where `begin` lies in an earlier one)
          before += here;
          continue;
        }
      }
      if (pass == 0 ? b % warps != warp : warp != 0) {
        if (pass == 1) break;
        continue;
      }
      const int s = b * 32 + lane;
      if (pass == 0 || batches > 1)
        mine = s < q.count ? load_seq(q, s, err) : SeqInfo{0, 0, 0};
      descends |= s < q.count && q.q_starts[s + 1] < q.q_starts[s];
      // units of one head of each lane's sequence
      const int tiles = tiles_of(mine, p);
      uint32_t one = tiles == 1 ? tile_units(mine, 0, p) + p.extra : 0;
      unsigned many = __ballot_sync(0xffffffffu, tiles > 1);
#pragma unroll 1
      while (many) {
        const int src = __ffs(many) - 1;
        many &= many - 1;
        const SeqInfo o{0, __shfl_sync(0xffffffffu, mine.q_len, src),
                        __shfl_sync(0xffffffffu, mine.kv_len, src)};
        const int n = __shfl_sync(0xffffffffu, tiles, src);
        uint32_t sum = 0;
#pragma unroll 1
        for (int i = lane; i < n; i += 32) sum += tile_units(o, i, p) + p.extra;
        sum = __reduce_add_sync(0xffffffffu, sum);
        if (lane == src) one = sum;
      }
      const uint32_t upto = warp_inclusive(one) * heads;
      if (pass == 0) {
        if (lane == 31) sm->batch[b] = upto;
        continue;
      }
      // the sequence, the head and the tile that hold the first unit
      uint32_t at = begin - before;
      const int src = __ffs(__ballot_sync(0xffffffffu, upto > at)) - 1;
      at -= __shfl_sync(0xffffffffu, upto - one * heads, src);
      const uint32_t per_head = __shfl_sync(0xffffffffu, one, src);
      const SeqInfo o{0, __shfl_sync(0xffffffffu, mine.q_len, src),
                      __shfl_sync(0xffffffffu, mine.kv_len, src)};
      const int n = __shfl_sync(0xffffffffu, tiles, src);
      const uint32_t h = at / per_head;
      at -= h * per_head;
      int t0 = 0;
      uint32_t u, sum;
      unsigned past;
#pragma unroll 1
      for (;; t0 += 32) {
        u = t0 + lane < n ? tile_units(o, t0 + lane, p) + p.extra : 0;
        sum = warp_inclusive(u);
        past = __ballot_sync(0xffffffffu, sum > at);
        if (past || t0 >= n) break;
        at -= __shfl_sync(0xffffffffu, sum, 31);
      }
      const int i = past ? __ffs(past) - 1 : 0;
      if (lane == i) {
        sm->range.s = b * 32 + src;
        sm->range.h = static_cast<int>(h);
        sm->range.tile = t0 + i;
        sm->range.at = static_cast<int>(at - (sum - u));
      }
      break;
    }
    if (__syncthreads_or(descends)) batches = 0;       // (load_seq has set the error bit)
    if (pass == 0) {
      uint32_t total = 0;
#pragma unroll 1
      for (int b = 0; b < batches; ++b) total += sm->batch[b];
      // the units in equal shares, over no more CTAs than min_units leaves work for
      const uint32_t used = min(ctas, max(1u, total / p.min_units));
      const uint32_t share = total / used, extra = total - share * used;
      begin = share * cta + min(cta, extra);
      if (threadIdx.x == 0) sm->range.left = cta < used ? share + (cta < extra) : 0;
      if (cta >= used) begin = total;                  // in no batch
    }
  }
  return sm->range;
}

// Walks a range item by item.
struct Walk {
  Range r;
  SeqInfo seq;
  int units;          // of the item
  int unit0, count;   // the range's part of them

  __device__ Walk(const Range& range, const Seqs& q, int heads, const Plan& p, unsigned int* err)
      : r(range) {
    if (r.left > 0) {
      seq = load_seq(q, r.s, err);
      settle(q, heads, p, err);
    }
  }
  __device__ bool more() const { return r.left > 0; }
  __device__ bool begins() const { return unit0 == 0; }
  __device__ bool ends() const { return unit0 + count == units; }
  __device__ void next(const Seqs& q, int heads, const Plan& p, unsigned int* err) {
    step(q, heads, p, err);
    settle(q, heads, p, err);
  }

 private:
  // On to the first item of which the range holds more than the `extra`.
  __device__ void settle(const Seqs& q, int heads, const Plan& p, unsigned int* err) {
    while (r.left > 0) {
      units = tile_units(seq, r.tile, p);
      const int end = static_cast<int>(min(static_cast<uint32_t>(units + p.extra - r.at), r.left)) + r.at;
      unit0 = max(0, r.at - p.extra);
      count = max(0, end - p.extra) - unit0;
      if (count > 0) return;
      step(q, heads, p, err);
    }
  }
  __device__ void step(const Seqs& q, int heads, const Plan& p, unsigned int* err) {
    const uint32_t here = units + p.extra - r.at;
    r.at = 0;
    if (here >= r.left) {
      r.left = 0;
      return;
    }
    r.left -= here;
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

// `many`: items of several tiles, whose rows lie in few parts each.
int run_join(bool many, const Attend& p, const Parts& parts, const Plan& plan, int ctas,
             int device, cudaStream_t stream);

}  // namespace attn
}  // namespace nvfp4
