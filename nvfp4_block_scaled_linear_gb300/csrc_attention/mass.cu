// mass.cu -- the attention weight that each cached key receives from the new
// tokens:  out[j] = mass[j] + sum over rows r that see j of 2^(c_r q_r . k_j - L_r)
// with c_r the scores' scale times log2 e and L_r = lse_r log2 e.
//
// The keys stay and the queries pass by: a warp keeps 16 keys' rows in
// registers as the warp MMA's A operand, loaded once and straight from the
// pages (a lane's 16-byte pieces are its operands when the k index inside an MMA
// is permuted alike for the queries), and the query rows come through shared
// memory, 32 at a time for the block's 8 warps.  Every row of scores is then a
// column of the accumulator, so a key's sum stays with one lane group from the
// first row to the last: no atomics, one order.
//
// For few rows (run_mass has the bounds; mass_tc.cu takes more): a single token's call reads
// the keys once and is bound by that.  A row's weight is added in fp32 as it is.
// Measured at 24 query and 4 key/value heads of 256: 8 sequences of one token (42
// MB of keys) 17.0 us, 2.6 TB/s; a block lives for one copy of its keys, so the
// latency of length, page and row shows.
//
// Over an e4m3 cache the codes are widened to f16 (exact) as they are loaded,
// and each query row is scaled by a power of two (attend_warp.cu says why).
#include <cuda_fp16.h>

#include <algorithm>

#include "common.cuh"

namespace nvfp4 {
namespace attn {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kStageRows = 32;                // query rows in shared memory at a time

template <int kDim, bool kE4m3>
__global__ void __launch_bounds__(kThreads) mass_kernel(const Mass p) {
  constexpr int kPitch = kDim * 2 + 16;                    // bytes of a query row
  constexpr int kSteps = kDim / 16;
  constexpr int kBlockKeys = kWarps * 16;
  __shared__ __align__(16) uint8_t q_sm[2][kStageRows * kPitch];
  __shared__ __align__(16) float2 row_sm[2][kStageRows];   // (c, L) of a row, read in pairs
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int s = blockIdx.z, kvh = blockIdx.y;
  const SeqInfo si = load_seq(p.seqs, s, p.err);
  const int key0 = blockIdx.x * kBlockKeys;
  const int64_t out0 = (int64_t(s) * p.cache.heads + kvh) * p.room;
  const int my_key = key0 + warp * 16;
  const int before = si.kv_len - si.q_len;                 // keys before the first new token
  // the rows of this head's group, token by token; those that see key0 on
  const int rows = si.q_len * p.group;
  const int row0 = max(0, key0 - before) * p.group / kStageRows * kStageRows;
  const bool any = key0 < si.kv_len && row0 < rows;

  // ---- the keys: A operands, steps in an order of k that fits 16-byte pieces
  uint32_t a[kSteps][4];
  if (any) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int key = my_key + half * 8 + g;
      int64_t page = p.cache.pages;
      int in_page = 0;
      if (key < si.kv_len) {
        const int n = key / p.cache.page_size;
        page = checked_page(p.seqs.table[int64_t(s) * p.seqs.width + n], p.cache.pages, p.err);
        in_page = key - n * p.cache.page_size;
      }
      const bool valid = page != p.cache.pages;
      const int64_t off = valid ? page * p.cache.ks[0] + in_page * p.cache.ks[1] + kvh * p.cache.ks[2] : 0;
      constexpr int kPieces = kDim * (kE4m3 ? 1 : 2) / 64;     // 16-byte pieces of a lane
      const uint8_t* row = static_cast<const uint8_t*>(p.cache.k) + off * (kE4m3 ? 1 : 2) + t * 16;
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (valid) v = *reinterpret_cast<const uint4*>(row + i * 64);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        if (kE4m3) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            a[(4 * i + j) % kSteps][half] = e4m3x2_to_f16x2(w[j] & 0xFFFFu);
            a[(4 * i + j) % kSteps][2 + half] = e4m3x2_to_f16x2(w[j] >> 16);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            a[(2 * i + j) % kSteps][half] = w[2 * j];
            a[(2 * i + j) % kSteps][2 + half] = w[2 * j + 1];
          }
        }
      }
    }
  }

  // ---- the rows: 8 threads to each, one stage ahead in registers
  const float c0 = p.scale * 1.44269504088896f *
                   (kE4m3 && p.cache.k_scale ? p.cache.k_scale[kvh] : 1.f);
  constexpr int kVec = kDim / 64;                          // 16-byte pieces of a thread
  const int my_row = tid >> 3, my_piece = tid & 7;
  uint4 next[kVec];
  float next_lse = 0.f;
  auto fetch = [&](int r) {
    const int tok = r / p.group, gi = r - tok * p.group;
    const bool valid = r < rows;
    const int64_t token = si.q0 + tok;
    const int head = kvh * p.group + gi;
    const __nv_bfloat16* src = p.q.data + token * p.q.ts + head * p.q.hs + my_piece * 8;
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      next[i] = valid ? *reinterpret_cast<const uint4*>(src + i * 64) : make_uint4(0, 0, 0, 0);
    next_lse = valid ? p.lse[token * p.q_heads + head] : 0.f;
  };
  auto put = [&](int b) {
    float c = c0;
    if (kE4m3) {
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const uint32_t w[4] = {next[i].x, next[i].y, next[i].z, next[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) top = fmaxf(top, fmaxf(fabsf(bf16_lo(w[j])), fabsf(bf16_hi(w[j]))));
      }
#pragma unroll
      for (int d = 4; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      int e = 141 - static_cast<int>(__float_as_uint(top) >> 23);
      e = top == 0.f || top > 3.4e38f ? 0 : min(e, 100);
      const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
      c *= __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        uint32_t w[4] = {next[i].x, next[i].y, next[i].z, next[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = f32x2_to_f16x2(bf16_lo(w[j]) * up, bf16_hi(w[j]) * up);
        next[i] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      *reinterpret_cast<uint4*>(&q_sm[b][my_row * kPitch + (i * 8 + my_piece) * 16]) = next[i];
    // (a row of lse -inf has no weight to give)
    if (my_piece == 0)
      row_sm[b][my_row] =
          make_float2(c, next_lse == -INFINITY ? INFINITY : next_lse * 1.44269504088896f);
  };

  float sum[2] = {0.f, 0.f};
  if (any) {
    fetch(row0 + my_row);
    put(0);
    __syncthreads();
    int b = 0;
    for (int r0 = row0; r0 < rows; r0 += kStageRows, b ^= 1) {
      const bool more = r0 + kStageRows < rows;
      if (more) fetch(r0 + kStageRows + my_row);
      // rows that see this warp's last key, and so all of them, need no mask
      const bool mask = r0 + kStageRows > rows ||
                        r0 < max(0, my_key + 15 - before) * p.group;
#pragma unroll 1
      for (int n = 0; n < kStageRows / 8; ++n) {
        if (r0 + n * 8 >= rows) break;
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        const uint8_t* qr = &q_sm[b][(n * 8 + g) * kPitch];
#pragma unroll
        for (int i = 0; i < kSteps; i += kE4m3 ? 4 : 2) {
          // the pieces of this lane, in the order of the keys'
          uint32_t w[8];
          const uint4 lo = *reinterpret_cast<const uint4*>(qr + (kE4m3 ? (i / 4 * 4 + t) * 32 : (i / 2 * 4 + t) * 16));
          w[0] = lo.x, w[1] = lo.y, w[2] = lo.z, w[3] = lo.w;
          if (kE4m3) {
            const uint4 hi = *reinterpret_cast<const uint4*>(qr + (i / 4 * 4 + t) * 32 + 16);
            w[4] = hi.x, w[5] = hi.y, w[6] = hi.z, w[7] = hi.w;
          }
#pragma unroll
          for (int j = 0; j < (kE4m3 ? 4 : 2); ++j) {
            const uint32_t(&am)[4] = a[(i + j) % kSteps];
            if (kE4m3)
              mma_f16_16816(d, am[0], am[1], am[2], am[3], w[2 * j], w[2 * j + 1]);
            else
              mma_bf16_16816(d, am[0], am[1], am[2], am[3], w[2 * j], w[2 * j + 1]);
          }
        }
        // columns 2t, 2t + 1 of this tile: rows of queries
        const float4 cl = *reinterpret_cast<const float4*>(&row_sm[b][n * 8 + 2 * t]);
        const int r = r0 + n * 8 + 2 * t;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float e0 = ex2(fmaf(d[2 * half], cl.x, -cl.y));
          float e1 = ex2(fmaf(d[2 * half + 1], cl.z, -cl.w));
          if (mask) {
            const int least = max(0, my_key + half * 8 + g - before) * p.group;
            if (r < least || r >= rows) e0 = 0.f;
            if (r + 1 < least || r + 1 >= rows) e1 = 0.f;
          }
          sum[half] += e0 + e1;
        }
      }
      if (more) put(b ^ 1);
      __syncthreads();
    }
  }
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    float x = sum[half];
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    x += __shfl_xor_sync(0xffffffffu, x, 2);
    const int key = my_key + half * 8 + g;
    if (t == 0 && key < p.room)
      p.out[out0 + key] = key < si.kv_len ? (p.mass ? p.mass[out0 + key] : 0.f) + x : 0.f;
  }
}

template <int kDim, bool kE4m3>
int run(const Mass& p, cudaStream_t stream) {
  constexpr int keys = kWarps * 16;
  const int64_t blocks = (p.room + keys - 1) / keys;
  if (blocks > INT32_MAX || p.cache.heads > 65535 || p.seqs.count > 65535) return NVFP4_ERR_SHAPE;
  return launch(mass_kernel<kDim, kE4m3>,
                dim3(static_cast<unsigned>(blocks), p.cache.heads, p.seqs.count), dim3(kThreads), 0,
                stream, p);
}

}  // namespace

int run_mass(const Mass& p, const Device& d, cudaStream_t stream) {
  const bool f8 = p.cache.e4m3;
  // This kernel's time grows with every 32 rows, that of mass_tc.cu stands still
  // up to 128 and is higher from the start, over e4m3 pages by the widening of K.
  // 32771 keys of 256: bf16 30 rows 28.5 us here against 33.2, 48 rows 34.3
  // against 33.3, 60 rows 39.0 against 33.0; e4m3 96 rows 38.9 against 64.7, 192
  // rows 61.5 against 71.1, 252 rows 77.4 against 67.5.
  // (No tokens: no query tile to copy, and only what was received before to hand on.)
  if (p.seqs.tokens > 0 && int64_t(p.max_q_len) * p.group > (f8 ? 192 : 32))
    return run_mass_tc(p, d, stream);
  switch (p.cache.dim) {
    case 64:
      return f8 ? run<64, true>(p, stream) : run<64, false>(p, stream);
    case 128:
      return f8 ? run<128, true>(p, stream) : run<128, false>(p, stream);
    default:
      return f8 ? run<256, true>(p, stream) : run<256, false>(p, stream);
  }
}

}  // namespace attn
}  // namespace nvfp4
