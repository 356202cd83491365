// join.cu -- the partial results of items that several CTAs shared, joined:
//   out = sum_i 2^(L_i - L) out_i,  2^L = sum_i 2^(L_i)
// in the CTAs' order.  A block looks after one row of the item that begins, and
// does not end, in one CTA's range.  A few KB per row: bound by the latency of
// its four dependent loads (note, end, sums, outputs), so each is one round.
// Behind one token over 4099 keys it ends some 3 us after the grid before it.
// Behind many rows it is the number of blocks that counts: a block for each of
// 152 x 128 rows of 256 took 33 us from a cold L2, 4 rows a block 14.
#include "schedule.cuh"

namespace nvfp4 {
namespace attn {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxParts = 512;

// kMany: many rows in few parts each, so the block's groups of threads take a
// row each; else they share the parts of one.
template <int kDim, bool kMany>
__global__ void __launch_bounds__(kThreads) join_kernel(const Attend p, const Parts parts,
                                                        const Plan plan, int ctas) {
  constexpr int kCols = kDim / 4;                // threads of one part, 4 columns each
  constexpr int kWays = kThreads / kCols;        // parts (or rows) read at a time
  __shared__ float weight[kMaxParts];
  __shared__ float4 sum_sm[kWays][kCols];
  __shared__ float total_sm;
  griddep_wait();
  griddep_launch_dependents();
  const int way = threadIdx.x / kCols, col = threadIdx.x % kCols;
  const int c = blockIdx.x, r = kMany ? blockIdx.y * kWays + way : blockIdx.y;
  const int lane = threadIdx.x & 31;
  const int4 note = parts.note[c];
  if (!(note.x & kPart1)) return;
  const SeqInfo si = load_seq(p.seqs, note.y, p.err);
  // the CTA in which the item ends
  int last = ctas;
  for (int i = c + 1; i < ctas; i += 32) {
    const int f = i + lane < ctas ? parts.note[i + lane].x : 0;
    const unsigned ends = __ballot_sync(0xffffffffu, f & kPart0Ends);
    if (ends) {
      last = i + __ffs(ends) - 1;
      break;
    }
  }
  const int n = last - c + 1;
  if (last == ctas || n > kMaxParts) return;
  const int tile_tokens = parts.tile_rows / p.group;
  const int sub = r / parts.tile_rows, rr = r - sub * parts.tile_rows;
  const int tok = rr / p.group, g = rr - tok * p.group;
  const int ti = note.w * plan.tile_tokens + sub * tile_tokens + tok;
  if (tok >= tile_tokens || ti >= si.q_len) return;
  const int64_t t = si.q0 + ti;
  const int h = note.z * p.group + g;
  if constexpr (kMany) {
    float top = -INFINITY;
    for (int i = 0; i < n; ++i) top = fmaxf(top, parts.lse2[parts.row(c + i, i == 0, r)]);
    const float base = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
    for (int i = 0; i < n; ++i) {
      const int64_t at = parts.row(c + i, i == 0, r);
      const float4 x = *reinterpret_cast<const float4*>(parts.out + at * kDim + col * 4);
      const float w = exp2f(parts.lse2[at] - base);
      sum += w;
      o.x = fmaf(w, x.x, o.x), o.y = fmaf(w, x.y, o.y);
      o.z = fmaf(w, x.z, o.z), o.w = fmaf(w, x.w, o.w);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    if (p.lse && col == 0) p.lse[t * p.q_heads + h] = (base + log2f(sum)) * 0.693147180559945f;
    *reinterpret_cast<uint2*>(p.out.data + t * p.out.ts + h * p.out.hs + col * 4) =
        make_uint2(f32x2_to_bf16x2(o.x * inv, o.y * inv), f32x2_to_bf16x2(o.z * inv, o.w * inv));
    return;
  }
  if (threadIdx.x < 32) {
    float top = -INFINITY;
    for (int i = lane; i < n; i += 32) {
      const float l = parts.lse2[parts.row(c + i, i == 0, r)];
      weight[i] = l;
      top = fmaxf(top, l);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const float base = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
    for (int i = lane; i < n; i += 32) {
      const float w = exp2f(weight[i] - base);
      weight[i] = w;
      sum += w;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == 0) {
      total_sm = sum;
      if (p.lse) p.lse[t * p.q_heads + h] = (base + log2f(sum)) * 0.693147180559945f;
    }
  }
  __syncthreads();
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int i = way; i < n; i += kWays) {
    const float w = weight[i];
    const float4 x = *reinterpret_cast<const float4*>(
        parts.out + parts.row(c + i, i == 0, r) * kDim + col * 4);
    o.x = fmaf(w, x.x, o.x), o.y = fmaf(w, x.y, o.y);
    o.z = fmaf(w, x.z, o.z), o.w = fmaf(w, x.w, o.w);
  }
  sum_sm[way][col] = o;
  __syncthreads();
  if (way != 0) return;
#pragma unroll
  for (int i = 1; i < kWays; ++i) {
    const float4 x = sum_sm[i][col];
    o.x += x.x, o.y += x.y, o.z += x.z, o.w += x.w;
  }
  const float inv = total_sm == 0.f ? 0.f : 1.f / total_sm;
  *reinterpret_cast<uint2*>(p.out.data + t * p.out.ts + h * p.out.hs + col * 4) =
      make_uint2(f32x2_to_bf16x2(o.x * inv, o.y * inv), f32x2_to_bf16x2(o.z * inv, o.w * inv));
}

}  // namespace

template <bool kMany>
static int run(const Attend& p, const Parts& parts, const Plan& plan, int ctas, int device,
               cudaStream_t stream) {
  auto* kernel = p.cache.dim == 256   ? join_kernel<256, kMany>
                 : p.cache.dim == 128 ? join_kernel<128, kMany>
                                      : join_kernel<64, kMany>;
  // The attention kernels leave the SMs with all memory given to shared memory;
  // blocks that ask for another split could only start when those have ended.
  static std::atomic<bool> ready[3][kMaxDevices];
  std::atomic<bool>& set = ready[p.cache.dim / 128][device];
  if (!set.load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared) != cudaSuccess) {
      cudaGetLastError();
      return NVFP4_ERR_LAUNCH;
    }
    set.store(true, std::memory_order_release);
  }
  const int rows = kMany ? kThreads * 4 / p.cache.dim : 1;       // of a block
  return launch(kernel, dim3(ctas, parts.rows / rows), dim3(kThreads), 0, stream, p,
                parts, plan, ctas);
}

int run_join(bool many, const Attend& p, const Parts& parts, const Plan& plan, int ctas,
             int device, cudaStream_t stream) {
  return many ? run<true>(p, parts, plan, ctas, device, stream)
              : run<false>(p, parts, plan, ctas, device, stream);
}

}  // namespace attn
}  // namespace nvfp4
