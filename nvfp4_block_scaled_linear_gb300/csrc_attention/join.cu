// join.cu -- the partial results of items that several CTAs shared, joined:
//   out = sum_i 2^(L_i - L) out_i,  2^L = sum_i 2^(L_i)
// in the CTAs' order.  A block looks after some rows of the item that begins,
// and does not end, in one CTA's range.  A few KB per row; bound by the
// latency of its two rounds of loads.
#include "schedule.cuh"

namespace nvfp4 {
namespace attn {
namespace {

constexpr int kThreads = 256;

template <int kDim>
__global__ void __launch_bounds__(kThreads) join_kernel(const Attend p, const Parts parts,
                                                        const Plan plan, int ctas) {
  constexpr int kPerRow = kDim / 4;              // threads of one row, 4 columns each
  griddep_wait();
  griddep_launch_dependents();
  const int c = blockIdx.x, lane = threadIdx.x & 31;
  const int4 note = parts.note[c];
  if (!(note.x & kPart1)) return;
  const SeqInfo si = load_seq(p.seqs, note.y, p.err);
  const int r = blockIdx.y * (kThreads / kPerRow) + threadIdx.x / kPerRow;
  const int col = (threadIdx.x % kPerRow) * 4;
  const int tok = r / p.group, g = r - tok * p.group;
  const int ti = note.w * plan.tile_tokens + tok;
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
  if (last == ctas || tok >= plan.tile_tokens || ti >= si.q_len) return;
  float top = parts.lse2[parts.row(c, 1, r)];
#pragma unroll 4
  for (int i = c + 1; i <= last; ++i) top = fmaxf(top, parts.lse2[parts.row(i, 0, r)]);
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
  const float base = top == -INFINITY ? 0.f : top;
#pragma unroll 4
  for (int i = c; i <= last; ++i) {
    const int64_t row = parts.row(i, i == c, r);
    const float w = exp2f(parts.lse2[row] - base);
    const float4 x = *reinterpret_cast<const float4*>(parts.out + row * kDim + col);
    sum += w;
    o.x = fmaf(w, x.x, o.x), o.y = fmaf(w, x.y, o.y);
    o.z = fmaf(w, x.z, o.z), o.w = fmaf(w, x.w, o.w);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int64_t t = si.q0 + ti;
  const int h = note.z * p.group + g;
  *reinterpret_cast<uint2*>(p.out.data + t * p.out.ts + h * p.out.hs + col) =
      make_uint2(f32x2_to_bf16x2(o.x * inv, o.y * inv), f32x2_to_bf16x2(o.z * inv, o.w * inv));
  if (p.lse && col == 0)
    p.lse[t * p.q_heads + h] = (base + log2f(sum)) * 0.693147180559945f;
}

}  // namespace

int run_join(const Attend& p, const Parts& parts, const Plan& plan, int ctas,
             cudaStream_t stream) {
  const int rows = kThreads / (p.cache.dim / 4);
  auto* kernel = p.cache.dim == 256   ? join_kernel<256>
                 : p.cache.dim == 128 ? join_kernel<128>
                                      : join_kernel<64>;
  return launch(kernel, dim3(ctas, (parts.rows + rows - 1) / rows), dim3(kThreads), 0, stream, p,
                parts, plan, ctas);
}

}  // namespace attn
}  // namespace nvfp4
