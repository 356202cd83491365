// norm_rope.cu -- RMS norm of every query and key head, position rotation,
// and the store of key and value rows in the paged cache, in one pass.
//
//   y = x * rsqrt(mean(x^2) + eps) * weight              (fp32)
//   (a, b) = (y[i], y[i + rot/2]) -> (a cos - b sin, b cos + a sin), i < rot/2
//
// Bound by bytes: every head is read once and written once.  A lane holds 8
// elements: in the rotated dimensions 4 and the 4 they are paired with, so that
// the rotation needs no other lane, beyond them 8 consecutive ones; a head takes
// dim/8 lanes, and the sum of squares that many lanes' shuffles.  A warp takes
// kSteps rows of heads of one token, all loaded before the first is used, so
// that the row of the cosine table and the two weight rows are read once for
// them and enough bytes are in flight.  A block is one token (or part of one):
// blocks that went on to further tokens, loading the next while working on one,
// took twice the registers and measured 73 us against 56.
//
// Measured at head_dim 256, 24 query and 4 key/value heads: 8192 tokens into
// e4m3 pages 56 us, 4.5 TB/s; one token 2.1 us.  What is missing to the copy
// rate of 6.7 TB/s is each warp's latency: token -> position -> cosine row, and
// the loads and stores of a warp do not overlap each other.
#include "common.cuh"

namespace nvfp4 {
namespace attn {
namespace {

constexpr int kMaxThreads = 128;

__device__ __forceinline__ void unpack4(const uint2 w, float* f) {
  f[0] = bf16_lo(w.x), f[1] = bf16_hi(w.x), f[2] = bf16_lo(w.y), f[3] = bf16_hi(w.y);
}
__device__ __forceinline__ uint2 pack4(const float* f) {
  return make_uint2(f32x2_to_bf16x2(f[0], f[1]), f32x2_to_bf16x2(f[2], f[3]));
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// kDim: the head's width; a warp's step covers 256 / kDim heads.  A warp's heads
// are all query, all key or all value heads.
template <int kDim, int kSteps>
__global__ void __launch_bounds__(kMaxThreads, 8) norm_rope_kernel(const NormRope p, int q_warps,
                                                                int k_warps) {
  constexpr int kLanes = kDim / 8, kPerStep = 32 / kLanes;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, li = lane % kLanes;
  const int64_t t = blockIdx.x;
  const int w = blockIdx.y * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int kind = w < q_warps ? 0 : w < q_warps + k_warps ? 1 : 2;      // query, key, value
  const int h0 = (w - (kind > 0 ? q_warps : 0) - (kind > 1 ? k_warps : 0)) * (kSteps * kPerStep) +
                 lane / kLanes;
  const int heads = kind == 0 ? p.q_heads : p.kv_heads;
  const Heads src = kind == 0 ? p.q : kind == 1 ? p.k : p.v;
  // this lane's two fours of elements
  const bool turns = kind < 2 && li * 8 < p.rot;
  const int at0 = turns ? li * 4 : li * 8, at1 = turns ? p.rot / 2 + li * 4 : li * 8 + 4;
  if (kind == 2 && !p.store) return;

  uint2 x[kSteps][2];
  const __nv_bfloat16* in = src.data + t * src.ts + h0 * src.hs;
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    x[s][0] = x[s][1] = make_uint2(0, 0);
    if (h0 + s * kPerStep < heads) {
      x[s][0] = *reinterpret_cast<const uint2*>(in + at0);
      x[s][1] = *reinterpret_cast<const uint2*>(in + at1);
      in += kPerStep * src.hs;
    }
  }
  float2 wt[4];
  if (kind < 2) {
    const __nv_bfloat16* weight = kind == 0 ? p.q_weight : p.k_weight;
    float f[8];
    unpack4(*reinterpret_cast<const uint2*>(weight + at0), f);
    unpack4(*reinterpret_cast<const uint2*>(weight + at1), f + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) wt[i] = make_float2(f[2 * i], f[2 * i + 1]);
  }
  float4 cs = make_float4(1.f, 1.f, 1.f, 1.f), sn = make_float4(0.f, 0.f, 0.f, 0.f);
  if (turns) {
    const int64_t pos = p.positions[t];
    if (pos >= 0 && pos < p.max_position) {
      const float* row = p.cos_sin + pos * p.rot + at0;
      cs = *reinterpret_cast<const float4*>(row);
      sn = *reinterpret_cast<const float4*>(row + p.rot / 2);
    } else {
      atomicOr(p.err, NVFP4_ATTENTION_BAD_INDEX);
    }
  }
  // where the first of the warp's rows goes, and the step to the next
  const bool to_cache = kind > 0 && p.store;
  const bool narrow = to_cache && p.cache.e4m3;
  int64_t off, next;
  void* out;
  bool stored = true;
  if (to_cache) {
    const int64_t slot = p.slots[t];
    stored = slot >= 0 && slot < p.cache.pages * p.cache.page_size;
    if (!stored && slot != -1) atomicOr(p.err, NVFP4_ATTENTION_BAD_INDEX);
    const int64_t page = slot >> 31 ? slot / p.cache.page_size
                                    : static_cast<uint32_t>(slot) / static_cast<uint32_t>(p.cache.page_size);
    const int64_t in_page = slot - page * p.cache.page_size;
    off = kind == 2 ? page * p.cache.vs[0] + in_page * p.cache.vs[1] + h0 * p.cache.vs[2]
                    : page * p.cache.ks[0] + in_page * p.cache.ks[1] + h0 * p.cache.ks[2];
    next = kPerStep * (kind == 2 ? p.cache.vs[2] : p.cache.ks[2]);
    out = kind == 2 ? p.cache.v : p.cache.k;
  } else {
    const Heads dst = kind == 0 ? p.q_out : p.k_out;
    off = t * dst.ts + h0 * dst.hs;
    next = kPerStep * dst.hs;
    out = dst.data;
  }

#pragma unroll
  for (int s = 0; s < kSteps; ++s, off += next) {
    const int h = h0 + s * kPerStep;
    float y[8];
    unpack4(x[s][0], y);
    unpack4(x[s][1], y + 4);
    if (kind < 2) {
      float2 sq = mul2(make_float2(y[0], y[1]), make_float2(y[0], y[1]));
#pragma unroll
      for (int i = 2; i < 8; i += 2) {
        sq.x = fmaf(y[i], y[i], sq.x);
        sq.y = fmaf(y[i + 1], y[i + 1], sq.y);
      }
      float sum = sq.x + sq.y;
#pragma unroll
      for (int m = kLanes / 2; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
      const float r = rsqrtf(sum * (1.f / kDim) + p.eps);
      float2 z[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        z[i] = mul2(mul2(make_float2(y[2 * i], y[2 * i + 1]), make_float2(r, r)), wt[i]);
      // (lanes that do not turn: cosine 1, sine 0)
      if (turns) {
        const float c4[4] = {cs.x, cs.y, cs.z, cs.w}, s4[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = i & 1 ? z[i >> 1].y : z[i >> 1].x;
          const float b = i & 1 ? z[2 + (i >> 1)].y : z[2 + (i >> 1)].x;
          y[i] = a * c4[i] - b * s4[i];
          y[i + 4] = b * c4[i] + a * s4[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) y[2 * i] = z[i].x, y[2 * i + 1] = z[i].y;
      }
    }
    if (h >= heads || !stored) continue;
    if (narrow) {
      const float* scales = kind == 2 ? p.cache.v_scale : p.cache.k_scale;
      const float scale = scales ? scales[h] : 1.f;
      uint32_t c[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        c[i] = __nv_cvt_float2_to_fp8x2(make_float2(y[2 * i] / scale, y[2 * i + 1] / scale),
                                        __NV_SATFINITE, __NV_E4M3);
      uint8_t* row = static_cast<uint8_t*>(out) + off;
      *reinterpret_cast<uint32_t*>(row + at0) = c[0] | c[1] << 16;
      *reinterpret_cast<uint32_t*>(row + at1) = c[2] | c[3] << 16;
    } else {
      __nv_bfloat16* row = static_cast<__nv_bfloat16*>(out) + off;
      *reinterpret_cast<uint2*>(row + at0) = pack4(y);
      *reinterpret_cast<uint2*>(row + at1) = pack4(y + 4);
    }
  }
}

}  // namespace

template <int kDim, int kSteps>
static int run(const NormRope& p, cudaStream_t stream) {
  constexpr int kPerWarp = kSteps * (256 / kDim);
  const int q_warps = (p.q_heads + kPerWarp - 1) / kPerWarp;
  const int k_warps = (p.kv_heads + kPerWarp - 1) / kPerWarp;
  // a block per token, or several where it has more heads than one holds
  const int warps = q_warps + k_warps * (p.store ? 2 : 1);
  const int blocks = (warps * 32 + kMaxThreads - 1) / kMaxThreads;
  const int threads = (warps + blocks - 1) / blocks * 32;
  return launch(norm_rope_kernel<kDim, kSteps>, dim3(static_cast<unsigned>(p.tokens), blocks),
                dim3(threads), 0, stream, p, q_warps, k_warps);
}

template <int kDim>
static int run(const NormRope& p, const Device& d, cudaStream_t stream) {
  // Few tokens: latency, so fewer rows one after the other in a warp.  More than
  // an SM's one: bytes in flight.  At head_dim 256, 24 and 4 heads: one token 2.1
  // us with 2 steps, 2.6 with 4; 8192 tokens into e4m3 pages 65 against 56.
  return p.tokens <= d.num_sms ? run<kDim, 2>(p, stream) : run<kDim, 4>(p, stream);
}

int run_norm_rope(const NormRope& p, const Device& d, cudaStream_t stream) {
  return p.dim == 256 ? run<256>(p, d, stream)
       : p.dim == 128 ? run<128>(p, d, stream)
                      : run<64>(p, d, stream);
}

}  // namespace attn
}  // namespace nvfp4
