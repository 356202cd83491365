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
// them and enough bytes are in flight to reach the memory's rate.
#include "common.cuh"

namespace nvfp4 {
namespace attn {
namespace {

constexpr int kSteps = 4;
constexpr int kThreads = 128;

__device__ __forceinline__ void unpack4(const uint2 w, float* f) {
  f[0] = bf16_lo(w.x), f[1] = bf16_hi(w.x), f[2] = bf16_lo(w.y), f[3] = bf16_hi(w.y);
}
__device__ __forceinline__ uint2 pack4(const float* f) {
  return make_uint2(f32x2_to_bf16x2(f[0], f[1]), f32x2_to_bf16x2(f[2], f[3]));
}

// kDim: the head's width; a warp's step covers 256 / kDim heads.
template <int kDim>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const NormRope p, int warps_per_token,
                                                             int heads) {
  constexpr int kLanes = kDim / 8, kPerStep = 32 / kLanes;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, li = lane % kLanes;
  const int64_t w = (int64_t(blockIdx.x) * kThreads + threadIdx.x) >> 5;
  const int64_t t = w / warps_per_token;
  if (t >= p.tokens) return;
  const int h0 = static_cast<int>(w - t * warps_per_token) * (kSteps * kPerStep) + lane / kLanes;
  // this lane's two fours of elements
  const bool turns = li * 8 < p.rot;
  const int at0 = turns ? li * 4 : li * 8, at1 = turns ? p.rot / 2 + li * 4 : li * 8 + 4;

  uint2 x[kSteps][2];
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int h = h0 + s * kPerStep;
    x[s][0] = x[s][1] = make_uint2(0, 0);
    if (h < heads) {
      const Heads& src = h < p.q_heads ? p.q : h < p.q_heads + p.kv_heads ? p.k : p.v;
      const int hh = h < p.q_heads ? h
                     : h < p.q_heads + p.kv_heads ? h - p.q_heads
                                                  : h - p.q_heads - p.kv_heads;
      const __nv_bfloat16* row = src.data + t * src.ts + hh * src.hs;
      x[s][0] = *reinterpret_cast<const uint2*>(row + at0);
      x[s][1] = *reinterpret_cast<const uint2*>(row + at1);
    }
  }
  uint2 qw[2], kw[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    qw[i] = *reinterpret_cast<const uint2*>(p.q_weight + (i ? at1 : at0));
    kw[i] = *reinterpret_cast<const uint2*>(p.k_weight + (i ? at1 : at0));
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
  const float c4[4] = {cs.x, cs.y, cs.z, cs.w}, s4[4] = {sn.x, sn.y, sn.z, sn.w};
  int64_t page = -1;
  int in_page = 0;
  if (p.store) {
    const int64_t slot = p.slots[t];
    if (slot >= 0 && slot < p.cache.pages * p.cache.page_size) {
      page = slot / p.cache.page_size;
      in_page = static_cast<int>(slot - page * p.cache.page_size);
    } else if (slot != -1) {
      atomicOr(p.err, NVFP4_ATTENTION_BAD_INDEX);
    }
  }

#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int h = h0 + s * kPerStep;
    const bool is_q = h < p.q_heads, is_v = h >= p.q_heads + p.kv_heads;
    float y[8];
    unpack4(x[s][0], y);
    unpack4(x[s][1], y + 4);
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sq = fmaf(y[i], y[i], sq);
#pragma unroll
    for (int m = kLanes / 2; m > 0; m >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, m);
    if (!is_v) {
      const float r = rsqrtf(sq * (1.f / kDim) + p.eps);
      float wt[8];
      unpack4(is_q ? qw[0] : kw[0], wt);
      unpack4(is_q ? qw[1] : kw[1], wt + 4);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = y[i] * r * wt[i];
      if (turns) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = y[i], b = y[i + 4];
          y[i] = a * c4[i] - b * s4[i];
          y[i + 4] = b * c4[i] + a * s4[i];
        }
      }
    }
    if (h >= heads) continue;
    const int hh = is_q ? h : is_v ? h - p.q_heads - p.kv_heads : h - p.q_heads;
    if (is_q || !p.store) {
      const Heads& dst = is_q ? p.q_out : p.k_out;
      __nv_bfloat16* row = dst.data + t * dst.ts + hh * dst.hs;
      *reinterpret_cast<uint2*>(row + at0) = pack4(y);
      *reinterpret_cast<uint2*>(row + at1) = pack4(y + 4);
      continue;
    }
    if (page < 0) continue;
    const int64_t* st = is_v ? p.cache.vs : p.cache.ks;
    const int64_t off = page * st[0] + in_page * st[1] + hh * st[2];
    void* base = is_v ? p.cache.v : p.cache.k;
    if (p.cache.e4m3) {
      const float* scales = is_v ? p.cache.v_scale : p.cache.k_scale;
      const float scale = scales ? scales[hh] : 1.f;
      uint32_t c[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        c[i] = __nv_cvt_float2_to_fp8x2(make_float2(y[2 * i] / scale, y[2 * i + 1] / scale),
                                        __NV_SATFINITE, __NV_E4M3);
      uint8_t* row = static_cast<uint8_t*>(base) + off;
      *reinterpret_cast<uint32_t*>(row + at0) = c[0] | c[1] << 16;
      *reinterpret_cast<uint32_t*>(row + at1) = c[2] | c[3] << 16;
    } else {
      __nv_bfloat16* row = static_cast<__nv_bfloat16*>(base) + off;
      *reinterpret_cast<uint2*>(row + at0) = pack4(y);
      *reinterpret_cast<uint2*>(row + at1) = pack4(y + 4);
    }
  }
}

}  // namespace

int run_norm_rope(const NormRope& p, const Device&, cudaStream_t stream) {
  const int heads = p.q_heads + p.kv_heads * (p.store ? 2 : 1);
  const int per_warp = kSteps * (256 / p.dim);
  const int wpt = (heads + per_warp - 1) / per_warp;
  const int64_t blocks = (p.tokens * wpt * 32 + kThreads - 1) / kThreads;
  if (blocks > INT32_MAX) return NVFP4_ERR_SHAPE;
  auto* kernel = p.dim == 256   ? norm_rope_kernel<256>
                 : p.dim == 128 ? norm_rope_kernel<128>
                                : norm_rope_kernel<64>;
  return launch(kernel, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, stream, p, wpt,
                heads);
}

}  // namespace attn
}  // namespace nvfp4
