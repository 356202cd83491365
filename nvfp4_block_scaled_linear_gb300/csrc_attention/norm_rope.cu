// norm_rope.cu -- RMS norm of every query and key head, position rotation,
// and the store of key and value rows in the paged cache, in one pass.
//
//   y = x * rsqrt(mean(x^2) + eps) * weight              (fp32)
//   (a, b) = (y[i], y[i + rot/2]) -> (a cos - b sin, b cos + a sin), i < rot/2
//
// Bound by bytes: every head is read once and written once.  A lane holds 8
// consecutive elements (one 16-byte access), so a head takes dim/8 lanes and
// the sum of squares that many lanes' shuffles; the rotation's partner sits
// rot/16 lanes away and arrives by one shuffle per element.  A warp takes
// kSteps rows of heads of one token, all loaded before the first is used, so
// that the row of the cosine table and the two weight rows are read once for
// them and enough bytes are in flight to reach the memory's rate.
#include "common.cuh"

namespace nvfp4 {
namespace attn {
namespace {

constexpr int kSteps = 4;
constexpr int kThreads = 128;

__device__ __forceinline__ void unpack8(const uint4 w, float (&f)[8]) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(v[i]);
    f[2 * i + 1] = bf16_hi(v[i]);
  }
}

// dim: the head's width; a warp's step covers 256 / dim heads.
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

  uint4 x[kSteps];
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int h = h0 + s * kPerStep;
    x[s] = make_uint4(0, 0, 0, 0);
    if (h < heads) {
      const Heads& src = h < p.q_heads ? p.q : h < p.q_heads + p.kv_heads ? p.k : p.v;
      const int hh = h < p.q_heads ? h
                     : h < p.q_heads + p.kv_heads ? h - p.q_heads
                                                  : h - p.q_heads - p.kv_heads;
      x[s] = *reinterpret_cast<const uint4*>(src.data + t * src.ts + hh * src.hs + li * 8);
    }
  }
  const uint4 qw = *reinterpret_cast<const uint4*>(p.q_weight + li * 8);
  const uint4 kw = *reinterpret_cast<const uint4*>(p.k_weight + li * 8);
  // cosines and signed sines of this lane's elements: identity outside the
  // rotated dimensions
  const int half = p.rot / 16;                        // lanes holding the first of each pair
  float cs[8], sn[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) cs[i] = 1.f, sn[i] = 0.f;
  int partner = lane;
  if (li < 2 * half) {
    const int64_t pos = p.positions[t];
    partner = li < half ? lane + half : lane - half;
    if (pos >= 0 && pos < p.max_position) {
      const float* row = p.cos_sin + pos * p.rot + (li < half ? li : li - half) * 8;
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        const float4 c = *reinterpret_cast<const float4*>(row + i);
        const float4 s = *reinterpret_cast<const float4*>(row + p.rot / 2 + i);
        cs[i] = c.x, cs[i + 1] = c.y, cs[i + 2] = c.z, cs[i + 3] = c.w;
        sn[i] = s.x, sn[i + 1] = s.y, sn[i + 2] = s.z, sn[i + 3] = s.w;
      }
      if (li < half) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sn[i] = -sn[i];
      }
    } else {
      atomicOr(p.err, NVFP4_ATTENTION_BAD_INDEX);
    }
  }
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
    unpack8(x[s], y);
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sq = fmaf(y[i], y[i], sq);
#pragma unroll
    for (int m = kLanes / 2; m > 0; m >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, m);
    const float r = rsqrtf(sq * (1.f / kDim) + p.eps);
    float wt[8];
    unpack8(is_q ? qw : kw, wt);
    float n[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) n[i] = y[i] * r * wt[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float other = __shfl_sync(0xffffffffu, n[i], partner);
      const float turned = partner == lane ? n[i] : fmaf(other, sn[i], n[i] * cs[i]);
      if (!is_v) y[i] = turned;
    }
    if (h >= heads) continue;
    const int hh = is_q ? h : is_v ? h - p.q_heads - p.kv_heads : h - p.q_heads;
    if (is_q || !p.store) {
      const Heads& dst = is_q ? p.q_out : p.k_out;
      *reinterpret_cast<uint4*>(dst.data + t * dst.ts + hh * dst.hs + li * 8) =
          make_uint4(f32x2_to_bf16x2(y[0], y[1]), f32x2_to_bf16x2(y[2], y[3]),
                     f32x2_to_bf16x2(y[4], y[5]), f32x2_to_bf16x2(y[6], y[7]));
      continue;
    }
    if (page < 0) continue;
    const int64_t* st = is_v ? p.cache.vs : p.cache.ks;
    const int64_t off = page * st[0] + in_page * st[1] + hh * st[2] + li * 8;
    void* base = is_v ? p.cache.v : p.cache.k;
    if (p.cache.e4m3) {
      const float* scales = is_v ? p.cache.v_scale : p.cache.k_scale;
      const float scale = scales ? scales[hh] : 1.f;
      uint32_t c[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        c[i] = __nv_cvt_float2_to_fp8x2(make_float2(y[2 * i] / scale, y[2 * i + 1] / scale),
                                        __NV_SATFINITE, __NV_E4M3);
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(base) + off) =
          make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
    } else {
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + off) =
          make_uint4(f32x2_to_bf16x2(y[0], y[1]), f32x2_to_bf16x2(y[2], y[3]),
                     f32x2_to_bf16x2(y[4], y[5]), f32x2_to_bf16x2(y[6], y[7]));
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
