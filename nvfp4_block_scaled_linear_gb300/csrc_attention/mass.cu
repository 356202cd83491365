// mass.cu -- the attention weight that each cached key receives from the new
// tokens, one warp per sequence, key/value head and key.
#include "common.cuh"

namespace nvfp4 {
namespace attn {
namespace {

constexpr int kThreads = 128;

template <int kDim>
__global__ void __launch_bounds__(kThreads) mass_kernel(const Mass p) {
  constexpr int kPer = kDim / 32;
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t(blockIdx.x) * kThreads + threadIdx.x) >> 5;
  const int64_t sh = w / p.room;
  const int j = static_cast<int>(w - sh * p.room);
  const int s = static_cast<int>(sh / p.cache.heads), kvh = static_cast<int>(sh % p.cache.heads);
  if (s >= p.seqs.count) return;
  const SeqInfo si = load_seq(p.seqs, s, p.err);
  float sum = 0.f;
  int64_t page = p.cache.pages;
  if (j < si.kv_len)
    page = checked_page(p.seqs.table[int64_t(s) * p.seqs.width + j / p.cache.page_size],
                        p.cache.pages, p.err);
  if (page != p.cache.pages) {
    const float ks = (p.cache.k_scale ? p.cache.k_scale[kvh] : 1.f) * p.scale;
    const int64_t ko = page * p.cache.ks[0] + (j % p.cache.page_size) * p.cache.ks[1] +
                       kvh * p.cache.ks[2] + lane;
    float k[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      k[i] = ks * (p.cache.e4m3
                       ? e4m3_to_f32(static_cast<const uint8_t*>(p.cache.k)[ko + i * 32])
                       : __bfloat162float(static_cast<const __nv_bfloat16*>(p.cache.k)[ko + i * 32]));
    // the first new token that sees key j
    for (int i = max(0, j - (si.kv_len - si.q_len)); i < si.q_len; ++i) {
      const int64_t t = si.q0 + i;
      for (int g = 0; g < p.group; ++g) {
        const int h = kvh * p.group + g;
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < kPer; ++e)
          x = fmaf(k[e], __bfloat162float(p.q.data[t * p.q.ts + h * p.q.hs + e * 32 + lane]), x);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
        sum += expf(x - p.lse[t * p.q_heads + h]);
      }
    }
  }
  if (lane == 0)
    p.out[w] = j < si.kv_len ? (p.mass ? p.mass[w] : 0.f) + sum : 0.f;
}

}  // namespace

int run_mass(const Mass& p, const Device&, cudaStream_t stream) {
  const int64_t blocks = (p.room * p.seqs.count * p.cache.heads * 32 + kThreads - 1) / kThreads;
  if (blocks > INT32_MAX) return NVFP4_ERR_SHAPE;
  auto* kernel = p.cache.dim == 256   ? mass_kernel<256>
                 : p.cache.dim == 128 ? mass_kernel<128>
                                      : mass_kernel<64>;
  return launch(kernel, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, stream, p);
}

}  // namespace attn
}  // namespace nvfp4
