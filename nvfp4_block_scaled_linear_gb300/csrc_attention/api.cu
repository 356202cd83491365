// api.cu -- the C ABI of include/nvfp4_attention.h: validation on the host,
// the per-device set-up and the attention error word.
#include <climits>
#include <cmath>
#include <mutex>
#include <utility>

#include "common.cuh"

namespace {

__device__ unsigned int g_attention_error;
__device__ unsigned int g_attention_error_read;

__global__ void read_attention_error_kernel(int clear) {
  g_attention_error_read =
      clear ? atomicExch(&g_attention_error, 0u) : atomicOr(&g_attention_error, 0u);
}

using nvfp4::attn::kMaxDevices;
struct Slot {
  bool ready = false, supported = false;
  nvfp4::attn::Device d;
};
Slot g_devices[kMaxDevices];
std::mutex g_device_mutex;

bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

// A stride counts only where its dimension has more than one element.
int check_heads(const nvfp4_heads* h, int64_t tokens, int64_t count) {
  if (!h || !h->data) return NVFP4_ERR_INVALID;
  if (misaligned(h->data)) return NVFP4_ERR_MISALIGNED;
  for (const auto& [stride, size] : {std::pair(h->token_stride, tokens), {h->head_stride, count}}) {
    if (size <= 1) continue;
    if (stride <= 0) return NVFP4_ERR_INVALID;
    if (stride % 8 != 0) return NVFP4_ERR_MISALIGNED;
    if (stride >= (int64_t(1) << 38)) return NVFP4_ERR_SHAPE;     // the copy engine's limit
  }
  return NVFP4_OK;
}

int check_cache(const nvfp4_kv_cache* c) {
  if (!c || !c->k || !c->v) return NVFP4_ERR_INVALID;
  if (c->type != NVFP4_CACHE_BF16 && c->type != NVFP4_CACHE_E4M3) return NVFP4_ERR_INVALID;
  if (c->num_pages <= 0 || c->num_pages > INT_MAX || c->page_size <= 0 || c->kv_heads <= 0)
    return NVFP4_ERR_INVALID;
  if (c->type == NVFP4_CACHE_BF16 && (c->k_scale || c->v_scale)) return NVFP4_ERR_INVALID;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return NVFP4_ERR_SHAPE;
  if (c->page_size % 16 != 0) return NVFP4_ERR_SHAPE;
  if (misaligned(c->k) || misaligned(c->v)) return NVFP4_ERR_MISALIGNED;
  const int size = c->type == NVFP4_CACHE_BF16 ? 2 : 1;
  for (int i = 0; i < 3; ++i) {
    if (c->k_stride[i] <= 0 || c->v_stride[i] <= 0) return NVFP4_ERR_INVALID;
    if (c->k_stride[i] * size % 16 != 0 || c->v_stride[i] * size % 16 != 0)
      return NVFP4_ERR_MISALIGNED;
    // the copy engine's limit on a stride
    if (c->k_stride[i] >= (int64_t(1) << 38) || c->v_stride[i] >= (int64_t(1) << 38))
      return NVFP4_ERR_SHAPE;
  }
  return NVFP4_OK;
}

int check_seqs(const nvfp4_sequences* s, bool queries) {
  if (!s || s->count < 0 || s->table_width <= 0) return NVFP4_ERR_INVALID;
  if (s->count > 0 && (!s->block_table || !s->kv_lens)) return NVFP4_ERR_INVALID;
  if (queries && s->count > 0 && (!s->q_starts || s->max_q_len < 0)) return NVFP4_ERR_INVALID;
  if (queries && s->count > NVFP4_ATTENTION_MAX_SEQUENCES) return NVFP4_ERR_SHAPE;
  return NVFP4_OK;
}

int check_groups(int64_t tokens, int32_t q_heads, int32_t kv_heads) {
  if (tokens < 0 || q_heads <= 0) return NVFP4_ERR_INVALID;
  if (tokens > INT_MAX / 2) return NVFP4_ERR_SHAPE;
  if (q_heads % kv_heads != 0 || q_heads / kv_heads > 128) return NVFP4_ERR_SHAPE;
  return NVFP4_OK;
}

nvfp4::attn::Heads heads(const nvfp4_heads* h, int64_t tokens, int64_t count, int dim) {
  if (!h) return {};
  return {static_cast<__nv_bfloat16*>(h->data), tokens > 1 ? h->token_stride : dim * count,
          count > 1 ? h->head_stride : dim};
}

nvfp4::attn::Cache cache_of(const nvfp4_kv_cache* c) {
  nvfp4::attn::Cache r{};
  if (!c) return r;
  r.k = c->k;
  r.v = c->v;
  r.k_scale = c->k_scale;
  r.v_scale = c->v_scale;
  r.pages = c->num_pages;
  for (int i = 0; i < 3; ++i) {
    r.ks[i] = c->k_stride[i];
    r.vs[i] = c->v_stride[i];
  }
  r.page_size = c->page_size;
  r.heads = c->kv_heads;
  r.dim = c->head_dim;
  r.e4m3 = c->type == NVFP4_CACHE_E4M3;
  return r;
}

nvfp4::attn::Seqs seqs_of(const nvfp4_sequences* s, int64_t tokens, int page_size) {
  return {s->block_table, s->kv_lens, s->q_starts, s->count, s->table_width,
          static_cast<int>(tokens), int64_t(s->table_width) * page_size};
}

}  // namespace

namespace nvfp4 {
namespace attn {

int device(Device* out) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    cudaGetLastError();
    return NVFP4_ERR_DEVICE;
  }
  std::lock_guard<std::mutex> lock(g_device_mutex);
  Slot& s = g_devices[dev];
  if (!s.ready) {
    int major = 0, minor = 0, sms = 0;
    void* err = nullptr;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
      cudaGetLastError();
      return NVFP4_ERR_DEVICE;
    }
    s.supported = major == 10 && minor == 3;
    if (s.supported && cudaGetSymbolAddress(&err, g_attention_error) != cudaSuccess) {
      cudaGetLastError();
      return NVFP4_ERR_DEVICE;
    }
    s.d.id = dev;
    s.d.num_sms = sms;
    s.d.err = static_cast<unsigned int*>(err);
    s.ready = true;
  }
  if (!s.supported) return NVFP4_ERR_DEVICE;
  *out = s.d;
  return NVFP4_OK;
}

}  // namespace attn
}  // namespace nvfp4

using namespace nvfp4::attn;

extern "C" {

int nvfp4_qk_norm_rope(const nvfp4_heads* q, const nvfp4_heads* k, const nvfp4_heads* v,
                       int64_t tokens, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                       const void* q_weight, const void* k_weight, float eps,
                       const float* cos_sin, int64_t max_position, int32_t rotary_dim,
                       const int64_t* positions, const nvfp4_heads* q_out,
                       const nvfp4_heads* k_out, const nvfp4_kv_cache* cache,
                       const int64_t* slots, void* stream) {
  if (tokens < 0 || q_heads <= 0 || kv_heads <= 0 || rotary_dim < 0 || !(eps >= 0.f))
    return NVFP4_ERR_INVALID;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return NVFP4_ERR_SHAPE;
  if (rotary_dim % 16 != 0 || rotary_dim > head_dim || tokens > INT_MAX ||
      int64_t(q_heads) + 2 * int64_t(kv_heads) > 65535)
    return NVFP4_ERR_SHAPE;
  if (!q_weight || !k_weight || (k_out != nullptr) == (cache != nullptr)) return NVFP4_ERR_INVALID;
  if (misaligned(q_weight) || misaligned(k_weight)) return NVFP4_ERR_MISALIGNED;
  if (cache) {
    if (const int st = check_cache(cache)) return st;
    if (cache->kv_heads != kv_heads || cache->head_dim != head_dim) return NVFP4_ERR_SHAPE;
  } else if (v || slots) {
    return NVFP4_ERR_INVALID;
  }
  if (rotary_dim > 0) {
    if (max_position <= 0) return NVFP4_ERR_INVALID;
    if (tokens > 0 && (!cos_sin || !positions)) return NVFP4_ERR_INVALID;
    if (misaligned(cos_sin)) return NVFP4_ERR_MISALIGNED;
  }
  if (tokens == 0) return NVFP4_OK;
  for (const nvfp4_heads* h : {q, q_out})
    if (const int st = check_heads(h, tokens, q_heads)) return st;
  for (const nvfp4_heads* h : {k, cache ? v : k_out})
    if (const int st = check_heads(h, tokens, kv_heads)) return st;
  if (cache && !slots) return NVFP4_ERR_INVALID;
  Device d;
  if (const int st = device(&d)) return st;
  NormRope p{};
  p.q = heads(q, tokens, q_heads, head_dim);
  p.k = heads(k, tokens, kv_heads, head_dim);
  p.v = heads(v, tokens, kv_heads, head_dim);
  p.q_out = heads(q_out, tokens, q_heads, head_dim);
  p.k_out = heads(k_out, tokens, kv_heads, head_dim);
  p.q_weight = static_cast<const __nv_bfloat16*>(q_weight);
  p.k_weight = static_cast<const __nv_bfloat16*>(k_weight);
  p.cos_sin = cos_sin;
  p.positions = positions;
  p.slots = slots;
  p.cache = cache_of(cache);
  p.tokens = tokens;
  p.max_position = max_position;
  p.q_heads = q_heads;
  p.kv_heads = kv_heads;
  p.dim = head_dim;
  p.rot = rotary_dim;
  p.store = cache != nullptr;
  p.eps = eps;
  p.err = d.err;
  return run_norm_rope(p, d, static_cast<cudaStream_t>(stream));
}

int64_t nvfp4_paged_attention_workspace(int32_t head_dim) {
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return 0;
  Device d;
  if (device(&d) != NVFP4_OK) return 0;
  return attend_workspace(head_dim, d);
}

int nvfp4_paged_attention(const nvfp4_heads* q, int64_t tokens, int32_t q_heads,
                          const nvfp4_kv_cache* cache, const nvfp4_sequences* seqs, float scale,
                          const nvfp4_heads* out, float* lse, void* workspace,
                          int64_t workspace_bytes, void* stream) {
  if (const int st = check_cache(cache)) return st;
  if (const int st = check_groups(tokens, q_heads, cache->kv_heads)) return st;
  if (const int st = check_seqs(seqs, true)) return st;
  if (!(scale > 0.f && scale < INFINITY)) return NVFP4_ERR_INVALID;
  if (tokens == 0 || seqs->count == 0) return NVFP4_OK;
  if (const int st = check_heads(q, tokens, q_heads)) return st;
  if (const int st = check_heads(out, tokens, q_heads)) return st;
  if (!workspace) return NVFP4_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(workspace) & 31u) return NVFP4_ERR_MISALIGNED;
  Device d;
  if (const int st = device(&d)) return st;
  if (workspace_bytes < attend_workspace(cache->head_dim, d)) return NVFP4_ERR_TOO_LARGE;
  Attend p{};
  p.q = heads(q, tokens, q_heads, cache->head_dim);
  p.out = heads(out, tokens, q_heads, cache->head_dim);
  p.cache = cache_of(cache);
  p.seqs = seqs_of(seqs, tokens, cache->page_size);
  p.q_heads = q_heads;
  p.group = q_heads / cache->kv_heads;
  p.max_q_len = seqs->max_q_len;
  p.scale = scale;
  p.lse = lse;
  p.workspace = workspace;
  p.err = d.err;
  return run_attend(p, d, static_cast<cudaStream_t>(stream));
}

int nvfp4_attention_mass(const nvfp4_heads* q, int64_t tokens, int32_t q_heads,
                         const nvfp4_kv_cache* cache, const nvfp4_sequences* seqs, float scale,
                         const float* lse, const float* mass, float* out, int64_t room,
                         void* stream) {
  if (const int st = check_cache(cache)) return st;
  if (const int st = check_groups(tokens, q_heads, cache->kv_heads)) return st;
  if (const int st = check_seqs(seqs, true)) return st;
  if (room <= 0 || !(scale > 0.f && scale < INFINITY)) return NVFP4_ERR_INVALID;
  if (room > INT_MAX) return NVFP4_ERR_SHAPE;
  if (seqs->count == 0) return NVFP4_OK;
  if (!out) return NVFP4_ERR_INVALID;
  if (tokens > 0) {
    if (const int st = check_heads(q, tokens, q_heads)) return st;
    if (!lse) return NVFP4_ERR_INVALID;
  }
  Device d;
  if (const int st = device(&d)) return st;
  Mass p{};
  p.q = heads(q, tokens, q_heads, cache->head_dim);
  p.cache = cache_of(cache);
  p.seqs = seqs_of(seqs, tokens, cache->page_size);
  p.q_heads = q_heads;
  p.group = q_heads / cache->kv_heads;
  p.max_q_len = seqs->max_q_len;
  p.scale = scale;
  p.lse = lse;
  p.mass = mass;
  p.out = out;
  p.room = room;
  p.err = d.err;
  // a length beyond the mass's rows is out of range as well
  if (p.seqs.max_kv > room) p.seqs.max_kv = room;
  return run_mass(p, d, static_cast<cudaStream_t>(stream));
}

int nvfp4_cache_evict(const nvfp4_kv_cache* cache, const nvfp4_sequences* seqs,
                      const float* mass, int64_t room, int32_t keep, int32_t recent,
                      const nvfp4_kv_cache* to, const int32_t* to_table, int32_t to_width,
                      int32_t* index, float* new_mass, int32_t* new_lens, void* stream) {
  if (const int st = check_cache(cache)) return st;
  if (const int st = check_cache(to)) return st;
  if (const int st = check_seqs(seqs, false)) return st;
  if (to->type != cache->type) return NVFP4_ERR_INVALID;
  if (to->kv_heads != cache->kv_heads || to->head_dim != cache->head_dim) return NVFP4_ERR_SHAPE;
  if (room <= 0 || keep < 1 || recent < 0 || recent > keep || to_width <= 0)
    return NVFP4_ERR_INVALID;
  if (room > INT_MAX || int64_t(to_width) * to->page_size < keep) return NVFP4_ERR_SHAPE;
  if (seqs->count == 0) return NVFP4_OK;
  if (!mass || !to_table || !index || !new_mass || !new_lens) return NVFP4_ERR_INVALID;
  Device d;
  if (const int st = device(&d)) return st;
  Evict p{};
  p.from = cache_of(cache);
  p.to = cache_of(to);
  p.table = seqs->block_table;
  p.kv_lens = seqs->kv_lens;
  p.to_table = to_table;
  p.count = seqs->count;
  p.width = seqs->table_width;
  p.to_width = to_width;
  p.mass = mass;
  p.room = room;
  p.keep = keep;
  p.recent = recent;
  p.index = index;
  p.new_mass = new_mass;
  p.new_lens = new_lens;
  p.err = d.err;
  return run_evict(p, d, static_cast<cudaStream_t>(stream));
}

int nvfp4_attention_status(unsigned int* bits, int clear) {
  if (!bits) return NVFP4_ERR_INVALID;
  Device d;
  if (const int st = device(&d)) return st;
  if (cudaDeviceSynchronize() != cudaSuccess) {
    cudaGetLastError();
    return NVFP4_ERR_DEVICE;
  }
  read_attention_error_kernel<<<1, 1>>>(clear);
  if (cudaGetLastError() != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess ||
      cudaMemcpyFromSymbol(bits, g_attention_error_read, sizeof(*bits)) != cudaSuccess) {
    cudaGetLastError();
    return NVFP4_ERR_DEVICE;
  }
  return NVFP4_OK;
}

}  // extern "C"
