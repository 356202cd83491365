/*
 * nvfp4_attention.h -- C ABI of the attention block's operators in
 * libnvfp4_linear.so (GB300, sm_103a): what a full-attention layer does
 * between its stacked q/k/v projection and its output projection.
 *
 *   nvfp4_qk_norm_rope     RMS norm of every query and key head and the
 *                          position rotation, in one pass, with the key and
 *                          value rows stored in a paged cache
 *   nvfp4_paged_attention  softmax attention of new tokens over that cache
 *   nvfp4_attention_mass   the attention weight that each cached key received
 *   nvfp4_cache_evict      the keys with the most weight kept, and their rows
 *                          moved together
 *
 * Conventions are those of nvfp4_linear.h: every buffer belongs to the
 * caller, nothing is allocated, calls are asynchronous on `stream`, validate
 * on the host before launching anything, may be captured into a CUDA graph,
 * and return an NVFP4_* status.  Kernels are launched with programmatic
 * dependent launch and read and write memory only after the kernel before
 * them in the stream has completed.
 *
 * Values that only the device holds (lengths, page numbers, slots,
 * positions) are checked by the kernels: one that is out of range sets
 * NVFP4_ATTENTION_BAD_INDEX in the device's attention error word, readable
 * with nvfp4_attention_status(), and the access it would have made is left
 * out.  The results of a call that set the bit are unspecified for the
 * sequence or token concerned.  A pipeline wait that times out sets
 * NVFP4_ATTENTION_TIMEOUT instead of faulting.
 *
 * Every integer tensor is dense (unit stride); heads and cache rows may be
 * strided views, their last dimension dense.
 */
#ifndef NVFP4_ATTENTION_H
#define NVFP4_ATTENTION_H

#include <stdint.h>

#include "nvfp4_linear.h"

#ifdef __cplusplus
extern "C" {
#endif

/* bf16 [tokens, heads, head_dim] on the device; strides in elements, each
 * positive and a multiple of 8 (that of a dimension of one is not read); data
 * 16-byte aligned. */
typedef struct nvfp4_heads {
  void* data;
  int64_t token_stride;
  int64_t head_stride;
} nvfp4_heads;

#define NVFP4_CACHE_BF16 0
#define NVFP4_CACHE_E4M3 1

/* A paged key/value cache.  k and v are [num_pages, page_size, kv_heads,
 * head_dim] on the device, 16-byte aligned, with the strides (in elements)
 * of the first three dimensions given; every stride is a multiple of 16
 * bytes.  head_dim is 64, 128 or 256; page_size is a multiple of 16.
 * An E4M3 row stands for its codes times its head's scale: k_scale and
 * v_scale are device fp32 [kv_heads], positive, or NULL for 1 (always NULL
 * with BF16). */
typedef struct nvfp4_kv_cache {
  void* k;
  void* v;
  int64_t num_pages;
  int64_t k_stride[3]; /* page, slot, head */
  int64_t v_stride[3];
  const float* k_scale;
  const float* v_scale;
  int32_t type; /* NVFP4_CACHE_* */
  int32_t page_size;
  int32_t kv_heads;
  int32_t head_dim;
} nvfp4_kv_cache;

/* The most sequences of one attention call.  (Its work, counted in 16 keys for
 * each few tokens and each key/value head of the longest sequence that the
 * block table has room for, has to stay below 2^32 as well: NVFP4_ERR_SHAPE.) */
#define NVFP4_ATTENTION_MAX_SEQUENCES 8192

/* A batch of sequences over a cache.  Sequence s holds its first kv_lens[s]
 * keys in the pages block_table[s][0..], key j in slot j % page_size of page
 * block_table[s][j / page_size].  Its new tokens are rows q_starts[s] to
 * q_starts[s + 1] - 1 of the token dimension; they are its last keys, so the
 * i-th of n new tokens sees keys 0 .. kv_lens[s] - n + i (none when that is
 * negative). */
typedef struct nvfp4_sequences {
  const int32_t* block_table; /* device [count, table_width] */
  const int32_t* kv_lens;     /* device [count], 0 <= kv_lens <= table_width * page_size */
  const int32_t* q_starts;    /* device [count + 1], ascending within [0, tokens] */
  int32_t count;
  int32_t table_width;
  int32_t max_q_len; /* the longest sequence's new tokens: chooses the kernel, not the result */
} nvfp4_sequences;

#define NVFP4_ATTENTION_TIMEOUT 1u
#define NVFP4_ATTENTION_BAD_INDEX 2u

/* For every token t and head: y = x * rsqrt(mean(x^2) + eps) * weight, then
 * for i < rotary_dim / 2 the pair (y[i], y[i + rotary_dim / 2]) becomes
 * (a cos - b sin, b cos + a sin) with cos = cos_sin[positions[t]][i] and
 * sin = cos_sin[positions[t]][rotary_dim / 2 + i]; the other dimensions stay.
 * Computed in fp32, rounded once (to nearest even) to the output's type.
 *   q, k, v      bf16 heads; q_heads, kv_heads, kv_heads of them.
 *   q_weight, k_weight   bf16 [head_dim].
 *   cos_sin      fp32 [max_position, rotary_dim]; rotary_dim a multiple of
 *                16, 0 <= rotary_dim <= head_dim (0: no rotation).
 *   positions    int64 [tokens].
 *   q_out        bf16 heads; may be q itself.
 *   k_out        bf16 heads (may be k itself), or NULL with a cache.
 *   cache, slots With a cache, token t's key and value rows go to slot
 *                slots[t] % page_size of page slots[t] / page_size (int64
 *                [tokens]; -1: the token's rows are not stored).  An E4M3
 *                cache takes e4m3(y / scale), saturating at 448.  Slots must
 *                be distinct.  v and slots are NULL without a cache.
 * tokens == 0 is a no-op. */
int nvfp4_qk_norm_rope(const nvfp4_heads* q, const nvfp4_heads* k, const nvfp4_heads* v,
                       int64_t tokens, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                       const void* q_weight, const void* k_weight, float eps,
                       const float* cos_sin, int64_t max_position, int32_t rotary_dim,
                       const int64_t* positions, const nvfp4_heads* q_out,
                       const nvfp4_heads* k_out, const nvfp4_kv_cache* cache,
                       const int64_t* slots, void* stream);

/* out[t, h] = sum_j p_j v_j with p the softmax of scale * q[t, h] . k_j over
 * the keys that t sees, the query heads sharing key/value heads in equal
 * consecutive groups; lse[t, h] = log sum_j exp(scale * q . k_j).  A token
 * that sees no key gets 0 and -inf.  Rows of the cache at or past a
 * sequence's length are never used, whatever they hold.  Scores, maxima and
 * sums are fp32; the weights are rounded to the cache's operand type (bf16,
 * or f16 over an E4M3 cache, in which weights down to 2^-36 of a row's largest
 * count) before they meet the values; out is rounded once to bf16.
 *   scale        positive and finite.
 *   q, out       bf16 [tokens, q_heads, head_dim] heads; q_heads a multiple
 *                of cache->kv_heads, at most 128 times it.
 *   lse          fp32 [tokens, q_heads], or NULL.
 *   workspace    32-byte aligned device memory of at least
 *                nvfp4_paged_attention_workspace() bytes; its contents need
 *                no set-up and mean nothing between calls, but calls that
 *                may overlap on the GPU need one each.
 * tokens outside every sequence are left alone, and so are all tokens where
 * q_starts descends anywhere (NVFP4_ATTENTION_BAD_INDEX). */
int nvfp4_paged_attention(const nvfp4_heads* q, int64_t tokens, int32_t q_heads,
                          const nvfp4_kv_cache* cache, const nvfp4_sequences* seqs, float scale,
                          const nvfp4_heads* out, float* lse, void* workspace,
                          int64_t workspace_bytes, void* stream);

/* Bytes of workspace that a call with this head_dim needs on the current
 * device (the same for every batch); 0 if head_dim is not supported. */
int64_t nvfp4_paged_attention_workspace(int32_t head_dim);

/* out[s, h, j] = mass[s, h, j] + sum over the tokens t of sequence s that see
 * key j and the query heads g of group h of exp(scale * q[t, g] . k_j -
 * lse[t, g]), for j < kv_lens[s]; 0 for the other j < room.  lse is what
 * nvfp4_paged_attention wrote for the same q, cache and scale; where it is
 * -inf the token's head adds nothing.  mass and out
 * are fp32 [count, kv_heads, room], room >= the longest kv_lens; mass may be
 * NULL (nothing received before) or out itself.  Sums in fp32 in a fixed
 * order. */
int nvfp4_attention_mass(const nvfp4_heads* q, int64_t tokens, int32_t q_heads,
                         const nvfp4_kv_cache* cache, const nvfp4_sequences* seqs, float scale,
                         const float* lse, const float* mass, float* out, int64_t room,
                         void* stream);

/* Cut every sequence to at most `keep` keys.  With n = kv_lens[s], m =
 * min(n, keep) and e = min(recent, m), each key/value head keeps the newest e
 * keys and, of the others, the m - e with the largest mass (the lower index
 * first among equals; NaN above every number), in their order in the
 * sequence.  Key r of those kept:
 *   index[s, h, r] = its place in the source, r < m; -1 for m <= r < keep
 *   new_mass[s, h, r] = its mass; 0 for m <= r < keep
 *   its key and value rows are copied to slot r % page_size of page
 *   to_table[s][r / page_size] of `to`
 * and new_lens[s] = m.  `to` has the source's type, kv_heads and head_dim
 * (its own page size, strides and scales: an E4M3 row's codes are taken over
 * where the head's scales are equal, else its values are rounded once to the
 * new scale, saturating at 448) and its pages named in to_table are none of
 * those the sequences still hold.
 *   mass         fp32 [count, kv_heads, room].
 *   seqs         block_table, kv_lens, count and table_width are read.
 *   to_table     int32 [count, to_width], to_width * to->page_size >= keep.
 *   index        int32 [count, kv_heads, keep]; new_mass fp32, the same;
 *   new_lens     int32 [count].
 * 0 <= recent <= keep, keep >= 1. */
int nvfp4_cache_evict(const nvfp4_kv_cache* cache, const nvfp4_sequences* seqs,
                      const float* mass, int64_t room, int32_t keep, int32_t recent,
                      const nvfp4_kv_cache* to, const int32_t* to_table, int32_t to_width,
                      int32_t* index, float* new_mass, int32_t* new_lens, void* stream);

/* Read the current device's attention error word (OR of the
 * NVFP4_ATTENTION_* bits set since it was last cleared) into *bits; clear it
 * if `clear` is non-zero.  Synchronises with the whole device first. */
int nvfp4_attention_status(unsigned int* bits, int clear);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_ATTENTION_H */
