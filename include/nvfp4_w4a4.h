/*
 * nvfp4_w4a4.h -- C ABI of the NVFP4 x NVFP4 operators in libnvfp4_linear.so
 * (GB300, sm_103a): layers whose activations are NVFP4 as well as their
 * weights (the W4A4 form of the compressed-tensors checkpoints, whose
 * input_global_scale is the activations' global scale).
 *
 *   nvfp4_add_rms_norm      the residual's addition and the RMS norm of each
 *                           row, into bf16 or into NVFP4 rows
 *   nvfp4_quantize_rows     bf16 rows into NVFP4 rows
 *   nvfp4_linear_w4a4       NVFP4 rows times an NVFP4 weight into bf16; of a
 *                           gate/up pair silu(gate) * up, into bf16 or into
 *                           NVFP4 rows for the next product
 *   nvfp4_w4a4_scale_layout a weight's scales in the order the product reads
 *
 * Conventions are those of nvfp4_linear.h: every buffer belongs to the
 * caller, nothing is allocated, calls are asynchronous on `stream`, validate
 * on the host before launching anything, may be captured into a CUDA graph,
 * and return an NVFP4_* status.  Kernels are launched with programmatic
 * dependent launch; nvfp4_linear_w4a4 reads the weight's codes and scales
 * before the kernel ahead of it in the stream has completed, so that kernel
 * must not write them; and where it is a call of this library too, which may
 * itself have started early, nor may the call ahead of that one, and so on up
 * to a kernel of another kind, a copy or a wait on the host.
 * nvfp4_w4a4_scale_layout is the exception: it lets nothing start before its
 * own end and may stand anywhere ahead, directly as well.  Everything else is
 * read and written after the kernel ahead.
 *
 * NVFP4 rows [M, K] stand for  e2m1(code[m,k]) * e4m3(scale[m, k/16]) /
 * global_scale.  Codes: uint8 [M, K/2], the low nibble holding the even k.
 * Scales, of rows and of weights alike: blocks of 128 rows x 64 k, 512 bytes
 * each, [ceil(rows/128)][K/64][512], where the scale of row r and of 16-block
 * j of a block lies at byte (r % 32) * 16 + (r / 32) * 4 + j: the order that
 * the tensor core takes them in.  A rows' buffer has room for whole blocks;
 * places of rows beyond M are never written and may hold anything.
 *
 * Quantisation, in fp32 with round-to-nearest-even, per 16 values v of a row:
 *   scale = e4m3((max|v| * global_scale) / 6), saturating at 448;
 *   code = e2m1((v * global_scale) / scale), saturating at 6; the codes are
 *   zeros where the scale rounds to 0 (a zero's sign is not kept);
 *   where max|v| * global_scale is not finite the scale is NaN and the codes
 *   are zeros: every product of that row is NaN.
 * Scales are never negative; rows from elsewhere must not hold negative ones
 * either (the product takes scales as unsigned).
 */
#ifndef NVFP4_W4A4_H
#define NVFP4_W4A4_H

#include <stdint.h>

#include "nvfp4_linear.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bits of the operators' device error word (nvfp4_w4a4_status). */
#define NVFP4_W4A4_TIMEOUT 1u       /* a pipeline wait gave up */

/* Widest row that nvfp4_add_rms_norm takes. */
#define NVFP4_W4A4_MAX_NORM 32768

/* NVFP4 rows on the device; codes and scales 16-byte aligned. */
typedef struct nvfp4_rows {
  uint8_t* codes;
  uint8_t* scales;
  float global_scale;             /* positive and finite */
} nvfp4_rows;

/* Bytes of the scales of `rows` rows of K: ceil(rows/128) * 128 * K/16 (0
 * where rows < 0 or K is not a positive multiple of 256). */
int64_t nvfp4_w4a4_scale_bytes(int64_t rows, int64_t K);

/* The scales of a weight, w_scale[N, K/16] as nvfp4_linear.h has them, in the
 * order above (blocked, 16-byte aligned, nvfp4_w4a4_scale_bytes(N, K) bytes).
 * *refused (device) is set to 1 where a scale is below zero or NaN, which the
 * product has no meaning for (its scales are unsigned), and left alone
 * otherwise; -0 becomes 0.  blocked overlaps nothing.  N % 128 == 0, K % 256
 * == 0. */
int nvfp4_w4a4_scale_layout(const uint8_t* w_scale, int64_t N, int64_t K, uint8_t* blocked,
                            unsigned int* refused, void* stream);

/* out = x (bf16 [M, K], row_stride elements from row to row, a multiple of 8;
 * 16-byte aligned) in NVFP4 with out->global_scale, apart from x.  K % 256
 * == 0. */
int nvfp4_quantize_rows(const void* x, int64_t row_stride, int64_t M, int64_t K,
                        const nvfp4_rows* out, void* stream);

/* r = x + residual (rounded to bf16; x itself where residual is NULL), into
 * residual_out (may be NULL), and
 *   y = r * rsqrt(mean(r^2) + eps) * weight      (fp32, rounded once)
 * (the mean: the fp32 sum over K, rounded once; a finite row whose squares pass
 * fp32's range, magnitudes from 1.8e19 / sqrt(K) on, gives zeros)
 * into y (bf16) or, where `rows` is given, into NVFP4 rows; exactly one of the
 * two is.  x, residual, residual_out, y: bf16 [M, K], 16-byte aligned, strides
 * in elements, multiples of 8; weight: bf16 [K].  An output may be one of the
 * inputs (same pointer and stride); otherwise outputs overlap neither inputs
 * nor one another (NVFP4_ERR_INVALID).
 * K % 16 == 0 (into NVFP4 rows K % 256 == 0), K <= NVFP4_W4A4_MAX_NORM. */
int nvfp4_add_rms_norm(const void* x, int64_t x_stride, const void* residual,
                       int64_t residual_stride, const void* weight, float eps, int64_t M,
                       int64_t K, void* residual_out, int64_t residual_out_stride, void* y,
                       int64_t y_stride, const nvfp4_rows* rows, void* stream);

/* An NVFP4 weight [N, K], N % 128 == 0, K % 256 == 0, stacked from up to 8
 * segments with global scales of their own (host arrays; segment_rows[i] rows
 * each, multiples of 16, summing to N).  scales: as nvfp4_w4a4_scale_layout
 * leaves them. */
typedef struct nvfp4_weight {
  const uint8_t* codes;           /* w_packed of nvfp4_linear.h, 16-byte aligned */
  const uint8_t* scales;
  int64_t N, K;
  int32_t segments;
  float global_scale[8];          /* positive and finite */
  int64_t segment_rows[8];
} nvfp4_weight;

/* y[M, N] bf16 = a . w^T.  With `swiglu` the weight holds gate rows [0, N/2)
 * and up rows [N/2, N) (N % 256 == 0) and the result [M, N/2] is
 * silu(g) * u, silu(g) = g / (1 + exp(-g)) in fp32, from the products
 * before any rounding; into y, or into NVFP4 rows `out` where that is given
 * (N % 512 == 0).  y: row-major, contiguous, 16-byte aligned.  Outputs must
 * not overlap inputs (NVFP4_ERR_INVALID).  The products of the global scales
 * must have reciprocals in fp32's normal range (NVFP4_ERR_INVALID).  Sums are
 * fp32, in an order that depends on the sizes (M rounded up to 8 among them)
 * and nothing else. */
int nvfp4_linear_w4a4(const nvfp4_rows* a, int64_t M, const nvfp4_weight* w, int32_t swiglu,
                      void* y, const nvfp4_rows* out, void* stream);

/* The current device's error word of these operators into *bits; cleared if
 * `clear` is non-zero.  Synchronises with the whole device.  */
int nvfp4_w4a4_status(unsigned int* bits, int clear);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_W4A4_H */
