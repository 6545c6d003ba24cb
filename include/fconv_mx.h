/*
 * fconv_mx.h -- MXFP4 (microscaled 4-bit floating point) on AMD MI355X
 * (gfx950): quantisation, its inverse, and the product of two quantised
 * matrices with the float epilogue of fconv.h.
 *
 * Format (OCP microscaling, e2m1 elements, e8m0 scales, blocks of 32 along a
 * row).  For block b of a row, with m = max |x| over the block:
 *   e    = floor(log2 m) - 2, at least -127      (m = 0: e = -127)
 *   code = x * 2^-e rounded to the nearest of {0, .5, 1, 1.5, 2, 3, 4, 6} and
 *          their negatives, ties to the even code, magnitudes above 6 to 6
 *   the block stands for code * 2^e; its scale byte is e + 127.
 * A block that holds an infinity or a NaN has the scale byte 255 and stands
 * for 32 NaNs.  The last block of a row may be short (cols need not be a
 * multiple of 32).
 *
 * A quantised matrix lives in ONE device buffer of fconv_mx_bytes(rows, cols)
 * bytes, in the order in which the matrix cores read it: row tiles of 16
 * rows, k tiles of 128 columns.
 *   codes   byte ((r/16 * KT + c/128) * 1024 + (c%128/32 * 16 + r%16) * 16
 *           + c%32/2), the low half for even c;   KT = ceil(cols/128)
 *   scales  follow the codes: byte ((r/16 * KS + c/512) * 256
 *           + (c%128/32 * 16 + r%16) * 4 + c%512/128);  KS = ceil(cols/512)
 * Rows past the last one and columns past cols (to whole tiles) hold zeros.
 * fconv_mx_layout lays out plain row-major codes and scales, as checkpoints
 * hold them.
 *
 * Conventions as in fconv.h: status codes only; every check happens before
 * anything is enqueued; the caller owns every buffer; plans are host objects
 * that runs never modify.
 */
#ifndef FCONV_MX_H
#define FCONV_MX_H

#include "fconv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of the buffer that holds a quantised [rows, cols] matrix.  Errors:
 * FCONV_ERR_INVALID_ARG (rows < 0, cols < 1, bytes NULL),
 * FCONV_ERR_UNSUPPORTED (cols above 2^22). */
FCONV_API fconv_status fconv_mx_bytes(int32_t rows, int32_t cols, size_t* bytes);

/* x [rows, cols] (fconv_dtype FCONV_BF16 or FCONV_FP32; row r at element
 * r * ldx, ldx >= cols) into the buffer `mx`.  Rows of any alignment that the
 * element type has.  `mx` is 16-byte aligned and does not overlap x.  This one
 * and the two below: FCONV_ERR_INVALID_ARG (rows < 0, cols < 1, a stride below
 * cols or past the address space, NULL, an overlap), FCONV_ERR_UNSUPPORTED
 * (dtype, cols above 2^22, more than 2^23 - 8 tiles of 16 rows x 512 columns),
 * FCONV_ERR_MISALIGNED, FCONV_ERR_DEVICE; rows of 0 are a no-op. */
FCONV_API fconv_status fconv_mx_quantize(void* stream, const void* x, int64_t ldx, int32_t rows,
                                         int32_t cols, int32_t dtype, void* mx);

/* The values that `mx` stands for, into y [rows, cols] (row r at r * ldy),
 * exact in fp32; in bf16 exact too, except below its smallest normal, where
 * they round to nearest even.  Scale bytes 253 and 254, which quantisation
 * never makes, can stand for magnitudes of 2^128 and more: those become
 * infinities. */
FCONV_API fconv_status fconv_mx_dequantize(void* stream, const void* mx, int32_t rows,
                                           int32_t cols, int32_t dtype, void* y, int64_t ldy);

/* Row-major codes [rows, ceil(cols/32)*16] (two to a byte, low half first)
 * and scales [rows, ceil(cols/32)] into the buffer `mx`.  Codes past cols are
 * taken as zero.  Codes 4-byte aligned. */
FCONV_API fconv_status fconv_mx_layout(void* stream, const void* codes, const void* scales,
                                       int32_t rows, int32_t cols, void* mx);

/* y[m, n] = act( sum_k X[m, k] * W[n, k]  + bias[n] ), X and W quantised
 * matrices; sums in fp32 by the matrix cores.  dtype: the type of y and of an
 * unquantised x (FCONV_BF16 or FCONV_FP32).  ops: [BIAS], [RELU | LEAKY_RELU |
 * CLIPPED_RELU | CLAMP], each optional, this order (fconv_op of fconv.h). */
typedef struct {
  int32_t M, N, K;
  int32_t dtype;
  int32_t n_ops;
  int32_t ops[FCONV_MAX_OPS];
  uint32_t flags; /* 0 */
} fconv_mx_desc;

typedef struct fconv_mx_plan_s* fconv_mx_plan;

/* Per-run arguments.
 *   x      device, [M, K] of the plan dtype, row m at element m * ldx; the run
 *          quantises it (by the rule above) on the way.  Or NULL, and
 *   x_mx   device, the quantised [M, K] matrix
 *   w_mx   device, the quantised [N, K] matrix
 *   bias   device, fp32 [N] (needed iff BIAS op)
 *   y      device, [M, N] of the plan dtype, row m at element m * ldy
 *   workspace / workspace_bytes: device scratch of at least
 *          fconv_mx_plan_workspace_size bytes (may be NULL when that is 0)
 *   activ_alpha, activ_beta: as in fconv_args
 * x, y and bias have their element type's alignment; x_mx, w_mx and the
 * workspace are 16-byte aligned.  y overlaps nothing else. */
typedef struct {
  const void* x;
  int64_t ldx;
  const void* x_mx;
  const void* w_mx;
  const float* bias;
  void* y;
  int64_t ldy;
  void* workspace;
  size_t workspace_bytes;
  float activ_alpha;
  float activ_beta;
} fconv_mx_args;

/* Host only.  M may be 0 (every run is then a no-op).  Errors:
 * FCONV_ERR_INVALID_ARG (NULL, M < 0, N < 1, K < 1),
 * FCONV_ERR_UNSUPPORTED (dtype, ops, flags, K above 2^22, or more than 2^23 - 8 output
 * tiles of 128 x 128 or tiles of 16 rows x 512 columns of x). */
FCONV_API fconv_status fconv_mx_plan_create(const fconv_mx_desc* desc, fconv_mx_plan* out);
FCONV_API fconv_status fconv_mx_plan_workspace_size(fconv_mx_plan plan, size_t* bytes);

/* Enqueues the product on `stream`.  Errors: FCONV_ERR_INVALID_ARG (NULL plan,
 * args or needed pointer, both or neither of x and x_mx, ldx < K, ldy < N, an
 * overlap, activation arguments as in fconv_plan_run), FCONV_ERR_MISALIGNED,
 * FCONV_ERR_WORKSPACE, FCONV_ERR_DEVICE. */
FCONV_API fconv_status fconv_mx_plan_run(fconv_mx_plan plan, void* stream,
                                         const fconv_mx_args* args);

/* Name of the product kernel that a run launches, given x or given x_mx; NULL
 * for a NULL plan. */
FCONV_API const char* fconv_mx_plan_kernel_name(fconv_mx_plan plan);
FCONV_API const char* fconv_mx_plan_quantized_kernel_name(fconv_mx_plan plan);
FCONV_API fconv_status fconv_mx_plan_destroy(fconv_mx_plan plan);

#ifdef __cplusplus
}
#endif

#endif /* FCONV_MX_H */
