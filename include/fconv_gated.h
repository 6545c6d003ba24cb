/*
 * fconv_gated.h -- gated feed-forward layer on AMD MI355X (gfx950) and its
 * gradients.
 *
 *   g[t, f] = sum_d x[t, d] w[f, d]            t < T, f < F, d < D
 *   u[t, f] = sum_d x[t, d] w[F + f, d]
 *   y[t, f] = act(g[t, f]) u[t, f]
 *   dg = dy u act'(g)      du = dy act(g)
 *   dx[t, d] = sum_f dg[t, f] w[f, d] + du[t, f] w[F + f, d]
 *   dw[f, d] = sum_t dg[t, f] x[t, d]          dw[F + f, d] = sum_t du[t, f] x[t, d]
 *
 *   FCONV_ACT_SILU       act(g) = g / (1 + exp(-g))
 *   FCONV_ACT_GELU       act(g) = g / 2 (1 + erf(g / sqrt 2))
 *   FCONV_ACT_GELU_TANH  act(g) = g / 2 (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3)))
 *   FCONV_ACT_RELU       act(g) = max(g, 0), act'(0) = 0
 *
 * Both projections, the activation and the product are one kernel.  dtype is
 * the type of x, w, y, dy, dx and dw (FCONV_BF16 or FCONV_FP32); products are
 * summed in fp32 by the matrix cores, activations are fp32.  For the gradients
 * the forward pass can keep g and u, in fp32; with FCONV_BF16, dg and du are
 * rounded to bf16 before they are multiplied.  All roundings are to nearest
 * even.  Results do not depend on the order in which workgroups run.
 *
 * With FCONV_BF16 and D a multiple of 8, tiles copy rows of x and w that lie on 16
 * bytes (address and row stride).  With others forward, and with such a w dx, takes
 * the general kernel, which takes two to six times as long where there are many
 * tokens; dw copies x to such rows first.  Rows of bf16 that begin or end inside a
 * dword may be read with the rest of it, also before the first element and behind the
 * last one; nothing depends on that.
 *
 * Conventions as in fconv.h: status codes only; every check happens before
 * anything is enqueued; the caller owns every buffer; plans are host objects
 * that runs never modify.
 */
#ifndef FCONV_GATED_H
#define FCONV_GATED_H

#include "fconv.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { FCONV_ACT_SILU, FCONV_ACT_GELU, FCONV_ACT_GELU_TANH, FCONV_ACT_RELU };

typedef struct {
  int32_t T, D, F;
  int32_t dtype;
  int32_t activation;
  uint32_t flags; /* 0 */
} fconv_gated_desc;

typedef struct fconv_gated_plan_s* fconv_gated_plan;

/* Device pointers of a run; rows are dense, row r at element r * ld.
 *   x [T, D], w [2 F, D]: the gate's rows, then the other projection's
 *   forward:   writes y [T, F], and kept (fconv_gated_plan_kept_size bytes,
 *              16-byte aligned) unless that is NULL
 *   backward:  reads kept (of the forward pass on the same x and w) and
 *              dy [T, F]; writes dx [T, D] and dw [2 F, D], either may be NULL
 *   workspace  at least fconv_gated_plan_*_workspace_size bytes, 16-byte aligned
 *              (may be NULL where that is 0)
 * Every other pointer has its element type's alignment.  What is written
 * overlaps nothing else. */
typedef struct {
  const void* x;
  int64_t ldx;
  const void* w;
  int64_t ldw;
  void* y;
  int64_t ldy;
  void* kept;
  const void* dy;
  int64_t lddy;
  void* dx;
  int64_t lddx;
  void* dw;
  int64_t lddw;
  void* workspace;
  size_t workspace_bytes;
} fconv_gated_args;

/* Host only.  T may be 0 (backward then writes dw = 0).  Errors:
 * FCONV_ERR_INVALID_ARG (NULL, T < 0, D < 1, F < 1), FCONV_ERR_UNSUPPORTED
 * (dtype, activation, flags, D or F above 2^20, T above 4194240, T * D, 2 T * F or
 * 2 F * D above 2^33, more than 2^28 tiles of 64 x 64 values of [g u] or dx). */
FCONV_API fconv_status fconv_gated_plan_create(const fconv_gated_desc* desc, fconv_gated_plan* out);
FCONV_API fconv_status fconv_gated_plan_kept_size(fconv_gated_plan plan, size_t* bytes);
FCONV_API fconv_status fconv_gated_plan_forward_workspace_size(fconv_gated_plan plan, size_t* bytes);
FCONV_API fconv_status fconv_gated_plan_backward_workspace_size(fconv_gated_plan plan, size_t* bytes);

/* Enqueue on `stream`.  Errors: FCONV_ERR_INVALID_ARG (NULL plan, args or
 * needed pointer, a row stride below the row's length or above 2^21, an overlap,
 * no output), FCONV_ERR_MISALIGNED, FCONV_ERR_WORKSPACE, FCONV_ERR_DEVICE. */
FCONV_API fconv_status fconv_gated_plan_forward(fconv_gated_plan plan, void* stream, const fconv_gated_args* args);
FCONV_API fconv_status fconv_gated_plan_backward(fconv_gated_plan plan, void* stream, const fconv_gated_args* args);

/* The products of a plan.  Name of the kernel, "_packed" where rows are copied
 * to 16-byte boundaries first, of a run whose operands are aligned as torch
 * allocates them with dense rows; NULL for a NULL plan, another product, or a
 * plan of no tokens. */
enum { FCONV_GATED_FORWARD, FCONV_GATED_DX, FCONV_GATED_DW };
FCONV_API const char* fconv_gated_plan_kernel_name(fconv_gated_plan plan, int32_t product);
/* Ranges of the product's sum, whose partial sums are joined (forward: 1). */
FCONV_API fconv_status fconv_gated_plan_ranges(fconv_gated_plan plan, int32_t product, int32_t* ranges);

FCONV_API fconv_status fconv_gated_plan_destroy(fconv_gated_plan plan);

#ifdef __cplusplus
}
#endif

#endif /* FCONV_GATED_H */
