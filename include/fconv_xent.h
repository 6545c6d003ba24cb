/*
 * fconv_xent.h -- softmax cross entropy of a linear output layer on AMD
 * MI355X (gfx950), and its gradient, without keeping the logits.
 *
 *   z[t, v] = sum_d h[t, d] w[v, d]                      t < T, v < V, d < D
 *   lse[t]  = log sum_v exp z[t, v]
 *   loss[t] = lse[t] - z[t, target[t]]
 *   g[t, v] = dloss[t] (exp(z[t, v] - lse[t]) - [v = target[t]])
 *   dh[t, d] = sum_v g[t, v] w[v, d]      dw[v, d] = sum_t g[t, v] h[t, d]
 *
 * A token whose target is ignore_index has loss 0 and no gradient, whatever
 * its h and dloss; its lse is computed all the same.  A target that is
 * neither that nor in [0, V) gives a NaN loss and NaN gradients.  An lse is
 * +inf where a logit is, -inf where all are, NaN where one is.  A dloss that is
 * infinite or NaN makes all of dw NaN, and dh of its token.
 *
 * dtype is the type of h, w, dh and dw (FCONV_BF16 or FCONV_FP32); products
 * are summed in fp32 by the matrix cores, loss, lse and dloss are fp32.  With
 * FCONV_BF16, softmax - onehot and h scaled by dloss / max |dloss| are rounded
 * to bf16 (to nearest even) before they are multiplied.
 * Results do not depend on the order in which workgroups run.
 *
 * Conventions as in fconv.h: status codes only; every check happens before
 * anything is enqueued; the caller owns every buffer; plans are host objects
 * that runs never modify.
 */
#ifndef FCONV_XENT_H
#define FCONV_XENT_H

#include "fconv.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  int32_t T, D, V;
  int32_t dtype;
  int64_t ignore_index;
  uint32_t flags; /* 0 */
} fconv_xent_desc;

typedef struct fconv_xent_plan_s* fconv_xent_plan;

/* Device pointers of a run; rows are dense, row r at element r * ld.
 *   h [T, D], w [V, D], target int64 [T]
 *   forward:   writes loss [T], lse [T]
 *   backward:  reads lse [T] (of the forward pass on the same h and w) and
 *              dloss [T]; writes dh [T, D] and dw [V, D], either may be NULL
 *   workspace  at least fconv_xent_plan_*_workspace_size bytes, 16-byte aligned
 * Every other pointer has its element type's alignment.  What is written
 * overlaps nothing else. */
typedef struct {
  const void* h;
  int64_t ldh;
  const void* w;
  int64_t ldw;
  const int64_t* target;
  float* loss;
  float* lse;
  const float* dloss;
  void* dh;
  int64_t lddh;
  void* dw;
  int64_t lddw;
  void* workspace;
  size_t workspace_bytes;
} fconv_xent_args;

/* Host only.  T may be 0 (backward then writes dw = 0).  Errors:
 * FCONV_ERR_INVALID_ARG (NULL, T < 0, D < 1, V < 1), FCONV_ERR_UNSUPPORTED
 * (dtype, flags, D above 2^20, V above 2^24, T above 4194240, T * D above 2^33,
 * or more than 2^28 tiles of 64 x 64 logits: T * V above about 2^40). */
FCONV_API fconv_status fconv_xent_plan_create(const fconv_xent_desc* desc, fconv_xent_plan* out);
FCONV_API fconv_status fconv_xent_plan_forward_workspace_size(fconv_xent_plan plan, size_t* bytes);
FCONV_API fconv_status fconv_xent_plan_backward_workspace_size(fconv_xent_plan plan, size_t* bytes);

/* Enqueue on `stream`.  Errors: FCONV_ERR_INVALID_ARG (NULL plan, args or
 * needed pointer, a row stride below D or above 2^21, an overlap, no output),
 * FCONV_ERR_MISALIGNED, FCONV_ERR_WORKSPACE, FCONV_ERR_DEVICE. */
FCONV_API fconv_status fconv_xent_plan_forward(fconv_xent_plan plan, void* stream,
                                               const fconv_xent_args* args);
FCONV_API fconv_status fconv_xent_plan_backward(fconv_xent_plan plan, void* stream,
                                                const fconv_xent_args* args);

/* The products of a plan: the forward pass's logits, the backward pass's (which
 * leave it as softmax - onehot), dh and dw.  Name of the kernel, "_packed" where
 * rows of w are copied to 16-byte boundaries first, of a run whose operands are
 * aligned as torch allocates them with dense rows; NULL for a NULL plan, another
 * product, or a plan of no tokens. */
enum { FCONV_XENT_LOGITS, FCONV_XENT_GRAD, FCONV_XENT_DH, FCONV_XENT_DW };
FCONV_API const char* fconv_xent_plan_kernel_name(fconv_xent_plan plan, int32_t product);
/* Pieces of the vocabulary that the product is taken in, and ranges of its sum. */
FCONV_API fconv_status fconv_xent_plan_division(fconv_xent_plan plan, int32_t product, int32_t* pieces,
                                                int32_t* ranges);

FCONV_API fconv_status fconv_xent_plan_destroy(fconv_xent_plan plan);

#ifdef __cplusplus
}
#endif

#endif /* FCONV_XENT_H */
