/*
 * fconv_embed.h -- embedding lookup on AMD MI355X (gfx950) and its gradient.
 *
 *   y[t, d]  = scale w[token[t], d]                      t < T, d < D
 *   dw[v, d] = scale sum over t with token[t] = v of dy[t, d]      v < V
 *
 * A token that is ignore_index has y = 0 and no gradient, whatever its dy
 * holds.  A token that is neither that nor in [0, V) has a row of NaN, and no
 * gradient.  Rows of dw without a token are zeros; with FCONV_EMBED_ADD the
 * gradient is added to what dw holds, and rows without a token stay as they are
 * (a table that an output layer shares, whose gradient is there already).
 *
 * dtype is the type of w, y, dy and dw (FCONV_BF16 or FCONV_FP32).  scale is
 * fp32; with scale 1 rows are copied bit by bit.  The products and sums are
 * fp32, rounded once (to nearest even).  A row's sum is taken in an order that
 * the tokens alone determine: results do not depend on how workgroups run.
 *
 * Conventions as in fconv.h: status codes only; every check happens before
 * anything is enqueued; the caller owns every buffer; plans are host objects
 * that runs never modify.
 */
#ifndef FCONV_EMBED_H
#define FCONV_EMBED_H

#include "fconv.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  int32_t T, D, V;
  int32_t dtype;
  int64_t ignore_index;
  float scale;
  uint32_t flags; /* 0 */
} fconv_embed_desc;

typedef struct fconv_embed_plan_s* fconv_embed_plan;

enum { FCONV_EMBED_ADD = 1 };

/* Device pointers of a run; rows are dense, row r at element r * ld.
 *   token int64 [T]
 *   forward:   reads w [V, D], writes y [T, D]
 *   backward:  reads dy [T, D], writes dw [V, D]; run_flags 0 or FCONV_EMBED_ADD
 *   workspace  (backward) at least fconv_embed_plan_workspace_size bytes,
 *              16-byte aligned (may be NULL where that is 0)
 * Every other pointer has its element type's alignment.  What is written
 * overlaps nothing else. */
typedef struct {
  const int64_t* token;
  const void* w;
  int64_t ldw;
  void* y;
  int64_t ldy;
  const void* dy;
  int64_t lddy;
  void* dw;
  int64_t lddw;
  uint32_t run_flags;
  void* workspace;
  size_t workspace_bytes;
} fconv_embed_args;

/* Host only.  T may be 0 (backward then writes dw = 0, or adds nothing).
 * Errors: FCONV_ERR_INVALID_ARG (NULL, T < 0, D < 1, V < 1, a scale that is not
 * finite), FCONV_ERR_UNSUPPORTED (dtype, flags, D above 2^20, V above 2^24, T above
 * 4194240, T * D or V * D above 2^33). */
FCONV_API fconv_status fconv_embed_plan_create(const fconv_embed_desc* desc, fconv_embed_plan* out);
FCONV_API fconv_status fconv_embed_plan_workspace_size(fconv_embed_plan plan, size_t* bytes);

/* Enqueue on `stream`.  Errors: FCONV_ERR_INVALID_ARG (NULL plan, args or
 * needed pointer, a row stride below D or above 2^21, an overlap, another flag),
 * FCONV_ERR_MISALIGNED, FCONV_ERR_WORKSPACE, FCONV_ERR_DEVICE. */
FCONV_API fconv_status fconv_embed_plan_forward(fconv_embed_plan plan, void* stream, const fconv_embed_args* args);
FCONV_API fconv_status fconv_embed_plan_backward(fconv_embed_plan plan, void* stream, const fconv_embed_args* args);

FCONV_API fconv_status fconv_embed_plan_destroy(fconv_embed_plan plan);

#ifdef __cplusplus
}
#endif

#endif /* FCONV_EMBED_H */
