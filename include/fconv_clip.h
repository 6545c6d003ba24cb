/*
 * fconv_clip.h -- norm of many gradients together on AMD MI355X (gfx950), and
 * their clipping by it.
 *
 *   norm = sqrt(sum over all tensors i and their elements e of in[i][e]^2)
 *   by   = min(1, max_norm / (norm + eps)), 1 for an infinite max_norm
 *   out[i][e] = by in[i][e]
 *
 * Squares are summed in 64 bits, so no gradient is too large or too small for
 * them; norm is fp32 (infinite where it is past that).  by is fp32; out is
 * rounded once, to nearest even.  With by = 1, in is copied bit by bit to an
 * out beside it, and stays untouched in place.  A NaN makes norm, by and all of
 * out NaN; an infinity makes norm infinite and by 0 (out 0, NaN for the
 * infinity); with an infinite max_norm neither does.  Results do not depend on
 * the order in which workgroups run.
 *
 * Conventions as in fconv.h: status codes only; every check happens before
 * anything is enqueued; the caller owns every buffer; plans are host objects
 * that runs never modify.
 */
#ifndef FCONV_CLIP_H
#define FCONV_CLIP_H

#include "fconv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A tensor's elements lie one after another in memory, in any order of its
 * dimensions; numel may be 0. */
typedef struct {
  int64_t numel;
  int32_t dtype; /* FCONV_BF16 or FCONV_FP32 */
} fconv_clip_tensor;

typedef struct fconv_clip_plan_s* fconv_clip_plan;

/* Host arrays of the plan's number of device pointers, read before the call
 * returns; each pointer has its element type's alignment (NULL where numel is 0).
 *   in         the gradients
 *   out        clip: each in[i] itself or a tensor that overlaps nothing
 *   max_norm   clip: 0 or more
 *   norm       written, unless given_norm is there
 *   given_norm clip: the norm, instead of that of `in` (of all ranks' gradients,
 *              where each has a part of them), or NULL
 *   workspace  at least fconv_clip_plan_workspace_size bytes, 16-byte aligned;
 *              not needed with given_norm
 * in, norm, given_norm and workspace overlap nothing that is written. */
typedef struct {
  const void* const* in;
  void* const* out;
  float max_norm;
  float* norm;
  const float* given_norm;
  void* workspace;
  size_t workspace_bytes;
} fconv_clip_args;

/* Host only; `tensors` is copied.  n may be 0 (the norm is then 0).  Errors:
 * FCONV_ERR_INVALID_ARG (NULL, n < 0, numel < 0, eps negative or not finite),
 * FCONV_ERR_UNSUPPORTED (dtype, n above 2^20, numel above 2^40, all together
 * above 2^43). */
FCONV_API fconv_status fconv_clip_plan_create(const fconv_clip_tensor* tensors, int32_t n, float eps,
                                              fconv_clip_plan* out);
FCONV_API fconv_status fconv_clip_plan_workspace_size(fconv_clip_plan plan, size_t* bytes);
/* The plan's tensors, as given (host memory of the plan). */
FCONV_API fconv_status fconv_clip_plan_tensors(fconv_clip_plan plan, const fconv_clip_tensor** tensors, int32_t* n);

/* Enqueue on `stream`: norm writes args->norm, clip that and args->out.  Errors:
 * FCONV_ERR_INVALID_ARG (NULL plan, args or needed pointer, max_norm negative or
 * NaN, an overlap, no memory for the host's list of ranges), FCONV_ERR_MISALIGNED,
 * FCONV_ERR_WORKSPACE, FCONV_ERR_DEVICE. */
FCONV_API fconv_status fconv_clip_plan_norm(fconv_clip_plan plan, void* stream, const fconv_clip_args* args);
FCONV_API fconv_status fconv_clip_plan_clip(fconv_clip_plan plan, void* stream, const fconv_clip_args* args);

FCONV_API fconv_status fconv_clip_plan_destroy(fconv_clip_plan plan);

#ifdef __cplusplus
}
#endif

#endif /* FCONV_CLIP_H */
