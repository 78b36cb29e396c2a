/*
 * ssm_layernorm.h: layer norm over the last dimension, with the residual sum
 * that a block has in front of it, and its backward pass.
 *
 * For each of `rows` rows of `dim` elements:
 *     s    = x + residual (rounded to the activation dtype), or x
 *     mean = sum(s) / dim,  rstd = 1 / sqrt(sum((s - mean)^2) / dim + eps)
 *     y    = (s - mean) * rstd * weight + bias
 * The norm reads the rounded sum: the residual stream as the next block and
 * the backward pass see it. Sums and statistics are float32.
 *
 * Conventions: as in ssm_scan.h (device pointers, dense row-major, status
 * codes found on the host before anything is launched, asynchronous on
 * `stream`), and:
 *   - x, residual, y, sum, dy, dsum, dx: [rows, dim], activation dtype;
 *     weight, bias, dweight, dbias: [dim] float32; mean, rstd: [rows] float32.
 *   - `device` is the CUDA device of every pointer and must be current.
 *   - The calls keep nothing and allocate nothing: they may run at once on
 *     several streams and threads, each with its own workspace, and be captured
 *     into CUDA graphs.
 *   - Every result is the same on every run (no atomics).
 *   - dim is 1..SSM_LAYERNORM_MAX_DIM (else SSM_ERR_UNSUPPORTED). Pointers are
 *     aligned to their element size; rows of whole 16-byte groups with every
 *     buffer 16-byte aligned move 16 bytes at a time.
 */
#ifndef SSM_LAYERNORM_H
#define SSM_LAYERNORM_H

#include <stddef.h>

#include "ssm_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SSM_LAYERNORM_MAX_DIM 8192

/*
 * ssm_layernorm_fwd: y, and where not NULL the sum, mean and rstd.
 *   residual     : NULL means s = x (and sum must be NULL).
 *   weight, bias : NULL means 1 and 0.
 * y may be x or residual itself, and sum may too (each element is read before
 * it is written). Nothing else that is written may overlap anything
 * (SSM_ERR_INVALID), y and sum each other included.
 */
SSM_API int ssm_layernorm_fwd(int device, const void *x, const void *residual,
                              const float *weight, const float *bias,
                              float eps, void *y, void *sum, float *mean,
                              float *rstd, int64_t rows, int64_t dim,
                              int dtype, struct CUstream_st *stream);

/*
 * ssm_layernorm_workspace: bytes of device memory ssm_layernorm_bwd needs for
 * these sizes when dweight or dbias is asked for.
 */
SSM_API int ssm_layernorm_workspace(int device, int64_t rows, int64_t dim,
                                    int dtype, size_t *bytes);

/*
 * ssm_layernorm_bwd: gradients of sum(dy * y) + sum(dsum * s):
 *   x          : what the norm read: x, or the forward's sum.
 *   mean, rstd : the forward's.
 *   dsum       : NULL means 0 (the gradient that reaches s from behind it).
 *   dx         : the gradient of s, which is that of x and of residual.
 *   dweight, dbias : NULL means not wanted.
 *   workspace  : at least ssm_layernorm_workspace bytes, used until the call
 *                is done on `stream`; NULL when neither sum is wanted.
 * dx may be dy, x or dsum itself. Nothing else that is written, the workspace
 * included, may overlap anything (SSM_ERR_INVALID).
 */
SSM_API int ssm_layernorm_bwd(int device, const void *dy, const void *x,
                              const float *mean, const float *rstd,
                              const float *weight, const void *dsum, void *dx,
                              float *dweight, float *dbias, void *workspace,
                              size_t workspace_bytes, int64_t rows,
                              int64_t dim, int dtype,
                              struct CUstream_st *stream);

#ifdef __cplusplus
}
#endif

#endif /* SSM_LAYERNORM_H */
