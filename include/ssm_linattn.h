/*
 * ssm_linattn.h: linear attention with a decay for each head: the state-space
 * recurrence whose retention is one number per head and step, so that a
 * prompt's steps are matrix products.
 *
 * For each sequence b and head h, with g = log_decay[b,t,h] +
 * head_log_decay[h] and a state S of [dk, dv]:
 *     S_t = exp(g_t) * S_{t-1} + k_t (outer) v_t
 *     y_t = scale * q_t S_t                       (read after the update)
 * Heads h share the q and k of group h / (heads / groups), as the channels of
 * the selective scan share C and B.
 *
 * Conventions: as in ssm_scan.h (device pointers, row-major, status codes
 * found on the host before anything is launched, asynchronous on `stream`),
 * and:
 *   - q, k: [batch, seqlen, groups, dk], v, y, dy: [batch, seqlen, heads, dv],
 *     log_decay: [batch, seqlen, heads], all of the activation dtype;
 *     head_log_decay: [heads] float32; lengths: [batch] int32; h0, h_last,
 *     state and their gradients: [batch, heads, dk, dv] float32.
 *   - q, k and v may be slices of wider rows: dims.q_stride, k_stride and
 *     v_stride are the elements from one token to the next (0: dense), and a
 *     sequence is seqlen of them. All else is dense.
 *   - Either decay may be NULL (0). A log decay of -infinity, or one below
 *     -87 (where its exponential is about to leave float32's normal numbers),
 *     starts the state anew at its token, whatever the state held. Others are finite numbers; positive
 *     ones are taken as they are, but where their sum over 128 tokens in a row
 *     passes 88 (a growth beyond float32), results may be infinite or NaN even
 *     if a token-by-token sum in float32 would not be.
 *   - lengths: NULL means every sequence has seqlen tokens. Else sequence b has
 *     lengths[b] of them (values outside 0..seqlen count as the nearer bound):
 *     what stands behind is not read into any result, whatever it holds; the
 *     rows of y and of the gradients there are written as zeros, and h_last is
 *     the state behind the last token (h0 for an empty sequence).
 *   - q, k and v are finite within the lengths. An infinity or NaN there
 *     reaches all that depends on it, and may reach any row of its sequence
 *     and head: the products of a chunk of 64 or 128 steps multiply what is
 *     masked by 0.
 *   - Buffers that must not overlap are taken from their first element to
 *     their last; SSM_ERR_INVALID where two do.
 *   - `device` is the CUDA device of every pointer and must be current.
 *   - The calls keep nothing and allocate nothing: they may run at once on
 *     several streams and threads, each with its own workspace, and be captured
 *     into CUDA graphs.
 *   - Every result is the same on every run (no atomics).
 *   - dk is 1..128, dv 1..SSM_LINATTN_MAX_VALUE (backward: 1..128), else
 *     SSM_ERR_UNSUPPORTED. Pointers are aligned to their element size, and
 *     outputs with an even row of dv (gradients: dk or dv) to two elements.
 *     Rows that start on 16-byte boundaries are read 16 bytes at a time.
 *   - float32 results (the states, the decays' gradients, and everything with
 *     float32 activations) are float32-accurate; with bfloat16 activations y,
 *     dq, dk, dv and dlog_decay are off by their rounding at the end and little
 *     else (what the sums leave out is 2^-16 of a term at most).
 */
#ifndef SSM_LINATTN_H
#define SSM_LINATTN_H

#include <stddef.h>

#include "ssm_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    int64_t batch;    /* > 0 */
    int64_t seqlen;   /* > 0 */
    int64_t heads;    /* > 0, of v and y */
    int64_t groups;   /* > 0, of q and k; divides heads */
    int64_t dk;       /* elements of a q or k row */
    int64_t dv;       /* elements of a v or y row */
    int64_t q_stride; /* elements from a token to the next; 0: dense */
    int64_t k_stride;
    int64_t v_stride;
} ssm_linattn_dims;

#define SSM_LINATTN_MAX_VALUE 256

/*
 * ssm_linattn_workspace: bytes of device memory ssm_linattn_fwd (backward ==
 * 0) or ssm_linattn_bwd (backward == 1) needs for these dims on `device`,
 * whatever its other arguments; 0 where none is needed. What a backward call
 * does without may be added to the 1:
 *   SSM_LINATTN_NO_HEAD_GRADIENT  : dhead_log_decay will be NULL;
 *   SSM_LINATTN_NO_DECAY_GRADIENT : dlog_decay and dhead_log_decay will be.
 */
#define SSM_LINATTN_NO_HEAD_GRADIENT 2
#define SSM_LINATTN_NO_DECAY_GRADIENT 4

SSM_API int ssm_linattn_workspace(int device, ssm_linattn_dims dims, int dtype,
                                  int backward, size_t *bytes);

/*
 * ssm_linattn_fwd: a prompt.
 *   h0     : NULL means a zero state in front.
 *   h_last : NULL means the last state is not written. It may be h0.
 *   workspace : at least ssm_linattn_workspace bytes, 16-byte aligned, used
 *            until the call is done on `stream`; NULL where that is 0.
 * y and h_last must not overlap each other or (else) an input, nor the
 * workspace any of these.
 */
SSM_API int ssm_linattn_fwd(int device, const void *q, const void *k,
                            const void *v, const void *log_decay,
                            const float *head_log_decay, float scale,
                            const int32_t *lengths, const float *h0, void *y,
                            float *h_last, void *workspace,
                            size_t workspace_bytes, ssm_linattn_dims dims,
                            int dtype, struct CUstream_st *stream);

/*
 * ssm_linattn_step: one token of every sequence (dims.seqlen must be 1): the
 * state is updated in place and read. state and y must not overlap each other
 * or an input.
 */
SSM_API int ssm_linattn_step(int device, const void *q, const void *k,
                             const void *v, const void *log_decay,
                             const float *head_log_decay, float scale,
                             float *state, void *y, ssm_linattn_dims dims,
                             int dtype, struct CUstream_st *stream);

/*
 * ssm_linattn_bwd: gradients of sum(dy * y) + sum(dh_last * h_last).
 *   inputs : as ssm_linattn_fwd; dy dense; dh_last NULL means 0.
 *   dq, dk : [batch, seqlen, groups, dk] dense, activation dtype, required:
 *            sums over each group's heads, in order, in float32.
 *   dv     : [batch, seqlen, heads, dv] dense, activation dtype, required.
 *   dlog_decay      : [batch, seqlen, heads] activation dtype, or NULL;
 *   dhead_log_decay : [heads] float32, or NULL; each only with its input.
 *            Without either, dq and dk take fewer products.
 *   dh0    : [batch, heads, dk, dv] float32, or NULL.
 *   workspace : as above, for the backward call.
 * The log decays' gradients at a token that starts the state anew are 0.
 * No output, and not the workspace, may overlap another or an input.
 */
SSM_API int ssm_linattn_bwd(int device, const void *q, const void *k,
                            const void *v, const void *log_decay,
                            const float *head_log_decay, float scale,
                            const int32_t *lengths, const float *h0,
                            const void *dy, const float *dh_last, void *dq,
                            void *dk, void *dv, void *dlog_decay,
                            float *dhead_log_decay, float *dh0,
                            void *workspace, size_t workspace_bytes,
                            ssm_linattn_dims dims, int dtype,
                            struct CUstream_st *stream);

/*
 * ssm_linattn_sync_status: wait for `stream`, then report whether a bounded
 * wait inside a kernel of ssm_linattn_fwd or ssm_linattn_bwd gave up on
 * `device` since the previous report (SSM_ERR_TIMEOUT: the results of those
 * calls are invalid; no input leads there), SSM_ERR_CUDA on an asynchronous
 * CUDA error, else SSM_OK. Resets the status, which all streams share.
 */
SSM_API int ssm_linattn_sync_status(int device, struct CUstream_st *stream);

#ifdef __cplusplus
}
#endif

#endif /* SSM_LINATTN_H */
