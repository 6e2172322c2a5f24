/*
 * dwseq.h -- C ABI of the sequence operators that stand beside the convolutions of
 * dwconv.h in libdwconv.so: causal linear attention with a decay for each head, group norm
 * with an activation over channels-last tensors, and activation checkpoints in 8 bits.
 *
 * Conventions of dwconv.h hold: device pointers owned by the caller, work enqueued on
 * `stream` without waiting, a status of enum dw_status, every argument checked before any
 * HIP call, nothing allocated and nothing kept after a call, arithmetic and sums in fp32 or
 * wider, 16-bit results rounded to nearest-even once.  Results do not depend on timing: no
 * atomics are used.  Tensors may have more than 2^31 elements; one size is at most 2^30, an
 * offset within a tensor at most 2^46 elements, and b h at most 2^20; limits of single operators stand
 * at them (DW_ETOOLARGE past any).
 */
#ifndef DWSEQ_H
#define DWSEQ_H

#include "dwconv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest key and value size of a head. */
#define DWSEQ_MAX_HEAD 256

/*
 * Decayed linear attention.  For every batch entry and head, with d = exp(log_decay[head]):
 *
 *   S_i = d S_(i-1) + k_i v_i',   o_i = scale q_i S_i        (i = 0 .. length - 1)
 *
 * q (b, t, hq, dk), k (b, t, hk, dk), v (b, t, hv, dv): element type `dtype`; the last
 *   dimension is contiguous, the others have the strides (in elements, >= 0) given in strides[0..8] = q's batch, token and head stride, then k's, then v's.  hq, hk and hv
 *   divide h; head j of the h uses head j / (h / hq) of q, and so on.
 * log_decay (h) float: <= 0; minus infinity keeps nothing of the past.
 * state (b, h, dk, dv) float or NULL (zeros): S before the first token.
 * lengths (b) int32 or NULL (all t): the tokens of each entry, taken into [0, t].  Tokens past
 *   it are not read; their output rows are zero and they leave the state as it is.
 * o (b, t, h, dv) contiguous, of `dtype`.
 * state_out (b, h, dk, dv) float: S after the last token; may be `state` itself.  May be NULL.
 * workspace: at least decayattn_workspace_bytes(0, ...), 256-byte aligned (NULL if that is 0).
 *
 * b, t >= 0 (0: nothing but the state is written); dk, dv in [1, DWSEQ_MAX_HEAD].
 * A value that is not finite spreads to the other tokens of its 64-token chunk and after it.
 */
int decayattn_fwd(const void *q, const void *k, const void *v, const float *log_decay,
                  const float *state, const int32_t *lengths, void *o, float *state_out,
                  void *workspace, size_t workspace_bytes, int64_t b, int64_t t, int64_t h,
                  int64_t hq, int64_t hk, int64_t hv, int64_t dk, int64_t dv,
                  const int64_t *strides, float scale, int dtype, void *stream);

/*
 * Gradients of decayattn_fwd.  do_ (b, t, h, dv) is o's gradient, of `dtype`, with its
 * strides in strides[9..11]; rows past a length are not read.  dstate_out (b, h, dk, dv) float
 * or NULL (zeros) is the gradient of the state after the last token.
 * dq, dk_, dv_: contiguous (b, t, hq, dk), (b, t, hk, dk), (b, t, hv, dv) of `dtype`; a head
 *   that several share gets the sum, added in fp32; rows past a length are zero.
 * dstate (b, h, dk, dv) float or NULL: the gradient of the state before the first token.
 *   log_decay is a constant: it gets no gradient.
 */
int decayattn_bwd(const void *q, const void *k, const void *v, const float *log_decay,
                  const void *do_, const float *state, const int32_t *lengths,
                  const float *dstate_out, void *dq, void *dk_, void *dv_, float *dstate,
                  void *workspace, size_t workspace_bytes, int64_t b, int64_t t, int64_t h,
                  int64_t hq, int64_t hk, int64_t hv, int64_t dk, int64_t dv,
                  const int64_t *strides, float scale, int dtype, void *stream);

/* Bytes of workspace of decayattn_fwd (pass 0) or decayattn_bwd (pass 1).  Host only. */
int decayattn_workspace_bytes(int pass, int64_t b, int64_t t, int64_t h, int64_t hq, int64_t hk,
                              int64_t hv, int64_t dk, int64_t dv, int dtype, size_t *bytes);

/*
 * One more token: state is updated in place (S = d S + k v') and o = scale q S.
 * q (b, hq, dk), k (b, hk, dk), v (b, hv, dv), strides[0..5] = q's batch and head stride, then
 * k's, then v's; o (b, h, dv) contiguous; state (b, h, dk, dv) float, contiguous but for its
 * batch stride state_stride (in elements, >= h dk dv).
 */
int decayattn_step(const void *q, const void *k, const void *v, const float *log_decay,
                   float *state, void *o, int64_t b, int64_t h, int64_t hq, int64_t hk,
                   int64_t hv, int64_t dk, int64_t dv, const int64_t *strides,
                   int64_t state_stride, float scale, int dtype, void *stream);

/*
 * 8-bit checkpoint of x (rows, c), contiguous.  Along a row each 32 values (the last ones of a row
 * may be fewer) share a step 2^e, the smallest power of two, at least 2^-126, by which the largest
 * finite magnitude rounds to at most 127; a value becomes the nearest whole number of steps, ties to
 * even.  codes (rows, c) signed bytes; exps (rows, ceil(c / 32)) signed bytes, the e of each block.
 * Code -128 stands for a value that is not finite; it comes back as a NaN.  There may be 2^32 - 256 blocks.
 */
int act8_pack(const void *x, int8_t *codes, int8_t *exps, int64_t rows, int64_t c, int dtype,
              void *stream);

/* y (rows, c) of `dtype`: code * 2^e, rounded to nearest-even, at most the type's largest finite value. */
int act8_unpack(const int8_t *codes, const int8_t *exps, void *y, int64_t rows, int64_t c, int dtype,
                void *stream);

enum dw_act { DW_ACT_NONE = 0, DW_ACT_SILU = 1, DW_ACT_GELU = 2 /* z Phi(z), by erf */ };

/*
 * Group norm with an activation over x (n, l, c), contiguous, channels last: mean and variance
 * over the l positions and the c / groups channels of each group,
 * xhat = (x - mean) / sqrt(variance + eps), y = act(xhat gamma + beta).
 * gamma, beta (c) and y (n, l, c) of x's type; mean, rstd (n, groups) float.
 * codes, exps: NULL, or where x's 8-bit checkpoint goes, as act8_pack with rows = n l.
 * Sizes: c at most 2^24 - 256; n < 2^24, or with l = 1 and c / groups <= 512 any n.  Some shapes past these are
 * served too, others have a launch of 2^32 threads or of more than 65535 workgroups along the groups (DW_ETOOLARGE).
 * workspace: groupnorm_act_workspace_bytes(0, ...), 256-byte aligned (NULL if that is 0).
 */
int groupnorm_act_fwd(const void *x, const void *gamma, const void *beta, void *y, float *mean,
                      float *rstd, int8_t *codes, int8_t *exps, void *workspace,
                      size_t workspace_bytes, int64_t n, int64_t l, int64_t c, int64_t groups,
                      float eps, int act, int dtype, void *stream);

/*
 * Gradients of groupnorm_act_fwd for y's gradient dy (n, l, c): dx (n, l, c), dgamma and dbeta (c), of
 * `dtype`.  The input is x, or where x is NULL its checkpoint (codes, exps): xhat is then taken from
 * the checkpoint's values with the given mean and rstd.  workspace: pass 1.  With n = 0 dgamma and
 * dbeta are not written.
 */
int groupnorm_act_bwd(const void *dy, const void *x, const int8_t *codes, const int8_t *exps,
                      const float *mean, const float *rstd, const void *gamma, const void *beta,
                      void *dx, void *dgamma, void *dbeta, void *workspace, size_t workspace_bytes,
                      int64_t n, int64_t l, int64_t c, int64_t groups, int act, int dtype,
                      void *stream);

/* Bytes of workspace of groupnorm_act_fwd (pass 0) or groupnorm_act_bwd (pass 1).  Host only. */
int groupnorm_act_workspace_bytes(int pass, int64_t n, int64_t l, int64_t c, int64_t groups,
                                  int dtype, size_t *bytes);

#ifdef __cplusplus
}
#endif

#endif /* DWSEQ_H */
