// dw_seq.hpp -- what the sequence operators (decayed attention, group norm with an
// activation, 8-bit checkpoints) share: launch descriptions and the host interface
// between the C entry points (dw_seq_api.hip) and the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dw {

// Strides of a (batch, token, head, size) tensor in elements; its size dimension is contiguous.
struct SeqStride {
    int64_t b, t, h;
};

struct AttnSizes {
    int64_t b, t;
    int h, hq, hk, hv, dk, dv;
    int dtype;
};

// One pass over a sequence: o_i = query_i Z_i with Z the decayed sum of key value'.
// The forward is one such pass; the three gradients are three, with the tensors'
// parts exchanged and, for two of them, the tokens taken from last to first.
struct AttnRole {
    const void *q, *k, *v;      // query, key, value
    SeqStride qs, ks, vs;
    int qrep, krep, vrep;       // query heads per own head of each tensor
    int dk, dv;                 // sizes of query/key and of value
    int dkp, dvp;               // the sizes with which the rows lie in memory: multiples of 8
    int wide_o;                 // o is written four elements at a time
    float s_intra, s_inter, s_upd;  // factors of in-chunk products, of query x state, of the state's update
    int reverse;                // tokens from the sequence's last to its first
    const float *zin;           // state before the first chunk (per batch and head, or per segment); may be null
    int64_t zin_pair, zin_seg;  // its strides from (batch, head) to the next and from segment to segment
    int zin_row, zin_col;       // its strides along key and value sizes (a transposed state swaps them)
    float *zout;                // state after the last token, (dk, dv) for each (batch, head); may be null
    void *o;                    // output rows, (b, t, h, dv) contiguous; of float where o_f32
    int o_f32;
};

struct AttnPlan {
    int dkp;         // key rows of the kernels' tiles, the same in every launch of a call
    int chunk;       // tokens of a chunk
    int nseg;        // segments of a sequence that separate workgroups take
    int seg_chunks;  // chunks of a segment
};

struct AttnLaunch {
    AttnRole role[3];
    int nroles;
    const float *log_decay;
    const int32_t *lengths;  // may be null
    int64_t t;
    int b, h;
    int dkp, nseg, seg_chunks;
    int nvb;  // value blocks of 128 columns: the most over the roles
};

// Kernels' launchers: kOk, kErrHip or kErrUnsupported (dw_internal.hpp).
AttnPlan attn_plan(const AttnSizes &s, int nroles);
int attn_out_launch(const AttnLaunch &l, int dtype, hipStream_t stream);
// Every segment's own state from zero into the role's seg (pair, segment, dk, dv); q of the one or two roles is not read.
int attn_state_launch(const AttnLaunch &l, float *const seg[2], int dtype, hipStream_t stream);
// Turns the segments' own states (pair, segment, dk, dv) into the states before each segment.
struct AttnScan {
    float *seg;
    const float *zin;  // state before the first segment; may be null
    float *zout;       // state after the last; may be null
};
// Of one state, or of two of the same size at once (two.seg not null).
int attn_scan_launch(const AttnScan &one, const AttnScan &two, const float *log_decay, const int32_t *lengths, int b, int h,
                     int64_t t, int dk, int dv, int nseg, int64_t seg_tokens, hipStream_t stream);
// out (b, t, heads, d rounded up to 8) = x with zeros after each row.
int attn_widen_launch(const void *x, const SeqStride &st, void *out, int64_t b, int64_t t, int heads, int d, int dtype,
                      hipStream_t stream);
// out (rows, hs, d) = sum of in (rows, hs * rep, d) over the rep heads that share one.
int attn_share_launch(const float *in, void *out, int64_t rows, int hs, int rep, int d, int dtype, hipStream_t stream);
int attn_step_launch(const void *q, const void *k, const void *v, const float *log_decay, float *state, void *o,
                     const AttnSizes &s, const int64_t *strides, int64_t state_stride, float scale, hipStream_t stream);

// 8-bit checkpoints (dw_act8.hpp): rows of c values.
int64_t act8_blocks(int64_t rows, int64_t c);  // workgroups of a launch, at most
int act8_pack_launch(const void *x, int8_t *codes, int8_t *exps, int64_t rows, int64_t c, int dtype, hipStream_t stream);
int act8_unpack_launch(const int8_t *codes, const int8_t *exps, void *y, int64_t rows, int64_t c, int dtype,
                       hipStream_t stream);

// Group norm with an activation over (n, l, c).
struct NormSizes {
    int64_t n, l, c;
    int groups, act, dtype;
    float eps;
};
// Bytes of workspace of the forward (pass 0) or the backward (pass 1).
int64_t norm_workspace(int pass, const NormSizes &s);
// Whether a pass's launches hold these sizes.
bool norm_grid_ok(int pass, const NormSizes &s);
int norm_fwd_launch(const NormSizes &s, const void *x, const void *gamma, const void *beta, void *y, float *mean,
                    float *rstd, int8_t *codes, int8_t *exps, void *ws, hipStream_t stream);
int norm_bwd_launch(const NormSizes &s, const void *dy, const void *x, const int8_t *codes, const int8_t *exps,
                    const float *mean, const float *rstd, const void *gamma, const void *beta, void *dx, void *dgamma,
                    void *dbeta, void *ws, hipStream_t stream);

}  // namespace dw
