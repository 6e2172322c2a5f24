// dw_seq_api.hip -- the extern "C" entry points declared in include/dwseq.h.
//
// Every argument is validated on the host before any HIP call, as in dw_api.hip.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <initializer_list>

#include "dw_internal.hpp"
#include "dw_seq.hpp"
#include "dwseq.h"

namespace {

constexpr int64_t kMaxSize = int64_t{1} << 30;
constexpr int64_t kMaxStride = int64_t{1} << 42;
constexpr int64_t kMaxElems = int64_t{1} << 46;  // of a tensor: byte offsets stay far inside 64 bits
constexpr int64_t kMaxPairs = int64_t{1} << 20;   // (batch, head) pairs: launches of fewer than 2^32 threads
constexpr int64_t kMaxGroups = (int64_t{1} << 24) - 1;  // workgroups of 256 threads, likewise

int64_t elem_size(int dtype) { return dtype == DW_F32 ? 4 : 2; }
bool known(int dtype) { return dtype == DW_F32 || dtype == DW_F16 || dtype == DW_BF16; }
bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// The product of sizes in [0, 2^30], or -1 past `most`.
int64_t product(std::initializer_list<int64_t> sizes, int64_t most) {
    int64_t p = 1;
    for (int64_t s : sizes) {
        if (s == 0) return 0;
        if (p > most / s) return -1;
        p *= s;
    }
    return p;
}

struct Span {
    const void *p;
    int64_t bytes;
};
bool overlap(const Span &a, const Span &b) {
    if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + b.bytes && y < x + a.bytes;
}

int map_launch(int rc) { return rc == dw::kOk ? DW_OK : rc == dw::kErrUnsupported ? DW_EUNSUPPORTED : DW_EHIP; }

// ---------------------------------------------------------------- decayed attention
int check_attn(int64_t b, int64_t t, int64_t h, int64_t hq, int64_t hk, int64_t hv, int64_t dk, int64_t dv, int dtype,
               dw::AttnSizes *s) {
    if (!known(dtype)) return DW_EDTYPE;
    if (b < 0 || t < 0 || h < 1 || hq < 1 || hk < 1 || hv < 1 || dk < 1 || dv < 1) return DW_ESHAPE;
    for (int64_t v : {b, t, h, hq, hk, hv, dk, dv})
        if (v > kMaxSize) return DW_ETOOLARGE;
    if (h % hq || h % hk || h % hv || dk > DWSEQ_MAX_HEAD || dv > DWSEQ_MAX_HEAD) return DW_EHEADS;
    if (product({b, t, h, dk > dv ? dk : dv}, kMaxElems) < 0 || product({b, h, dk, dv}, kMaxElems) < 0 ||
        product({b, h}, kMaxPairs) < 0)
        return DW_ETOOLARGE;
    *s = {b, t, static_cast<int>(h), static_cast<int>(hq), static_cast<int>(hk), static_cast<int>(hv),
          static_cast<int>(dk), static_cast<int>(dv), dtype};
    return DW_OK;
}

// Strides of tensors whose dimensions but the last have these sizes.
int check_strides(const int64_t *strides, std::initializer_list<int64_t> sizes) {
    if (!strides) return DW_EPTR;
    const int n = static_cast<int>(sizes.size());
    for (int i = 0; i < n; ++i)
        if (strides[i] < 0 || strides[i] > kMaxStride) return DW_ESTRIDE;
    for (int i = 0; i < n; ++i)
        if (strides[i] > 0 && sizes.begin()[i] - 1 > kMaxElems / strides[i]) return DW_ETOOLARGE;
    return DW_OK;
}

// The bytes from a strided (b, t, heads, d) tensor's first element to its last.
Span span_of(const void *p, const dw::SeqStride &st, int64_t b, int64_t t, int64_t heads, int64_t d, int64_t e) {
    if (b == 0 || t == 0) return {p, 0};
    return {p, ((b - 1) * st.b + (t - 1) * st.t + (heads - 1) * st.h + d) * e};
}
int64_t round256(int64_t n) { return (n + 255) / 256 * 256; }

// Where a call's workspace parts lie, in bytes.
struct AttnSpace {
    int64_t seg[2];    // the segments' states: (key, value), and for the gradients (query, do)
    int64_t share[3];  // per-head gradients of shared q, k, v heads in fp32; -1: none
    int64_t wide[4];   // q, k, v, do with rows rounded up to eight elements; -1: as they are
    int64_t bytes;
};
bool odd(int64_t d) { return d % 8 != 0; }
int up8(int d) { return (d + 7) / 8 * 8; }
AttnSpace attn_space(int pass, const dw::AttnSizes &s, const dw::AttnPlan &p) {
    AttnSpace w{{0, 0}, {-1, -1, -1}, {-1, -1, -1, -1}, 0};
    const int64_t states = round256(s.b * s.h * p.nseg * s.dk * s.dv * 4);
    for (int i = 0; i <= pass; ++i) {
        w.seg[i] = w.bytes;
        if (p.nseg > 1) w.bytes += states;
    }
    if (pass == 1) {
        const int heads[3] = {s.hq, s.hk, s.hv}, size[3] = {s.dk, s.dk, s.dv};
        for (int i = 0; i < 3; ++i)
            if (heads[i] != s.h) {
                w.share[i] = w.bytes;
                w.bytes += round256(s.b * s.t * s.h * size[i] * 4);
            }
    }
    const int heads[4] = {s.hq, s.hk, s.hv, s.h}, size[4] = {s.dk, s.dk, s.dv, s.dv};
    for (int i = 0; i < 3 + pass; ++i)
        if (odd(size[i])) {
            w.wide[i] = w.bytes;
            w.bytes += round256(s.b * s.t * heads[i] * up8(size[i]) * elem_size(s.dtype));
        }
    return w;
}

int check_workspace(const void *workspace, size_t have, int64_t need) {
    if (need > 0 && (!workspace || have < static_cast<size_t>(need) || !aligned(workspace, 256))) return DW_EWORKSPACE;
    return DW_OK;
}

// A tensor as the kernels read it.
struct Part {
    const void *p;
    dw::SeqStride st;
    int rep, d, dp;
};
// The tensor itself, or a copy of it with rows rounded up to eight elements.
int part_of(Part *out, const void *p, const dw::SeqStride &st, int heads, int d, int64_t copy, void *workspace,
            const dw::AttnSizes &s, hipStream_t stream) {
    *out = {p, st, s.h / heads, d, up8(d)};
    if (copy < 0 || s.t == 0) return dw::kOk;
    out->p = static_cast<char *>(workspace) + copy;
    out->st = {s.t * heads * out->dp, int64_t{heads} * out->dp, out->dp};
    return dw::attn_widen_launch(p, st, static_cast<char *>(workspace) + copy, s.b, s.t, heads, d, s.dtype, stream);
}

// The tensors' parts in a role.
dw::AttnRole role_of(const Part &q, const Part &k, const Part &v) {
    dw::AttnRole r{};
    r.q = q.p, r.k = k.p, r.v = v.p;
    r.qs = q.st, r.ks = k.st, r.vs = v.st;
    r.qrep = q.rep, r.krep = k.rep, r.vrep = v.rep;
    r.dk = k.d, r.dv = v.d;
    r.dkp = k.dp, r.dvp = v.dp;
    return r;
}
void set_output(dw::AttnRole *r, void *o, bool f32, int64_t e) {
    r->o = o;
    r->o_f32 = f32;
    r->wide_o = r->dv % 4 == 0 && aligned(o, f32 || e == 4 ? 16 : 8);
}
void set_state(dw::AttnRole *r, const float *z, int64_t pair, int64_t seg, bool transposed) {
    r->zin = z;
    r->zin_pair = pair;
    r->zin_seg = seg;
    r->zin_row = transposed ? 1 : r->dv;
    r->zin_col = transposed ? r->dk : 1;
}

dw::AttnLaunch launch_of(const dw::AttnSizes &s, const dw::AttnPlan &p, const float *log_decay, const int32_t *lengths) {
    dw::AttnLaunch l{};
    l.log_decay = log_decay;
    l.lengths = lengths;
    l.t = s.t;
    l.b = static_cast<int>(s.b);
    l.h = s.h;
    l.dkp = p.dkp;
    l.nseg = p.nseg;
    l.seg_chunks = p.seg_chunks;
    return l;
}
void add_role(dw::AttnLaunch *l, const dw::AttnRole &r) {
    l->role[l->nroles++] = r;
    const int nvb = (r.dv + 127) / 128;
    if (nvb > l->nvb) l->nvb = nvb;
}

// ---------------------------------------------------------------- norms and checkpoints
int check_act8(const void *x, const void *codes, const void *exps, int64_t rows, int64_t c, int dtype) {
    if (!known(dtype)) return DW_EDTYPE;
    if (rows < 0 || c < 1) return DW_ESHAPE;
    if (rows > kMaxElems || c > kMaxSize || product({rows, c}, kMaxElems) < 0) return DW_ETOOLARGE;
    if (rows == 0) return DW_OK;
    if (dw::act8_blocks(rows, c) > kMaxGroups) return DW_ETOOLARGE;
    return x && codes && exps && aligned(x, elem_size(dtype)) ? DW_OK : DW_EPTR;
}
Span codes_span(const void *codes, int64_t rows, int64_t c) { return {codes, rows * c}; }
Span exps_span(const void *exps, int64_t rows, int64_t c) { return {exps, rows * ((c + 31) / 32)}; }

int check_norm(int pass, int64_t n, int64_t l, int64_t c, int64_t groups, int act, int dtype, dw::NormSizes *s) {
    if (!known(dtype)) return DW_EDTYPE;
    if (n < 0 || l < 1 || c < 1 || groups < 1) return DW_ESHAPE;
    for (int64_t v : {n, l, c, groups})
        if (v > kMaxSize) return DW_ETOOLARGE;
    if (c % groups) return DW_EGROUPS;
    if (act != DW_ACT_NONE && act != DW_ACT_SILU && act != DW_ACT_GELU) return DW_EGROUPS;
    if (product({n, l, c}, kMaxElems) < 0) return DW_ETOOLARGE;
    *s = {n, l, c, static_cast<int>(groups), act, dtype, 0.f};
    return n == 0 || dw::norm_grid_ok(pass, *s) ? DW_OK : DW_ETOOLARGE;
}

// Every output against every input and every other output.
template <int NO, int NI> bool any_overlap(const Span (&outs)[NO], const Span (&ins)[NI]) {
    for (int i = 0; i < NO; ++i) {
        for (const Span &in : ins)
            if (overlap(outs[i], in)) return true;
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i], outs[j])) return true;
    }
    return false;
}

}  // namespace

extern "C" {

int decayattn_workspace_bytes(int pass, int64_t b, int64_t t, int64_t h, int64_t hq, int64_t hk, int64_t hv, int64_t dk,
                              int64_t dv, int dtype, size_t *bytes) {
    if (!bytes || (pass != 0 && pass != 1)) return pass != 0 && pass != 1 ? DW_ESHAPE : DW_EPTR;
    dw::AttnSizes s;
    const int rc = check_attn(b, t, h, hq, hk, hv, dk, dv, dtype, &s);
    if (rc != DW_OK) return rc;
    *bytes = static_cast<size_t>(attn_space(pass, s, dw::attn_plan(s, pass ? 3 : 1)).bytes);
    return DW_OK;
}

int decayattn_fwd(const void *q, const void *k, const void *v, const float *log_decay, const float *state,
                  const int32_t *lengths, void *o, float *state_out, void *workspace, size_t workspace_bytes, int64_t b,
                  int64_t t, int64_t h, int64_t hq, int64_t hk, int64_t hv, int64_t dk, int64_t dv,
                  const int64_t *strides, float scale, int dtype, void *stream) {
    dw::AttnSizes s;
    int rc = check_attn(b, t, h, hq, hk, hv, dk, dv, dtype, &s);
    if (rc == DW_OK) rc = check_strides(strides, {b, t, hq, b, t, hk, b, t, hv});
    if (rc != DW_OK) return rc;
    if (b == 0) return DW_OK;
    const int64_t e = elem_size(dtype), states = b * h * dk * dv * 4;
    if (!log_decay || !aligned(log_decay, 4) || !aligned(state, 4) || !aligned(state_out, 4) || !aligned(lengths, 4))
        return DW_EPTR;
    if (t > 0)
        for (const void *p : {q, k, v, static_cast<const void *>(o)})
            if (!p || !aligned(p, e)) return DW_EPTR;
    const dw::AttnPlan plan = dw::attn_plan(s, 1);
    const AttnSpace space = attn_space(0, s, plan);
    rc = check_workspace(workspace, workspace_bytes, space.bytes);
    if (rc != DW_OK) return rc;
    const dw::SeqStride qs{strides[0], strides[1], strides[2]}, ks{strides[3], strides[4], strides[5]},
        vs{strides[6], strides[7], strides[8]};
    const Span outs[] = {{o, b * t * h * dv * e}, {state_out, states}, {space.bytes ? workspace : nullptr, space.bytes}};
    const Span ins[] = {span_of(q, qs, b, t, hq, dk, e), span_of(k, ks, b, t, hk, dk, e), span_of(v, vs, b, t, hv, dv, e),
                        {log_decay, h * 4}, {lengths, b * 4}, {state == state_out ? nullptr : state, states}};
    for (int i = 0; i < 3; ++i) {
        for (const Span &in : ins)
            if (overlap(outs[i], in)) return DW_EALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i], outs[j])) return DW_EALIAS;
    }
    if ((overlap(outs[0], {state, states})) || overlap(outs[2], {state, states})) return DW_EALIAS;

    const hipStream_t st = static_cast<hipStream_t>(stream);
    dw::AttnLaunch l = launch_of(s, plan, log_decay, lengths);
    Part pq, pk, pv;
    rc = part_of(&pq, q, qs, s.hq, s.dk, space.wide[0], workspace, s, st);
    if (rc == dw::kOk) rc = part_of(&pk, k, ks, s.hk, s.dk, space.wide[1], workspace, s, st);
    if (rc == dw::kOk) rc = part_of(&pv, v, vs, s.hv, s.dv, space.wide[2], workspace, s, st);
    if (rc != dw::kOk) return map_launch(rc);
    dw::AttnRole r = role_of(pq, pk, pv);
    r.s_intra = r.s_inter = scale;
    r.s_upd = 1.f;
    set_output(&r, o, false, e);
    float *seg = reinterpret_cast<float *>(static_cast<char *>(workspace) + space.seg[0]);
    const int64_t size = dk * dv;
    if (plan.nseg > 1) set_state(&r, seg, plan.nseg * size, size, false);
    else set_state(&r, state, size, 0, false), r.zout = state_out;
    add_role(&l, r);
    if (plan.nseg > 1) {
        float *const segs[2] = {seg, nullptr};
        rc = dw::attn_state_launch(l, segs, dtype, st);
        if (rc == dw::kOk)
            rc = dw::attn_scan_launch({seg, state, state_out}, {}, log_decay, lengths, l.b, l.h, t, s.dk, s.dv, plan.nseg,
                                      static_cast<int64_t>(plan.seg_chunks) * plan.chunk, st);
        if (rc != dw::kOk) return map_launch(rc);
    }
    return map_launch(dw::attn_out_launch(l, dtype, st));
}

int decayattn_bwd(const void *q, const void *k, const void *v, const float *log_decay, const void *do_,
                  const float *state, const int32_t *lengths, const float *dstate_out, void *dq, void *dk_, void *dv_,
                  float *dstate, void *workspace, size_t workspace_bytes, int64_t b, int64_t t, int64_t h, int64_t hq,
                  int64_t hk, int64_t hv, int64_t dk, int64_t dv, const int64_t *strides, float scale, int dtype,
                  void *stream) {
    dw::AttnSizes s;
    int rc = check_attn(b, t, h, hq, hk, hv, dk, dv, dtype, &s);
    if (rc == DW_OK) rc = check_strides(strides, {b, t, hq, b, t, hk, b, t, hv, b, t, h});
    if (rc != DW_OK) return rc;
    if (b == 0) return DW_OK;
    const int64_t e = elem_size(dtype), states = b * h * dk * dv * 4;
    if (!log_decay || !aligned(log_decay, 4) || !aligned(state, 4) || !aligned(dstate, 4) || !aligned(dstate_out, 4) ||
        !aligned(lengths, 4))
        return DW_EPTR;
    if (t > 0)
        for (const void *p : {q, k, v, do_, static_cast<const void *>(dq), static_cast<const void *>(dk_),
                              static_cast<const void *>(dv_)})
            if (!p || !aligned(p, e)) return DW_EPTR;
    const dw::AttnPlan plan = dw::attn_plan(s, 3);
    const AttnSpace space = attn_space(1, s, plan);
    rc = check_workspace(workspace, workspace_bytes, space.bytes);
    if (rc != DW_OK) return rc;
    const dw::SeqStride qs{strides[0], strides[1], strides[2]}, ks{strides[3], strides[4], strides[5]},
        vs{strides[6], strides[7], strides[8]}, os{strides[9], strides[10], strides[11]};
    const Span outs[] = {{dq, b * t * hq * dk * e}, {dk_, b * t * hk * dk * e}, {dv_, b * t * hv * dv * e},
                         {space.bytes ? workspace : nullptr, space.bytes}, {dstate, states}};
    const Span ins[] = {span_of(q, qs, b, t, hq, dk, e), span_of(k, ks, b, t, hk, dk, e), span_of(v, vs, b, t, hv, dv, e),
                        span_of(do_, os, b, t, h, dv, e), {log_decay, h * 4}, {lengths, b * 4}, {state, states},
                        {dstate_out, states}};
    for (int i = 0; i < 5; ++i) {
        for (const Span &in : ins)
            if (overlap(outs[i], in)) return DW_EALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i], outs[j])) return DW_EALIAS;
    }

    const hipStream_t st = static_cast<hipStream_t>(stream);
    char *ws = static_cast<char *>(workspace);
    const int64_t size = dk * dv, seg_tokens = static_cast<int64_t>(plan.seg_chunks) * plan.chunk;
    Part pq, pk, pv, po;
    rc = part_of(&pq, q, qs, s.hq, s.dk, space.wide[0], workspace, s, st);
    if (rc == dw::kOk) rc = part_of(&pk, k, ks, s.hk, s.dk, space.wide[1], workspace, s, st);
    if (rc == dw::kOk) rc = part_of(&pv, v, vs, s.hv, s.dv, space.wide[2], workspace, s, st);
    if (rc == dw::kOk) rc = part_of(&po, do_, os, s.h, s.dv, space.wide[3], workspace, s, st);
    if (rc != dw::kOk) return map_launch(rc);
    const float *z[2] = {state, dstate_out};
    int64_t pair = size, step = 0;
    if (plan.nseg > 1) {
        float *const seg[2] = {reinterpret_cast<float *>(ws + space.seg[0]), reinterpret_cast<float *>(ws + space.seg[1])};
        dw::AttnLaunch l = launch_of(s, plan, log_decay, lengths);
        dw::AttnRole r = role_of(pq, pk, pv);
        r.s_upd = 1.f;
        add_role(&l, r);
        r = role_of(pk, pq, po);
        r.s_upd = scale;
        r.reverse = 1;
        add_role(&l, r);
        rc = dw::attn_state_launch(l, seg, dtype, st);
        if (rc == dw::kOk)
            rc = dw::attn_scan_launch({seg[0], state, nullptr}, {seg[1], dstate_out, dstate}, log_decay, lengths, l.b, l.h, t,
                                      s.dk, s.dv, plan.nseg, seg_tokens, st);
        if (rc != dw::kOk) return map_launch(rc);
        z[0] = seg[0], z[1] = seg[1];
        pair = plan.nseg * size, step = size;
    }
    void *const out[3] = {dq, dk_, dv_};
    dw::AttnLaunch l = launch_of(s, plan, log_decay, lengths);
    for (int i = 0; i < 3; ++i) {
        dw::AttnRole r = i == 0 ? role_of(po, pv, pk) : i == 1 ? role_of(pv, po, pq) : role_of(pk, pq, po);
        r.s_intra = scale;
        r.s_inter = i == 0 ? scale : 1.f;
        r.s_upd = i == 0 ? 1.f : scale;
        r.reverse = i != 0;
        set_state(&r, z[i != 0], pair, step, i != 2);
        if (i == 2 && plan.nseg == 1) r.zout = dstate;
        const bool shared = space.share[i] >= 0;
        set_output(&r, shared ? ws + space.share[i] : out[i], shared, e);
        add_role(&l, r);
    }
    rc = dw::attn_out_launch(l, dtype, st);
    const int heads[3] = {s.hq, s.hk, s.hv}, sizes[3] = {s.dk, s.dk, s.dv};
    for (int i = 0; i < 3 && rc == dw::kOk; ++i)
        if (space.share[i] >= 0 && t > 0)
            rc = dw::attn_share_launch(reinterpret_cast<const float *>(ws + space.share[i]), out[i], b * t, heads[i],
                                       s.h / heads[i], sizes[i], dtype, st);
    return map_launch(rc);
}

int decayattn_step(const void *q, const void *k, const void *v, const float *log_decay, float *state, void *o, int64_t b,
                   int64_t h, int64_t hq, int64_t hk, int64_t hv, int64_t dk, int64_t dv, const int64_t *strides,
                   int64_t state_stride, float scale, int dtype, void *stream) {
    dw::AttnSizes s;
    int rc = check_attn(b, 1, h, hq, hk, hv, dk, dv, dtype, &s);
    if (rc == DW_OK) rc = check_strides(strides, {b, hq, b, hk, b, hv});
    if (rc != DW_OK) return rc;
    if (state_stride < h * dk * dv || state_stride > kMaxStride) return DW_ESTRIDE;
    if (b - 1 > kMaxElems / state_stride) return DW_ETOOLARGE;
    if (b == 0) return DW_OK;
    const int64_t e = elem_size(dtype);
    for (const void *p : {q, k, v, static_cast<const void *>(o)})
        if (!p || !aligned(p, e)) return DW_EPTR;
    if (!log_decay || !state || !aligned(log_decay, 4) || !aligned(state, 4)) return DW_EPTR;
    const dw::SeqStride qs{strides[0], 0, strides[1]}, ks{strides[2], 0, strides[3]}, vs{strides[4], 0, strides[5]};
    const Span outs[] = {{o, b * h * dv * e}, {state, ((b - 1) * state_stride + h * dk * dv) * 4}};
    const Span ins[] = {span_of(q, qs, b, 1, hq, dk, e), span_of(k, ks, b, 1, hk, dk, e), span_of(v, vs, b, 1, hv, dv, e),
                        {log_decay, h * 4}};
    for (const Span &out : outs)
        for (const Span &in : ins)
            if (overlap(out, in)) return DW_EALIAS;
    if (overlap(outs[0], outs[1])) return DW_EALIAS;
    return map_launch(dw::attn_step_launch(q, k, v, log_decay, state, o, s, strides, state_stride, scale,
                                           static_cast<hipStream_t>(stream)));
}

int act8_pack(const void *x, int8_t *codes, int8_t *exps, int64_t rows, int64_t c, int dtype, void *stream) {
    const int rc = check_act8(x, codes, exps, rows, c, dtype);
    if (rc != DW_OK || rows == 0) return rc;
    const Span outs[] = {codes_span(codes, rows, c), exps_span(exps, rows, c)};
    const Span ins[] = {{x, rows * c * elem_size(dtype)}};
    if (any_overlap(outs, ins)) return DW_EALIAS;
    return map_launch(dw::act8_pack_launch(x, codes, exps, rows, c, dtype, static_cast<hipStream_t>(stream)));
}

int act8_unpack(const int8_t *codes, const int8_t *exps, void *y, int64_t rows, int64_t c, int dtype, void *stream) {
    const int rc = check_act8(y, codes, exps, rows, c, dtype);
    if (rc != DW_OK || rows == 0) return rc;
    const Span outs[] = {{y, rows * c * elem_size(dtype)}};
    const Span ins[] = {codes_span(codes, rows, c), exps_span(exps, rows, c)};
    if (any_overlap(outs, ins)) return DW_EALIAS;
    return map_launch(dw::act8_unpack_launch(codes, exps, y, rows, c, dtype, static_cast<hipStream_t>(stream)));
}

int groupnorm_act_workspace_bytes(int pass, int64_t n, int64_t l, int64_t c, int64_t groups, int dtype, size_t *bytes) {
    if (pass != 0 && pass != 1) return DW_ESHAPE;
    if (!bytes) return DW_EPTR;
    dw::NormSizes s;
    const int rc = check_norm(pass, n, l, c, groups, DW_ACT_NONE, dtype, &s);
    if (rc != DW_OK) return rc;
    *bytes = static_cast<size_t>(dw::norm_workspace(pass, s));
    return DW_OK;
}

int groupnorm_act_fwd(const void *x, const void *gamma, const void *beta, void *y, float *mean, float *rstd, int8_t *codes,
                      int8_t *exps, void *workspace, size_t workspace_bytes, int64_t n, int64_t l, int64_t c,
                      int64_t groups, float eps, int act, int dtype, void *stream) {
    dw::NormSizes s;
    int rc = check_norm(0, n, l, c, groups, act, dtype, &s);
    if (rc != DW_OK || n == 0) return rc;
    s.eps = eps;
    const int64_t e = elem_size(dtype), rows = n * l;
    for (const void *p : {x, gamma, beta, static_cast<const void *>(y)})
        if (!p || !aligned(p, e)) return DW_EPTR;
    if (!mean || !rstd || !aligned(mean, 4) || !aligned(rstd, 4) || !codes != !exps) return DW_EPTR;
    if (codes) {
        rc = check_act8(x, codes, exps, rows, c, dtype);
        if (rc != DW_OK) return rc;
    }
    const int64_t need = dw::norm_workspace(0, s);
    rc = check_workspace(workspace, workspace_bytes, need);
    if (rc != DW_OK) return rc;
    const Span outs[] = {{y, rows * c * e}, {mean, n * groups * 4}, {rstd, n * groups * 4}, codes_span(codes, rows, c),
                         exps_span(exps, rows, c), {need ? workspace : nullptr, need}};
    const Span ins[] = {{x, rows * c * e}, {gamma, c * e}, {beta, c * e}};
    if (any_overlap(outs, ins)) return DW_EALIAS;
    return map_launch(dw::norm_fwd_launch(s, x, gamma, beta, y, mean, rstd, codes, exps, need ? workspace : nullptr,
                                          static_cast<hipStream_t>(stream)));
}

int groupnorm_act_bwd(const void *dy, const void *x, const int8_t *codes, const int8_t *exps, const float *mean,
                      const float *rstd, const void *gamma, const void *beta, void *dx, void *dgamma, void *dbeta,
                      void *workspace, size_t workspace_bytes, int64_t n, int64_t l, int64_t c, int64_t groups, int act,
                      int dtype, void *stream) {
    dw::NormSizes s;
    int rc = check_norm(1, n, l, c, groups, act, dtype, &s);
    if (rc != DW_OK || n == 0) return rc;
    const int64_t e = elem_size(dtype), rows = n * l;
    for (const void *p : {dy, gamma, beta, static_cast<const void *>(dx), static_cast<const void *>(dgamma),
                          static_cast<const void *>(dbeta)})
        if (!p || !aligned(p, e)) return DW_EPTR;
    if (!mean || !rstd || !aligned(mean, 4) || !aligned(rstd, 4)) return DW_EPTR;
    if (x ? (codes || exps || !aligned(x, e)) : (!codes || !exps)) return DW_EPTR;
    const int64_t need = dw::norm_workspace(1, s);
    rc = check_workspace(workspace, workspace_bytes, need);
    if (rc != DW_OK) return rc;
    const Span outs[] = {{dx, rows * c * e}, {dgamma, c * e}, {dbeta, c * e}, {need ? workspace : nullptr, need}};
    const Span ins[] = {{dy, rows * c * e}, {x, rows * c * e}, codes_span(codes, rows, c), exps_span(exps, rows, c),
                        {mean, n * groups * 4}, {rstd, n * groups * 4}, {gamma, c * e}, {beta, c * e}};
    if (any_overlap(outs, ins)) return DW_EALIAS;
    return map_launch(dw::norm_bwd_launch(s, dy, x, codes, exps, mean, rstd, gamma, beta, dx, dgamma, dbeta, workspace,
                                          static_cast<hipStream_t>(stream)));
}

}  // extern "C"
