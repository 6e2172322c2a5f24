// dw_norm.hip -- group norm with an activation over channels-last tensors, and its gradients:
//
//   xhat = (x - mean) rstd,  z = xhat gamma + beta,  y = act(z);  mean and variance over the l
//   positions and the channels of a group, for each of the n samples.
//   dz = dy act'(z), g = dz gamma,  dx = rstd (g - mean(g) - xhat mean(g xhat)),
//   dgamma = sum dz xhat, dbeta = sum dz over samples and positions.
//
// Memory bound: x in and y out forward, x (or its 8-bit checkpoint) and dy in and dx out
// backward.  Two forms:
//  - one position (l = 1): a group is a run of adjacent values, held in the registers of one to 64
//    lanes, so the tensors are read once and the variance is taken about the exact mean;
//  - otherwise a pass for the sums and a pass for the result, over slabs of positions.  A thread
//    keeps eight channels and strides over rows; its sums are taken about its first values, and
//    (count, mean, M2) triples are joined about the common mean, so that a mean far from zero or
//    a few large values cost no digits.
// 16384 rows of 1024 bf16 with SiLU: 14.3 us, 4.7 TB/s, where about 70 vector cycles a value, two
// transcendentals among them, weigh as much as memory; 64 x 3136 x 128 fp16 in two passes: 14 and 19 us.
// Sums are fp32, in a fixed order.  A value keeps its own subtraction of the mean: folding the mean
// into the offset would lose what beta - mean rstd gamma cancels.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "dw_act8.hpp"
#include "dw_internal.hpp"
#include "dw_seq.hpp"
#include "dwseq.h"

namespace dw {
namespace {

// The normal distribution's Phi(z), and exp(-z^2 / 2) into e.  With x = |z| / sqrt(2) and
// t = 1 / (1 + 0.45 x), erfc(x) exp(x^2) = t Q(t): Q is a polynomial of degree 9 fitted to the least
// largest relative error (3.2e-8 over all x >= 0; 1.7e-7 with its steps in fp32), so the tail keeps its
// digits, and the exponential is the one that the slope needs too.  About 25 issue slots without a
// branch, where erff and a second exp took about 60.
__device__ __forceinline__ float normal_cdf(float z, float *e) {
    const float t = __builtin_amdgcn_rcpf(fmaf(0.31819805f, fabsf(z), 1.f));
    float q = -0.041399103f;
    q = fmaf(q, t, 0.19072266f);
    q = fmaf(q, t, -0.30064568f);
    q = fmaf(q, t, 0.14246328f);
    q = fmaf(q, t, -0.022394108f);
    q = fmaf(q, t, 0.11996298f);
    q = fmaf(q, t, 0.1752496f);
    q = fmaf(q, t, 0.22827192f);
    q = fmaf(q, t, 0.25388315f);
    q = fmaf(q, t, 0.25388533f);
    *e = __expf(-0.5f * z * z);
    const float half = 0.5f * q * t * *e;
    return z >= 0.f ? 1.f - half : half;
}
// 1 / sqrt(v) for v > 0: the hardware's estimate (1 ulp) and a Newton step, where a square root and a division
// with their checks take about 25 instructions.  Estimates that a step would spoil stay: infinity and zero.
__device__ __forceinline__ float inverse_root(float v) {
    const float r = __builtin_amdgcn_rsqf(v), h = 0.5f * r, e = fmaf(-(v * r), h, 0.5f);
    return v >= 0x1p-100f && v <= 0x1p100f ? fmaf(r, e, r) : 1.f / sqrtf(v);
}
// A few values' activation; one branch for all.
template <int N> __device__ __forceinline__ void act_of(float (&z)[N], int act) {
    if (act == DW_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] *= __builtin_amdgcn_rcpf(1.f + __expf(-z[i]));
    } else if (act == DW_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float e;
            z[i] *= normal_cdf(z[i], &e);
        }
    }
}
// d times the activation's slope at z.
template <int N> __device__ __forceinline__ void times_slope(float (&d)[N], const float (&z)[N], int act) {
    if (act == DW_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float s = __builtin_amdgcn_rcpf(1.f + __expf(-z[i]));
            d[i] *= s * (1.f + z[i] * (1.f - s));
        }
    } else if (act == DW_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float e;
            const float c = normal_cdf(z[i], &e);
            d[i] *= fmaf(z[i] * 0.39894228f, e, c);
        }
    }
}

// Sum over `lanes` adjacent lanes (a power of two, the same for the whole wave), in each of them.
// Within 16 lanes the partner's value comes by DPP (quads exchanged, then half rows and rows mirrored,
// which pairs lanes whose sums are already equal), beyond by lane swaps: no LDS.
template <int CTRL> __device__ __forceinline__ float dpp(float v) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float group_sum(float v, int lanes) {
    if (lanes > 1) v += dpp<0xb1>(v);    // quad_perm 1 0 3 2
    if (lanes > 2) v += dpp<0x4e>(v);    // quad_perm 2 3 0 1
    if (lanes > 4) v += dpp<0x141>(v);   // row_half_mirror
    if (lanes > 8) v += dpp<0x140>(v);   // row_mirror
    if (lanes > 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    if (lanes > 32) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    return v;
}
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
    v = max(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0xb1, 0xf, 0xf, true)));
    return max(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x4e, 0xf, 0xf, true)));
}

// n values of a row (n <= 8, zeros after), as they are in memory until they are used: no branches, so
// that the loads of several rows are in flight together.  FULL: n is 8 or 0 in every lane, and with 0
// the values are some that exist.  Where there is nothing to read, p is an address that may be read.
template <typename T, bool FULL> struct Unit {
    T v[8];
    __device__ __forceinline__ void load(const T *p, int n) {
        if constexpr (FULL) {
            __builtin_memcpy(v, p, sizeof(v));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = p[min(i, max(n, 1) - 1)];
        }
    }
    __device__ __forceinline__ void get(float (&x)[8], int n) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = FULL || i < n ? to_f32(v[i]) : 0.f;
    }
};

// The backward's view of the input: the tensor itself, or its checkpoint.
template <typename T, bool CK, bool FULL> struct Input {
    const T *x;
    const int8_t *codes, *exps;
    int64_t c, nb;
    struct Held {
        Unit<T, FULL> x;
    };
    __device__ __forceinline__ void load(Held &h, int64_t row, int ch, int n) const { h.x.load(x + row * c + ch, n); }
    __device__ __forceinline__ void get(const Held &h, float (&v)[8], int ch, int n) const { h.x.get(v, n); }
};
template <typename T, bool FULL> struct Input<T, true, FULL> {
    const T *x;
    const int8_t *codes, *exps;
    int64_t c, nb;
    struct Held {
        int8_t q[8], lo, hi;  // codes, and the exponents of the first and the last value's blocks
    };
    __device__ __forceinline__ void load(Held &h, int64_t row, int ch, int n) const {
        const int8_t *p = codes + row * c + ch, *e = exps + row * nb;
        if constexpr (FULL) {
            __builtin_memcpy(h.q, p, 8);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) h.q[i] = p[min(i, max(n, 1) - 1)];
        }
        h.lo = e[ch >> 5];
        h.hi = e[(ch + max(n, 1) - 1) >> 5];
    }
    __device__ __forceinline__ void get(const Held &h, float (&v)[8], int ch, int n) const {
        if (FULL && h.lo == h.hi) {  // one step for all eight
            uint2 q;
            __builtin_memcpy(&q, h.q, 8);
            act8_values(q, h.lo, largest_finite<float>(), v);
            return;
        }
        const float lo = act8_step(h.lo), hi = act8_step(h.hi);
        const int edge = 32 - (ch & 31);  // values before the next block
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = FULL || i < n ? act8_value(h.q[i], i < edge ? lo : hi, largest_finite<float>()) : 0.f;
    }
};

// ---------------------------------------------------------------- one position
// u lanes hold a group: lane j of them channels 8 j .. 8 j + 7 of it.  A workgroup takes gb groups
// of `rows` rows at a time and strides over the rows, so a thread keeps its channels.
struct TokenGrid {
    int u, gb, rows;     // lanes of a group, groups and rows of a workgroup
    int gblocks, blocks; // workgroups along the groups and along the rows
};
struct TokenArgs {
    int64_t n;
    int c, groups, cg, u, gb, rows, act;
    float eps;
};
struct TokenPlace {
    int g, ch, n;  // group, first channel (one that exists), channels (0: none)
    int64_t row;
};
__device__ __forceinline__ TokenPlace token_place(const TokenArgs &a) {
    const int slot = threadIdx.x / a.u, j = threadIdx.x % a.u;
    const int r = slot / a.gb;
    TokenPlace p;
    p.g = min(static_cast<int>(blockIdx.y) * a.gb + slot % a.gb, a.groups - 1);
    p.n = r < a.rows && static_cast<int>(blockIdx.y) * a.gb + slot % a.gb < a.groups ? max(0, min(8, a.cg - 8 * j)) : 0;
    p.ch = p.g * a.cg + (p.n > 0 ? 8 * j : 0);
    p.row = static_cast<int64_t>(blockIdx.x) * a.rows + min(r, a.rows - 1);
    return p;
}

// FULL: groups of whole units.  UN rows of a thread are in flight at once.
template <typename T, bool CK, bool FULL, int UN>
__global__ __launch_bounds__(kThreads) void norm_token_fwd_kernel(TokenArgs a, const T *x, const T *gamma, const T *beta, T *y,
                                                                  float *mean, float *rstd, int8_t *codes, int8_t *exps) {
    const TokenPlace p = token_place(a);
    float gm[8], bt[8];
    load_upto8(gamma + p.ch, p.n, gm);
    load_upto8(beta + p.ch, p.n, bt);
    const float inv = 1.f / a.cg;
    const int64_t step = static_cast<int64_t>(gridDim.x) * a.rows;
    for (int64_t first = p.row; first - p.row < a.n; first += UN * step) {  // the same turns in every lane
        Unit<T, FULL> raw[UN];
#pragma unroll
        for (int k = 0; k < UN; ++k) raw[k].load(x + min(first + k * step, a.n - 1) * a.c + p.ch, p.n);
#pragma unroll
        for (int k = 0; k < UN; ++k) {
            const int64_t row = first + k * step;
            if (row >= a.n) break;  // a group's lanes leave together
            float v[8];
            raw[k].get(v, p.n);
            // a lane without channels adds nothing
            const float sum = ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
            const float m = group_sum(p.n > 0 ? sum : 0.f, a.u) * inv;
            float d[8], s = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                d[i] = FULL || i < p.n ? v[i] - m : 0.f;
                s = fmaf(d[i], d[i], s);
            }
            const float rs = inverse_root(group_sum(p.n > 0 ? s : 0.f, a.u) * inv + a.eps);
            if constexpr (CK) {  // groups of whole blocks of 32: four adjacent lanes hold one
                const int e = act8_exponent(quad_max(act8_top(v)));
                const uint2 q = act8_codes(v, e);
                if (p.n > 0) {
                    __builtin_memcpy(codes + row * a.c + p.ch, &q, 8);
                    if (p.ch % 32 == 0) exps[(row * a.c + p.ch) / 32] = static_cast<int8_t>(e);
                }
            }
            if (p.n == 0) continue;
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] = d[i] * (rs * gm[i]) + bt[i];
            act_of(d, a.act);
            store_upto8(y + row * a.c + p.ch, FULL ? 8 : p.n, d);
            if (threadIdx.x % a.u == 0) {
                mean[row * a.groups + p.g] = m;
                rstd[row * a.groups + p.g] = rs;
            }
        }
    }
}

constexpr int kTokenBwd = 512;  // threads of the backward's workgroups: fewer rows of partial sums
// part: (workgroups along the rows, 2, c): the sums of dz xhat and of dz over a workgroup's rows
template <typename T, bool CK, bool FULL>
__global__ __launch_bounds__(kTokenBwd) void norm_token_bwd_kernel(TokenArgs a, const T *dy, Input<T, CK, FULL> in, const T *gamma,
                                                                   const T *beta, const float *mean, const float *rstd, T *dx,
                                                                   float *part) {
    constexpr int UN = 2;  // rows of a thread in flight
    __shared__ float sum[2][8][kTokenBwd];
    const TokenPlace p = token_place(a);
    float gm[8], bt[8], sg[8], sb[8];
    load_upto8(gamma + p.ch, p.n, gm);
    load_upto8(beta + p.ch, p.n, bt);
#pragma unroll
    for (int i = 0; i < 8; ++i) sg[i] = sb[i] = 0.f;
    const float inv = 1.f / a.cg;
    const int64_t step = static_cast<int64_t>(gridDim.x) * a.rows;
    for (int64_t first = p.row; first - p.row < a.n; first += UN * step) {
        typename Input<T, CK, FULL>::Held raw[UN];
        Unit<T, FULL> rawd[UN];
        float ms[UN], rss[UN];
#pragma unroll
        for (int k = 0; k < UN; ++k) {
            const int64_t row = min(first + k * step, a.n - 1);
            in.load(raw[k], row, p.ch, p.n);
            rawd[k].load(dy + row * a.c + p.ch, p.n);
            ms[k] = mean[row * a.groups + p.g];
            rss[k] = rstd[row * a.groups + p.g];
        }
#pragma unroll
        for (int k = 0; k < UN; ++k) {
            const int64_t row = first + k * step;
            if (row >= a.n) break;  // a group's lanes leave together
            float v[8], d[8], z[8];
            in.get(raw[k], v, p.ch, p.n);
            rawd[k].get(d, p.n);
            float s1 = 0.f, s2 = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] = (v[i] - ms[k]) * rss[k];
                z[i] = v[i] * gm[i] + bt[i];
            }
            times_slope(d, z, a.act);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (!FULL && i >= p.n) continue;
                sg[i] = fmaf(d[i], v[i], sg[i]);
                sb[i] += d[i];
                d[i] *= gm[i];
                s1 += d[i];
                s2 = fmaf(d[i], v[i], s2);
            }
            s1 = group_sum(p.n > 0 ? s1 : 0.f, a.u) * inv;
            s2 = group_sum(p.n > 0 ? s2 : 0.f, a.u) * inv;
            if (p.n == 0) continue;
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] = (d[i] - s1 - v[i] * s2) * rss[k];
            store_upto8(dx + row * a.c + p.ch, FULL ? 8 : p.n, d);
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[0][i][threadIdx.x] = sg[i], sum[1][i][threadIdx.x] = sb[i];
    __syncthreads();
    const int width = a.gb * a.u;
    if (static_cast<int>(threadIdx.x) < width) {
        for (int r = 1; r < a.rows; ++r)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sg[i] += sum[0][i][threadIdx.x + r * width];
                sb[i] += sum[1][i][threadIdx.x + r * width];
            }
        float *to = part + static_cast<int64_t>(blockIdx.x) * 2 * a.c + p.ch;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < p.n) to[i] = sg[i], to[a.c + i] = sb[i];
    }
}

// ---------------------------------------------------------------- maps that fit
// A workgroup takes whole groups of a sample, all positions of them, in registers: the tensors are read
// once and the variance is taken about the exact mean.  A lane keeps V consecutive channels of one group
// (V divides the channels of a group) and every R-th row, K of them at most.  Workgroups of one sample
// follow each other on one XCD (workgroup w runs on XCD w mod 8), so that the parts of a memory line
// that several of them read come from its L2.  (512 groups of 784 x 9 fp32 values: forward 13 us,
// backward 17, against 20 and 26 in the two passes below.)
struct SlabGrid {
    int v, threads, gb, rows;  // channels of a lane, threads, groups of a workgroup, rows at a time
};
struct SlabArgs {
    int64_t n;
    int l, c, groups, cg, gb, rows, act;
    float eps;
};
struct SlabPlace {
    int64_t sample;
    int g, ch, r, slot;  // group, first channel, first row (l or more: none), place among the group's lanes
    int gl, lanes;       // the group within the workgroup and a group's lanes
    bool live;
};
template <int V> __device__ __forceinline__ bool slab_place(const SlabArgs &a, SlabPlace *p) {
    const int per = a.groups / a.gb;  // workgroups of a sample
    const uint32_t y = blockIdx.x >> 3;
    p->sample = static_cast<int64_t>(y / per) * 8 + (blockIdx.x & 7u);
    if (p->sample >= a.n) return false;
    const int units = a.cg / V, width = a.gb * units, lr = threadIdx.x % width;
    const int r = threadIdx.x / width;
    p->live = r < a.rows;
    p->gl = lr / units;
    p->g = static_cast<int>(y % per) * a.gb + p->gl;
    p->ch = p->g * a.cg + (lr % units) * V;
    p->r = p->live ? r : a.l;
    p->lanes = a.rows * units;
    p->slot = p->gl * p->lanes + r * units + lr % units;
    return true;
}
// The sums over each group's lanes of a value pair, in every lane of the group.
__device__ __forceinline__ float2 slab_sum(float2 v, const SlabPlace &p, int gb, float2 *red, float2 *res) {
    const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
    if (gb == 1) {  // a wave's lanes are all of one group
        v = make_float2(group_sum(p.live ? v.x : 0.f, 64), group_sum(p.live ? v.y : 0.f, 64));
        __syncthreads();  // the sums before these have been read
        if (lane == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        float2 s = red[0];
        for (int w = 1; w < waves; ++w) s.x += red[w].x, s.y += red[w].y;
        return s;
    }
    if (p.live) red[p.slot] = v;
    __syncthreads();
    for (int g = threadIdx.x >> 6; g < gb; g += waves) {
        float2 s = make_float2(0.f, 0.f);
        for (int e = lane; e < p.lanes; e += 64) s.x += red[g * p.lanes + e].x, s.y += red[g * p.lanes + e].y;
        s = make_float2(group_sum(s.x, 64), group_sum(s.y, 64));
        if (lane == 0) res[g] = s;
    }
    __syncthreads();
    return res[p.gl];
}
template <typename T, int V> struct Few { T v[V]; };
// Keeps the compiler from holding the values' conversions to fp32 from one use to the next.
template <typename T, int V> __device__ __forceinline__ void as_stored(Few<T, V> &f) {
    if constexpr (sizeof(f) % 4 == 0 && sizeof(T) < 4) {
        uint32_t w[sizeof(f) / 4];
        __builtin_memcpy(w, &f, sizeof(f));
#pragma unroll
        for (uint32_t &x : w) asm volatile("" : "+v"(x));
        __builtin_memcpy(&f, w, sizeof(f));
    }
}

template <typename T, int V, int K>
__global__ __launch_bounds__(1024) void norm_slab_fwd_kernel(SlabArgs a, const T *x, const T *gamma, const T *beta, T *y,
                                                             float *mean, float *rstd) {
    __shared__ float2 red[1024], res[1024];
    SlabPlace p;
    if (!slab_place<V>(a, &p)) return;
    const int64_t row0 = p.sample * a.l;
    Few<T, V> raw[K], rg, rb;
#pragma unroll
    for (int k = 0; k < K; ++k)  // rows past the last read it again
        if (k * a.rows < a.l) __builtin_memcpy(&raw[k], x + (row0 + min(p.r + k * a.rows, a.l - 1)) * a.c + p.ch, sizeof(raw[k]));
    __builtin_memcpy(&rg, gamma + p.ch, sizeof(rg));
    __builtin_memcpy(&rb, beta + p.ch, sizeof(rb));
    const float inv = 1.f / (static_cast<float>(a.l) * a.cg);
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
        if (k * a.rows < a.l) {
            as_stored(raw[k]);
            float t = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) t += to_f32(raw[k].v[i]);
            s += p.r + k * a.rows < a.l ? t : 0.f;
        }
    const float m = slab_sum(make_float2(s, 0.f), p, a.gb, red, res).x * inv;
    s = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
        if (k * a.rows < a.l) {
            as_stored(raw[k]);
            float t = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float d = to_f32(raw[k].v[i]) - m;
                t = fmaf(d, d, t);
            }
            s += p.r + k * a.rows < a.l ? t : 0.f;
        }
    const float rs = inverse_root(slab_sum(make_float2(s, 0.f), p, a.gb, red, res).x * inv + a.eps);
    if (!p.live) return;
    if (p.slot == p.gl * p.lanes) {
        mean[p.sample * a.groups + p.g] = m;
        rstd[p.sample * a.groups + p.g] = rs;
    }
    float gm[V], bt[V];
#pragma unroll
    for (int i = 0; i < V; ++i) gm[i] = to_f32(rg.v[i]) * rs, bt[i] = to_f32(rb.v[i]);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int r = p.r + k * a.rows;
        if (r >= a.l) break;
        float z[V];
        Few<T, V> o;
        as_stored(raw[k]);
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] = (to_f32(raw[k].v[i]) - m) * gm[i] + bt[i];
        act_of(z, a.act);
#pragma unroll
        for (int i = 0; i < V; ++i) o.v[i] = from_f32<T>(z[i]);
        __builtin_memcpy(y + (row0 + r) * a.c + p.ch, &o, sizeof(o));
    }
}

// part: (sample, 2, c): the sums of dz xhat and of dz over a sample's positions
template <typename T, int V, int K, bool CK>
__global__ __launch_bounds__(1024) void norm_slab_bwd_kernel(SlabArgs a, const T *dy, const T *x, const int8_t *codes,
                                                             const int8_t *exps, const T *gamma, const T *beta,
                                                             const float *mean, const float *rstd, T *dx, float *part) {
    extern __shared__ float chan[];  // [channel][2][row]: V * 2 floats a thread
    __shared__ float2 red[1024], res[1024];
    SlabPlace p;
    if (!slab_place<V>(a, &p)) return;
    const int64_t row0 = p.sample * a.l, nb = (a.c + 31) / 32;
    using X = typename std::conditional<CK, int8_t, T>::type;
    Few<X, V> rawx[K];
    Few<T, V> rawd[K], rg, rb;
    int8_t e[CK ? K : 1];
#pragma unroll
    for (int k = 0; k < K; ++k)
        if (k * a.rows < a.l) {
            const int64_t row = row0 + min(p.r + k * a.rows, a.l - 1), at = row * a.c + p.ch;
            if constexpr (CK) {
                __builtin_memcpy(&rawx[k], codes + at, sizeof(rawx[k]));
                e[k] = exps[row * nb + (p.ch >> 5)];  // V divides 32: one block's values
            } else {
                __builtin_memcpy(&rawx[k], x + at, sizeof(rawx[k]));
            }
            __builtin_memcpy(&rawd[k], dy + at, sizeof(rawd[k]));
        }
    __builtin_memcpy(&rg, gamma + p.ch, sizeof(rg));
    __builtin_memcpy(&rb, beta + p.ch, sizeof(rb));
    const float m = mean[p.sample * a.groups + p.g], rs = rstd[p.sample * a.groups + p.g];
    float gm[V], bt[V], sg[V], sb[V];
#pragma unroll
    for (int i = 0; i < V; ++i) gm[i] = to_f32(rg.v[i]), bt[i] = to_f32(rb.v[i]), sg[i] = sb[i] = 0.f;
    // xhat and dz of a row.  Of fp32 tensors they take the registers of x and dy; from 16 bits they would take
    // twice those and are made twice.
    constexpr bool kHeld = sizeof(T) == 4;
    float hx[kHeld ? K : 1][V], hd[kHeld ? K : 1][V];
    auto row_of = [&](int k, float (&xh)[V], float (&d)[V]) {
        float z[V];
        as_stored(rawx[k]);
        as_stored(rawd[k]);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float v;
            if constexpr (CK) v = act8_value(rawx[k].v[i], act8_step(e[k]), largest_finite<float>());
            else v = to_f32(rawx[k].v[i]);
            xh[i] = (v - m) * rs;
            z[i] = xh[i] * gm[i] + bt[i];
            d[i] = to_f32(rawd[k].v[i]);
        }
        times_slope(d, z, a.act);
    };
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (p.r + k * a.rows >= a.l) break;
        float xh[V], d[V];
        row_of(k, xh, d);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            sg[i] = fmaf(d[i], xh[i], sg[i]);
            sb[i] += d[i];
            if constexpr (kHeld) hx[k][i] = xh[i], hd[k][i] = d[i];
        }
    }
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        s.x = fmaf(gm[i], sb[i], s.x);
        s.y = fmaf(gm[i], sg[i], s.y);
    }
    const int width = a.gb * a.cg, ch0 = (p.g - p.gl) * a.cg;
    if (p.live)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float *q = chan + (p.ch - ch0 + i) * 2 * a.rows + threadIdx.x / (width / V);
            q[0] = sg[i];
            q[a.rows] = sb[i];
        }
    s = slab_sum(s, p, a.gb, red, res);  // its barriers also publish chan
    const float inv = 1.f / (static_cast<float>(a.l) * a.cg);
    s.x *= inv;
    s.y *= inv;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int r = p.r + k * a.rows;
        if (r >= a.l) break;
        float xh[V], d[V];
        if constexpr (kHeld) {
#pragma unroll
            for (int i = 0; i < V; ++i) xh[i] = hx[k][i], d[i] = hd[k][i];
        } else {
            row_of(k, xh, d);
        }
        Few<T, V> o;
#pragma unroll
        for (int i = 0; i < V; ++i) o.v[i] = from_f32<T>((d[i] * gm[i] - s.x - xh[i] * s.y) * rs);
        __builtin_memcpy(dx + (row0 + r) * a.c + p.ch, &o, sizeof(o));
    }
    const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
    for (int i = threadIdx.x >> 6; i < 2 * width; i += waves) {
        float t = 0.f;
        for (int r = lane; r < a.rows; r += 64) t += chan[i * a.rows + r];
        t = group_sum(t, 64);
        if (lane == 0) part[p.sample * 2 * a.c + (i & 1) * a.c + ch0 + (i >> 1)] = t;
    }
}

// ---------------------------------------------------------------- maps
// A workgroup takes `rows` positions of one sample and a span of whole groups, 2048 channels at a
// time: tx units of eight channels by ty rows of threads.
struct MapGrid {
    int gb, gblocks;    // groups of a workgroup, workgroups along the groups
    int tx, ty, steps;  // threads along channels and rows; 2048-channel steps of a span
    int splits, rows;   // workgroups along the positions, positions of each
    bool join;          // the passes for the result join the slabs' sums themselves
};
struct MapArgs {
    int l, rows, c, groups, cg, gb, tx, ty, steps, splits, act, join;
    float eps;
};
struct MapPlace {
    int64_t sample, row0;    // the sample and its slab's first row among all (sample, position) rows
    int split, count;        // the slab and its positions
    int g0, ng, ch0, width;  // groups and channels of the span
    int tx, ty;
};
__device__ __forceinline__ MapPlace map_place(const MapArgs &a) {
    MapPlace p;
    p.sample = blockIdx.x / a.splits;
    p.split = blockIdx.x % a.splits;
    p.row0 = p.sample * a.l + p.split * a.rows;
    p.count = min(a.rows, a.l - p.split * a.rows);
    p.g0 = blockIdx.y * a.gb;
    p.ng = min(a.gb, a.groups - p.g0);
    p.ch0 = p.g0 * a.cg;
    p.width = p.ng * a.cg;
    p.tx = threadIdx.x % a.tx;
    p.ty = threadIdx.x / a.tx;
    return p;
}
// A thread's unit in a step of the span: its first channel there (one that exists) and its channels.
struct MapUnit {
    int at, n;
};
__device__ __forceinline__ MapUnit map_unit(const MapArgs &a, const MapPlace &p, int st) {
    const int at = 8 * (st * kThreads + p.tx), n = p.ty < a.ty ? max(0, min(8, p.width - at)) : 0;
    return {n > 0 ? at : 0, n};
}
// The group (in the span) of each of a unit's channels.
struct UnitGroups {
    int g[8];
};
__device__ __forceinline__ UnitGroups unit_groups(const MapUnit &m, int cg) {
    UnitGroups u;
    int g = m.at / cg, left = cg - m.at % cg;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        u.g[i] = i < m.n ? g : 0;
        if (--left == 0) ++g, left = cg;
    }
    return u;
}

constexpr int kSpan = 8 * kThreads;  // channels of a step
// Rows of a thread in flight: 64 bytes of a tensor.
template <typename T> constexpr int rows_in_flight() { return sizeof(T) == 4 ? 2 : 4; }

// Lanes that share a group's sums: a power of two, at most 64, all groups at once where they fit.
__device__ __forceinline__ int lanes_of(int groups) {
    int lanes = 64;
    while (lanes > 1 && lanes * groups > kThreads) lanes >>= 1;
    return lanes;
}

// stat: (sample, group, split, 2): mean and sum of squares about it
template <typename T, bool FULL>
__global__ __launch_bounds__(kThreads) void norm_map_stat_kernel(MapArgs a, const T *x, float *stat) {
    constexpr int kRows = rows_in_flight<T>();
    __shared__ float sm[kSpan], sq[kSpan];  // [ty][channel], then [channel]: means and sums of squares
    const MapPlace p = map_place(a);
    const int each = p.count / a.ty, more = p.count % a.ty;  // rows of a row of threads: each, or one more
    float gmean = 0.f, gsq = 0.f;                            // of a span of several steps: one group
    for (int st = 0; st < a.steps; ++st) {
        const MapUnit m = map_unit(a, p, st);
        const int w = min(p.width - st * kSpan, 8 * a.tx);
        const T *q = x + p.row0 * a.c + p.ch0 + m.at;
        float s1[8], s2[8], x0[8];
        Unit<T, FULL> raw[kRows];
#pragma unroll
        for (int k = 0; k < kRows; ++k) raw[k].load(q + static_cast<int64_t>(min(p.ty + k * a.ty, p.count - 1)) * a.c, m.n);
        raw[0].get(x0, m.n);
#pragma unroll
        for (int i = 0; i < 8; ++i) s1[i] = s2[i] = 0.f;
        for (int r = p.ty; r < p.count; r += kRows * a.ty) {
            Unit<T, FULL> now[kRows];
#pragma unroll
            for (int k = 0; k < kRows; ++k) now[k] = raw[k];
            if (const int to = r + kRows * a.ty; to < p.count) {  // in flight while these are added
#pragma unroll
                for (int k = 0; k < kRows; ++k) raw[k].load(q + static_cast<int64_t>(min(to + k * a.ty, p.count - 1)) * a.c, m.n);
            }
#pragma unroll
            for (int k = 0; k < kRows; ++k) {
                if (r + k * a.ty >= p.count) break;
                float v[8];
                now[k].get(v, m.n);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float d = v[i] - x0[i];
                    s1[i] += d;
                    s2[i] = fmaf(d, d, s2[i]);
                }
            }
        }
        const int mine = each + (p.ty < more);
        const float inv = mine > 0 ? 1.f / mine : 0.f;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < m.n) {
                const float d = s1[i] * inv, e = s2[i] - s1[i] * d;
                sm[p.ty * w + 8 * p.tx + i] = x0[i] + d;
                sq[p.ty * w + 8 * p.tx + i] = e < 0.f ? 0.f : e;
            }
        __syncthreads();
        // a channel's rows of threads, then a group's channels, joined about their common means
        const float all = 1.f / p.count;
        for (int ch = threadIdx.x; ch < w; ch += kThreads) {
            float s = 0.f, q2 = 0.f;
            for (int ty = 0; ty < a.ty; ++ty) s = fmaf(static_cast<float>(each + (ty < more)), sm[ty * w + ch], s);
            const float mu = s * all;
            for (int ty = 0; ty < a.ty; ++ty) {
                const float d = sm[ty * w + ch] - mu;
                const int k = each + (ty < more);
                if (k > 0) q2 += sq[ty * w + ch] + static_cast<float>(k) * d * d;
            }
            sm[ch] = mu;  // row 0 of the threads: read by this thread alone
            sq[ch] = q2;
        }
        __syncthreads();
        const int lanes = lanes_of(p.ng), part = min(a.cg, w);  // channels of a group in this step
        for (int g0 = 0; g0 < p.ng; g0 += kThreads / lanes) {
            const int g = g0 + static_cast<int>(threadIdx.x) / lanes, j = threadIdx.x % lanes;
            const int entries = g < p.ng ? part : 0;
            float s = 0.f, q2 = 0.f;
            for (int e = j; e < entries; e += lanes) s += sm[g * a.cg + e];
            const float mu = group_sum(s, lanes) / part;
            for (int e = j; e < entries; e += lanes) {
                const float d = sm[g * a.cg + e] - mu;
                q2 += sq[g * a.cg + e] + p.count * (d * d);
            }
            q2 = group_sum(q2, lanes);
            if (a.steps > 1) {  // one group over several steps: join with the steps before
                const float before = static_cast<float>(st) * kSpan, sum = before + part, d = mu - gmean;
                gmean += d * (part / sum);
                gsq += q2 + d * d * (p.count * (before * (part / sum)));
                if (st + 1 < a.steps) continue;
            } else {
                gmean = mu;
                gsq = q2;
            }
            if (g < p.ng && j == 0) {
                float *to = stat + ((p.sample * a.groups + p.g0 + g) * a.splits + p.split) * 2;
                to[0] = gmean;
                to[1] = gsq;
            }
        }
    }
}

// Mean and rstd of a group from its slabs' (mean, sum of squares), by `lanes` adjacent lanes.
__device__ __forceinline__ float2 join_slabs(const float *q, int splits, int l, int rows, int cg, float eps, int j, int lanes) {
    float s = 0.f, q2 = 0.f;
    for (int k = j; k < splits; k += lanes) s = fmaf(static_cast<float>(min(rows, l - k * rows)), q[2 * k], s);
    const float m = group_sum(s, lanes) / static_cast<float>(l);
    for (int k = j; k < splits; k += lanes) {
        const float d = q[2 * k] - m;
        q2 += q[2 * k + 1] + static_cast<float>(min(rows, l - k * rows)) * cg * d * d;
    }
    return make_float2(m, inverse_root(group_sum(q2, lanes) / (static_cast<float>(l) * cg) + eps));
}
// A group's sums of g and of g xhat from its slabs', as means.
__device__ __forceinline__ float2 join_means(const float *q, int splits, int l, int cg, int j, int lanes) {
    float s1 = 0.f, s2 = 0.f;
    for (int k = j; k < splits; k += lanes) s1 += q[2 * k], s2 += q[2 * k + 1];
    const float inv = 1.f / (static_cast<float>(l) * cg);
    return make_float2(group_sum(s1, lanes) * inv, group_sum(s2, lanes) * inv);
}
// The same for all groups of all samples in a launch of its own, `lanes` lanes to each: for the
// forward with eps, for the backward without.
template <bool BWD>
__global__ __launch_bounds__(kThreads) void norm_map_join_kernel(const float *q, float2 *out, float *mean, float *rstd,
                                                                 int64_t items, int l, int rows, int cg, int splits, int lanes,
                                                                 float eps) {
    const int64_t item = static_cast<int64_t>(blockIdx.x) * (kThreads / lanes) + threadIdx.x / lanes;
    const int j = threadIdx.x % lanes, mine = item < items ? splits : 0;
    const float *p = q + (item < items ? item : 0) * splits * 2;
    const float2 r = BWD ? join_means(p, mine, l, cg, j, lanes) : join_slabs(p, mine, l, rows, cg, eps, j, lanes);
    if (item < items && j == 0) {
        if (BWD) out[item] = r;
        else mean[item] = r.x, rstd[item] = r.y;
    }
}

template <typename T, bool CK, bool FULL>
__global__ __launch_bounds__(kThreads) void norm_map_fwd_kernel(MapArgs a, const T *x, const T *gamma, const T *beta,
                                                                const float *stat, float *mean, float *rstd, T *y,
                                                                int8_t *codes, int8_t *exps) {
    constexpr int kRows = rows_in_flight<T>();
    __shared__ float2 ms[kSpan];  // the span's groups: at most one for each channel
    const MapPlace p = map_place(a);
    const int64_t item0 = p.sample * a.groups + p.g0;
    Unit<T, FULL> raw[kRows];
    auto load = [&](const MapUnit &u, int r0) {
#pragma unroll
        for (int k = 0; k < kRows; ++k)
            raw[k].load(x + (p.row0 + min(r0 + k * a.ty + p.ty, p.count - 1)) * a.c + p.ch0 + u.at, u.n);
    };
    load(map_unit(a, p, 0), 0);  // in flight while the groups' statistics are joined
    if (a.join) {
        const int lanes = lanes_of(p.ng);
        for (int g0 = 0; g0 < p.ng; g0 += kThreads / lanes) {
            const int g = g0 + static_cast<int>(threadIdx.x) / lanes, j = threadIdx.x % lanes;
            const int gi = min(g, p.ng - 1);
            const float2 r = join_slabs(stat + (item0 + gi) * a.splits * 2, a.splits, a.l, a.rows, a.cg, a.eps, j, lanes);
            if (g < p.ng && j == 0) {
                ms[g] = r;
                if (p.split == 0) mean[item0 + g] = r.x, rstd[item0 + g] = r.y;
            }
        }
    } else {
        for (int g = threadIdx.x; g < p.ng; g += kThreads) ms[g] = make_float2(mean[item0 + g], rstd[item0 + g]);
    }
    __syncthreads();
    for (int st = 0; st < a.steps; ++st) {
        const MapUnit u = map_unit(a, p, st);
        const UnitGroups ug = unit_groups(u, a.cg);
        float gm[8], bt[8], m[8];
        load_upto8(gamma + p.ch0 + u.at, u.n, gm);
        load_upto8(beta + p.ch0 + u.at, u.n, bt);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            m[i] = ms[ug.g[i]].x;
            gm[i] *= ms[ug.g[i]].y;
        }
        const int64_t off0 = p.row0 * a.c + p.ch0 + u.at;
        for (int r0 = 0; r0 < p.count; r0 += kRows * a.ty) {  // the same turns in every lane
            if (st > 0 && r0 == 0) load(u, r0);
            Unit<T, FULL> now[kRows];
#pragma unroll
            for (int k = 0; k < kRows; ++k) now[k] = raw[k];
            if (r0 + kRows * a.ty < p.count) load(u, r0 + kRows * a.ty);  // in flight while these are worked on
#pragma unroll
            for (int k = 0; k < kRows; ++k) {
                const int r = r0 + k * a.ty + p.ty;
                const bool live = u.n > 0 && r < p.count;
                const int64_t off = off0 + static_cast<int64_t>(r) * a.c;
                float v[8];
                now[k].get(v, u.n);
                if constexpr (CK) {  // rows of whole blocks of 32: four adjacent lanes hold one
                    const int e = act8_exponent(quad_max(act8_top(v)));
                    const uint2 q = act8_codes(v, e);
                    if (live) {
                        __builtin_memcpy(codes + off, &q, 8);
                        if (off % 32 == 0) exps[off / 32] = static_cast<int8_t>(e);
                    }
                }
                if (!live) continue;
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = (v[i] - m[i]) * gm[i] + bt[i];
                act_of(v, a.act);
                store_upto8(y + off, FULL ? 8 : u.n, v);
            }
        }
    }
}

// part: (sample, split, 2, c): the sums of dz xhat and of dz over a slab's positions.
// gpart: (sample, group, split, 2): the sums of g and of g xhat.
template <typename T, bool CK, bool FULL>
__global__ __launch_bounds__(kThreads) void norm_map_sum_kernel(MapArgs a, const T *dy, Input<T, CK, FULL> in, const T *gamma,
                                                                const T *beta, const float *mean, const float *rstd,
                                                                float *part, float *gpart) {
    constexpr int kRows = rows_in_flight<T>();
    __shared__ float sum[2][kSpan];
    const MapPlace p = map_place(a);
    float t1 = 0.f, t2 = 0.f;  // of a span of several steps: one group
    for (int st = 0; st < a.steps; ++st) {
        const MapUnit u = map_unit(a, p, st);
        const int w = min(p.width - st * kSpan, 8 * a.tx);
        const UnitGroups ug = unit_groups(u, a.cg);
        float gm[8], bt[8], m[8], rs[8], sg[8], sb[8];
        typename Input<T, CK, FULL>::Held raw[kRows];
        Unit<T, FULL> rawd[kRows];
        auto load = [&](int r0) {
#pragma unroll
            for (int k = 0; k < kRows; ++k) {
                const int64_t row = p.row0 + min(r0 + k * a.ty, p.count - 1);
                in.load(raw[k], row, p.ch0 + u.at, u.n);
                rawd[k].load(dy + row * a.c + p.ch0 + u.at, u.n);
            }
        };
        load(p.ty);
        load_upto8(gamma + p.ch0 + u.at, u.n, gm);
        load_upto8(beta + p.ch0 + u.at, u.n, bt);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t g = p.sample * a.groups + p.g0 + ug.g[i];
            m[i] = mean[g];
            rs[i] = rstd[g];
            sg[i] = sb[i] = 0.f;
        }
        for (int r0 = p.ty; r0 < p.count; r0 += kRows * a.ty) {
            if (r0 != p.ty) load(r0);
#pragma unroll
            for (int k = 0; k < kRows; ++k) {
                if (r0 + k * a.ty >= p.count) break;
                float v[8], d[8], z[8];
                in.get(raw[k], v, p.ch0 + u.at, u.n);
                rawd[k].get(d, u.n);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[i] = (v[i] - m[i]) * rs[i];
                    z[i] = v[i] * gm[i] + bt[i];
                }
                times_slope(d, z, a.act);
#pragma unroll
                for (int i = 0; i < 8; ++i) {  // what lies past a unit's channels is not written below
                    sg[i] = fmaf(d[i], v[i], sg[i]);
                    sb[i] += d[i];
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < u.n) sum[0][p.ty * w + 8 * p.tx + i] = sg[i], sum[1][p.ty * w + 8 * p.tx + i] = sb[i];
        __syncthreads();
        float *to = part + static_cast<int64_t>(blockIdx.x) * 2 * a.c + p.ch0 + st * kSpan;
        for (int ch = threadIdx.x; ch < w; ch += kThreads) {
            float s = 0.f, b = 0.f;
            for (int ty = 0; ty < a.ty; ++ty) s += sum[0][ty * w + ch], b += sum[1][ty * w + ch];
            to[ch] = s;
            to[a.c + ch] = b;
            const float g = to_f32(gamma[p.ch0 + st * kSpan + ch]);
            sum[0][ch] = s * g;  // row 0 of the threads: read by this thread alone
            sum[1][ch] = b * g;
        }
        __syncthreads();
        const int lanes = lanes_of(p.ng), mine = min(a.cg, w);
        for (int g0 = 0; g0 < p.ng; g0 += kThreads / lanes) {
            const int g = g0 + static_cast<int>(threadIdx.x) / lanes, j = threadIdx.x % lanes;
            const int entries = g < p.ng ? mine : 0;
            float s1 = 0.f, s2 = 0.f;
            for (int e = j; e < entries; e += lanes) s1 += sum[1][g * a.cg + e], s2 += sum[0][g * a.cg + e];
            s1 = group_sum(s1, lanes);
            s2 = group_sum(s2, lanes);
            if (a.steps > 1) {
                t1 += s1;
                t2 += s2;
                if (st + 1 < a.steps) continue;
                s1 = t1, s2 = t2;
            }
            if (g < p.ng && j == 0) {
                float *o = gpart + ((p.sample * a.groups + p.g0 + g) * a.splits + p.split) * 2;
                o[0] = s1;
                o[1] = s2;
            }
        }
    }
}

template <typename T, bool CK, bool FULL>
__global__ __launch_bounds__(kThreads) void norm_map_bwd_kernel(MapArgs a, const T *dy, Input<T, CK, FULL> in, const T *gamma,
                                                                const T *beta, const float *mean, const float *rstd,
                                                                const float *gpart, const float2 *means, T *dx) {
    constexpr int kRows = rows_in_flight<T>();
    __shared__ float2 ms[kSpan];
    const MapPlace p = map_place(a);
    const int64_t item0 = p.sample * a.groups + p.g0;
    typename Input<T, CK, FULL>::Held raw[kRows];
    Unit<T, FULL> rawd[kRows];
    auto load = [&](const MapUnit &u, int r0) {
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int64_t row = p.row0 + min(r0 + k * a.ty, p.count - 1);
            in.load(raw[k], row, p.ch0 + u.at, u.n);
            rawd[k].load(dy + row * a.c + p.ch0 + u.at, u.n);
        }
    };
    load(map_unit(a, p, 0), p.ty);  // in flight while the groups' sums are joined
    if (a.join) {
        const int lanes = lanes_of(p.ng);
        for (int g0 = 0; g0 < p.ng; g0 += kThreads / lanes) {
            const int g = g0 + static_cast<int>(threadIdx.x) / lanes, j = threadIdx.x % lanes;
            const float2 r = join_means(gpart + (item0 + min(g, p.ng - 1)) * a.splits * 2, a.splits, a.l, a.cg, j, lanes);
            if (g < p.ng && j == 0) ms[g] = r;
        }
    } else {
        for (int g = threadIdx.x; g < p.ng; g += kThreads) ms[g] = means[item0 + g];
    }
    __syncthreads();
    for (int st = 0; st < a.steps; ++st) {
        const MapUnit u = map_unit(a, p, st);
        if (u.n == 0) continue;
        const UnitGroups ug = unit_groups(u, a.cg);
        float gm[8], bt[8], m[8], rs[8], m1[8], m2[8];
        load_upto8(gamma + p.ch0 + u.at, u.n, gm);
        load_upto8(beta + p.ch0 + u.at, u.n, bt);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            m[i] = mean[item0 + ug.g[i]];
            rs[i] = rstd[item0 + ug.g[i]];
            m1[i] = ms[ug.g[i]].x;
            m2[i] = ms[ug.g[i]].y;
        }
        for (int r0 = p.ty; r0 < p.count; r0 += kRows * a.ty) {
            if (st > 0 || r0 != p.ty) load(u, r0);
#pragma unroll
            for (int k = 0; k < kRows; ++k) {
                if (r0 + k * a.ty >= p.count) break;
                float v[8], d[8], z[8];
                in.get(raw[k], v, p.ch0 + u.at, u.n);
                rawd[k].get(d, u.n);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[i] = (v[i] - m[i]) * rs[i];
                    z[i] = v[i] * gm[i] + bt[i];
                }
                times_slope(d, z, a.act);
#pragma unroll
                for (int i = 0; i < 8; ++i) d[i] = (d[i] * gm[i] - m1[i] - v[i] * m2[i]) * rs[i];
                store_upto8(dx + (p.row0 + r0 + k * a.ty) * a.c + p.ch0 + u.at, FULL ? 8 : u.n, d);
            }
        }
    }
}

constexpr int kColumnThreads = 1024;
// Column sums of part (rows, 2, c): workgroup (i, k) takes 32 columns and the k-th `chunk` of rows.  Into
// out (chunks, 2, c) where that is given, else into dgamma and dbeta.
template <typename T>
__global__ __launch_bounds__(kColumnThreads) void norm_column_kernel(const float *part, float *out, T *dgamma, T *dbeta,
                                                                     int64_t rows, int64_t chunk, int c) {
    __shared__ float sum[32][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + tx, last = min(rows, (blockIdx.y + int64_t{1}) * chunk);
    float s = 0.f;
    if (col < 2 * static_cast<int64_t>(c)) {
#pragma unroll 8
        for (int64_t r = blockIdx.y * chunk + ty; r < last; r += 32) s += part[r * 2 * c + col];
    }
    sum[ty][tx] = s;
    __syncthreads();
    if (ty == 0 && col < 2 * static_cast<int64_t>(c)) {
        float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int r = 0; r < 32; ++r) v[r & 3] += sum[r][tx];
        const float all = (v[0] + v[1]) + (v[2] + v[3]);
        if (out) out[static_cast<int64_t>(blockIdx.y) * 2 * c + col] = all;
        else (col < c ? dgamma : dbeta)[col < c ? col : col - c] = from_f32<T>(all);
    }
}

int done() { return hipGetLastError() == hipSuccess ? kOk : kErrHip; }

// A group of one position in at most 64 lanes of eight channels.
bool token_form(const NormSizes &s) { return s.l == 1 && s.c / s.groups <= 512; }
// Rows of a thread in flight in the forward: more waves of one row each cover the waits better (16384 rows
// of 1024 bf16 values: one row 16.1 us, two 17.1, four 19.5).
constexpr int kTokenRows = 1;

TokenGrid token_grid(const NormSizes &s, int pass) {
    TokenGrid t;
    const int cg = static_cast<int>(s.c / s.groups), units = (cg + 7) / 8, threads = pass ? kTokenBwd : kThreads;
    t.u = 1;
    while (t.u < units) t.u *= 2;
    t.gb = std::min(s.groups, threads / t.u);
    t.rows = std::max(1, threads / t.u / t.gb);
    t.gblocks = (s.groups + t.gb - 1) / t.gb;
    const int64_t un = pass ? 2 : kTokenRows, full = (s.n + t.rows * un - 1) / (t.rows * un);
    // the backward's workgroups each leave a row of partial sums: few enough that these stay small
    const int64_t want = std::max<int64_t>(1, (pass ? 512 : 4096) / t.gblocks);
    t.blocks = static_cast<int>(std::min(full, want));
    return t;
}
TokenArgs token_args(const NormSizes &s, const TokenGrid &t) {
    return {s.n, static_cast<int>(s.c), s.groups, static_cast<int>(s.c / s.groups), t.u, t.gb, t.rows, s.act, s.eps};
}

// Rows that a lane of a slab holds: 40 registers of the forward's tensor, 16 of each of the backward's.
constexpr int slab_rows(int bytes, int pass) {
    const int regs = bytes < 4 ? 1 : bytes / 4, k = (pass ? 16 : 40) / regs;
    return k < 16 ? k : 16;
}
// The slab's form of a pass; threads 0 where the groups do not fit.  A workgroup takes as many groups as
// fit the fewest threads.  A 128-byte line that several workgroups read has to stay in their XCD's L2 from
// the first to the last of them: rows of less than 64 bytes are taken only of tensors that the L2s hold
// (32 MB).  Measured, forward: 16 x 784 x 288 fp32 (14 MB, 36-byte rows) 13 us against 20 us in two
// passes; 64 x 3136 x 128 fp16 (51 MB, 32-byte rows) 37 us against 34.
SlabGrid slab_grid(const NormSizes &s, int pass) {
    SlabGrid g{0, 0, 0, 0};
    const int e = s.dtype == DW_F32 ? 4 : 2;
    const int64_t cg = s.c / s.groups;
    g.v = 16 / e;
    while (cg % g.v) g.v /= 2;
    const int k = slab_rows(g.v * e, pass);
    const int64_t units = cg / g.v;
    const bool resident = s.n * s.l * s.c * e <= (32 << 20);
    for (int threads : {256, 512, 1024})
        for (int gb = static_cast<int>(std::min<int64_t>(s.groups, threads / units)); gb >= 1; --gb) {
            const int64_t width = gb * units;
            if (gb < s.groups && width * g.v * e < (resident ? 32 : 64)) break;
            const int64_t rows = std::min<int64_t>(threads / width, s.l);
            if (rows * k < s.l || s.groups % gb) continue;
            if ((s.n + 7) / 8 * 8 * (s.groups / gb) * threads > UINT32_MAX) continue;  // threads of the launch
            g.threads = threads;
            g.gb = gb;
            g.rows = static_cast<int>(rows);
            return g;
        }
    return g;
}
SlabArgs slab_args(const NormSizes &s, const SlabGrid &g) {
    return {s.n, static_cast<int>(s.l), static_cast<int>(s.c), s.groups, static_cast<int>(s.c / s.groups), g.gb, g.rows, s.act,
            s.eps};
}
uint32_t slab_blocks(const NormSizes &s, const SlabGrid &g) {
    return static_cast<uint32_t>((s.n + 7) / 8 * 8 * (s.groups / g.gb));
}
template <typename T, int V>
void slab_fwd(const NormSizes &s, const SlabGrid &g, const T *x, const T *gamma, const T *beta, T *y, float *mean, float *rstd,
              hipStream_t st) {
    hipLaunchKernelGGL((norm_slab_fwd_kernel<T, V, slab_rows(V * sizeof(T), 0)>), dim3(slab_blocks(s, g)), dim3(g.threads), 0, st,
                       slab_args(s, g), x, gamma, beta, y, mean, rstd);
}
template <typename T, bool CK, int V>
void slab_bwd(const NormSizes &s, const SlabGrid &g, const T *dy, const T *x, const int8_t *codes, const int8_t *exps,
              const T *gamma, const T *beta, const float *mean, const float *rstd, T *dx, float *part, hipStream_t st) {
    hipLaunchKernelGGL((norm_slab_bwd_kernel<T, V, slab_rows(V * sizeof(T), 1), CK>), dim3(slab_blocks(s, g)), dim3(g.threads),
                       g.threads * V * 8, st, slab_args(s, g), dy, x, codes, exps, gamma, beta, mean, rstd, dx, part);
}

MapGrid map_grid(const NormSizes &s) {
    MapGrid m;
    const int64_t cg = s.c / s.groups;
    m.gb = static_cast<int>(std::min<int64_t>(s.groups, std::max<int64_t>(1, kSpan / cg)));
    m.gblocks = (s.groups + m.gb - 1) / m.gb;
    const int64_t width = m.gb * cg;
    m.steps = static_cast<int>((width + kSpan - 1) / kSpan);
    m.tx = static_cast<int>(std::min<int64_t>(kThreads, (width + 7) / 8));
    m.ty = kThreads / m.tx;
    // about 1024 workgroups, of at least the rows a thread has in flight
    const int64_t want = std::max<int64_t>(1, 1024 / std::max<int64_t>(1, s.n * m.gblocks));
    const int64_t most = std::max<int64_t>(1, s.l / ((s.dtype == DW_F32 ? 2 : 4) * m.ty));
    const int64_t splits = std::min(want, most);
    m.rows = static_cast<int>((s.l + splits - 1) / splits);
    m.splits = static_cast<int>((s.l + m.rows - 1) / m.rows);
    // each workgroup of the second pass joins its groups' slabs again: while that is little work, it
    // saves a launch
    m.join = static_cast<int64_t>(m.splits) * m.gb <= 4096;
    return m;
}
MapArgs map_args(const NormSizes &s, const MapGrid &m) {
    return {static_cast<int>(s.l), m.rows, static_cast<int>(s.c), s.groups, static_cast<int>(s.c / s.groups), m.gb, m.tx, m.ty,
            m.steps, m.splits, s.act, m.join, s.eps};
}

// Whether the four lanes of every block of 32 channels are neighbours in the maps' form.
bool whole_blocks(const NormSizes &s) { return s.c % 32 == 0 && map_grid(s).gb * (s.c / s.groups) % 32 == 0; }

// Lanes for items of `work` entries: a power of two, each lane about `each` of them.
int lanes_for(int64_t work, int each) {
    int lanes = 1;
    while (lanes < 64 && static_cast<int64_t>(lanes) * each < work) lanes *= 2;
    return lanes;
}
uint32_t lane_blocks(int64_t items, int lanes) { return static_cast<uint32_t>((items * lanes + kThreads - 1) / kThreads); }

int64_t part_rows(const NormSizes &s) {
    return token_form(s) ? token_grid(s, 1).blocks : slab_grid(s, 1).threads ? s.n : s.n * map_grid(s).splits;
}
// The two-pass form of maps.
bool two_pass(const NormSizes &s, int pass) { return !token_form(s) && !slab_grid(s, pass).threads; }
int64_t round256(int64_t n) { return (n + 255) / 256 * 256; }
// Workgroups of norm_column_kernel along the 2 c columns.
uint32_t column_blocks(int64_t c) { return static_cast<uint32_t>((2 * c + 31) / 32); }
// Chunks of the rows of partial sums: a workgroup adds 32 rows at a time, and few columns alone would
// leave the card empty.
int column_chunks(int64_t rows) { return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(64, rows / 512))); }

// Where the backward's workspace parts lie, in bytes.
struct BwdSpace {
    int64_t gpart, means, mid, bytes;
};
BwdSpace bwd_space(const NormSizes &s) {
    BwdSpace w;
    w.gpart = round256(part_rows(s) * 2 * s.c * 4);
    const bool two = two_pass(s, 1);
    w.means = w.gpart + (two ? round256(s.n * s.groups * map_grid(s).splits * 8) : 0);
    w.mid = w.means + (two && !map_grid(s).join ? round256(s.n * s.groups * 8) : 0);
    const int chunks = column_chunks(part_rows(s));
    w.bytes = w.mid + (chunks > 1 ? round256(chunks * 2 * s.c * 4) : 0);
    return w;
}

template <typename T, bool CK, bool FULL>
int fwd(const NormSizes &s, const void *x, const void *gamma, const void *beta, void *y, float *mean, float *rstd,
        int8_t *codes, int8_t *exps, void *ws, hipStream_t st) {
    const T *x_ = static_cast<const T *>(x), *g = static_cast<const T *>(gamma), *b = static_cast<const T *>(beta);
    if (token_form(s)) {
        const TokenGrid t = token_grid(s, 0);
        hipLaunchKernelGGL((norm_token_fwd_kernel<T, CK, FULL, kTokenRows>), dim3(t.blocks, t.gblocks),
                           dim3(kThreads), 0, st, token_args(s, t), x_, g, b, static_cast<T *>(y), mean, rstd, codes, exps);
        return done();
    }
    if (const SlabGrid sg = slab_grid(s, 0); sg.threads) {
        auto f = sg.v == 1 ? slab_fwd<T, 1> : sg.v == 2 ? slab_fwd<T, 2> : sg.v == 4 ? slab_fwd<T, 4> : slab_fwd<T, 16 / sizeof(T)>;
        f(s, sg, x_, g, b, static_cast<T *>(y), mean, rstd, st);
        return done();
    }
    const MapGrid m = map_grid(s);
    const MapArgs a = map_args(s, m);
    const dim3 grid(static_cast<uint32_t>(s.n * m.splits), m.gblocks);
    float *stat = static_cast<float *>(ws);
    hipLaunchKernelGGL((norm_map_stat_kernel<T, FULL>), grid, dim3(kThreads), 0, st, a, x_, stat);
    if (!m.join) {
        const int64_t items = s.n * s.groups;
        const int lanes = lanes_for(m.splits, 4);
        hipLaunchKernelGGL((norm_map_join_kernel<false>), dim3(lane_blocks(items, lanes)), dim3(kThreads), 0, st, stat, nullptr,
                           mean, rstd, items, a.l, a.rows, a.cg, a.splits, lanes, s.eps);
    }
    hipLaunchKernelGGL((norm_map_fwd_kernel<T, CK, FULL>), grid, dim3(kThreads), 0, st, a, x_, g, b, stat, mean, rstd,
                       static_cast<T *>(y), codes, exps);
    return done();
}

template <typename T, bool CK, bool FULL>
int bwd(const NormSizes &s, const void *dy, const void *x, const int8_t *codes, const int8_t *exps, const float *mean,
        const float *rstd, const void *gamma, const void *beta, void *dx, void *dgamma, void *dbeta, void *ws,
        hipStream_t st) {
    const T *dy_ = static_cast<const T *>(dy), *g = static_cast<const T *>(gamma), *b = static_cast<const T *>(beta);
    const Input<T, CK, FULL> in{static_cast<const T *>(x), codes, exps, s.c, (s.c + 31) / 32};
    const BwdSpace space = bwd_space(s);
    char *w = static_cast<char *>(ws);
    float *part = static_cast<float *>(ws);
    const int64_t rows = part_rows(s);
    if (token_form(s)) {
        const TokenGrid t = token_grid(s, 1);
        hipLaunchKernelGGL((norm_token_bwd_kernel<T, CK, FULL>), dim3(t.blocks, t.gblocks), dim3(kTokenBwd), 0, st,
                           token_args(s, t), dy_, in, g, b, mean, rstd, static_cast<T *>(dx), part);
    } else if (const SlabGrid sg = slab_grid(s, 1); sg.threads) {
        auto f = sg.v == 1 ? slab_bwd<T, CK, 1> : sg.v == 2 ? slab_bwd<T, CK, 2> : sg.v == 4 ? slab_bwd<T, CK, 4>
                                                                                             : slab_bwd<T, CK, 16 / sizeof(T)>;
        f(s, sg, dy_, static_cast<const T *>(x), codes, exps, g, b, mean, rstd, static_cast<T *>(dx), part, st);
    } else {
        const MapGrid m = map_grid(s);
        const MapArgs a = map_args(s, m);
        const dim3 grid(static_cast<uint32_t>(s.n * m.splits), m.gblocks);
        float *gpart = reinterpret_cast<float *>(w + space.gpart);
        float2 *means = reinterpret_cast<float2 *>(w + space.means);
        hipLaunchKernelGGL((norm_map_sum_kernel<T, CK, FULL>), grid, dim3(kThreads), 0, st, a, dy_, in, g, b, mean, rstd, part,
                           gpart);
        if (!m.join) {
            const int64_t items = s.n * s.groups;
            const int lanes = lanes_for(m.splits, 4);
            hipLaunchKernelGGL((norm_map_join_kernel<true>), dim3(lane_blocks(items, lanes)), dim3(kThreads), 0, st, gpart, means,
                               nullptr, nullptr, items, a.l, a.rows, a.cg, a.splits, lanes, 0.f);
        }
        hipLaunchKernelGGL((norm_map_bwd_kernel<T, CK, FULL>), grid, dim3(kThreads), 0, st, a, dy_, in, g, b, mean, rstd, gpart,
                           means, static_cast<T *>(dx));
    }
    T *dg = static_cast<T *>(dgamma), *db = static_cast<T *>(dbeta);
    const uint32_t cols = column_blocks(s.c);
    const int c = static_cast<int>(s.c), chunks = column_chunks(rows);
    if (chunks == 1) {
        hipLaunchKernelGGL((norm_column_kernel<T>), dim3(cols), dim3(kColumnThreads), 0, st, part, nullptr, dg, db, rows, rows, c);
        return done();
    }
    float *mid = reinterpret_cast<float *>(w + space.mid);
    const int64_t chunk = (rows + chunks - 1) / chunks;
    hipLaunchKernelGGL((norm_column_kernel<T>), dim3(cols, chunks), dim3(kColumnThreads), 0, st, part, mid, dg, db, rows, chunk, c);
    hipLaunchKernelGGL((norm_column_kernel<T>), dim3(cols), dim3(kColumnThreads), 0, st, mid, nullptr, dg, db,
                       static_cast<int64_t>(chunks), static_cast<int64_t>(chunks), c);
    return done();
}

template <typename F> int by_type(int dtype, F f) {
    if (dtype == DW_F32) return f(float{});
    if (dtype == DW_F16) return f(__half{});
    return f(bf16_t{});
}
// Units of eight channels without a rest: of a group for one position, of a span for maps.
bool full_units(const NormSizes &s) {
    const int64_t cg = s.c / s.groups;
    return token_form(s) ? cg % 8 == 0 : s.c % 8 == 0 && map_grid(s).gb * cg % 8 == 0;
}

}  // namespace

int64_t norm_workspace(int pass, const NormSizes &s) {
    if (s.n == 0) return 0;
    if (pass == 0) return two_pass(s, 0) ? round256(s.n * s.groups * map_grid(s).splits * 8) : 0;
    return bwd_space(s).bytes;
}

// What a pass's launches hold: 2^32 - 1 threads, 65535 workgroups along the groups.  The slabs' form is taken only
// where its launch does; the join's own launch, of at most 64 lanes a group, is of at most 1024 / 3 spans of at most
// kSpan groups (three slabs or more, see map_grid()).
bool norm_grid_ok(int pass, const NormSizes &s) {
    if (pass == 1 && int64_t{column_blocks(s.c)} * kColumnThreads > UINT32_MAX) return false;
    if (token_form(s)) return token_grid(s, pass).gblocks <= 65535;
    if (!two_pass(s, pass)) return true;
    const MapGrid m = map_grid(s);
    return m.gblocks <= 65535 && s.n * m.splits * kThreads <= UINT32_MAX;
}

int norm_fwd_launch(const NormSizes &s, const void *x, const void *gamma, const void *beta, void *y, float *mean,
                    float *rstd, int8_t *codes, int8_t *exps, void *ws, hipStream_t st) {
    return by_type(s.dtype, [&](auto tag) {
        using T = decltype(tag);
        // the norm's own pass packs where a block's lanes are neighbours; elsewhere x is packed by itself
        const bool inside = codes && (token_form(s) ? (s.c / s.groups) % 32 == 0 : two_pass(s, 0) && whole_blocks(s));
        if (inside) return fwd<T, true, true>(s, x, gamma, beta, y, mean, rstd, codes, exps, ws, st);
        if (codes) {
            const int rc = act8_pack_launch(x, codes, exps, s.n * s.l, s.c, s.dtype, st);
            if (rc != kOk) return rc;
        }
        return full_units(s) ? fwd<T, false, true>(s, x, gamma, beta, y, mean, rstd, nullptr, nullptr, ws, st)
                             : fwd<T, false, false>(s, x, gamma, beta, y, mean, rstd, nullptr, nullptr, ws, st);
    });
}

int norm_bwd_launch(const NormSizes &s, const void *dy, const void *x, const int8_t *codes, const int8_t *exps,
                    const float *mean, const float *rstd, const void *gamma, const void *beta, void *dx, void *dgamma,
                    void *dbeta, void *ws, hipStream_t st) {
    return by_type(s.dtype, [&](auto tag) {
        using T = decltype(tag);
        auto f = codes ? (full_units(s) ? bwd<T, true, true> : bwd<T, true, false>)
                       : (full_units(s) ? bwd<T, false, true> : bwd<T, false, false>);
        return f(s, dy, x, codes, exps, mean, rstd, gamma, beta, dx, dgamma, dbeta, ws, st);
    });
}

}  // namespace dw
