// dw_decayattn.hip -- causal linear attention with a decay for each head:
//
//   S_i = d S_(i-1) + k_i v_i',   o_i = scale q_i S_i,   d = exp(log_decay[head]) in [0, 1].
//
// Chunks of C tokens turn the recurrence into products for the matrix cores.  With Z the state
// before a chunk and i, j positions inside it (n of them within the sequence's length):
//
//   P_ij = (q_i . k_j) d^(i-j) for j <= i, 0 otherwise
//   o_i  = s_inter d^(i+1-r) q_i Z + s_intra sum_j P_ij v_j
//   Z'   = d^n Z + sum_j s_upd d^(n-1-j+r) k_j v_j'
//
// r = 0 runs the forward.  The gradients are the same pass with the tensors' parts exchanged:
// dq_i = scale sum_(j<=i) d^(i-j) (do_i . v_j) k_j takes (do, v, k) as (query, key, value);
// dv_j = scale sum_(i>=j) d^(i-j) (k_j . q_i) do_i takes (k, q, do) with the tokens from last to
// first, dk_j takes (v, do, q) likewise.  There Z has been multiplied by d once more than the
// sum that the gradient needs (the gradient of the state before token j, not after it): r = 1.
//
// A long sequence is cut into segments for separate workgroups when there are few heads:
// decay_state_kernel sums each segment's own state, decay_scan_kernel turns those into the
// states before each segment, decay_out_kernel does the rest.
//
// Arithmetic.  Every product runs on v_mfma_f32_*_bf16 with fp32 sums.  An operand is a sum of
// bf16 planes, each the upper 16 bits of what the planes before it leave (the upper half of a
// binary32 is a bf16), so a bf16 tensor is one plane, fp16 two and fp32 three, all exact and
// none able to overflow, which fp16 operands could in a state or in P.  P and Z, held in fp32,
// enter a 16-bit output's products as two planes, an fp32 output's as three; decayed values enter a
// state that is returned as three, one that only 16-bit outputs see as two.  Two planes are a rounding
// to 16 bits (2^-16): the second is rounded to nearest, and not cut off, so that no output leans to one
// side (cut off, bf16 outputs of positive inputs were 7.3e-6 too small on average and fp16 ones 1.7e-5).
// It is 2^-8 of a bf16 output's own rounding and 2^-5 of an fp16 one's; a third plane would take the LDS
// of the second workgroup on a CU.  Of the plane products only those above the planes' own
// rounding are made: orders i + j <= 1 for 16-bit outputs, <= 2 for fp32 and for the state; an fp16
// tensor's first plane is rounded to nearest too, so that the products left out have either sign.
// Against fp32 matrix instructions (1/16 of the bf16 rate) the six products of fp32 cost 3/8.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "dw_common.hpp"
#include "dw_internal.hpp"
#include "dw_seq.hpp"
#include "dwconv.h"

namespace dw {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(1))) char global_char;

// A workgroup has eight waves, 16 value columns each; two workgroups fit a CU.  With four waves of 32
// columns (half the LDS reads) the matrix and vector pipes were idle half of the time.  What bounds the output pass is
// vector and matrix issue: a chunk of 64 tokens of 128 x 128 bf16 heads is 460 and 81 instructions a wave, 3.8 us for
// a workgroup alone on its CU and twice that for two (gradients of 8 x 4096 tokens, 8 heads: 242 us).
constexpr int kWG = 512;
constexpr int kVB = 128;  // value columns of a workgroup

template <typename T> struct Planes;
template <> struct Planes<bf16_t> { static constexpr int N = 1, O = 2; };
template <> struct Planes<__half> { static constexpr int N = 2, O = 2; };
template <> struct Planes<float> { static constexpr int N = 3, O = 3; };

// Threads that take a row of W elements, eight each: a power of two.
constexpr int row_threads(int W) { return W <= 64 ? 8 : W <= 128 ? 16 : 32; }
// Steps in which a workgroup takes C such rows.
constexpr int row_steps(int C, int W) { return C * row_threads(W) > kWG ? C * row_threads(W) / kWG : 1; }

// The kernels' tiles.  C: tokens of a chunk, 64 where two workgroups' tiles then fit a CU's
// LDS.  Row strides are 8, 24 or 40 banks past a multiple of
// the 64: 16-byte reads of 16 rows then run without bank conflicts (4 banks past cost 4 cycles a read,
// measured), and so do the transposing reads of 8 rows in a row.
template <typename T, int DKP> struct Tile {
    static constexpr int NP = Planes<T>::N, NO = Planes<T>::O;
    static constexpr int C = NP == 1 && DKP <= 128 ? 64 : 32;
    static constexpr int KS = DKP + 16, VS = kVB + 16, PS = C + 16;
    static constexpr int NU = row_steps(C, DKP), NV = row_steps(C, kVB);
    static constexpr int waves = DKP <= 128 && NP < 3 ? 4 : 2;  // of a SIMD: two workgroups where they fit
};

// Eight consecutive elements of a row as they are in memory.
template <typename T> struct Raw8 { uint32_t w[sizeof(T) * 2]; };

union Frag {
    uint4 q;
    uint32_t w[4];
    uint2 d[2];
    s16x4 s[2];
    bf16x8 v;
};

// A scalar that stays in a register: the compiler would load a launch's argument again in every turn, and
// that load's wait is one for the LDS reads in flight too.
template <typename V> __device__ __forceinline__ V held(V v) {
#ifdef __OPTIMIZE__  // unoptimised code has no value in a scalar register from one statement to the next
    asm volatile("" : "+s"(v));
#endif
    return v;
}
// The wave's index as a scalar.
__device__ __forceinline__ int wave_index() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }
// The thread's index as a value that the compiler does not follow: what a loop derives from it is
// computed again in each turn.  Held across turns those addresses would take the registers that the
// state and the loads in flight need, and their reloads from scratch wait for the loads before them.
__device__ __forceinline__ int fresh_thread() {
    int t = threadIdx.x;
    asm volatile("" : "+v"(t));
    return t;
}

__device__ __forceinline__ f32x4 mfma(const Frag &a, const Frag &b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.v, c, 0, 0, 0);
}

// The next bf16 planes of a and b in one word (a in the low half); a and b become what is left, exactly.
__device__ __forceinline__ uint32_t peel2(float &a, float &b) {
    const uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
    a -= __uint_as_float(x & 0xffff0000u);
    b -= __uint_as_float(y & 0xffff0000u);
    return __builtin_amdgcn_perm(y, x, 0x07060302u);
}
// The same with a and b rounded to nearest; what is left is of either sign, and exact.
__device__ __forceinline__ uint32_t round2(float &a, float &b) {
    const uint32_t w = pack2<bf16_t>(a, b);
    a -= __uint_as_float(w << 16);
    b -= __uint_as_float(w & 0xffff0000u);
    return w;
}
// The p-th of a value pair's N planes.  Two planes do not hold an fp32 value: the second is rounded to nearest (the
// first is cut off, for the rounding of a value near fp32's largest would be infinite).  Three do, cut off.
template <int N> __device__ __forceinline__ uint32_t plane2(int p, float &a, float &b) {
    return N == 2 && p == 1 ? pack2<bf16_t>(a, b) : peel2(a, b);
}
// Eight values as N planes.
template <int N> __device__ __forceinline__ void split8(float (&x)[8], Frag (&f)[N]) {
#pragma unroll
    for (int p = 0; p < N; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i) f[p].w[i] = plane2<N>(p, x[2 * i], x[2 * i + 1]);
}

__device__ __forceinline__ float raw_value(const Raw8<float> &r, int i) { return __uint_as_float(r.w[i]); }
__device__ __forceinline__ float raw_value(const Raw8<__half> &r, int i) {
    const uint16_t h = static_cast<uint16_t>(r.w[i / 2] >> (16 * (i & 1)));
    return __half2float(__builtin_bit_cast(__half, h));
}

template <typename T, int NP> __device__ __forceinline__ void raw_planes(const Raw8<T> &r, Frag (&f)[NP]) {
    if constexpr (std::is_same<T, bf16_t>::value) {
        f[0].q = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
    } else {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = raw_value(r, i);
        if constexpr (NP == 2) {  // fp16's 11 bits: the first eight to nearest, the rest exact
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[0].w[i] = round2(x[2 * i], x[2 * i + 1]);
                f[1].w[i] = peel2(x[2 * i], x[2 * i + 1]);
            }
        } else {
            split8<NP>(x, f);
        }
    }
}

// d^m for m tokens, from the exponent in 64 bits: exact to 2^-23 for any m.
__device__ __forceinline__ float decay_power(double g2, int m) {
    const double p = g2 * m, y = p < -1000.0 ? -1000.0 : p > 1000.0 ? 1000.0 : p, whole = rint(y);
    return ldexpf(exp2f(static_cast<float>(y - whole)), static_cast<int>(whole));
}
// log2 of the decay; a decay of zero becomes one whose every power but the 0th is zero.
__device__ __forceinline__ double log2_decay(float g) {
    return (g < -1e30f ? -1e30 : static_cast<double>(g)) * 1.4426950408889634;
}

// Where a tensor's rows of one (batch, head) lie: d, a multiple of 8, elements, `pitch` bytes apart.
struct Rows {
    const char *p;
    int64_t pitch;
    int d;
};

// A workgroup's share of a pass.
struct Where {
    int pair, b, h, seg, vb;
    int len;          // the sequence's length
    float log_decay;  // loaded with it: both wait for the same memory
    int64_t first;    // first position of the segment
    int64_t end;      // first position past it
};

// Workgroups of one (batch, head, segment) read the same rows in their roles and value blocks:
// they are neighbours on one XCD (workgroup w runs on XCD w mod 8) and share its L2.
template <int C>
__device__ __forceinline__ bool locate(const AttnLaunch &l, int *role, Where *w) {
    const uint32_t x = blockIdx.x, xcd = x & 7u;
    uint32_t y = x >> 3;
    const uint32_t inner = l.nroles * l.nvb;
    const uint32_t g = (y / inner) * 8 + xcd;
    y %= inner;
    *role = y / l.nvb;
    w->vb = y % l.nvb;
    w->pair = g / l.nseg;
    w->seg = g % l.nseg;
    if (w->pair >= l.b * l.h || w->vb * kVB >= l.role[*role].dv) return false;
    w->b = w->pair / l.h;
    w->h = w->pair % l.h;
    int64_t len = l.t;
    w->log_decay = l.log_decay[w->h];
    if (l.lengths) len = min(static_cast<int64_t>(max(l.lengths[w->b], 0)), l.t);
    w->len = static_cast<int>(len);
    w->first = static_cast<int64_t>(w->seg) * l.seg_chunks * C;
    w->end = min(l.t, w->first + static_cast<int64_t>(l.seg_chunks) * C);
    return true;
}

template <typename T>
__device__ __forceinline__ Rows rows_of(const void *p, const SeqStride &s, const Where &w, int rep, int d, int col = 0) {
    return {reinterpret_cast<const char *>(static_cast<const T *>(p) + w.b * s.b + (w.h / rep) * s.h + col),
            s.t * static_cast<int64_t>(sizeof(T)), d - col};
}

constexpr int64_t kNearPitch = int64_t{1} << 24;  // rows whose offsets within a chunk fit 32 bits

// A tile's rows (n > 0 of C) into registers: thread and step i give row i R + thread / RT, and a
// unit of eight elements of it.  No branches, so that all loads are in flight at once; what lies
// outside reads a row or unit that does exist and is cleared when it is staged.  A whole tile's
// addresses are a scalar for each step and one lane offset.  They need no alignment: gfx950 loads
// take any address.
template <typename T, int C, int W, int NU>
__device__ __forceinline__ void load_tile(int tid, Raw8<T> (&raw)[NU], const Rows &m, int64_t first, int n, int len,
                                          bool reverse) {
    constexpr int RT = row_threads(W), R = kWG / RT < C ? kWG / RT : C;
    const int c8 = tid % RT, row = R * RT < kWG ? min(tid / RT, R - 1) : tid / RT;
    const uint32_t unit = (8 * c8 < m.d ? c8 : 0) * static_cast<uint32_t>(8 * sizeof(T));
    const int64_t low = reverse ? len - first - n : first;  // the tile's first row in memory
    if (n == C && m.pitch <= kNearPitch) {
        const int pitch = static_cast<int>(m.pitch), step = reverse ? -R * pitch : R * pitch;
        const uint32_t at = static_cast<uint32_t>(reverse ? R - 1 - row : row) * static_cast<uint32_t>(pitch) + unit;
        const char *base = m.p + low * m.pitch + (reverse ? (NU - 1) * R * pitch : 0);
#pragma unroll
        for (int i = 0; i < NU; ++i) __builtin_memcpy(&raw[i], base + static_cast<int64_t>(i) * step + at, sizeof(raw[i]));
    } else {
#pragma unroll
        for (int i = 0; i < NU; ++i) {
            const int r = min(i * R + row, n - 1);
            __builtin_memcpy(&raw[i], m.p + (low + (reverse ? n - 1 - r : r)) * m.pitch + unit, sizeof(raw[i]));
        }
    }
}
// How a tile lies in LDS.  Query: of each 32 columns, column 16 b + 4 q + e goes to place 8 q + 4 b + e, and
// of each two units of eight columns the first comes second in odd rows.  Key: they are exchanged so in rows 8
// to 15 of each 16.  Without the exchanges the query's 8-byte writes of two rows, and the 8-byte reads of
// 16 rows of keys, meet in half of the banks.
enum Layout { kPlain, kQuery, kKey };
// Stages a tile's rows as planes in LDS, zeros past its rows and their ends.
template <typename T, int NP, int C, int W, int S, Layout LAYOUT, int NU>
__device__ __forceinline__ void stage(int tid, uint16_t *lds, Raw8<T> (&raw)[NU], int n, int d) {
    constexpr int RT = row_threads(W), R = kWG / RT;
    const int c8 = tid % RT, row = tid / RT;
    if (n < C || d < W) {
#pragma unroll
        for (int i = 0; i < NU; ++i) {
            const bool live = i * R + row < n && 8 * c8 < d;
#pragma unroll
            for (uint32_t &w : raw[i].w) w = live ? w : 0u;
        }
    }
    if ((8 * RT > W && 8 * c8 >= W) || (R > C && row >= C)) return;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
        Frag f[NP];
        raw_planes<T, NP>(raw[i], f);
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            uint16_t *to = lds + (p * C + i * R + row) * S;
            if (LAYOUT == kQuery) {  // columns 8 c8 .. 8 c8 + 7: b = c8 / 2 mod 2, q = 2 (c8 mod 2) and the next
                const int flip = 8 * ((i * R + row) & 1);
                to += 32 * (c8 >> 2) + 16 * (c8 & 1) + 4 * ((c8 >> 1) & 1);
                *reinterpret_cast<uint2 *>(to + flip) = f[p].d[0];
                *reinterpret_cast<uint2 *>(to + 8 - flip) = f[p].d[1];
            } else {
                const int flip = LAYOUT == kKey ? ((i * R + row) >> 3) & 1 : 0;
                *reinterpret_cast<uint4 *>(to + 8 * (c8 ^ flip)) = f[p].q;
            }
        }
    }
}

// The order in which a chunk's tokens enter the products over tokens.  A transposing read gives a
// lane four rows of one column; 32 lanes take eight rows that follow each other, which lie in different
// LDS banks.  So of each 16 tokens, place 8 h + 4 b + e holds token 8 b + 4 h + e.
__device__ __forceinline__ int token_at(int place) {
    return (place & ~12) | ((place & 4) << 1) | ((place & 8) >> 1);
}

// Column c0 + lane % 16 of the 32 rows from r0 of a row-major LDS tile as a fragment: its eight values
// are places 8 (lane / 16) + 0..7 of token_at().  Each group of 16 lanes reads four rows of 16 columns,
// lane i giving the address of columns 4 (i % 4) of row i / 4.
template <Layout LAYOUT> __device__ __forceinline__ Frag column_frag(int lane, const uint16_t *lds, int stride, int r0, int c0) {
    const int i = lane & 15;
    const uint16_t *p = lds + (r0 + 16 * (lane >> 5) + 4 * ((lane >> 4) & 1) + (i >> 2)) * stride + c0;
    const int at = 4 * (i & 3);
    Frag f;
    f.s[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + at));
    f.s[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 8 * stride + (LAYOUT == kKey ? at ^ 8 : at)));
    return f;
}

// Value i of accumulator tile m is row 16 m + i + 4 (lane / 16) of the state, column lane % 16 of the
// wave's.

// z from a state of dk x dv (element (r, c) at r rs + c cs) or to one; zeros outside.  A whole state
// takes a scalar address for each value and one lane offset; of a transposed one (rs = 1) the four rows of a
// tile are one load.  All loads are in flight at once.
template <int DKP>
__device__ __forceinline__ void load_state(f32x4 (&z)[DKP / 16], const float *p, int col, int dk, int dv, int rs, int cs) {
    const int up = 4 * ((fresh_thread() & 63) >> 4);
    if (rs == 1 && dk % 4 == 0) {
        const float *first = p + min(col, dv - 1) * cs;
        const int rows = (col < dv ? dk : 0) - up;
#pragma unroll
        for (int m = 0; m < DKP / 16; ++m) __builtin_memcpy(&z[m], first + min(16 * m + up, dk - 4), sizeof(z[m]));
#pragma unroll
        for (int m = 0; m < DKP / 16; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) z[m][i] = 16 * m < rows ? z[m][i] : 0.f;
    } else if (dk == DKP && __all(col < dv)) {
        const uint32_t at = static_cast<uint32_t>(up * rs + col * cs);
#pragma unroll
        for (int m = 0; m < DKP / 16; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) z[m][i] = (p + (16 * m + i) * rs)[at];
    } else {
        const int in = min(col, dv - 1) * cs, rows = (col < dv ? dk : 0) - up;
#pragma unroll
        for (int m = 0; m < DKP / 16; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) z[m][i] = p[min(16 * m + i + up, dk - 1) * rs + in];
#pragma unroll
        for (int m = 0; m < DKP / 16; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) z[m][i] = 16 * m + i < rows ? z[m][i] : 0.f;
    }
}
template <int DKP> __device__ __forceinline__ void store_state(float *p, const f32x4 (&z)[DKP / 16], int col, int dk, int dv) {
    const int up = 4 * ((fresh_thread() & 63) >> 4);
    const uint32_t at = static_cast<uint32_t>(up * dv + col);
    if (col >= dv) return;
    if (dk == DKP) {
#pragma unroll
        for (int m = 0; m < DKP / 16; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) (p + (16 * m + i) * dv)[at] = z[m][i];
    } else {
#pragma unroll
        for (int m = 0; m < DKP / 16; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (16 * m + i + up < dk) (p + (16 * m + i) * dv)[at] = z[m][i];
    }
}

// Adds a chunk to the state: z[m] += K' (w V) over the chunk's tokens, w V as NV planes.  wv holds the
// tokens' weights in the order of token_at().
template <typename T, int DKP, int NV, int NP = Tile<T, DKP>::NP>
__device__ __forceinline__ void add_chunk(int lane, f32x4 (&z)[DKP / 16], const uint16_t *kt,
                                          const Frag (&vf)[Tile<T, DKP>::C / 32][NP], const float *wv) {
    using L = Tile<T, DKP>;
    const int quad = lane >> 4;
#pragma unroll
    for (int ks = 0; ks < L::C / 32; ++ks) {
        float x[8];
        const float4 w0 = *reinterpret_cast<const float4 *>(wv + 32 * ks + 8 * quad);
        const float4 w1 = *reinterpret_cast<const float4 *>(wv + 32 * ks + 8 * quad + 4);
        const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float v[NP];
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                const uint32_t word = vf[ks][p].w[i / 2];
                v[p] = __uint_as_float(i & 1 ? word & 0xffff0000u : word << 16);
            }
#pragma unroll
            for (int p = NP - 1; p > 0; --p) v[p - 1] += v[p];
            x[i] = v[0] * w[i];
        }
        Frag f[NV];
        split8<NV>(x, f);
#pragma unroll
        for (int m = 0; m < DKP / 16; m += 2) {  // two tiles at a time: no product waits for the one before
#pragma unroll
            for (int p = NP - 1; p >= 0; --p) {
                const Frag k0 = column_frag<kKey>(lane, kt + p * L::C * L::KS, L::KS, 32 * ks, 16 * m);
                const Frag k1 = column_frag<kKey>(lane, kt + p * L::C * L::KS, L::KS, 32 * ks, 16 * m + 16);
#pragma unroll
                for (int j = NV - 1 - p; j >= 0; --j) {
                    z[m] = mfma(k0, f[j], z[m]);
                    z[m + 1] = mfma(k1, f[j], z[m + 1]);
                }
            }
        }
    }
}

template <typename T, int DKP>
__global__ __launch_bounds__(kWG, (Tile<T, DKP>::waves)) void decay_state_kernel(AttnLaunch l, float *seg0,
                                                                                   float *seg1) {
    using L = Tile<T, DKP>;
    __shared__ __align__(16) uint16_t kt[L::NP * L::C * L::KS];
    __shared__ __align__(16) uint16_t vt[L::NP * L::C * L::VS];
    __shared__ __align__(16) float wv[L::C];
    int ri;
    Where w;
    if (!locate<L::C>(l, &ri, &w)) return;
    const AttnRole &r = l.role[ri];
    const int wave = wave_index();
    const int64_t seg_end = min(w.end, static_cast<int64_t>(w.len));
    const Rows kr = rows_of<T>(r.k, r.ks, w, r.krep, r.dkp);
    const Rows vr = rows_of<T>(r.v, r.vs, w, r.vrep, r.dvp, w.vb * kVB);
    const double g2 = log2_decay(w.log_decay);
    const bool active = 16 * wave < vr.d;
    f32x4 z[DKP / 16] = {};

    Raw8<T> rk[L::NU], rv[L::NV];
    auto load = [&](int tid, int64_t base) {
        const int n = static_cast<int>(min(static_cast<int64_t>(L::C), seg_end - base));
        load_tile<T, L::C, DKP>(tid, rk, kr, base, n, w.len, r.reverse);
        load_tile<T, L::C, kVB>(tid, rv, vr, base, n, w.len, r.reverse);
    };
    if (w.first < seg_end) load(threadIdx.x, w.first);
    for (int64_t base = w.first; base < seg_end; base += L::C) {
        const int tid = fresh_thread(), lane = tid & 63;
        const int n = static_cast<int>(min(static_cast<int64_t>(L::C), seg_end - base));
        stage<T, L::NP, L::C, DKP, L::KS, kKey>(tid, kt, rk, n, kr.d);
        stage<T, L::NP, L::C, kVB, L::VS, kPlain>(tid, vt, rv, n, vr.d);
        // weights to the segment's end: no state is ever scaled, so no rounding piles up
        if (tid < L::C) {
            const int64_t left = seg_end - 1 - base - token_at(tid);
            wv[tid] = left < 0 ? 0.f : r.s_upd * decay_power(g2, static_cast<int>(left) + r.reverse);
        }
        __syncthreads();
        if (base + L::C < seg_end) load(tid, base + L::C);
        if (active) {
            Frag vf[L::C / 32][L::NP];
#pragma unroll
            for (int ks = 0; ks < L::C / 32; ++ks)
#pragma unroll
                for (int p = 0; p < L::NP; ++p)
                    vf[ks][p] = column_frag<kPlain>(lane, vt + p * L::C * L::VS, L::VS, 32 * ks, 16 * wave);
            add_chunk<T, DKP, 3>(lane, z, kt, vf, wv);
        }
        __syncthreads();
    }
    float *seg = ri == 0 ? seg0 : seg1;
    seg += (static_cast<int64_t>(w.pair) * l.nseg + w.seg) * r.dk * r.dv;
    store_state<DKP>(seg, z, w.vb * kVB + 16 * wave + (threadIdx.x & 15), r.dk, r.dv);
}

// One thread follows V elements of a (batch, head)'s state over the segments, the next eight segments' in
// flight; a gradient's two states go by blockIdx.z.  64-bit powers and sums: it reads and writes memory and
// little else.  (Two states of 64 heads of 128 x 128 over 4 segments, 67 MB: one element a thread 25 us, two
// 20, four 14; one state of 16 heads over 32 segments 16, 13 and 13.)
template <int V>
__global__ __launch_bounds__(kThreads) void decay_scan_kernel(AttnScan one, AttnScan two, const float *log_decay,
                                                              const int32_t *lengths, int h, int64_t t, int size, int nseg,
                                                              int64_t seg_tokens) {
    struct Part {
        float v[V];
    };
    const int pair = blockIdx.y, e = (blockIdx.x * kThreads + threadIdx.x) * V;
    if (e >= size) return;
    float *const seg = blockIdx.z ? two.seg : one.seg, *const zout = blockIdx.z ? two.zout : one.zout;
    const float *const zin = blockIdx.z ? two.zin : one.zin;
    float *p = seg + static_cast<int64_t>(pair) * nseg * size + e;
    Part next[8], first{};
    auto load = [&](int s0) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (s0 + i < nseg) __builtin_memcpy(&next[i], p + static_cast<int64_t>(s0 + i) * size, sizeof(Part));
    };
    load(0);
    if (zin) __builtin_memcpy(&first, zin + static_cast<int64_t>(pair) * size + e, sizeof(Part));
    int64_t len = t;
    if (lengths) len = min(static_cast<int64_t>(max(lengths[pair / h], 0)), t);
    const float g = log_decay[pair % h];
    const double lg = g < -1e30f ? -1e30 : static_cast<double>(g), whole = exp(lg * seg_tokens);
    double carry[V];
#pragma unroll
    for (int j = 0; j < V; ++j) carry[j] = first.v[j];
    for (int s0 = 0; s0 < nseg; s0 += 8) {
        Part mine[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) mine[i] = next[i];
        if (s0 + 8 < nseg) load(s0 + 8);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (s0 + i >= nseg) break;
            Part before;
#pragma unroll
            for (int j = 0; j < V; ++j) before.v[j] = static_cast<float>(carry[j]);
            __builtin_memcpy(p + static_cast<int64_t>(s0 + i) * size, &before, sizeof(Part));
            const int64_t n = min(max(len - (s0 + i) * seg_tokens, int64_t{0}), seg_tokens);
            if (n > 0) {
                const double keep = n == seg_tokens ? whole : exp(lg * n);
#pragma unroll
                for (int j = 0; j < V; ++j) carry[j] = carry[j] * keep + mine[i].v[j];
            }
        }
    }
    if (zout) {
        Part last;
#pragma unroll
        for (int j = 0; j < V; ++j) last.v[j] = static_cast<float>(carry[j]);
        __builtin_memcpy(zout + static_cast<int64_t>(pair) * size + e, &last, sizeof(Part));
    }
}

// Where a wave's 16 columns of a (batch, head)'s output rows lie.
struct OutRows {
    global_char *p;  // known as global memory: held() hides where a pointer comes from
    int64_t pitch;  // bytes from a token's row to the next
    int left;       // columns from the wave's first to the row's end
    int f32;        // of float, whatever the inputs are
    int wide;       // four columns are written at a time
};
template <typename T> __device__ __forceinline__ OutRows out_rows(const AttnLaunch &l, const AttnRole &r, const Where &w, int col0) {
    const int e = r.o_f32 ? 4 : static_cast<int>(sizeof(T));
    const int64_t first = (w.b * l.t * l.h + w.h) * r.dv + col0;
    return {(global_char *)(static_cast<char *>(r.o) + first * e), static_cast<int64_t>(l.h) * r.dv * e, r.dv - col0, r.o_f32, r.wide_o};
}
// Whether the columns of every wave with some are 16, written four at a time within 32-bit offsets.
__device__ __forceinline__ bool plain(const OutRows &m, int dv) { return m.wide && dv % 16 == 0 && m.pitch <= kNearPitch; }
// Rows of outputs from their transpose o' (a query in each lane column, four consecutive value columns in
// four registers), zeros from row n on.
enum Store { kAnyRows, kWhole, kWholeF32 };  // whole: a whole chunk whose rows plain() allows, of T or of float
template <typename T, Store STORE, int QT>
__device__ __forceinline__ void store_rows(const OutRows &m, const f32x4 (&o)[QT], int lane, int64_t base, int len, bool reverse,
                                           int rows, int n) {
    const int quad = lane >> 4, l16 = lane & 15;
    if constexpr (STORE != kAnyRows) {  // a scalar address for each 16 rows and one lane offset
        const int pitch = static_cast<int>(m.pitch), step = reverse ? -16 * pitch : 16 * pitch;
        constexpr bool wide = STORE == kWholeF32 || std::is_same<T, float>::value;
        const uint32_t at = static_cast<uint32_t>(reverse ? 15 - l16 : l16) * static_cast<uint32_t>(pitch) + (wide ? 16 : 8) * quad;
        global_char *first = m.p + (reverse ? len - base - 16 : base) * m.pitch;
#pragma unroll
        for (int qt = 0; qt < QT; ++qt) {
            global_char *to = first + static_cast<int64_t>(qt) * step + at;
            if constexpr (wide) *(__attribute__((address_space(1))) f32x4 *)to = o[qt];
            else *(__attribute__((address_space(1))) u32x2 *)to = u32x2{pack2<T>(o[qt][0], o[qt][1]), pack2<T>(o[qt][2], o[qt][3])};
        }
        return;
    }
    const bool f32 = std::is_same<T, float>::value || m.f32;
    const int left = m.left - 4 * quad;
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) {
        const int i = 16 * qt + l16;
        const int64_t pos = base + i, row = i < n && reverse ? len - 1 - pos : pos;
        if (i >= rows) continue;
        float x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = i < n ? o[qt][j] : 0.f;
        if (f32) {
            float *p = (float *)(m.p + row * m.pitch) + 4 * quad;
            if (m.wide && left > 0) {
                *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < left) p[j] = x[j];
            }
        } else if constexpr (!std::is_same<T, float>::value) {
            T *p = (T *)(m.p + row * m.pitch) + 4 * quad;
            if (m.wide && left > 0) {
                *reinterpret_cast<uint2 *>(p) = make_uint2(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]));
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < left) p[j] = from_f32<T>(x[j]);
            }
        }
    }
}

// The state is kept as z = Z / d^(C age): a chunk then divides its tokens' weights instead of scaling
// the whole state, which is done once the factor has fallen under 2^-20 or after kAges chunks.  The
// factors come from a table of exact powers, so a long sequence piles up no rounding of d^C.
constexpr int kAges = 16;

// PRECISE: the state after the last token is wanted, so w V enters it as three planes; a state that
// only 16-bit outputs see is held to their two.
template <typename T, int DKP, bool PRECISE>
__global__ __launch_bounds__(kWG, (Tile<T, DKP>::waves)) void decay_out_kernel(AttnLaunch l) {
    using L = Tile<T, DKP>;
    constexpr int NP = L::NP, NO = L::NO, C = L::C, QT = C / 16;
    __shared__ __align__(16) uint16_t qs[NP * C * L::KS];  // kQuery
    __shared__ __align__(16) uint16_t kt[NP * C * L::KS];
    __shared__ __align__(16) uint16_t vt[NP * C * L::VS];
    __shared__ __align__(16) uint16_t pt[NO * C * L::PS];
    __shared__ __align__(16) float wv[C];
    __shared__ float pw[C + 1], pi[16 + C], pc[kAges + 1];
    int ri;
    Where w;
    if (!locate<C>(l, &ri, &w)) return;
    const AttnRole &r = l.role[ri];
    const int wave = wave_index();
    const Rows qr = rows_of<T>(r.q, r.qs, w, r.qrep, r.dkp);
    const Rows kr = rows_of<T>(r.k, r.ks, w, r.krep, r.dkp);
    const Rows vr = rows_of<T>(r.v, r.vs, w, r.vrep, r.dvp, w.vb * kVB);
    const bool active = 16 * wave < vr.d;
    const int col0 = w.vb * kVB + 16 * wave;  // the wave's columns of the state
    OutRows out = out_rows<T>(l, r, w, col0);
    out.p = held(out.p);
    out.pitch = held(out.pitch);
    const bool reverse = held(r.reverse);
    const float s_inter = held(r.s_inter), s_upd = held(r.s_upd);
    Raw8<T> rq[L::NU], rk[L::NU], rv[L::NV];
    auto load = [&](int tid, int64_t base) {
        const int n = static_cast<int>(min(static_cast<int64_t>(C), w.len - base));
        load_tile<T, C, DKP>(tid, rq, qr, base, n, w.len, reverse);
        load_tile<T, C, DKP>(tid, rk, kr, base, n, w.len, reverse);
        load_tile<T, C, kVB>(tid, rv, vr, base, n, w.len, reverse);
    };
    const int64_t live_end = min(w.end, static_cast<int64_t>(w.len));
    if (w.first < live_end) load(threadIdx.x, w.first);
    f32x4 z[DKP / 16] = {};
    if (r.zin)
        load_state<DKP>(z, r.zin + w.pair * r.zin_pair + w.seg * r.zin_seg, col0 + (threadIdx.x & 15), r.dk, r.dv, r.zin_row,
                        r.zin_col);
    {
        const double g2 = log2_decay(w.log_decay);
        // pw: powers; pi: s_intra times them, after 16 zeros for the places above the diagonal
        for (int i = threadIdx.x; i <= C; i += kWG) {
            const float p = decay_power(g2, i);
            pw[i] = p;
            if (i < C) pi[16 + i] = r.s_intra * p;
            if (i < 16) pi[i] = 0.f;
            if (i <= kAges) pc[i] = decay_power(g2, C * i);
        }
        // blocks of P above the diagonal are read as part of 32 keys and never written
        for (int i = threadIdx.x; i < NO * C * L::PS / 2; i += kWG) reinterpret_cast<uint32_t *>(pt)[i] = 0;
    }

    int age = 0;
    int64_t base = w.first;
    auto chunk = [&](auto how) {
        constexpr Store STORE = decltype(how)::value;
        constexpr bool WHOLE = STORE != kAnyRows;
        const int tid = fresh_thread(), lane = tid & 63, quad = lane >> 4, l16 = lane & 15;
        const int n = WHOLE ? C : static_cast<int>(min(static_cast<int64_t>(C), live_end - base));
        stage<T, NP, C, DKP, L::KS, kQuery>(tid, qs, rq, n, qr.d);
        stage<T, NP, C, DKP, L::KS, kKey>(tid, kt, rk, n, kr.d);
        stage<T, NP, C, kVB, L::VS, kPlain>(tid, vt, rv, n, vr.d);
        __syncthreads();
        if (base + C < live_end) load(tid, base + C);
        const float now = pc[age], next = pc[min(age + 1, kAges)];
        const bool keeps = __builtin_amdgcn_readfirstlane(n == C && age < kAges && next >= 0x1p-20f && next <= 0x1p20f);
        if (tid < C) {
            const int left = n - 1 - token_at(tid);
            wv[tid] = left >= 0 ? s_upd * pw[left + reverse] / (keeps ? next : 1.f) : 0.f;
        }

        // P: 16 x 16 blocks on and under the diagonal, shared out over the waves
        constexpr int B16 = C / 16;
#pragma unroll
        for (int i = 0; i < (B16 * (B16 + 1) / 2 + 7) / 8; ++i) {
            const int blk = 8 * i + wave;
            if (blk >= B16 * (B16 + 1) / 2) break;
            const int it = (blk >= 1) + (blk >= 3) + (blk >= 6), jt = blk - it * (it + 1) / 2;
            const uint16_t *kp = kt + (16 * jt + token_at(l16)) * L::KS + ((4 * quad) ^ (2 * (l16 & 4)));
            const uint16_t *qp = qs + (16 * it + l16) * L::KS + 8 * (quad ^ (l16 & 1));
            f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < DKP / 32; ++ks) {
                Frag kf[NP], qf[NP];
#pragma unroll
                for (int p = 0; p < NP; ++p) {
                    kf[p].d[0] = *reinterpret_cast<const uint2 *>(kp + p * C * L::KS + 32 * ks);
                    kf[p].d[1] = *reinterpret_cast<const uint2 *>(kp + p * C * L::KS + 32 * ks + 16);
                    qf[p].q = *reinterpret_cast<const uint4 *>(qp + p * C * L::KS + 32 * ks);
                }
#pragma unroll
                for (int p = NP - 1; p >= 0; --p)
#pragma unroll
                    for (int s = NO - 1 - p; s >= 0; --s)
                        if (s < NP) acc = mfma(kf[p], qf[s], acc);
            }
            // acc[e]: query 16 it + l16, the key at place 4 quad + e of block jt: token e + token_at(4 quad)
            const float *f = pi + 16 + 16 * (it - jt) + l16 - token_at(4 * quad);
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = f[-e] != 0.f ? acc[e] * f[-e] : 0.f;
#pragma unroll
            for (int p = 0; p < NO; ++p) {
                uint2 word;
                word.x = plane2<NO>(p, x[0], x[1]);
                word.y = plane2<NO>(p, x[2], x[3]);
                *reinterpret_cast<uint2 *>(pt + (p * C + 16 * it + l16) * L::PS + 16 * jt + 4 * quad) = word;
            }
        }
        // o' = z' q', the accumulators' own layout serving as the operand: their value i of tile m is row
        // 16 m + 4 quad + i, the order that kQuery gives q's columns
        f32x4 o[QT];
        if (WHOLE || active) {
#pragma unroll
            for (int ks = 0; ks < DKP / 32; ++ks) {
                float x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = z[2 * ks + i / 4][i & 3];
                Frag zf[NO];
                split8<NO>(x, zf);
#pragma unroll
                for (int p = NP - 1; p >= 0; --p) {
                    Frag qf[QT];
#pragma unroll
                    for (int qt = 0; qt < QT; ++qt)
                        qf[qt].q = *reinterpret_cast<const uint4 *>(qs + (p * C + 16 * qt + l16) * L::KS + 32 * ks + 8 * (quad ^ (l16 & 1)));
#pragma unroll
                    for (int s = NO - 1 - p; s >= 0; --s)
#pragma unroll
                        for (int qt = 0; qt < QT; ++qt)
                            o[qt] = mfma(zf[s], qf[qt], ks == 0 && p == NP - 1 && s == NO - 1 - p ? f32x4{} : o[qt]);
                }
            }
#pragma unroll
            for (int qt = 0; qt < QT; ++qt) {
                const float f = s_inter * now * pw[16 * qt + l16 + 1 - reverse];
#pragma unroll
                for (int i = 0; i < 4; ++i) o[qt][i] *= f;
            }
        }
        __syncthreads();
        if (WHOLE || active) {
            Frag vf[C / 32][NP];
#pragma unroll
            for (int ks = 0; ks < C / 32; ++ks)
#pragma unroll
                for (int p = 0; p < NP; ++p) vf[ks][p] = column_frag<kPlain>(lane, vt + p * C * L::VS, L::VS, 32 * ks, 16 * wave);
#pragma unroll
            for (int qt = 0; qt < QT; ++qt)
#pragma unroll
                for (int ks = 0; ks <= qt / 2; ++ks)
#pragma unroll
                    for (int s = NO - 1; s >= 0; --s) {
                        Frag pf;
                        pf.q = *reinterpret_cast<const uint4 *>(pt + (s * C + 16 * qt + l16) * L::PS + 32 * ks + 8 * quad);
#pragma unroll
                        for (int p = NO - 1 - s; p >= 0; --p)
                            if (p < NP) o[qt] = mfma(vf[ks][p], pf, o[qt]);
                    }
            store_rows<T, STORE>(out, o, lane, base, w.len, reverse, static_cast<int>(min(static_cast<int64_t>(C), w.end - base)), n);
            if (!keeps) {
                const float f = now * pw[n];
#pragma unroll
                for (int m = 0; m < DKP / 16; ++m)
#pragma unroll
                    for (int i = 0; i < 4; ++i) z[m][i] *= f;
            }
            add_chunk<T, DKP, PRECISE ? 3 : NO>(lane, z, kt, vf, wv);
        }
        age = keeps ? age + 1 : 0;
        __syncthreads();
    };
    // Whole chunks have a loop of their own: there the number of loads and stores in flight is known, so that
    // the wait for a chunk's rows is not one for the output rows stored after them.  A wave without columns
    // stores none and takes the other loop: the branch is the same for a whole wave, and the barriers as many.
    __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0): nothing in flight but what the loop starts
    if (active && plain(out, r.dv)) {
        if constexpr (!std::is_same<T, float>::value)
            if (out.f32)
                for (; base + C <= live_end; base += C) chunk(std::integral_constant<Store, kWholeF32>{});
        for (; base + C <= live_end; base += C) chunk(std::integral_constant<Store, kWhole>{});
    }
    for (; base < live_end; base += C) chunk(std::integral_constant<Store, kAnyRows>{});
    if (active) {
        const f32x4 none[QT] = {};
        for (; base < w.end; base += C)
            store_rows<T, kAnyRows>(out, none, threadIdx.x & 63, base, w.len, reverse,
                              static_cast<int>(min(static_cast<int64_t>(C), w.end - base)), 0);
    }
    if (PRECISE && r.zout) {
        const float f = age > 0 ? pc[age] : 1.f;
#pragma unroll
        for (int m = 0; m < DKP / 16; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) z[m][i] *= f;
        store_state<DKP>(r.zout + static_cast<int64_t>(w.pair) * r.dk * r.dv, z, col0 + (threadIdx.x & 15), r.dk, r.dv);
    }
}

// Rows of an odd size into rows of whole units of eight elements: out (rows, dp) from x
// (b, t, heads, d).
template <typename T>
__global__ __launch_bounds__(kThreads) void widen_kernel(const T *x, SeqStride st, T *out, int64_t total, int64_t t, int heads,
                                                         int d, int dp) {
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t row = i / dp, bt = row / heads, b = bt / t;
        const int c = static_cast<int>(i - row * dp);
        out[i] = c < d ? x[b * st.b + (bt - b * t) * st.t + (row - bt * heads) * st.h + c] : T{};
    }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void share_kernel(const float *in, T *out, int64_t total, int hs, int rep, int d) {
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t head = i / d;
        const float *p = in + head * rep * d + (i - head * d);
        float s = 0.f;
        for (int r = 0; r < rep; ++r) s += p[static_cast<int64_t>(r) * d];
        out[i] = from_f32<T>(s);
    }
}

// ---------------------------------------------------------------- one token
// A workgroup takes 32 columns of one head's state: 8 lanes of 4 columns, 32 rows at a time.  The
// state is read and written once, 128 bytes of a row together; the rest is small beside it.  (256 x 8
// heads of 128 x 128: 56 us, 4.8 TB/s; one user's 8 heads: 4.5 us.)
template <typename T, bool VEC>
__global__ __launch_bounds__(kThreads) void decay_step_kernel(const T *q, const T *k, const T *v, const float *log_decay,
                                                              float *state, T *o, int h, int qrep, int krep, int vrep,
                                                              int dk, int dv, SeqStride qs, SeqStride ks, SeqStride vs,
                                                              int64_t state_stride, float scale) {
    __shared__ float part[4][32];
    const int pair = blockIdx.x, b = pair / h, hh = pair % h;
    const int tx = threadIdx.x & 7, ty = threadIdx.x >> 3, c = blockIdx.y * 32 + 4 * tx;
    const float keep = expf(log_decay[hh]);
    const T *qp = q + b * qs.b + (hh / qrep) * qs.h, *kp = k + b * ks.b + (hh / krep) * ks.h;
    const T *vp = v + b * vs.b + (hh / vrep) * vs.h;
    float *sp = state + b * state_stride + static_cast<int64_t>(hh) * dk * dv + c;
    float x[4], sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = c + i < dv ? to_f32(vp[c + i]) : 0.f;
    for (int r = ty; r < dk; r += 32) {
        float *p = sp + static_cast<int64_t>(r) * dv;
        const float kr = to_f32(kp[r]), qr = to_f32(qp[r]);
        float s[4];
        if (VEC) {
            if (c < dv) {
                const float4 a = *reinterpret_cast<const float4 *>(p);
                s[0] = fmaf(a.x, keep, kr * x[0]), s[1] = fmaf(a.y, keep, kr * x[1]);
                s[2] = fmaf(a.z, keep, kr * x[2]), s[3] = fmaf(a.w, keep, kr * x[3]);
                *reinterpret_cast<float4 *>(p) = make_float4(s[0], s[1], s[2], s[3]);
            } else {
                s[0] = s[1] = s[2] = s[3] = 0.f;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[i] = 0.f;
                if (c + i < dv) p[i] = s[i] = fmaf(p[i], keep, kr * x[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] = fmaf(qr, s[i], sum[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        sum[i] += __shfl_xor(sum[i], 8);
        sum[i] += __shfl_xor(sum[i], 16);
        sum[i] += __shfl_xor(sum[i], 32);
    }
    if ((threadIdx.x & 63) < 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) part[threadIdx.x >> 6][4 * tx + i] = sum[i];
    }
    __syncthreads();
    const int oc = blockIdx.y * 32 + threadIdx.x;
    if (threadIdx.x < 32 && oc < dv) {
        const float y = (part[0][threadIdx.x] + part[1][threadIdx.x]) + (part[2][threadIdx.x] + part[3][threadIdx.x]);
        o[static_cast<int64_t>(pair) * dv + oc] = from_f32<T>(y * scale);
    }
}

int padded(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : d <= 192 ? 192 : 256; }
int chunk_of(int dtype, int dkp) { return dtype == DW_BF16 && dkp <= 128 ? 64 : 32; }
int done() { return hipGetLastError() == hipSuccess ? kOk : kErrHip; }

template <typename F> int by_type(int dtype, F f) {
    if (dtype == DW_F32) return f(float{});
    if (dtype == DW_F16) return f(__half{});
    return f(bf16_t{});
}
template <typename F> int by_size(int dkp, F f) {
    if (dkp == 64) return f(std::integral_constant<int, 64>{});
    if (dkp == 128) return f(std::integral_constant<int, 128>{});
    if (dkp == 192) return f(std::integral_constant<int, 192>{});
    return f(std::integral_constant<int, 256>{});
}
// Workgroups of a launch: whole rounds of the 8 XCDs (locate()).
uint32_t blocks_of(const AttnLaunch &l) {
    const uint64_t g = static_cast<uint64_t>(l.b) * l.h * l.nseg;
    return static_cast<uint32_t>((g + 7) / 8 * 8 * l.nroles * l.nvb);
}

}  // namespace

// Segments of a sequence.  Without them a workgroup walks a head's whole sequence; with them the
// keys and values are read twice, the segments' states go to memory and back, and two or three small
// launches are added.  The fewest microseconds of a simple account are taken: a chunk costs a workgroup
// u when it has its CU to itself, 2 u with another beside it; half of that for the segments'
// own states; four passes over those at 5 TB/s.  u is 4 for 64 tokens of 128 x 128 bf16 heads.  (Gradients of 8
// sequences of 4096 tokens, 8 heads: 1 segment 243 us, 2 290, 3 298, 4 267, 6 289, 8 282; 2 sequences of
// 16384, 8 heads: 8 segments 192 us, 11 155, 16 126, 22 139, 32 129, 64 150; gradients of 2 of 301, 4 heads, fp32: 1
// segment 48 us, 3 39, 5 29, 10 25.  The account takes 1, 16 and 10.)
AttnPlan attn_plan(const AttnSizes &s, int nroles) {
    const int dkp = padded(nroles > 1 ? std::max(s.dk, s.dv) : s.dk);
    AttnPlan p;
    p.dkp = dkp;
    p.chunk = chunk_of(s.dtype, dkp);
    const int64_t chunks = std::max<int64_t>(1, (s.t + p.chunk - 1) / p.chunk);
    const int64_t nvb = ((nroles > 1 ? std::max(s.dk, s.dv) : s.dv) + kVB - 1) / kVB, pairs = std::max<int64_t>(1, s.b * s.h);
    const double u = 4.0 * dkp / 128 * p.chunk / 64 * (s.dtype == DW_BF16 ? 1.0 : s.dtype == DW_F16 ? 1.6 : 3.0);
    const int64_t slots = dkp <= 128 && (s.dtype != DW_F32 || dkp <= 64) ? 512 : 256;
    auto walk = [&](int64_t groups, int64_t per) {
        const int64_t rest = groups % slots;
        return (groups / slots * per * (slots / 256) + (rest == 0 ? 0.0 : rest <= 256 ? 1.0 * per : 2.0 * per)) * u;
    };
    double best = 0;
    p.seg_chunks = static_cast<int>(chunks);
    const int64_t most = pairs <= 65535 ? 64 : 1;  // (batch, head) pairs of the scan's grid
    for (int64_t want = 1; want <= most && want <= chunks; ++want) {
        const int64_t per = (chunks + want - 1) / want, nseg = (chunks + per - 1) / per;
        if (nseg > 1 && pairs * nvb * nroles * nseg > 1 << 22) break;  // launches of fewer than 2^32 threads
        double cost = walk(pairs * nvb * nroles * nseg, per);
        if (nseg > 1) {
            const int64_t states = nroles > 1 ? 2 : 1;
            cost += 0.5 * walk(pairs * nvb * states * nseg, per) + pairs * nseg * states * s.dk * s.dv * 16 / 5e6 + 8.0;
        }
        if (want == 1 || cost < best) {
            best = cost;
            p.seg_chunks = static_cast<int>(per);
        }
    }
    p.nseg = static_cast<int>((chunks + p.seg_chunks - 1) / p.seg_chunks);
    return p;
}

int attn_out_launch(const AttnLaunch &l, int dtype, hipStream_t stream) {
    return by_type(dtype, [&](auto tag) {
        return by_size(l.dkp, [&](auto d) {
            using T = decltype(tag);
            bool precise = false;
            for (int i = 0; i < l.nroles; ++i) precise = precise || l.role[i].zout;
            // fp32's state has its three planes in either form: only one is compiled
            if (precise || std::is_same<T, float>::value)
                hipLaunchKernelGGL((decay_out_kernel<T, decltype(d)::value, true>), dim3(blocks_of(l)), dim3(kWG), 0, stream,
                                   l);
            else
                hipLaunchKernelGGL((decay_out_kernel<T, decltype(d)::value, std::is_same<T, float>::value>), dim3(blocks_of(l)),
                                   dim3(kWG), 0, stream, l);
            return done();
        });
    });
}

int attn_state_launch(const AttnLaunch &l, float *const seg[2], int dtype, hipStream_t stream) {
    return by_type(dtype, [&](auto tag) {
        return by_size(l.dkp, [&](auto d) {
            hipLaunchKernelGGL((decay_state_kernel<decltype(tag), decltype(d)::value>), dim3(blocks_of(l)), dim3(kWG),
                               0, stream, l, seg[0], seg[1]);
            return done();
        });
    });
}

int attn_scan_launch(const AttnScan &one, const AttnScan &two, const float *log_decay, const int32_t *lengths, int b, int h,
                     int64_t t, int dk, int dv, int nseg, int64_t seg_tokens, hipStream_t stream) {
    const int size = dk * dv, v = size % 4 ? 1 : 4;
    const auto kern = v == 4 ? decay_scan_kernel<4> : decay_scan_kernel<1>;
    hipLaunchKernelGGL(kern, dim3((size + kThreads * v - 1) / (kThreads * v), b * h, two.seg ? 2 : 1), dim3(kThreads), 0, stream,
                       one, two, log_decay, lengths, h, t, size, nseg, seg_tokens);
    return done();
}

int attn_share_launch(const float *in, void *out, int64_t rows, int hs, int rep, int d, int dtype, hipStream_t stream) {
    const int64_t total = rows * hs * d;
    const uint32_t blocks = static_cast<uint32_t>(std::min<int64_t>((total + kThreads - 1) / kThreads, 8192));
    return by_type(dtype, [&](auto tag) {
        using T = decltype(tag);
        hipLaunchKernelGGL(share_kernel<T>, dim3(blocks), dim3(kThreads), 0, stream, in, static_cast<T *>(out), total, hs,
                           rep, d);
        return done();
    });
}

int attn_widen_launch(const void *x, const SeqStride &st, void *out, int64_t b, int64_t t, int heads, int d, int dtype,
                      hipStream_t stream) {
    const int dp = (d + 7) / 8 * 8;
    const int64_t total = b * t * heads * dp;
    const uint32_t blocks = static_cast<uint32_t>(std::min<int64_t>((total + kThreads - 1) / kThreads, 8192));
    return by_type(dtype, [&](auto tag) {
        using T = decltype(tag);
        hipLaunchKernelGGL(widen_kernel<T>, dim3(blocks), dim3(kThreads), 0, stream, static_cast<const T *>(x), st,
                           static_cast<T *>(out), total, t, heads, d, dp);
        return done();
    });
}

int attn_step_launch(const void *q, const void *k, const void *v, const float *log_decay, float *state, void *o,
                     const AttnSizes &s, const int64_t *st, int64_t state_stride, float scale, hipStream_t stream) {
    const SeqStride qs{st[0], 0, st[1]}, ks{st[2], 0, st[3]}, vs{st[4], 0, st[5]};
    const bool vec = s.dv % 4 == 0 && reinterpret_cast<uintptr_t>(state) % 16 == 0 && state_stride % 4 == 0;
    const dim3 grid(static_cast<uint32_t>(s.b * s.h), (s.dv + 31) / 32);
    return by_type(s.dtype, [&](auto tag) {
        using T = decltype(tag);
        auto kern = vec ? decay_step_kernel<T, true> : decay_step_kernel<T, false>;
        hipLaunchKernelGGL(kern, grid, dim3(kThreads), 0, stream, static_cast<const T *>(q), static_cast<const T *>(k),
                           static_cast<const T *>(v), log_decay, state, static_cast<T *>(o), s.h, s.h / s.hq, s.h / s.hk,
                           s.h / s.hv, s.dk, s.dv, qs, ks, vs, state_stride, scale);
        return done();
    });
}

}  // namespace dw
