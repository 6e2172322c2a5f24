// dw_act8.hpp -- the 8-bit checkpoint format and reads of eight consecutive values, shared by the
// checkpoint's own kernels (dw_act8.hip) and the norms that write or read one (dw_norm.hip).
//
// Along a row of c values each 32 share a step 2^e: the smallest power of two (at least 2^-126)
// by which the largest finite magnitude rounds to at most 127.  A value is kept as the whole
// number of steps nearest to it, ties to even, in a signed byte; -128 stands for a value that is
// not finite and comes back as a NaN.  codes: (rows, c) bytes; exps: (rows, ceil(c / 32)) bytes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dw_common.hpp"

namespace dw {

// Eight values from memory that need only be aligned to its own type: global loads and stores of
// gfx950 take any address, so rows of an odd length are read as widely as others.
template <typename T> struct Wide8 { T v[8]; };
template <typename T> __device__ __forceinline__ void load8(const T *p, float (&x)[8]) {
    Wide8<T> r;
    __builtin_memcpy(&r, p, sizeof(r));
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = to_f32(r.v[i]);
}
template <typename T> __device__ __forceinline__ void store8(T *p, const float (&x)[8]) {
    Wide8<T> r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r.v[i] = from_f32<T>(x[i]);
    __builtin_memcpy(p, &r, sizeof(r));
}
// The first n of them (n <= 8); the rest are zero.
template <typename T> __device__ __forceinline__ void load_upto8(const T *p, int n, float (&x)[8]) {
    if (n >= 8) {
        load8(p, x);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = i < n ? to_f32(p[i]) : 0.f;
    }
}
template <typename T> __device__ __forceinline__ void store_upto8(T *p, int n, const float (&x)[8]) {
    if (n >= 8) {
        store8(p, x);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = from_f32<T>(x[i]);
    }
}

// The bits of the largest finite magnitude of eight values.
__device__ __forceinline__ uint32_t act8_top(const float (&x)[8]) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
    if (top >= 0x7f800000u) {  // hardly ever: some are not finite
        top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t a = __float_as_uint(x[i]) & 0x7fffffffu;
            top = max(top, a < 0x7f800000u ? a : 0u);
        }
    }
    return top;
}
// The step's exponent for a largest magnitude: in [-126, 122].
__device__ __forceinline__ int act8_exponent(uint32_t top) {
    // 2^(e - 1) <= top < 2^e for e = biased exponent - 126: 64 to 128 steps of 2^(e - 7)
    const int e = max(static_cast<int>(top >> 23) - 126, -119) - 7;
    return __uint_as_float(top) * __uint_as_float(static_cast<uint32_t>(127 - e) << 23) >= 127.5f ? e + 1 : e;
}
// Eight codes: the product is exact, and adding 3 * 2^22 leaves the nearest whole number, ties to
// even, in the low bits.  A value that is not finite leaves an infinity or a NaN, found by its exponent.
__device__ __forceinline__ uint2 act8_codes(const float (&x)[8], int e) {
    const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    uint32_t c[8], all = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        c[i] = __float_as_uint(fmaf(x[i], inv, 12582912.f));
        all = max(all, c[i] & 0x7fffffffu);
    }
    if (all >= 0x7f800000u) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if ((c[i] & 0x7f800000u) == 0x7f800000u) c[i] = 0x80u;
    }
    uint2 r;
    r.x = __builtin_amdgcn_perm(__builtin_amdgcn_perm(c[3], c[2], 0x0c0c0400u), __builtin_amdgcn_perm(c[1], c[0], 0x0c0c0400u),
                                0x05040100u);
    r.y = __builtin_amdgcn_perm(__builtin_amdgcn_perm(c[7], c[6], 0x0c0c0400u), __builtin_amdgcn_perm(c[5], c[4], 0x0c0c0400u),
                                0x05040100u);
    return r;
}
__device__ __forceinline__ float act8_step(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }
// Eight codes' values with step 2^e: (code + 128) step - 128 step, each product exact while 128 steps are at most the
// type's largest value.  The step of 2^121 of a block that reaches 2^127 makes 2^128 of them, which no fp32 holds.
__device__ __forceinline__ void act8_values(uint2 q, int e, float most, float (&v)[8]) {
    const float step = act8_step(e), low = -128.f * step;
    const uint32_t u[2] = {q.x ^ 0x80808080u, q.y ^ 0x80808080u};  // code + 128 as a byte: 0 stands for a NaN
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fmaf(static_cast<float>((u[i / 4] >> (8 * (i & 3))) & 0xffu), step, low);
    // hardly ever: a byte of zero in either word, or steps so large that a value, or `low`, may pass the type's largest
    const uint32_t zero = ((u[0] - 0x01010101u) & ~u[0] & 0x80808080u) | ((u[1] - 0x01010101u) & ~u[1] & 0x80808080u);
    if (zero != 0 || -low > most) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool nan = ((u[i / 4] >> (8 * (i & 3))) & 0xffu) == 0;
            const float w = static_cast<float>(static_cast<int8_t>((i < 4 ? q.x : q.y) >> (8 * (i & 3)))) * step;
            v[i] = nan ? __uint_as_float(0x7fc00000u) : fminf(fmaxf(w, -most), most);
        }
    }
}
// The value of one code.
__device__ __forceinline__ float act8_value(int code, float step, float most) {
    const float v = static_cast<float>(code) * step;
    return code == -128 ? __uint_as_float(0x7fc00000u) : fminf(fmaxf(v, -most), most);
}

template <typename T> __device__ __forceinline__ float largest_finite();
template <> __device__ __forceinline__ float largest_finite<float>() { return __uint_as_float(0x7f7fffffu); }
template <> __device__ __forceinline__ float largest_finite<__half>() { return 65504.f; }
template <> __device__ __forceinline__ float largest_finite<bf16_t>() { return __uint_as_float(0x7f7f0000u); }

}  // namespace dw
