// Microscaled 4-bit floating point (MX4): blocks of 32 values along a row,
// each value a 4-bit code (E2M1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign), each
// block one scale byte s that multiplies it by 2^(s - 127) (255: not a number).
// Two codes share a byte, the earlier one in the low half.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"
#include "linear_layer.h"

namespace ll {

constexpr int kMxBlock = 32;

// FP32 <-> storage types. The 16-bit types travel as raw patterns.
template <int TYPE> struct Elem { using type = uint16_t; };
template <> struct Elem<LL_TYPE_F32> { using type = float; };

template <int TYPE>
__device__ __forceinline__ float to_f32(typename Elem<TYPE>::type v)
{
    if constexpr (TYPE == LL_TYPE_F32)
        return v;
    else if constexpr (TYPE == LL_TYPE_F16)
        return (float)__builtin_bit_cast(_Float16, v);
    else
        return __builtin_bit_cast(float, (uint32_t)v << 16);
}

// Rounded once, to nearest even.
template <int TYPE>
__device__ __forceinline__ typename Elem<TYPE>::type from_f32(float v)
{
    if constexpr (TYPE == LL_TYPE_F32)
        return v;
    else if constexpr (TYPE == LL_TYPE_F16)
        return __builtin_bit_cast(uint16_t, (_Float16)v);
    else
        return __builtin_bit_cast(uint16_t, (__bf16)v);
}

// Eight values of a row from `src` on as they stand in memory, the first n of them
// inside it (n >= 8: all; n <= 0, or a null src: zeros). 16-byte loads at any
// alignment and one path for every lane: where the row ends inside the eight, its
// last eight are read (`wide`: the row has eight; else one by one), and raw_values
// puts them in their places, once they are there. (Read one by one, they hold up
// their workgroup: gradient of 8192 x 2100 bfloat16 110 us, of 8192 x 2104 65.)
template <int TYPE, int P>
__device__ __forceinline__ void raw_row(const typename Elem<TYPE>::type *src, int64_t n, bool wide, u32x4 (&v)[P])
{
    using T = typename Elem<TYPE>::type;
    constexpr int PER = 16 / (int)sizeof(T);
    static_assert(P * PER == 8, "eight values");
#pragma unroll
    for (int i = 0; i < P; ++i)
        v[i] = u32x4{0u, 0u, 0u, 0u};
    if (src == nullptr || n <= 0)
        return;
    if (wide) {
        src += n < 8 ? n - 8 : 0;
#pragma unroll
        for (int i = 0; i < P; ++i)
            v[i] = load16<u32x4>(src + i * PER);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) {
                uint32_t w = 0;
                __builtin_memcpy(&w, src + j, sizeof(T));
                v[j / PER][j % PER * (int)sizeof(T) / 4] |= w << (8 * (j * (int)sizeof(T) % 4));
            }
    }
}

template <int TYPE, int P>
__device__ __forceinline__ void raw_values(const u32x4 (&raw)[P], int64_t n, bool wide, float (&v)[8])
{
    constexpr int PER = 8 / P;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if constexpr (TYPE == LL_TYPE_F32)
            v[j] = __uint_as_float(raw[j / PER][j % PER]);
        else
            v[j] = to_f32<TYPE>((uint16_t)(raw[0][j / 2] >> (16 * (j & 1))));
    }
    if (wide && n > 0 && n < 8) {   // the row's last eight: n of them from 8 - n on
        const int s = 8 - (int)n;
#pragma unroll
        for (int d = 4; d >= 1; d >>= 1)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = (s & d) ? (j + d < 8 ? v[j + d] : 0.0f) : v[j];
    }
}

// E values of a row from `src` on, the first n of them inside it (n >= E: all);
// the others are 0. Whole groups take 16-byte loads at any alignment.
template <int TYPE, int E>
__device__ __forceinline__ void load_row(const typename Elem<TYPE>::type *src, int64_t n, float (&v)[E])
{
    using T = typename Elem<TYPE>::type;
    constexpr int PER = 16 / (int)sizeof(T);
    static_assert(E % PER == 0, "whole 16-byte chunks");
    if (n >= E) {
#pragma unroll
        for (int i = 0; i < E / PER; ++i) {
            const u32x4 raw = load16<u32x4>(src + i * PER);
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                if constexpr (sizeof(T) == 4)
                    v[i * PER + j] = __uint_as_float(raw[j]);   // (a bit_cast of a vector's element reads element 0)
                else
                    v[i * PER + j] = to_f32<TYPE>((uint16_t)(raw[j / 2] >> (16 * (j & 1))));
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < E; ++j)
            v[j] = j < n ? to_f32<TYPE>(src[j]) : 0.0f;
    }
}

// The first n (n >= E: all) of E values to a row, rounded to its type.
template <int TYPE, int E>
__device__ __forceinline__ void store_row(typename Elem<TYPE>::type *dst, int64_t n, const float (&v)[E])
{
    using T = typename Elem<TYPE>::type;
    constexpr int PER = 16 / (int)sizeof(T);
    static_assert(E % PER == 0, "whole 16-byte chunks");
    if (n >= E) {
#pragma unroll
        for (int i = 0; i < E / PER; ++i) {
            u32x4 raw;
            if constexpr (sizeof(T) == 4) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    raw[j] = __builtin_bit_cast(uint32_t, v[i * 4 + j]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    raw[j] = (uint32_t)from_f32<TYPE>(v[i * 8 + 2 * j]) |
                             (uint32_t)from_f32<TYPE>(v[i * 8 + 2 * j + 1]) << 16;
            }
            __builtin_memcpy(dst + i * PER, &raw, 16);
        }
    } else {
#pragma unroll
        for (int j = 0; j < E; ++j)
            if (j < n)
                dst[j] = from_f32<TYPE>(v[j]);
    }
}

// The scale byte of a block whose largest magnitude has the FP32 pattern
// `top`: floor(log2(top)) - 2 + 127, at least 0, so that the largest value
// lands in [4, 8) of the codes' range (codes stop at 6); 255 for a block that
// holds an infinity or a NaN, whose values have no 4-bit form. The exponent
// field of an FP32 subnormal is 0 and gives byte 0 too, as its logarithm does.
__device__ __forceinline__ uint32_t mx_scale(uint32_t top)
{
    const uint32_t e = top >> 23;
    return e == 255u ? 255u : e > 2u ? e - 2u : 0u;
}

// Eight codes of eight values under scale byte `s`, to nearest with ties to
// the even code, magnitudes past 6 to 6. The conversion reads the scale from
// the exponent field of an FP32 value (field 0: 2^-127).
__device__ __forceinline__ uint32_t mx_encode8(const float *v, uint32_t s)
{
    const float sc = __builtin_bit_cast(float, s << 23);
    uint32_t r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], sc, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], sc, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4], v[5], sc, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6], v[7], sc, 3);
    return s == 255u ? 0u : r;
}

}  // namespace ll
