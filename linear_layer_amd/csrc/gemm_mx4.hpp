// Device code shared by the kernels of the products with a 4-bit microscaled
// operand: the matrix instructions, the decoding of codes, checked loads and
// the epilogue.
#pragma once

#include "launch.hpp"
#include "lowp.hpp"
#include "mx4.hpp"

namespace ll {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Byte BA of sa scales a, byte BB of sb scales b.
template <int BA, int BB>
__device__ __forceinline__ f32x4 mma_mx4(const u32x4 &a, const u32x4 &b, const f32x4 &c, int sa, int sb)
{
    const i32x8 x = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    const i32x8 y = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, BA, sa, BB, sb);
}

__device__ __forceinline__ f32x4 mma_f16(const u32x4 &a, const u32x4 &b, const f32x4 &c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c,
                                                  0, 0, 0);
}

__device__ __forceinline__ f32x4 mma_bf16(const u32x4 &a, const u32x4 &b, const f32x4 &c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Eight codes (one dword) as 16-bit values; `sc` carries the scale byte in an
// FP32 exponent field.
template <bool BF16>
__device__ __forceinline__ u32x4 decode8(uint32_t q, float sc)
{
    u32x4 r;
    if constexpr (BF16) {
        r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, sc, 0));
        r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, sc, 1));
        r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, sc, 2));
        r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, sc, 3));
    } else {
        r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, sc, 0));
        r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, sc, 1));
        r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, sc, 2));
        r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, sc, 3));
    }
    return r;
}

// Eight binary16 values as two bfloat16 parts, hi + lo exactly: hi is the
// value's top 8 bits of fraction, the rest has 3. An infinity or a NaN stays
// in hi alone.
__device__ __forceinline__ void split8(const u32x4 &a, u32x4 &hi, u32x4 &lo)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t h[2], l[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float v = (float)__builtin_bit_cast(_Float16, (uint16_t)(a[j] >> (16 * e)));
            const uint32_t b = __builtin_bit_cast(uint32_t, v), t = b & 0xffff0000u;
            const float d = v - __builtin_bit_cast(float, t);
            h[e] = t >> 16;
            l[e] = (b & 0x7f800000u) == 0x7f800000u ? 0u : __builtin_bit_cast(uint32_t, d) >> 16;
        }
        hi[j] = h[0] | h[1] << 16;
        lo[j] = l[0] | l[1] << 16;
    }
}

// Turns a 4 x 4 matrix of dwords around, v[i] of the 16 lanes of group g being its
// element (g, i): afterwards v[i] of group g is element (i, g).
__device__ __forceinline__ void turn4(u32x4 &v)
{
    const auto a = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
    const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    v = u32x4{c[0], c[1], d[0], d[1]};
}

// Whether a scale byte keeps the decoded values exact in binary16.
__device__ __forceinline__ bool f16_scale_ok(uint32_t s) { return s - 104u <= 36u; }

// Scale bytes 253 and 254: values reach 6 * 2^127, past bfloat16 and FP32, and
// decode8 makes them infinite. Such a block is decoded 2^-4 lower instead, and its
// products (exact, and 2^-13 at least) enter their sum times 2^4. They are rare, so
// nothing looks for them before a sum has come out infinite or NaN, as any such value
// makes it (looked for in the loops they cost the bfloat16 products 2 to 7 %).
__device__ __forceinline__ bool far_scale(uint32_t s) { return s - 253u < 2u; }
// The scale to decode with, and what is left of it.
__device__ __forceinline__ float near_part(uint32_t s) { return __uint_as_float((far_scale(s) ? s - 4u : s) << 23); }
__device__ __forceinline__ float far_part(uint32_t s) { return far_scale(s) ? 16.0f : 1.0f; }

__device__ __forceinline__ bool finite(float v) { return __builtin_fabsf(v) < __builtin_inff(); }

// Whether sums are finite, by one comparison of theirs (false too where they overflow
// together, which costs a look at each).
__device__ __forceinline__ bool finite4(const f32x4 &v) { return finite(v[0] + v[1] + v[2] + v[3]); }
template <int M, int N>
__device__ __forceinline__ bool all_finite(const f32x4 (&v)[M][N])
{
    f32x4 t = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                t[r] += v[m][n][r];
    return finite4(t);
}

// One value through the epilogue.
__device__ __forceinline__ float finish(const MxParams &p, float v, const float *dst)
{
    return p.beta == 0.0f ? p.alpha * v : __builtin_fmaf(p.alpha, v, p.beta * *dst);
}

// Those columns lo .. hi-1 of four neighbouring ones through the epilogue (lo <= 0,
// hi >= 4: all).
__device__ __forceinline__ void finish4(const MxParams &p, const f32x4 &v, float *dst, int64_t lo, int64_t hi)
{
    if (lo <= 0 && hi >= 4) {
        f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
        if (p.beta != 0.0f)
            __builtin_memcpy(&o, dst, 16);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            o[j] = p.beta == 0.0f ? p.alpha * v[j] : __builtin_fmaf(p.alpha, v[j], p.beta * o[j]);
        __builtin_memcpy(dst, &o, 16);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j >= lo && j < hi)
                dst[j] = finish(p, v[j], dst + j);
    }
}

// Tile `id` of the order that walks tiles in groups of p.group_m tile rows,
// column by column, so that the tiles in work at a time share rows and columns.
__device__ __forceinline__ void mx_tile_of(const MxParams &p, int id, int &tm, int &tn)
{
    const int group = p.group_m * p.tiles_n;
    const int first = id / group * p.group_m, within = id % group;
    const int rows = min(p.tiles_m - first, p.group_m);
    tm = first + within % rows;
    tn = within / rows;
}

// The first `have` (1 .. 15) of 16 bytes of which they are the last; 0 behind them.
__device__ __forceinline__ u32x4 last_bytes(const u32x4 &v, int have)
{
    const uint64_t lo = v[0] | (uint64_t)v[1] << 32, hi = v[2] | (uint64_t)v[3] << 32;
    const int s = 8 * (16 - have);   // 8 .. 120
    const uint64_t l = s >= 64 ? hi >> (s & 63) : lo >> s | hi << (64 - s), h = s >= 64 ? 0 : hi >> s;
    return u32x4{(uint32_t)l, (uint32_t)(l >> 32), (uint32_t)h, (uint32_t)(h >> 32)};
}

// The 16 bytes of codes of block `blk` of a row of K values; values past K
// are 0. Where a row has less than a block left, the last 16 bytes of it are
// read and shifted (LONG: K >= 32), or it is read byte by byte.
template <bool LONG>
__device__ __forceinline__ u32x4 load_block(const uint8_t *row, int64_t blk, int K)
{
    const int64_t k = blk * kMxBlock;
    u32x4 v = {0u, 0u, 0u, 0u};
    if (k + kMxBlock <= K) {
        v = load16<u32x4>(row + k / 2);
    } else if (k < K) {
        const int n = (int)(K - k), bytes = (n + 1) / 2;
        if constexpr (LONG) {
            v = load16<u32x4>(row + ((int64_t)K + 1) / 2 - 16);
            if (n & 1)
                v[3] &= 0x0fffffffu;
            if (bytes < 16)
                v = last_bytes(v, bytes);
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                if (j < bytes) {
                    const uint32_t b = row[k / 2 + j] & (2 * j + 1 < n ? 0xffu : 0x0fu);
                    v[j / 4] |= b << (8 * (j % 4));
                }
            }
        }
    }
    return v;
}

// 16-bit values k .. k+7 of a row of K; 0 past K (LONG: K >= 8).
template <bool LONG>
__device__ __forceinline__ u32x4 load_halves(const uint8_t *row, int64_t k, int K)
{
    u32x4 v = {0u, 0u, 0u, 0u};
    if (k + 8 <= K) {
        v = load16<u32x4>(row + 2 * k);
    } else if (k < K) {
        if constexpr (LONG) {
            v = last_bytes(load16<u32x4>(row + 2 * ((int64_t)K - 8)), 2 * (int)(K - k));
        } else {
            const uint16_t *h = reinterpret_cast<const uint16_t *>(row) + k;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (k + j < K)
                    v[j / 2] |= (uint32_t)h[j] << (16 * (j % 2));
        }
    }
    return v;
}

// A sum that is not finite, over the blocks [b0, b1) of a row of 16-bit A and a row of
// B: taken again by vector FMAs if a block has a far scale and none is NaN.
template <int A, bool LONG>
__device__ __forceinline__ float far_dot(float sum, const uint8_t *a, const uint8_t *b, const uint8_t *sb, int b0, int b1,
                                         int K)
{
    bool far = false, nan = false;
#pragma unroll 1
    for (int blk = b0; blk < b1; ++blk) {
        const uint32_t s = sb[blk];
        far |= far_scale(s);
        nan |= s == 255u;
    }
    if (!far || nan)
        return sum;
    sum = 0.0f;
    auto half = [&](const uint16_t h) __attribute__((always_inline)) { return A == MXA_F16 ? to_f32<LL_TYPE_F16>(h) : to_f32<LL_TYPE_BF16>(h); };
    if constexpr (LONG) {
#pragma unroll 1
        for (int blk = b0; blk < b1; ++blk) {
            const u32x4 q = load_block<true>(b, blk, K);
            const uint32_t s = sb[blk];
            float part = 0.0f;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const u32x4 x = load_halves<true>(a, (int64_t)blk * kMxBlock + 8 * t, K), y = decode8<true>(q[t], near_part(s));
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    part = __builtin_fmaf(half((uint16_t)(x[j / 2] >> (16 * (j & 1)))),
                                          to_f32<LL_TYPE_BF16>((uint16_t)(y[j / 2] >> (16 * (j & 1)))), part);
            }
            sum = __builtin_fmaf(part, far_part(s), sum);
        }
    } else {   // K < 32: one block, value by value
#pragma unroll 1
        for (int k = 0; k < K; ++k) {
            const uint32_t y = decode8<true>(b[k / 2] >> (4 * (k & 1)) & 15u, near_part(sb[0]))[0];
            sum = __builtin_fmaf(half(reinterpret_cast<const uint16_t *>(a)[k]), to_f32<LL_TYPE_BF16>((uint16_t)y), sum);
        }
        sum *= far_part(sb[0]);
    }
    return sum;
}

// Four neighbouring sums of row m and columns n .. n+3 (those inside N), in LDS that
// the calling lane alone uses, and all four after far_dot had those that are not finite.
template <int A, bool LONG>
__device__ __forceinline__ f32x4 settle4(const MxParams &p, const f32x4 &v, float *at, int64_t m, int64_t n, int b0, int b1)
{
    *reinterpret_cast<f32x4 *>(at) = v;
#pragma unroll 1
    for (int j = 0; j < 4; ++j)
        if (n + j < p.N && !finite(at[j]))
            at[j] = far_dot<A, LONG>(at[j], p.A + m * p.lda, p.B + (n + j) * p.ldb, p.SB + (n + j) * p.ldsb, b0, b1, p.K);
    return *reinterpret_cast<f32x4 *>(at);
}

}  // namespace ll
