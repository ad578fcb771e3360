// What the kernels of the 16-bit layer's products share: the matrix instruction, copies into
// LDS and the order of 16-byte pieces in it, and the write-back of eight sums.
#pragma once

#include <type_traits>
#include <utility>

#include "linear16.hpp"

namespace ll {
namespace l16 {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

template <bool BF16> constexpr int kType16 = BF16 ? LL_TYPE_BF16 : LL_TYPE_F16;

template <bool BF16>
__device__ __forceinline__ f32x4 mma(const f16x8 &a, const f16x8 &b, const f32x4 &c)
{
    if constexpr (BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                       0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// 16-byte chunk c of row `row` of a ROWS stage, and unit u of k-row k of a COLS stage.
__device__ __forceinline__ int rows_swz(int row) { return (row >> 1) & 7; }
__device__ __forceinline__ int cols_swz(int k) { return 2 * (k & 3) + ((k >> 3) & 1); }

template <int... I, class F>
__device__ __forceinline__ void static_for_(std::integer_sequence<int, I...>, F f)
{
    (f(std::integral_constant<int, I>{}), ...);
}
// f(0), .., f(N - 1) with constants for arguments.
template <int N, class F>
__device__ __forceinline__ void static_for(F f)
{
    static_for_(std::make_integer_sequence<int, N>{}, f);
}

constexpr uint32_t kPastEnd = 0x80000000u;   // past the end of every buffer here: 256 rows of less than 2^21 values

// buffer_load_dwordx4 into LDS: this lane's 16 bytes at byte `off` of the buffer go to LDS
// byte lds_base + 16 * lane, zeros where they lie past its end. Inline assembly, so that the
// compiler does not take it for an LDS store that every LDS read must wait for; the caller
// waits for the copies before the barrier that publishes them. The compiler's hazard checks
// do not look inside: M0 may be used a wait state after its write, and a descriptor that a
// vector instruction wrote (v_readlane, of a spilled one) by a load only five later, but by a
// scalar instruction at once. Hence the two moves, which are the wait for M0 too.
__device__ __forceinline__ void lds_buffer_16(const u32x4 &buffer, uint32_t off, uint32_t lds_base)
{
    const uint64_t lo = (uint64_t)buffer[1] << 32 | buffer[0], hi = (uint64_t)buffer[3] << 32 | buffer[2];
    asm volatile("s_mov_b32 m0, %0\n\ts_mov_b64 s[92:93], %2\n\ts_mov_b64 s[94:95], %3\n\t"
                 "buffer_load_dwordx4 %1, s[92:95], 0 offen lds"
                 :
                 : "s"(lds_base), "v"(off), "s"(lo), "s"(hi)
                 : "memory", "m0", "s92", "s93", "s94", "s95");
}

// Eight values of a matrix of LL_TYPE_F32 or the 16-bit type, the first n of them inside it.
template <bool BF16>
__device__ __forceinline__ void load8(int type, const void *base, int64_t at, int64_t n, float (&v)[8])
{
    if (type == LL_TYPE_F32)
        load_row<LL_TYPE_F32, 8>(static_cast<const float *>(base) + at, n, v);
    else
        load_row<kType16<BF16>, 8>(static_cast<const uint16_t *>(base) + at, n, v);
}
template <bool BF16>
__device__ __forceinline__ void store8(int type, void *base, int64_t at, int64_t n, const float (&v)[8])
{
    if (type == LL_TYPE_F32)
        store_row<LL_TYPE_F32, 8>(static_cast<float *>(base) + at, n, v);
    else
        store_row<kType16<BF16>, 8>(static_cast<uint16_t *>(base) + at, n, v);
}

// Eight sums of row `row`, columns col .. col + 7, to the forward product's outputs. n of
// them are inside (8 or more: all); r: what is added after the activation. Lanes without a row
// (live false) take part in the blocks' maxima of their neighbours' row only.
template <bool BF16>
__device__ __forceinline__ void finish_fwd(const L16Params &p, float (&v)[8], const float (&bias)[8], const float (&r)[8],
                                           int64_t row, int col, int n, bool live)
{
#pragma unroll
    for (int e = 0; e < 8; ++e)
        v[e] += bias[e];
    if (p.ZQ != nullptr) {
        // blocks of 32: four neighbouring lanes, which are of one row
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            top = max(top, e < n ? __builtin_bit_cast(uint32_t, v[e]) & 0x7fffffffu : 0u);
        const uint32_t s = mx8_scale(max_of_quad(top));
        if (live) {
            const uint32_t lo = mx8_encode4(v[0], v[1], v[2], v[3], s), hi = mx8_encode4(v[4], v[5], v[6], v[7], s);
            const uint64_t q = (uint64_t)hi << 32 | lo;
            uint8_t *dst = p.ZQ + row * p.ldzq + col;
            if (n >= 8) {
                __builtin_memcpy(dst, &q, 8);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e < n)
                        dst[e] = (uint8_t)(q >> (8 * e));
            }
            if ((col & 31) == 0)
                p.ZS[row * p.ldzs + (col >> 5)] = (uint8_t)s;
        }
    }
    if (!live)
        return;
    if (p.Z != nullptr)
        store_row<kType16<BF16>, 8>(p.Z + row * p.ldz + col, n, v);
    with_activation(act_for(p.act, p.ctype == LL_TYPE_F32), [&](auto kind) __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = activate<decltype(kind)::value>(v[e]);
    });
#pragma unroll
    for (int e = 0; e < 8; ++e)
        v[e] += r[e];
    store8<BF16>(p.ctype, p.C, row * p.ldc + col, n, v);
}

}  // namespace l16
}  // namespace ll
