// Products with a 4-bit microscaled operand (MX4, see mx4.hpp):
//   C = alpha * A * B^T + beta * C,  B [N][K] in MX4, A [M][K] in MX4, binary16 or bfloat16,
// FP32 sums, FP32 C.
//
// With both operands in MX4 the inner product runs on the scaled matrix
// instruction v_mfma_scale_f32_16x16x128_f8f6f4. Its operand layout is the
// format's own: lane l holds row l % 16 of the block and the 32 values of
// k = 32 * (l / 16) .. +31, which is one 16-byte chunk of codes under one
// scale byte, so codes and scales go from memory to the instruction as they
// are. With 16-bit A the codes are turned into 16-bit values in registers,
// scale applied, and the product runs on the 16x16x32 instruction of A's type.
// A lane then holds a whole block of B, 32 values, and gives 8 of them to each
// of four instructions; the order of k inside an instruction is free as long as
// A's lanes follow it.
//
// An E2M1 value times a power of two is exact in bfloat16 (its subnormals
// included, which the matrix units keep). In binary16 it is exact for scale
// bytes 104 .. 140 only (2^-23 .. 2^13); past those the wave splits A's values
// into two bfloat16 parts instead (11 bits of fraction into 8 and 3) and
// multiplies twice, which is exact for every scale.
#include "linear_layer.h"
#include "launch.hpp"
#include "lowp.hpp"
#include "mx4.hpp"

namespace ll {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x4 mma_mx4(const u32x4 &a, const u32x4 &b, const f32x4 &c, int sa, int sb)
{
    const i32x8 x = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    const i32x8 y = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, 0, sa, 0, sb);
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

// Whether a scale byte keeps the decoded values exact in binary16.
__device__ __forceinline__ bool f16_scale_ok(uint32_t s) { return s - 104u <= 36u; }

// One value through the epilogue.
__device__ __forceinline__ float finish(const MxParams &p, float v, const float *dst)
{
    return p.beta == 0.0f ? p.alpha * v : __builtin_fmaf(p.alpha, v, p.beta * *dst);
}

// ---------------------------------------------------------------------------
// Streaming kernel: operands go from memory (or L2) straight into registers.
// A workgroup computes a (16 FM) x (16 FN) tile of C; its W waves take the K
// range in turns of 128 * J values, and their sums are added through LDS in
// wave order, so a result never depends on the run. This serves the products
// that read B once (a few rows of A, where HBM bounds them and nothing is
// shared), those too small to give the tile kernels a workgroup per CU, and
// every operand whose alignment rules out the direct-to-LDS copies: rows are
// read in 16-byte pieces at any alignment, the block that crosses K byte by
// byte.
//
// Rows past M or N read the last row instead; their sums are not stored.

// The 16 bytes of codes of block `blk` of a row of K values; values past K
// are 0.
__device__ __forceinline__ u32x4 load_block(const uint8_t *row, int64_t blk, int K)
{
    const int64_t k = blk * kMxBlock;
    u32x4 v = {0u, 0u, 0u, 0u};
    if (k + kMxBlock <= K) {
        v = load16<u32x4>(row + k / 2);
    } else if (k < K) {
        const int n = (int)(K - k);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            if (2 * j < n) {
                const uint32_t b = row[k / 2 + j] & (2 * j + 1 < n ? 0xffu : 0x0fu);
                v[j / 4] |= b << (8 * (j % 4));
            }
        }
    }
    return v;
}

// 16-bit values k .. k+7 of a row of K; 0 past K.
__device__ __forceinline__ u32x4 load_halves(const uint8_t *row, int64_t k, int K)
{
    u32x4 v = {0u, 0u, 0u, 0u};
    if (k + 8 <= K) {
        v = load16<u32x4>(row + 2 * k);
    } else if (k < K) {
        const uint16_t *h = reinterpret_cast<const uint16_t *>(row) + k;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (k + j < K)
                v[j / 2] |= (uint32_t)h[j] << (16 * (j % 2));
    }
    return v;
}

template <int A, int FM, int FN, int J, int W>
__global__ void __launch_bounds__(64 * W) gemm_mx4_stream_kernel(MxParams p)
{
    constexpr int BM = 16 * FM, BN = 16 * FN;
    constexpr int AC = A == MXA_MX4 ? 1 : 4;   // 16-byte chunks of A per lane and block
    __shared__ float part[W][BM * BN];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, r16 = lane & 15;
    const int id = block_index(blockIdx.x, gridDim.x);
    const int tm = id % p.tiles_m, tn = id / p.tiles_m;
    const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
    const int K = p.K;
    const int64_t nblk = (int64_t)(K - 1) / kMxBlock + 1;
    const int64_t nunit = (nblk + 4 * J - 1) / (4 * J);

    const uint8_t *arow[FM], *sarow[FM], *brow[FN], *sbrow[FN];
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        int64_t m = m0 + 16 * i + r16;
        m = m < p.M ? m : p.M - 1;
        arow[i] = p.A + m * p.lda;
        sarow[i] = A == MXA_MX4 ? p.SA + m * p.ldsa : nullptr;
    }
#pragma unroll
    for (int i = 0; i < FN; ++i) {
        int64_t n = n0 + 16 * i + r16;
        n = n < p.N ? n : p.N - 1;
        brow[i] = p.B + n * p.ldb;
        sbrow[i] = p.SB + n * p.ldsb;
    }

    struct Unit {
        u32x4 a[J][FM][AC], b[J][FN];
        uint32_t sa[J][A == MXA_MX4 ? FM : 1], sb[J][FN];
    };
    auto fetch = [&](Unit &u, int64_t unit) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int64_t blk = (unit * J + j) * 4 + g;
#pragma unroll
            for (int i = 0; i < FN; ++i) {
                u.b[j][i] = load_block(brow[i], blk, K);
                u.sb[j][i] = blk < nblk ? sbrow[i][blk] : 127u;
            }
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                if constexpr (A == MXA_MX4) {
                    u.a[j][i][0] = load_block(arow[i], blk, K);
                    u.sa[j][i] = blk < nblk ? sarow[i][blk] : 127u;
                } else {
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        u.a[j][i][t] = load_halves(arow[i], blk * kMxBlock + 8 * t, K);
                }
            }
        }
    };

    f32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    auto multiply = [&](const Unit &u) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            if constexpr (A == MXA_MX4) {
#pragma unroll
                for (int n = 0; n < FN; ++n)
#pragma unroll
                    for (int m = 0; m < FM; ++m)
                        acc[m][n] = mma_mx4(u.a[j][m][0], u.b[j][n], acc[m][n], (int)u.sa[j][m], (int)u.sb[j][n]);
            } else {
                bool wide = false;   // scales binary16 cannot take
                if constexpr (A == MXA_F16) {
#pragma unroll
                    for (int n = 0; n < FN; ++n)
                        wide |= !f16_scale_ok(u.sb[j][n]);
                    wide = __any(wide);
                }
#pragma unroll
                for (int n = 0; n < FN; ++n) {
                    const float sc = __builtin_bit_cast(float, u.sb[j][n] << 23);
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        if (A == MXA_F16 && !wide) {
                            const u32x4 b = decode8<false>(u.b[j][n][t], sc);
#pragma unroll
                            for (int m = 0; m < FM; ++m)
                                acc[m][n] = mma_f16(u.a[j][m][t], b, acc[m][n]);
                        } else {
                            const u32x4 b = decode8<true>(u.b[j][n][t], sc);
#pragma unroll
                            for (int m = 0; m < FM; ++m) {
                                if constexpr (A == MXA_F16) {
                                    u32x4 hi, lo;
                                    split8(u.a[j][m][t], hi, lo);
                                    acc[m][n] = mma_bf16(lo, b, acc[m][n]);
                                    acc[m][n] = mma_bf16(hi, b, acc[m][n]);
                                } else {
                                    acc[m][n] = mma_bf16(u.a[j][m][t], b, acc[m][n]);
                                }
                            }
                        }
                    }
                }
            }
        }
    };

    for (int64_t unit = wave; unit < nunit; unit += W) {
        Unit u;
        fetch(u, unit);
        multiply(u);
    }

    // lane l holds column l % 16 and rows 4 * (l / 16) .. +3 of a block
#pragma unroll
    for (int m = 0; m < FM; ++m)
#pragma unroll
        for (int n = 0; n < FN; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                part[wave][(16 * m + 4 * g + r) * BN + 16 * n + r16] = acc[m][n][r];
    __syncthreads();
#pragma unroll
    for (int i = tid; i < BM * BN; i += 64 * W) {
        const int64_t m = m0 + i / BN, n = n0 + i % BN;
        if (m >= p.M || n >= p.N)
            continue;
        float v = part[0][i];
#pragma unroll
        for (int w = 1; w < W; ++w)
            v += part[w][i];
        float *dst = p.C + m * p.ldc + n;
        *dst = finish(p, v, dst);
    }
}

template <int A, int FM, int FN, int J, int W>
static hipError_t launch_stream(MxParams p, hipStream_t s)
{
    p.tiles_m = cdiv(p.M, 16 * FM);
    p.tiles_n = cdiv(p.N, 16 * FN);
    const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
    if (tiles > max_grid_x(64 * W))
        return hipErrorInvalidValue;
    hipLaunchKernelGGL((gemm_mx4_stream_kernel<A, FM, FN, J, W>), dim3((unsigned)tiles), dim3(64 * W), 0, s, p);
    return hipGetLastError();
}

template <int A>
static hipError_t launch_a(const MxParams &p, int cus, hipStream_t s)
{
    if (p.M <= 16)
        return launch_stream<A, 1, 1, 1, 4>(p, s);
    return launch_stream<A, 4, 4, 1, 4>(p, s);
}

hipError_t launch_gemm_mx4(MxParams p, int a, int cus, hipStream_t s)
{
    if (a == MXA_MX4)
        return launch_a<MXA_MX4>(p, cus, s);
    if (a == MXA_F16)
        return launch_a<MXA_F16>(p, cus, s);
    return launch_a<MXA_BF16>(p, cus, s);
}

}  // namespace ll
