// The 16-bit layer for few rows: every weight is read once for at most 64 rows, so memory bounds
// the product and the matrix cores have time to spare.
//
// A workgroup of NW waves computes MT x 16 rows by NB x 16 columns. Its waves share the inner
// dimension out in turns of 64 values: wave w takes turns w, w + NW, ... and reads its operands
// straight into the matrix instruction's registers, 16 bytes a lane (the instruction has four
// lanes to a row, so a load covers 64 bytes of 16 rows of W and the next one the other half of
// their lines). W's rows of DEPTH turns are on their way at a time. X's rows come from L2, where
// the other workgroups' reads have brought them; lanes past the last row read that row again,
// which costs no traffic. At the end the waves' sums meet in LDS and are added in the waves'
// order, and the write-back is that of the tile kernel.
#include "launch.hpp"
#include "linear16_finish.hpp"

namespace ll {

using namespace l16;

constexpr int kTurn = 64;   // values of the inner dimension a wave takes at a time

// Eight values of a row from k on; zeros past K. VEC: rows are whole 16-byte pieces.
template <bool VEC>
__device__ __forceinline__ f16x8 load8_at(const uint16_t *row, int64_t k, int K)
{
    u32x4 v = {0u, 0u, 0u, 0u};
    if (VEC ? k < K : k + 8 <= K) {
        v = load16<u32x4>(row + k);
    } else if (!VEC) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (k + e < K)
                v[e / 2] |= (uint32_t)row[k + e] << (16 * (e % 2));
    }
    return __builtin_bit_cast(f16x8, v);
}

template <bool BF16, int MT, int NB, int NW, int DEPTH, bool VEC>
__global__ void __launch_bounds__(64 * NW) l16_rows_kernel(L16Params p, int tiles_n)
{
    constexpr int PITCH = NB * 16 + 4;
    __shared__ float part[NW][MT * 16 * PITCH];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    Chunk c{};
    const int id = blockIdx.x / tiles_n;
    if (id >= find_chunk(p.groups, p.M, MT * 16, id, c))
        return;
    const int m0 = c.begin + c.index * MT * 16, n0 = (int)(blockIdx.x % tiles_n) * NB * 16;
    const int grp = lane >> 4, r16 = lane & 15;
    const uint16_t *w = static_cast<const uint16_t *>(p.B) + c.group * p.stride_b;
    const uint16_t *wrow[NB], *xrow[MT];
#pragma unroll
    for (int j = 0; j < NB; ++j)
        wrow[j] = w + (int64_t)min(n0 + 16 * j + r16, p.N - 1) * p.ldb + 8 * grp;
#pragma unroll
    for (int i = 0; i < MT; ++i)
        xrow[i] = p.A + (int64_t)min(m0 + 16 * i + r16, c.end - 1) * p.lda + 8 * grp;
    const int K = p.K - 8 * grp;   // this lane's values of a row

    f32x4 acc[MT][NB];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
            acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // (turns past K load nothing and add zeros: every wave has as many)
    const int turns = cdiv(cdiv(p.K, kTurn), NW);
    f16x8 wv[DEPTH][2][NB], xv[DEPTH][2][MT];
    auto fetch = [&](int t, f16x8 (&wd)[2][NB], f16x8 (&xd)[2][MT]) __attribute__((always_inline)) {
        const int64_t k = ((int64_t)t * NW + wave) * kTurn;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int j = 0; j < NB; ++j)
                wd[h][j] = load8_at<VEC>(wrow[j], k + 32 * h, K);
#pragma unroll
            for (int i = 0; i < MT; ++i)
                xd[h][i] = load8_at<VEC>(xrow[i], k + 32 * h, K);
        }
    };
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
        fetch(d, wv[d], xv[d]);
    for (int t = 0; t < turns; t += DEPTH) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {   // (past the last turn: zeros)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int j = 0; j < NB; ++j)
                        acc[i][j] = mma<BF16>(wv[d][h][j], xv[d][h][i], acc[i][j]);
            fetch(t + d + DEPTH, wv[d], xv[d]);
        }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
            *reinterpret_cast<f32x4 *>(&part[wave][(16 * i + r16) * PITCH + 16 * j + 4 * grp]) = acc[i][j];
    __syncthreads();
    // eight columns a lane; four lanes are a block of 32
    constexpr int LPR = NB * 2;
    static_assert(LPR % 4 == 0, "whole blocks of Z's 8 bits");
    for (int s = tid; s < MT * 16 * LPR; s += 64 * NW) {
        const int rl = s / LPR, cl = s % LPR * 8, row = m0 + rl, col = n0 + cl, n = p.N - col;
        const bool live = row < c.end && n > 0;
        float v[8], bias[8], r[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = r[e] = 0.0f;
        load_row<LL_TYPE_F32, 8>(p.bias + (int64_t)c.group * p.N + col, p.bias != nullptr ? n : 0, bias);
        if (p.R != nullptr)
            load8<BF16>(p.ctype, p.R, (int64_t)row * p.ldr + col, live ? n : 0, r);
#pragma unroll
        for (int k = 0; k < NW; ++k) {
            const f32x4 lo = *reinterpret_cast<const f32x4 *>(&part[k][rl * PITCH + cl]);
            const f32x4 hi = *reinterpret_cast<const f32x4 *>(&part[k][rl * PITCH + cl + 4]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[e] += lo[e], v[4 + e] += hi[e];
        }
        finish_fwd<BF16>(p, v, bias, r, row, col, n, live);
    }
}

template <bool BF16, int MT, int NB, int NW, int DEPTH, bool VEC>
static hipError_t launch_mt(const L16Params &p, hipStream_t s)
{
    const int tiles_n = cdiv(p.N, NB * 16);
    const int64_t rows = p.groups.offsets == nullptr ? cdiv(p.M, MT * 16)
                                                     : (int64_t)(p.M / (MT * 16)) + (p.groups.n < p.M ? p.groups.n : p.M);
    if (rows * tiles_n > max_grid_x(64 * NW))
        return hipErrorInvalidValue;
    hipLaunchKernelGGL((l16_rows_kernel<BF16, MT, NB, NW, DEPTH, VEC>), dim3((unsigned)(rows * tiles_n)), dim3(64 * NW), 0, s,
                       p, tiles_n);
    return hipGetLastError();
}

template <bool BF16, bool VEC>
static hipError_t launch_rows16(const L16Params &p, hipStream_t s)
{
    const int each = cdiv(p.M, p.groups.n < p.M ? p.groups.n : p.M);
    if (each <= 16)
        return launch_mt<BF16, 1, 2, 8, 3, VEC>(p, s);
    if (each <= 32)
        return launch_mt<BF16, 2, 2, 8, 3, VEC>(p, s);
    return launch_mt<BF16, 4, 2, 8, 2, VEC>(p, s);
}

hipError_t launch_l16_rows(bool bf16, const L16Params &p, bool vec, hipStream_t s)
{
    if (vec)
        return bf16 ? launch_rows16<true, true>(p, s) : launch_rows16<false, true>(p, s);
    return bf16 ? launch_rows16<true, false>(p, s) : launch_rows16<false, false>(p, s);
}

}  // namespace ll
