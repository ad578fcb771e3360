// The residual step between two blocks of a network and its gradient:
//   x' = x + alpha * gate * (y * r_y * w_post),  r_y = (mean(y^2)  + eps)^(-1/2)
//   h  = x' * r_x * w_pre,                       r_x = (mean(x'^2) + eps)^(-1/2)
// per row of N values: y is the block's product (FP32), x the residual stream,
// gate, w_post, w_pre vectors over the columns. Sums, means and x' between the
// two norms are FP32; x' and h are rounded once each.
//
// Gradient, given dx' and dh. With u = y * r_y, n = x' * r_x and
// t = alpha * gate * w_post:
//   T  = dx' + r_x * (dh * w_pre - n * mean(dh * w_pre * n))   (all that reaches x')
//   dx = T,  dy = r_y * (T * t - u * mean(T * t * u))
//   dgate = alpha * w_post * S,  dw_post = alpha * gate * S,  S = sum over rows of T * u
//   dw_pre = sum over rows of dh * n
//
// Both are bound by HBM: a row is read once into registers and its sums go
// through one workgroup. Rows too long for the registers are read again. 8192 x 4096
// bfloat16 forward 70 us, 4.8 TB/s; 8191 x 4096 gradient 114 us, 4.7 TB/s, of which 8
// add the partial sums over rows (both from memory).
#include "linear_layer.h"
#include "lowp.hpp"
#include "mx4.hpp"

namespace ll {

// LDS of a workgroup's sums: a place for each of up to 16 waves, of `N` sums in turn.
template <int N>
struct Sums {
    float at[N][16];
    // Once, by every thread of a workgroup of more than one wave.
    __device__ __forceinline__ void clear()
    {
        if (threadIdx.x < 16 * N)
            (&at[0][0])[threadIdx.x] = 0.0f;
        __syncthreads();
    }
};

// The sums of V values over a workgroup, in every thread, by way of places SLOT ..
// SLOT + V - 1; where WAVE over the calling wave alone. The order is fixed: lanes by
// halving distance, then waves likewise. One barrier: a slot is used again only after
// a sum through another one.
template <bool WAVE, int SLOT, int V, int N>
__device__ __forceinline__ void block_sum(float (&v)[V], Sums<N> &lds)
{
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1)
            v[i] += __shfl_xor(v[i], d);
    }
    if constexpr (!WAVE) {
        static_assert(SLOT + V <= N, "places");
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                lds.at[SLOT + i][threadIdx.x >> 6] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < V; ++i) {
            v[i] = lds.at[SLOT + i][threadIdx.x & 15];
#pragma unroll
            for (int d = 8; d >= 1; d >>= 1)
                v[i] += __shfl_xor(v[i], d);
        }
    }
}

__device__ __forceinline__ float inv_rms(float sum, int n, float eps)
{
    return 1.0f / sqrtf(sum / (float)n + eps);
}

// Eight values of a column vector from c on; `one` where there is no vector.
__device__ __forceinline__ void load_vec(const float *v, int64_t c, int64_t n, float one, float (&o)[8])
{
    if (v == nullptr) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            o[j] = one;
    } else {
        load_row<LL_TYPE_F32, 8>(v + c, n - c, o);
    }
}

// A thread holds C groups of 8 neighbouring values, 8 columns times the workgroup's
// width (whole waves, as many as the row needs) apart. LONG: rows longer than 8 * NT * C, walked in several passes over memory,
// each sum in passes of its own.
// MAX 64: a row to a wave, four waves to a workgroup, no barrier.
// EARLY: the vectors are read with the row, not where they are used: with few rows
// nothing else hides their latency (4 x 4096 binary16 4.9 -> 4.0 us).
template <int TYPE, int MAX, int C, bool LONG, bool EARLY>
__global__ void __launch_bounds__(MAX == 64 ? 256 : MAX) rmsnorm_residual_kernel(NormParams p)
{
    using T = typename Elem<TYPE>::type;
    constexpr bool WAVE = MAX == 64;
    __shared__ Sums<2> lds;
    const int N = p.N, NT = WAVE ? 64 : (int)blockDim.x, tid = WAVE ? threadIdx.x & 63 : threadIdx.x;
    const int64_t rows = WAVE ? 4 : 1;
    if constexpr (!WAVE)
        lds.clear();
    for (int64_t m = blockIdx.x * rows + (WAVE ? threadIdx.x >> 6 : 0); m < p.M; m += gridDim.x * rows) {
        // without y or h a row has one sum: its slot is free for the next row once
        // every wave has read it (of a workgroup that has a next row, past 2^20 rows)
        if constexpr (!WAVE)
            if (m != blockIdx.x && (p.Y == nullptr || p.H == nullptr))
                __syncthreads();
        const float *y = p.Y != nullptr ? p.Y + m * p.ldy : nullptr;
        const T *x = static_cast<const T *>(p.X) + m * p.ldx;
        T *xo = p.XO != nullptr ? static_cast<T *>(p.XO) + m * p.ldxo : nullptr;
        T *h = p.H != nullptr ? static_cast<T *>(p.H) + m * p.ldh : nullptr;
        const int span = 8 * NT * C, passes = LONG ? cdiv(N, span) : 1;
        float yv[C][8], xv[C][8];
        auto load = [&](int pass) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int64_t col = (int64_t)pass * span + 8 * ((int64_t)c * NT + tid);
                load_row<TYPE, 8>(x + col, N - col, xv[c]);
                if (y != nullptr)
                    load_row<LL_TYPE_F32, 8>(y + col, N - col, yv[c]);
            }
        };
        float ry = 0.0f;
        float ew[EARLY ? C : 1][8], eg[EARLY ? C : 1][8], ep[EARLY ? C : 1][8];
        static_assert(!EARLY || !LONG, "one pass");
        if (!LONG)
            load(0);
        if constexpr (EARLY) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int64_t col = 8 * ((int64_t)c * NT + tid);
                load_vec(p.w_post, col, N, 1.0f, ew[c]);
                load_vec(p.gate, col, N, 1.0f, eg[c]);
                load_vec(p.w_pre, col, N, 1.0f, ep[c]);
            }
        }
        if (y != nullptr) {
            float s[1] = {0.0f};
            for (int pass = 0; pass < passes; ++pass) {
                if (LONG)
                    load(pass);
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        s[0] = __builtin_fmaf(yv[c][j], yv[c][j], s[0]);
            }
            block_sum<WAVE, 0>(s, lds);
            ry = inv_rms(s[0], N, p.eps);
        }
        // x' in xv; written where asked for
        auto residual = [&](int pass, bool store) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int64_t col = (int64_t)pass * span + 8 * ((int64_t)c * NT + tid);
                if (col >= N)
                    continue;
                if (y != nullptr) {
                    float w[8], g[8];
                    if constexpr (EARLY) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            w[j] = ew[c][j], g[j] = eg[c][j];
                    } else {
                        load_vec(p.w_post, col, N, 1.0f, w);
                        load_vec(p.gate, col, N, 1.0f, g);
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        xv[c][j] = __builtin_fmaf(p.alpha * g[j], yv[c][j] * ry * w[j], xv[c][j]);
                }
                if (store && xo != nullptr)
                    store_row<TYPE, 8>(xo + col, N - col, xv[c]);
            }
        };
        float s[1] = {0.0f};
        for (int pass = 0; pass < passes; ++pass) {
            if (LONG)
                load(pass);
            // in place (XO = X) a long row is written by its last pass only
            residual(pass, !LONG || h == nullptr);
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    s[0] = __builtin_fmaf(xv[c][j], xv[c][j], s[0]);
        }
        if (h == nullptr)
            continue;
        block_sum<WAVE, 1>(s, lds);
        const float rx = inv_rms(s[0], N, p.eps);
        for (int pass = 0; pass < passes; ++pass) {
            if (LONG) {
                load(pass);
                residual(pass, true);
            }
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int64_t col = (int64_t)pass * span + 8 * ((int64_t)c * NT + tid);
                if (col >= N)
                    continue;
                float w[8];
                if constexpr (EARLY) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        w[j] = ep[c][j];
                } else {
                    load_vec(p.w_pre, col, N, 1.0f, w);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    xv[c][j] = xv[c][j] * rx * w[j];
                store_row<TYPE, 8>(h + col, N - col, xv[c]);
            }
        }
    }
}

template <int TYPE>
static hipError_t norm_t(const NormParams &p, hipStream_t s)
{
    const int64_t most = 1 << 20;
    const int64_t groups = p.N <= 1024 ? ((int64_t)p.M + 3) / 4 : p.M;
    const dim3 grid((unsigned)(groups < most ? groups : most));
#define LL_NORM(MAX, C, LONG, EARLY, NT) \
    hipLaunchKernelGGL((rmsnorm_residual_kernel<TYPE, MAX, C, LONG, EARLY>), grid, dim3(NT), 0, s, p)
    // a thread to 8 columns, or 16 where there are rows to hide its latency; few
    // rows read everything at once (6061 x 4892 binary16 93 us, in a fixed 512 threads 102)
    const int one = cdiv(cdiv(p.N, 8), 64) * 64, two = cdiv(cdiv(p.N, 16), 64) * 64;
    if (p.N <= 512)
        LL_NORM(64, 1, false, true, 256);
    else if (p.N <= 1024)
        LL_NORM(64, 2, false, true, 256);
    else if (p.N <= 2048)
        LL_NORM(256, 1, false, true, one);
    else if (p.N <= 8192 && p.M <= 512)
        LL_NORM(1024, 1, false, true, one);
    else if (p.N <= 8192)
        LL_NORM(512, 2, false, false, two);
    else if (p.N <= 16384)
        LL_NORM(1024, 2, false, false, two);
    else
        LL_NORM(1024, 1, true, false, 1024);
#undef LL_NORM
    return hipGetLastError();
}

hipError_t launch_rmsnorm_residual(int type, const NormParams &p, hipStream_t s)
{
    if (type == LL_TYPE_F32)
        return norm_t<LL_TYPE_F32>(p, s);
    if (type == LL_TYPE_F16)
        return norm_t<LL_TYPE_F16>(p, s);
    return norm_t<LL_TYPE_BF16>(p, s);
}

// ---- gradient ---------------------------------------------------------------
//
// A workgroup walks rows blockIdx.x, blockIdx.x + grid, .. and keeps its
// columns' shares of S and of dw_pre's sum; it writes them once, as row
// blockIdx.x of `part` ([grid][2][N] floats), and a second launch adds the
// rows in order. No atomics: the result does not depend on the run.
//
// TEAMS: rows so short that one wave holds one are taken by TEAMS waves of a
// workgroup, a row each, and their shares added in wave order at the end
// (8192 x 512 bfloat16 39 -> 20 us).
template <int TYPE, int MAX, int C, int TEAMS>
__global__ void __launch_bounds__(MAX * TEAMS) rmsnorm_grad_kernel(NormGradParams p)
{
    using T = typename Elem<TYPE>::type;
    static_assert(TEAMS == 1 || (MAX == 64 && C == 1), "a team is a wave: its sums need no barrier");
    constexpr bool WAVE = MAX == 64;
    __shared__ Sums<4> lds;
    if constexpr (!WAVE)
        lds.clear();
    const int N = p.N, NT = WAVE ? 64 : (int)blockDim.x, tid = WAVE ? threadIdx.x & 63 : threadIdx.x;
    const int64_t stride = (int64_t)gridDim.x * TEAMS, first = (int64_t)blockIdx.x * TEAMS + (WAVE ? threadIdx.x >> 6 : 0);
    float sS[C][8], sP[C][8], t[C][8], wp[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int64_t col = 8 * ((int64_t)c * NT + tid);
        float g[8];
        load_vec(p.w_post, col, N, 1.0f, t[c]);
        load_vec(p.gate, col, N, 1.0f, g);
        load_vec(p.w_pre, col, N, 1.0f, wp[c]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            sS[c][j] = sP[c][j] = 0.0f;
            t[c][j] *= p.alpha * g[j];
        }
    }
    // The next row is on its way while this one is worked on, since the sums have
    // to wait for one another and the loads for nothing but memory (16-bit
    // 8191 x 4096 128 -> 108 us, 4.9 TB/s; a large copy reaches 5.1 to 5.5).
    constexpr int RAW = 8 / (16 / (int)sizeof(T));   // 16-byte pieces of 8 values
    u32x4 ry4[C][2], rx4[C][RAW], rd4[C][RAW], rk4[C][RAW];
    auto fetch = [&](int64_t m) __attribute__((always_inline)) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int64_t col = 8 * ((int64_t)c * NT + tid);
            raw_row<LL_TYPE_F32>(p.Y != nullptr ? p.Y + m * p.ldy + col : nullptr, N - col, N >= 8, ry4[c]);
            raw_row<TYPE>(static_cast<const T *>(p.X) + m * p.ldx + col, N - col, N >= 8, rx4[c]);
            raw_row<TYPE>(p.DXO != nullptr ? static_cast<const T *>(p.DXO) + m * p.lddxo + col : nullptr, N - col, N >= 8, rd4[c]);
            raw_row<TYPE>(p.DH != nullptr ? static_cast<const T *>(p.DH) + m * p.lddh + col : nullptr, N - col, N >= 8, rk4[c]);
        }
    };
    if (first < p.M)
        fetch(first);
    for (int64_t m = first; m < p.M; m += stride) {
        float yv[C][8], xv[C][8], dv[C][8], kv[C][8];
        float s[1] = {0.0f};
#pragma unroll
        for (int c = 0; c < C; ++c) {
            raw_values<LL_TYPE_F32>(ry4[c], N - 8 * ((int64_t)c * NT + tid), N >= 8, yv[c]);
            raw_values<TYPE>(rx4[c], N - 8 * ((int64_t)c * NT + tid), N >= 8, xv[c]);
            raw_values<TYPE>(rd4[c], N - 8 * ((int64_t)c * NT + tid), N >= 8, dv[c]);
            raw_values<TYPE>(rk4[c], N - 8 * ((int64_t)c * NT + tid), N >= 8, kv[c]);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                s[0] = __builtin_fmaf(yv[c][j], yv[c][j], s[0]);
        }
        if (m + stride < p.M)
            fetch(m + stride);
        block_sum<WAVE, 0>(s, lds);
        const float ry = inv_rms(s[0], N, p.eps_y);
        float q[2] = {0.0f, 0.0f};   // sums of x'^2 and of dh * w_pre * x'
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                yv[c][j] *= ry;   // u
                xv[c][j] = __builtin_fmaf(t[c][j], yv[c][j], xv[c][j]);
                q[0] = __builtin_fmaf(xv[c][j], xv[c][j], q[0]);
                q[1] = __builtin_fmaf(kv[c][j] * wp[c][j], xv[c][j], q[1]);
            }
        block_sum<WAVE, 1>(q, lds);
        const float rx = inv_rms(q[0], N, p.eps), mean_kn = q[1] * rx / (float)N;
        float z[1] = {0.0f};
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float n = xv[c][j] * rx;
                sP[c][j] = __builtin_fmaf(kv[c][j], n, sP[c][j]);
                dv[c][j] += rx * (kv[c][j] * wp[c][j] - n * mean_kn);   // T
                sS[c][j] = __builtin_fmaf(dv[c][j], yv[c][j], sS[c][j]);
                z[0] = __builtin_fmaf(dv[c][j] * t[c][j], yv[c][j], z[0]);
            }
        block_sum<WAVE, 3>(z, lds);
        const float mean_z = z[0] / (float)N;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int64_t col = 8 * ((int64_t)c * NT + tid);
            if (col >= N)
                continue;
            if (p.DX != nullptr)
                store_row<TYPE, 8>(static_cast<T *>(p.DX) + m * p.lddx + col, N - col, dv[c]);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                dv[c][j] = ry * (dv[c][j] * t[c][j] - yv[c][j] * mean_z);
            if (p.DY != nullptr)
                store_row<LL_TYPE_F32, 8>(p.DY + m * p.lddy + col, N - col, dv[c]);
        }
    }
    if constexpr (TEAMS > 1) {
        __shared__ float shares[TEAMS][2][8 * MAX + 8];
        float(*mine)[8 * MAX + 8] = shares[threadIdx.x / MAX];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            mine[0][j * MAX + tid] = sS[0][j], mine[1][j * MAX + tid] = sP[0][j];
        __syncthreads();
        if (threadIdx.x >= MAX)
            return;
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int w = 1; w < TEAMS; ++w)
                sS[0][j] += shares[w][0][j * MAX + tid], sP[0][j] += shares[w][1][j * MAX + tid];
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int64_t col = 8 * ((int64_t)c * NT + tid);
        if (col >= N)
            continue;
        float *row = p.part + (int64_t)blockIdx.x * 2 * N + col;
        store_row<LL_TYPE_F32, 8>(row, N - col, sS[c]);
        store_row<LL_TYPE_F32, 8>(row + N, N - col, sP[c]);
    }
}

// Rows too long for a workgroup's registers, in two launches. First each row's
// four numbers (r_y, r_x, mean(dh * w_pre * n), mean(T * t * u)), reading the
// row once for each sum.
struct RowStats {
    float ry, rx, mean_kn, mean_z;
};

// One group of 8 columns of a row, as the formulas name its values.
template <int TYPE>
struct GradCols {
    using T = typename Elem<TYPE>::type;
    float y[8], x[8], d[8], k[8], t[8], wp[8];
    __device__ __forceinline__ void vectors(const NormGradParams &p, int64_t col)
    {
        float g[8];
        load_vec(p.w_post, col, p.N, 1.0f, t);
        load_vec(p.gate, col, p.N, 1.0f, g);
        load_vec(p.w_pre, col, p.N, 1.0f, wp);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            t[j] *= p.alpha * g[j];
    }
    __device__ __forceinline__ void row(const NormGradParams &p, int64_t m, int64_t col)
    {
        const int64_t n = p.N - col;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            y[j] = d[j] = k[j] = 0.0f;
        if (p.Y != nullptr)
            load_row<LL_TYPE_F32, 8>(p.Y + m * p.ldy + col, n, y);
        load_row<TYPE, 8>(static_cast<const T *>(p.X) + m * p.ldx + col, n, x);
        if (p.DXO != nullptr)
            load_row<TYPE, 8>(static_cast<const T *>(p.DXO) + m * p.lddxo + col, n, d);
        if (p.DH != nullptr)
            load_row<TYPE, 8>(static_cast<const T *>(p.DH) + m * p.lddh + col, n, k);
    }
};

template <int TYPE, int NT>
__global__ void __launch_bounds__(NT) rmsnorm_grad_stats_kernel(NormGradParams p, RowStats *stats)
{
    __shared__ Sums<4> lds;
    lds.clear();
    const int64_t m = blockIdx.x;
    GradCols<TYPE> v;
    RowStats r;
    float s[1] = {0.0f}, q[2] = {0.0f, 0.0f}, z[1] = {0.0f};
    for (int64_t col = 8 * (int64_t)threadIdx.x; col < p.N; col += 8 * NT) {
        v.row(p, m, col);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            s[0] = __builtin_fmaf(v.y[j], v.y[j], s[0]);
    }
    block_sum<false, 0>(s, lds);
    r.ry = inv_rms(s[0], p.N, p.eps_y);
    for (int64_t col = 8 * (int64_t)threadIdx.x; col < p.N; col += 8 * NT) {
        v.row(p, m, col);
        v.vectors(p, col);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float x = __builtin_fmaf(v.t[j], v.y[j] * r.ry, v.x[j]);
            q[0] = __builtin_fmaf(x, x, q[0]);
            q[1] = __builtin_fmaf(v.k[j] * v.wp[j], x, q[1]);
        }
    }
    block_sum<false, 1>(q, lds);
    r.rx = inv_rms(q[0], p.N, p.eps);
    r.mean_kn = q[1] * r.rx / (float)p.N;
    for (int64_t col = 8 * (int64_t)threadIdx.x; col < p.N; col += 8 * NT) {
        v.row(p, m, col);
        v.vectors(p, col);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float u = v.y[j] * r.ry, n = __builtin_fmaf(v.t[j], u, v.x[j]) * r.rx;
            const float total = v.d[j] + r.rx * (v.k[j] * v.wp[j] - n * r.mean_kn);
            z[0] = __builtin_fmaf(total * v.t[j], u, z[0]);
        }
    }
    block_sum<false, 3>(z, lds);
    r.mean_z = z[0] / (float)p.N;
    if (threadIdx.x == 0)
        stats[m] = r;
}

// Then every column group on its own: 2048 columns and the rows
// blockIdx.y, blockIdx.y + grid y, .. to a workgroup.
template <int TYPE>
__global__ void __launch_bounds__(256) rmsnorm_grad_cols_kernel(NormGradParams p, const RowStats *stats)
{
    using T = typename Elem<TYPE>::type;
    const int64_t col = 8 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
    if (col >= p.N)
        return;
    GradCols<TYPE> v;
    v.vectors(p, col);
    float sS[8], sP[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        sS[j] = sP[j] = 0.0f;
    for (int64_t m = blockIdx.y; m < p.M; m += gridDim.y) {
        const RowStats r = stats[m];
        v.row(p, m, col);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float u = v.y[j] * r.ry, n = __builtin_fmaf(v.t[j], u, v.x[j]) * r.rx;
            sP[j] = __builtin_fmaf(v.k[j], n, sP[j]);
            v.d[j] += r.rx * (v.k[j] * v.wp[j] - n * r.mean_kn);
            sS[j] = __builtin_fmaf(v.d[j], u, sS[j]);
            v.y[j] = r.ry * (v.d[j] * v.t[j] - u * r.mean_z);
        }
        if (p.DX != nullptr)
            store_row<TYPE, 8>(static_cast<T *>(p.DX) + m * p.lddx + col, p.N - col, v.d);
        if (p.DY != nullptr)
            store_row<LL_TYPE_F32, 8>(p.DY + m * p.lddy + col, p.N - col, v.y);
    }
    float *row = p.part + (int64_t)blockIdx.y * 2 * p.N + col;
    store_row<LL_TYPE_F32, 8>(row, p.N - col, sS);
    store_row<LL_TYPE_F32, 8>(row + p.N, p.N - col, sP);
}

// The columns' sums over `rows` partial rows, then dgate, dw_post and dw_pre. A
// workgroup takes 16 columns; its threads, 4 quads of columns by 64, every 64th row,
// 8 of them in flight, and their sums are added in a fixed order (16 MB of 512
// partial rows of 4096: 8 us, with 32 columns to a workgroup 11). The launch's
// columns begin at `from`.
__global__ void __launch_bounds__(256) rmsnorm_grad_finish_kernel(NormGradParams p, int rows, int64_t from)
{
    __shared__ float sums[64][2][16 + 1];
    const int quad = threadIdx.x & 3, r0 = threadIdx.x >> 2;
    const int64_t col = from + (int64_t)blockIdx.x * 16 + 4 * quad, left = p.N - col;
    float a[4] = {0.0f, 0.0f, 0.0f, 0.0f}, b[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (left > 0) {
        for (int r = r0; r < rows; r += 512) {
            float u[8][4], v[8][4];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float *row = p.part + (int64_t)(r + 64 * i) * 2 * p.N + col;
                const int64_t n = r + 64 * i < rows ? left : 0;
                load_row<LL_TYPE_F32, 4>(row, n, u[i]);
                load_row<LL_TYPE_F32, 4>(row + p.N, n, v[i]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    a[j] += u[i][j], b[j] += v[i][j];
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
        sums[r0][0][4 * quad + j] = a[j], sums[r0][1][4 * quad + j] = b[j];
    __syncthreads();
    const int64_t c = from + (int64_t)blockIdx.x * 16 + (threadIdx.x & 15);
    const int which = threadIdx.x >> 4;
    if (which > 1 || c >= p.N)
        return;
    float t = 0.0f;
#pragma unroll
    for (int r = 0; r < 64; ++r)
        t += sums[r][which][threadIdx.x & 15];
    if (which == 0 && p.DGATE != nullptr)
        p.DGATE[c] = p.alpha * (p.w_post != nullptr ? p.w_post[c] : 1.0f) * t;
    if (which == 0 && p.DWPOST != nullptr)
        p.DWPOST[c] = p.alpha * (p.gate != nullptr ? p.gate[c] : 1.0f) * t;
    if (which == 1 && p.DWPRE != nullptr)
        p.DWPRE[c] = t;
}

// Rows that the registers of a workgroup hold, this one and the next (with 16384 in
// 1024 threads they spill: 4096 x 16384 bfloat16 502 us against 462 in two launches).
constexpr int kGradRegCols = 8192;
// Workgroups (rows of partial sums) of a gradient: two for each CU, four of short
// rows (8192 x 600 FP32 39 us, with two 52).
static int grad_groups(int M, int N)
{
    const int most = N <= 2048 ? 1024 : 512;
    return M < most ? M : most;
}
static int64_t grad_stats_bytes(int M, int N)
{
    return N > kGradRegCols ? ((int64_t)M * (int64_t)sizeof(RowStats) + 255) / 256 * 256 : 0;
}

int64_t rmsnorm_grad_workspace(int M, int N)
{
    return M <= 0 || N <= 0 ? 0 : grad_stats_bytes(M, N) + (int64_t)grad_groups(M, N) * 2 * N * 4;
}

template <int TYPE>
static hipError_t norm_grad_t(NormGradParams p, void *ws, hipStream_t s)
{
    p.part = reinterpret_cast<float *>(static_cast<char *>(ws) + grad_stats_bytes(p.M, p.N));
    const int groups = grad_groups(p.M, p.N);
    const dim3 grid((unsigned)groups);
#define LL_GRAD(MAX, C, TEAMS, NT) \
    hipLaunchKernelGGL((rmsnorm_grad_kernel<TYPE, MAX, C, TEAMS>), grid, dim3(NT), 0, s, p)
    // a thread to 8 columns up to 3584, to 16 past that (8192 rows of bfloat16: 2304 columns
    // 77 us against 85 with 16 a thread, 3328 96.5 and 97.3, 3840 110.4 and 108.9, 4096
    // 115.2 and 113.5; FP32 gains from 8 a little longer, 3840 154 and 163)
    const int one = cdiv(cdiv(p.N, 8), 64) * 64, two = cdiv(cdiv(p.N, 16), 64) * 64;
    if (p.M <= 0)
        ;   // no rows: the finishing launch writes zeros
    else if (p.N <= 512)
        LL_GRAD(64, 1, 4, 256);
    else if (p.N <= 2048)
        LL_GRAD(256, 1, 1, one);
    else if (p.N <= 3584)
        LL_GRAD(512, 1, 1, one);
    else if (p.N <= kGradRegCols)
        LL_GRAD(512, 2, 1, two);
    else {
        RowStats *stats = static_cast<RowStats *>(ws);
        const int slab = 1 << 20;   // rows of a launch: work items fit 32 bits
        for (int64_t m = 0; m < p.M; m += slab) {
            NormGradParams q = p;
            using T = typename Elem<TYPE>::type;
            q.Y = p.Y != nullptr ? p.Y + m * p.ldy : nullptr;
            q.X = static_cast<const T *>(p.X) + m * p.ldx;
            q.DXO = p.DXO != nullptr ? static_cast<const T *>(p.DXO) + m * p.lddxo : nullptr;
            q.DH = p.DH != nullptr ? static_cast<const T *>(p.DH) + m * p.lddh : nullptr;
            const int64_t rows = p.M - m < slab ? p.M - m : slab;
            hipLaunchKernelGGL((rmsnorm_grad_stats_kernel<TYPE, 1024>), dim3((unsigned)rows), dim3(1024), 0, s, q,
                               stats + m);
        }
        hipLaunchKernelGGL((rmsnorm_grad_cols_kernel<TYPE>),
                           dim3((unsigned)(((int64_t)p.N + 2047) / 2048), (unsigned)groups), dim3(256), 0, s, p,
                           stats);
    }
#undef LL_GRAD
    if (p.DGATE != nullptr || p.DWPOST != nullptr || p.DWPRE != nullptr) {
        constexpr int64_t cols = (int64_t)1 << 27;   // of a launch: work items fit 32 bits
        for (int64_t from = 0; from < p.N; from += cols) {
            const int64_t n = p.N - from < cols ? p.N - from : cols;
            hipLaunchKernelGGL(rmsnorm_grad_finish_kernel, dim3((unsigned)((n + 15) / 16)), dim3(256), 0, s, p, groups, from);
        }
    }
    return hipGetLastError();
}

hipError_t launch_rmsnorm_grad(int type, NormGradParams p, void *ws, hipStream_t s)
{
    p.eps_y = p.eps;
    // x' = x, or no rows: y is 0, so is t, and r_y a number, whatever eps, gate and w_post hold
    if (p.Y == nullptr || p.M <= 0) {
        p.w_post = p.gate = nullptr;
        p.alpha = 0.0f;
        p.eps_y = 1.0f;
    }
    if (type == LL_TYPE_F32)
        return norm_grad_t<LL_TYPE_F32>(p, ws, s);
    if (type == LL_TYPE_F16)
        return norm_grad_t<LL_TYPE_F16>(p, ws, s);
    return norm_grad_t<LL_TYPE_BF16>(p, ws, s);
}

}  // namespace ll
