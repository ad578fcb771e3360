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
// A lane then loads a whole block of B, 32 values in four dwords; turning the
// dwords around between the four groups of 16 lanes (turn4) gives each
// instruction one block, 8 values to a group, as A's rows are read in order.
//
// An E2M1 value times a power of two is exact in bfloat16 (its subnormals
// included, which the matrix units keep). In binary16 it is exact for scale
// bytes 104 .. 140 only (2^-23 .. 2^13); past those the wave splits A's values
// into two bfloat16 parts instead (11 bits of fraction into 8 and 3) and
// multiplies twice, which is exact too. The two largest scales pass bfloat16's
// range as well: see far_scale.
#include "linear_layer.h"
#include "gemm_mx4.hpp"

#include <algorithm>
#include <type_traits>

namespace ll {

// ---------------------------------------------------------------------------
// Streaming kernel: operands go from memory (or L2) straight into registers.
// A workgroup computes a (16 FM) x (16 FN) tile of C; its W waves take the K
// range in turns of 128 * J values, two of them in flight, and their sums are
// added through LDS in wave order, so a result never depends on the run. With
// a workspace K is first shared out over p.splits workgroups, whose sums the
// join kernel adds in order. This serves the products with few rows of A and
// those too small to give the tile kernels a workgroup per CU, at any
// alignment: rows are read in 16-byte pieces, the last one of a row from the
// row's last 16 bytes, shifted (LONG; a row of less than 32 values byte by byte).
// What bounds it is the rate at which a CU reads its rows of A and B from L2,
// 20 to 34 bytes a ns: hence tiles that are as high as M, wide enough not to read
// A too often, and as many workgroups as CUs (33 x 4096 x 11008 in binary16: 48 x 64
// tiles in four shares 15.2 us and 3.9 to join, 32 x 32 tiles in one 28).
//
// Rows past M or N read the last row instead; their sums are not stored. binary16
// A meets a scale past its range: the wave leaves the loop and does the rest of its
// share in bfloat16 parts.

template <int A, int FM, int FN, int J, int W, bool LONG>
__global__ void __launch_bounds__(64 * W) gemm_mx4_stream_kernel(MxParams p)
{
    constexpr bool MX = A == MXA_MX4;
    constexpr int BM = 16 * FM, BN = 16 * FN;
    __shared__ __attribute__((aligned(16))) float part[W][BM * BN];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, r16 = lane & 15;
    const int tiles = p.tiles_m * p.tiles_n, id = block_index(blockIdx.x, gridDim.x);
    const int split = id / tiles, tile = id - split * tiles;
    const int tm = tile % p.tiles_m, tn = tile / p.tiles_m;
    const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
    const int K = p.K;
    const int nblk = (K - 1) / kMxBlock + 1;
    const int all = (nblk + 4 * J - 1) / (4 * J);
    // this workgroup's units: all of them, or the split-th of p.splits shares
    const int begin = (int)((int64_t)all * split / p.splits), nunit = (int)((int64_t)all * (split + 1) / p.splits);

    const uint8_t *arow[FM], *sarow[FM], *brow[FN], *sbrow[FN];
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        int64_t m = m0 + 16 * i + r16;
        m = m < p.M ? m : p.M - 1;
        arow[i] = p.A + m * p.lda;
        sarow[i] = MX ? p.SA + m * p.ldsa : nullptr;
    }
#pragma unroll
    for (int i = 0; i < FN; ++i) {
        int64_t n = n0 + 16 * i + r16;
        n = n < p.N ? n : p.N - 1;
        brow[i] = p.B + n * p.ldb;
        sbrow[i] = p.SB + n * p.ldsb;
    }

    // J times four blocks. Lane group g has block g's codes of B, and of A in MX4;
    // of 16-bit A piece t is values 8 g .. +7 of block t, so that the four groups
    // read 64 bytes of a row at a time.
    struct Unit {
        u32x4 a[J][FM][MX ? 1 : 4], b[J][FN];
        uint32_t sa[J][MX ? FM : 1], sb[J][FN];
    };
    // The unit that K ends in.
    auto fetch_ragged = [&](Unit &u, int unit) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int first = (unit * J + j) * 4, blk = first + g;
#pragma unroll
            for (int i = 0; i < FN; ++i) {
                u.b[j][i] = load_block<LONG>(brow[i], blk, K);
                u.sb[j][i] = blk < nblk ? sbrow[i][blk] : 127u;
            }
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                if constexpr (MX) {
                    u.a[j][i][0] = load_block<LONG>(arow[i], blk, K);
                    u.sa[j][i] = blk < nblk ? sarow[i][blk] : 127u;
                } else {
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        u.a[j][i][t] = load_halves<LONG>(arow[i], (int64_t)(first + t) * kMxBlock + 8 * g, K);
                }
            }
        }
    };
    // A whole one, without a branch between its loads.
    auto fetch = [&](Unit &u, int unit) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int first = (unit * J + j) * 4;
#pragma unroll
            for (int i = 0; i < FN; ++i) {
                u.b[j][i] = load16<u32x4>(brow[i] + (int64_t)first * 16 + g * 16);
                u.sb[j][i] = sbrow[i][first + g];
            }
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                if constexpr (MX) {
                    u.a[j][i][0] = load16<u32x4>(arow[i] + (int64_t)first * 16 + g * 16);
                    u.sa[j][i] = sarow[i][first + g];
                } else {
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        u.a[j][i][t] = load16<u32x4>(arow[i] + (int64_t)(first + t) * 64 + 16 * g);
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

    // (WIDE: binary16 A against scales it cannot take, A's values in two parts)
    auto multiply = [&](const Unit &u, int j, auto w) __attribute__((always_inline)) {
        constexpr bool WIDE = decltype(w)::value;
        if constexpr (MX) {
#pragma unroll
            for (int n = 0; n < FN; ++n)
#pragma unroll
                for (int m = 0; m < FM; ++m)
                    acc[m][n] = mma_mx4<0, 0>(u.a[j][m][0], u.b[j][n], acc[m][n], (int)u.sa[j][m], (int)u.sb[j][n]);
        } else {
#pragma unroll
            for (int n = 0; n < FN; ++n) {
                u32x4 q = u.b[j][n], sc = {u.sb[j][n] << 23, u.sb[j][n] << 23, u.sb[j][n] << 23, u.sb[j][n] << 23};
                turn4(q);    // piece t: values 8 g .. +7 of block t
                turn4(sc);   // and its scale
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const u32x4 b = decode8<A == MXA_BF16 || WIDE>(q[t], __uint_as_float(sc[t]));
#pragma unroll
                    for (int m = 0; m < FM; ++m) {
                        if constexpr (WIDE) {
                            u32x4 hi, lo;
                            split8(u.a[j][m][t], hi, lo);
                            acc[m][n] = mma_bf16(lo, b, acc[m][n]);
                            acc[m][n] = mma_bf16(hi, b, acc[m][n]);
                        } else {
                            acc[m][n] = A == MXA_BF16 ? mma_bf16(u.a[j][m][t], b, acc[m][n])
                                                      : mma_f16(u.a[j][m][t], b, acc[m][n]);
                        }
                    }
                }
            }
        }
    };
    // The products of a unit; false, and none made, where a scale is past binary16.
    auto products = [&](const Unit &u) __attribute__((always_inline)) {
        if constexpr (A == MXA_F16) {
            bool wide = false;
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int n = 0; n < FN; ++n)
                    wide |= !f16_scale_ok(u.sb[j][n]);
            if (__any(wide))
                return false;
        }
#pragma unroll
        for (int j = 0; j < J; ++j)
            multiply(u, j, std::false_type{});
        return true;
    };

    // whole units, two in flight
    const int whole = min(K / (128 * J), nunit);
    Unit u0, u1;
    int unit = begin + wave, left = nunit;   // units from `left` on are still to do
    if (unit < whole)
        fetch(u0, unit);
    while (unit < whole) {
        const int second = unit + W;
        if (second < whole)
            fetch(u1, second);
        if (!products(u0)) {
            left = unit;
            break;
        }
        unit = second + W;
        if (unit < whole)
            fetch(u0, unit);
        if (second < whole && !products(u1)) {
            left = second;
            break;
        }
    }
    // the one that K ends in, and for binary16 A what its wave left
    if (left == nunit && whole < nunit && (whole - begin) % W == wave)
        left = whole;
    for (; left < nunit; left += W) {
        fetch_ragged(u0, left);
#pragma unroll
        for (int j = 0; j < J; ++j)
            multiply(u0, j, std::bool_constant<A == MXA_F16>{});
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
    constexpr int QUADS = BN / 4;
    if constexpr (!MX && W == 1)   // a lone wave looks at all its sums at once (5000 x 5000 x 128 in bfloat16 32.4 us, in the loop 33.6)
        if (__builtin_expect(__any(!all_finite(acc)), 0))
#pragma unroll 1
            for (int i = tid; i < BM * QUADS; i += 64) {
                const int64_t m = m0 + i / QUADS, n = n0 + i % QUADS * 4;
                float *at = &part[0][4 * i];
                if (m < p.M)
                    settle4<A, LONG>(p, *reinterpret_cast<f32x4 *>(at), at, m, n, begin * 4 * J, min(nunit * 4 * J, nblk));
            }
    for (int i = tid; i < BM * QUADS; i += 64 * W) {
        const int64_t m = m0 + i / QUADS, n = n0 + i % QUADS * 4;
        if (m >= p.M || n >= p.N)
            continue;
        f32x4 v = *reinterpret_cast<const f32x4 *>(&part[0][4 * i]);
#pragma unroll
        for (int w = 1; w < W; ++w) {
            const f32x4 u = *reinterpret_cast<const f32x4 *>(&part[w][4 * i]);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[j] += u[j];
        }
        if constexpr (!MX && W > 1)
            if (__builtin_expect(!finite4(v), 0))
                v = settle4<A, LONG>(p, v, &part[0][4 * i], m, n, begin * 4 * J, min(nunit * 4 * J, nblk));
        if (p.splits > 1) {
            float *dst = p.ws + ((int64_t)split * p.M + m) * p.N + n;
            if (n + 4 <= p.N) {
                __builtin_memcpy(dst, &v, 16);
            } else {
#pragma unroll
                for (int j = 0; j < 3; ++j)
                    if (n + j < p.N)
                        dst[j] = v[j];
            }
        } else {
            finish4(p, v, p.C + m * p.ldc + n, 0, p.N - n);
        }
    }
}

// C from the shares' sums, added in their order: four columns to a thread.
__global__ void __launch_bounds__(256) gemm_mx4_join_kernel(MxParams p, int quads, int64_t items)
{
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < items; i += (int64_t)gridDim.x * 256) {
        const int64_t m = i / quads, n = (i - m * quads) * 4;
        const float *src = p.ws + m * p.N + n;
        f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
        for (int s = 0; s < p.splits; ++s) {
            float v[4];
            load_row<LL_TYPE_F32, 4>(src + (int64_t)s * p.M * p.N, p.N - n, v);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                sum[j] += v[j];
        }
        finish4(p, sum, p.C + m * p.ldc + n, 0, p.N - n);
    }
}

// The part of a product from row m and column n on, `rows` x `cols` of it.
static MxParams part_of(MxParams p, int64_t m, int64_t n, int64_t rows, int64_t cols)
{
    p.A += m * p.lda;
    p.SA = p.SA != nullptr ? p.SA + m * p.ldsa : nullptr;
    p.B += n * p.ldb;
    p.SB += n * p.ldsb;
    p.C += m * p.ldc + n;
    p.M = (int)rows;
    p.N = (int)cols;
    return p;
}

template <int A, int FM, int FN, int J, int W, bool LONG = true>
static hipError_t launch_stream(const MxParams &whole, hipStream_t s)
{
    // launches of as many tiles as their work items can be counted (a product with
    // shares of K, whose workspace is laid out for all of it, has far fewer)
    constexpr int64_t most = max_grid_x(64 * W), BM = 16 * FM, BN = 16 * FN;
    const int64_t rows = std::min<int64_t>(whole.M, most * BM);
    const int64_t cols = std::min<int64_t>(whole.N, most / ((rows + BM - 1) / BM) * BN);
    for (int64_t m = 0; m < whole.M; m += rows)
        for (int64_t n = 0; n < whole.N; n += cols) {
            MxParams p = part_of(whole, m, n, std::min(rows, whole.M - m), std::min(cols, whole.N - n));
            p.tiles_m = cdiv(p.M, BM);
            p.tiles_n = cdiv(p.N, BN);
            hipLaunchKernelGGL((gemm_mx4_stream_kernel<A, FM, FN, J, W, LONG>),
                               dim3((unsigned)(p.tiles_m * p.tiles_n * p.splits)), dim3(64 * W), 0, s, p);
        }
    if (whole.splits > 1) {
        const int quads = cdiv(whole.N, 4);
        const int64_t items = (int64_t)whole.M * quads, groups = (items + 255) / 256;
        hipLaunchKernelGGL(gemm_mx4_join_kernel, dim3((unsigned)(groups < 1 << 20 ? groups : 1 << 20)), dim3(256), 0, s, whole,
                           quads, items);
    }
    return hipGetLastError();
}

// LDS of the row kernel: bytes of a plane of A (a piece of 8 values of every block
// of a row, whole turns of 64 blocks; 64 bytes past a multiple of 256, so that the
// pieces of a block lie on different banks), and in all.
__host__ __device__ constexpr int rows_plane(int nblk) { return (nblk + 63) / 64 * 1024 + 64; }
constexpr int rows_planes(int a) { return a == MXA_MX4 ? 1 : a == MXA_F16 ? 8 : 4; }
constexpr int64_t rows_lds(int a, int64_t K)
{
    const int64_t nblk = (K + kMxBlock - 1) / kMxBlock;
    return rows_planes(a) * ((nblk + 63) / 64 * 1024 + 64) + (a == MXA_MX4 ? (nblk + 63) / 64 * 64 : 0);
}

// ---------------------------------------------------------------------------
// Row kernel, for a decode step's one row of A: HBM bounds it, and
// memory serves whole rows better than the streaming kernel's 64 bytes of 16. With
// weights that cycle through more than the cache: B 28672 x 8192 24.7 us under a 4-bit
// row, 5.1 TB/s (streaming 32.4), 25.4 under a bfloat16 one (41.0), 29.7 under binary16,
// in two parts; B 11008 x 4096, 24 MB, 6.5, 7.3 and 8.3 (streaming 9.2 and 10.9 for the
// first two), and from the cache 3.8, 5.1 and 6.0. A wave takes R rows of B, 64 blocks of
// one at a time: lane l block l, a load of 1 KiB. The matrix instruction then has for
// its 16 rows of B 16 sets of four blocks of the same row, and for its 16 rows of A
// the same sets of A's: the sum of its result's diagonal is their inner
// product. What it computes beside the diagonal is not used; it still takes 16
// cycles (64 with 16-bit A, 128 with binary16) for a KiB of codes, more than four
// times HBM's rate.
// A lies in LDS as the instruction takes it: codes, or [piece of 8 values][block], so
// that neighbouring lanes read neighbouring 16 bytes. binary16 is split into two
// bfloat16 parts there (see split8), exact whatever the scales.
// KW waves of a workgroup share rows, and NW such groups take rows of their own.
// (With two rows of A it was no faster than the streaming kernel, with four slower.)
template <int A, int R, int KW, int NW>
__global__ void __launch_bounds__(64 * KW * NW) gemm_mx4_rows_kernel(MxParams p)
{
    constexpr bool MX = A == MXA_MX4;
    constexpr int NT = 64 * KW * NW, PL = rows_planes(A);
    extern __shared__ __attribute__((aligned(16))) uint8_t as[];
    __shared__ float sums[KW > 1 ? KW * NW : 1][R];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int K = p.K, nblk = (K - 1) / kMxBlock + 1, padded = (nblk + 63) & ~63;
    const int plane = rows_plane(nblk);
    uint8_t *const scales = as + PL * plane;   // MX: `padded` bytes
    const int64_t n0 = ((int64_t)block_index(blockIdx.x, gridDim.x) * NW + wave / KW) * R;

    const uint8_t *brow[R], *sbrow[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int64_t n = n0 + i < p.N ? n0 + i : p.N - 1;
        brow[i] = p.B + n * p.ldb;
        sbrow[i] = p.SB + n * p.ldsb;
    }
    // blocks past the row: codes 0 under scale 1
    struct Unit {
        u32x4 q[R];
        uint32_t s[R];
    };
    auto fetch = [&](Unit &u, int blk) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            u.q[i] = u32x4{0u, 0u, 0u, 0u};
            u.s[i] = 127u;
        }
        if (blk < K / kMxBlock) {
#pragma unroll
            for (int i = 0; i < R; ++i)
                u.q[i] = load16<u32x4>(brow[i] + (int64_t)blk * 16);
        } else if (blk < nblk) {
#pragma unroll
            for (int i = 0; i < R; ++i)
                u.q[i] = load_block<true>(brow[i], blk, K);
        }
        if (blk < nblk) {
#pragma unroll
            for (int i = 0; i < R; ++i)
                u.s[i] = sbrow[i][blk];
        }
    };
    constexpr int STEP = 64 * KW;   // blocks of a turn
    const int first = wave % KW * 64;
    Unit u0, u1;
    fetch(u0, first + lane);
    fetch(u1, first + STEP + lane);

    // A into LDS; 0 past its row
    if constexpr (MX) {
        for (int b = tid; b < padded; b += NT) {
            *reinterpret_cast<u32x4 *>(as + b * 16) = load_block<true>(p.A, b, K);
            scales[b] = b < nblk ? p.SA[b] : (uint8_t)127;
        }
    } else {
        for (int c = tid; c < 4 * padded; c += NT) {
            const u32x4 v = load_halves<true>(p.A, (int64_t)c * 8, K);
            uint8_t *at = as + (c & 3) * plane + (c >> 2) * 16;
            if constexpr (A == MXA_F16) {
                u32x4 hi, lo;
                split8(v, hi, lo);
                *reinterpret_cast<u32x4 *>(at) = hi;
                *reinterpret_cast<u32x4 *>(at + 4 * plane) = lo;
            } else {
                *reinterpret_cast<u32x4 *>(at) = v;
            }
        }
    }
    __syncthreads();

    f32x4 acc[R];
#pragma unroll
    for (int i = 0; i < R; ++i)
        acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    auto multiply = [&](const Unit &u, int blk) __attribute__((always_inline)) {
        if constexpr (MX) {
            const u32x4 a = *reinterpret_cast<const u32x4 *>(as + blk * 16);
            const int sa = scales[blk];
#pragma unroll
            for (int i = 0; i < R; ++i)
                acc[i] = mma_mx4<0, 0>(a, u.q[i], acc[i], sa, (int)u.s[i]);
        } else {
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                u32x4 a[PL / 4];
#pragma unroll
                for (int h = 0; h < PL / 4; ++h)
                    a[h] = *reinterpret_cast<const u32x4 *>(as + (4 * h + t) * plane + blk * 16);
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const u32x4 b = decode8<true>(u.q[i][t], __uint_as_float(u.s[i] << 23));
#pragma unroll
                    for (int h = PL / 4 - 1; h >= 0; --h)
                        acc[i] = mma_bf16(a[h], b, acc[i]);
                }
            }
        }
    };
    for (int base = first; base < nblk;) {
        multiply(u0, base + lane);
        if (base + 2 * STEP < nblk)
            fetch(u0, base + 2 * STEP + lane);
        base += STEP;
        if (base >= nblk)
            break;
        multiply(u1, base + lane);
        if (base + 2 * STEP < nblk)
            fetch(u1, base + 2 * STEP + lane);
        base += STEP;
    }

    // the diagonal: lane l has column l % 16 and rows 4 * (l / 16) .. +3
    const int r16 = lane & 15;
    const bool mine = (r16 >> 2) == lane >> 4;
    float sum = 0.0f;   // lane i: of row i
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const f32x4 d = acc[i];
        const float e = (r16 & 2) ? ((r16 & 1) ? d[3] : d[2]) : ((r16 & 1) ? d[1] : d[0]);
        float v = dpp_row_sum16(mine ? e : 0.0f);
        v += __shfl_xor(v, 16);
        v += __shfl_xor(v, 32);
        sum = lane == i ? v : sum;
    }
    if constexpr (KW > 1) {
        if (lane < R)
            sums[wave][lane] = sum;
        __syncthreads();
        if (wave % KW != 0)
            return;
    }
    const int64_t n = n0 + lane;
    if (lane < R && n < p.N) {
#pragma unroll
        for (int k = 1; k < KW; ++k)
            sum += sums[wave + k][lane];
        if constexpr (!MX)
            if (__builtin_expect(!finite(sum), 0))
                sum = far_dot<A, true>(sum, p.A, p.B + n * p.ldb, p.SB + n * p.ldsb, 0, nblk, K);
        p.C[n] = finish(p, sum, p.C + n);
    }
}

template <int A, int R, int KW, int NW>
static hipError_t launch_rows(const MxParams &whole, hipStream_t s)
{
    constexpr int64_t cols = max_grid_x(64 * KW * NW) * R * NW;   // of a launch
    for (int64_t n = 0; n < whole.N; n += cols) {
        const MxParams p = part_of(whole, 0, n, 1, std::min(cols, whole.N - n));
        hipLaunchKernelGGL((gemm_mx4_rows_kernel<A, R, KW, NW>), dim3((unsigned)cdiv(p.N, R * NW)), dim3(64 * KW * NW),
                           (unsigned)rows_lds(A, p.K), s, p);
    }
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// The plan of a product: which kernel, and for the streaming kernel in how many
// shares of K (one without a workspace).

enum Kernel : int { ROWS, ROWS_SHARED, TINY, SHORT, TILE_256, TILE_128, STREAM };   // from STREAM on: kStream's
struct Stream {
    int fm, fn;
    bool mx, h16;   // built for A in MX4, in 16 bits
};
constexpr Stream kStream[] = {{1, 1, true, true}, {2, 2, true, true}, {4, 4, true, false}, {1, 4, false, true},
                              {2, 4, false, true}, {3, 4, false, true}};
constexpr int kStreams = sizeof kStream / sizeof kStream[0];

struct Plan {
    int kernel, splits;
};

// Estimated times in us, from measurements on MI355X. The streaming kernel's
// follows the bytes that a CU's workgroups read (16-bit A: 64 x 4096 x 4096 270 KB in
// 14.4 us, 256 x 4096 x 4096 802 in 35.5, 128 x 11008 x 4096 1203 in 53; 4-bit A, in
// shorter loads: 48 x 11008 x 4096 278 KB in 17.3), or the turns of its eight waves
// (8 x 1000 x 8000 in 4 bits 12.2, in shares 9.8), the tiles' the stages of a round: 128 x 128 alone on a CU
// 15.7 us at K 4096 in 4 bits and 43 with 16-bit A, two to a CU 28.9 and 65; 256 x 256
// 47 and 114, in halves 20.3 and 49.
static Plan plan(int64_t M, int64_t N, int64_t K, int a, bool copies, bool workspace, int cus)
{
    if (K < 32)
        return {TINY, 1};
    // one row of A (its LDS copy within 60 KiB): two waves to a row of B where the
    // rows are long and few (4096 x 11008 6.9 against 7.4 us, 512 x 11008 4.4 against 5.7)
    if (M == 1 && K >= 512 && rows_lds(a, K) <= 61440)
        return {K > 2 * N ? ROWS_SHARED : ROWS, 1};
    const bool mx = a == MXA_MX4;
    auto tiles = [&](int64_t bm, int64_t bn) { return (double)((M + bm - 1) / bm) * (double)((N + bn - 1) / bn); };
    auto rounds = [](double n, double slots) { return (double)(int64_t)((n + slots - 1) / slots); };
    // K of one or two turns: one wave to a tile, since the others of a workgroup would
    // find nothing to do (5366 x 10986 x 128 in 4 bits 88 against 188 us, 1000 x 11008
    // x 32 20 against 59)
    if (K <= 256 && tiles(mx ? 64 : 32, 64) >= 2 * cus)
        return {SHORT, 1};
    Plan best = {STREAM, 1};
    double least = 1e30;
    auto offer = [&](double us, int kernel, int splits) {
        if (us < least) {
            least = us;
            best = {kernel, splits};
        }
    };
    const double arow = (double)(mx ? K / 2 + K / 32 : 2 * K), brow = (double)(K / 2 + K / 32);
    for (int i = 0; i < kStreams; ++i) {
        const Stream &c = kStream[i];
        if (!(mx ? c.mx : c.h16))
            continue;
        const double n = tiles(16 * c.fm, 16 * c.fn);
        const double bytes = (16 * c.fm < M ? 16 * c.fm : M) * arow + (16 * c.fn < N ? 16 * c.fn : N) * brow;
        for (int s = 1; s <= (workspace ? 16 : 1); ++s) {
            // a share has at least 8 blocks of four for its eight waves; the sums are
            // written and read again, and added by a second launch
            if (s > 1 && (K < 1024 * (int64_t)s || (double)M * (double)N * 4 * s > 6.4e7))
                break;
            // (two workgroups of a CU wait for their turns together)
            const double fill = rounds(n * s, cus) * bytes / s / (mx ? 20e3 : 26e3);
            const double wait = 1.15 * K / 1024 / s * (n * s > 2 * cus ? n * s / (2 * cus) : 1.0);
            offer(3.0 + (fill > wait ? fill : wait) + (s > 1 ? 4.5 + (double)M * (double)N * 8 * s / 3e6 : 0.0),
                  STREAM + i, s);
        }
    }
    if (M >= 128 && N >= 128 && K >= 512) {
        const double t = tiles(128, 128), k = (double)K / 4096, full = (double)(int64_t)(t / (2 * cus)), last = t - full * 2 * cus;
        offer(3.0 + k * (full * (mx ? 26.0 : 62.0) + (last > cus ? (mx ? 26.0 : 62.0) : last > 0 ? (mx ? 13.0 : 40.0) : 0.0)), TILE_128, 1);
    }
    if (copies && M >= 256 && N >= 256 && K >= 512) {
        const double t = tiles(256, 256), k = (double)K / 4096, full = (double)(int64_t)(t / cus), last = t - full * cus;
        offer(4.0 + k * (full * (mx ? 43.0 : 108.0) + (last > cus / 2 ? (mx ? 43.0 : 108.0) : last > 0 ? (mx ? 17.0 : 46.0) : 0.0)), TILE_256, 1);
    }
    return best;
}

int64_t mx4_workspace(int M, int N, int K, int a, int cus)
{
    if (M <= 0 || N <= 0 || K <= 0)
        return 0;
    int splits = 1;
    for (int copies = 0; copies < 2; ++copies) {
        const int n = plan(M, N, K, a, copies != 0, true, cus).splits;
        splits = n > splits ? n : splits;
    }
    return splits > 1 ? (int64_t)splits * M * N * 4 : 0;
}

const char *mx4_kernel_name(int M, int N, int K, int a, bool copies, bool workspace, int cus)
{
    static const char *const names[] = {"rows", "rows_shared", "tiny", "short", "tile_256x256", "tile_128x128",
                                        "stream_16x16", "stream_32x32", "stream_64x64", "stream_16x64", "stream_32x64", "stream_48x64"};
    static_assert(sizeof names / sizeof names[0] == STREAM + kStreams, "a name for each");
    return M <= 0 || N <= 0 || K <= 0 ? "" : names[plan(M, N, K, a, copies, workspace, cus).kernel];
}

template <int A>
static hipError_t launch_a(MxParams p, int cus, hipStream_t s)
{
    // copies take rows of whole 16-byte pieces and 32-bit offsets within a tile
    const bool copies = ((uintptr_t)p.A | (uintptr_t)p.B | (uintptr_t)p.lda | (uintptr_t)p.ldb) % 16 == 0 &&
                        p.lda < 1 << 24 && p.ldb < 1 << 24 && p.ldsa < 1 << 24 && p.ldsb < 1 << 24;
    const Plan q = plan(p.M, p.N, p.K, A, copies, p.ws != nullptr, cus);
    p.splits = q.splits;
    constexpr bool MX = A == MXA_MX4;
    switch (q.kernel) {
    case ROWS: return launch_rows<A, 2, 1, 8>(p, s);
    case ROWS_SHARED: return launch_rows<A, 2, 2, 4>(p, s);
    case TINY: return launch_stream<A, 1, 1, 1, 4, false>(p, s);
    case SHORT: return launch_stream<A, MX ? 4 : 2, 4, 1, 1>(p, s);
    case TILE_256: return launch_gemm_mx4_tile(p, A, MX_TILE_256, copies, cus, s);
    case TILE_128: return launch_gemm_mx4_tile(p, A, MX_TILE_128, copies, cus, s);
    case STREAM: return launch_stream<A, 1, 1, MX ? 2 : 1, 8>(p, s);
    case STREAM + 1: return launch_stream<A, 2, 2, 1, 8>(p, s);
    }
    if constexpr (MX) {
        return launch_stream<A, 4, 4, 1, 8>(p, s);
    } else {
        switch (q.kernel) {
        case STREAM + 3: return launch_stream<A, 1, 4, 1, 8>(p, s);
        case STREAM + 4: return launch_stream<A, 2, 4, 1, 8>(p, s);
        default: return launch_stream<A, 3, 4, 1, 8>(p, s);
        }
    }
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
