// The 16-bit layer for few rows: a weight is read once for as many rows as a workgroup has, 16, 32 or
// 64 by the groups' average, so memory bounds the product and the matrix cores have time to spare. (A
// group of more rows than that has its weight read again for each such chunk, mostly from the
// caches: 1024 rows of 64 experts of 4096 x 2048 evenly 227 us, all of them in one expert 86.)
//
// A workgroup of NW waves computes MT x 16 rows by 64 columns, over all of the inner dimension
// or a share of it. Its waves share that out in turns of 64 values, a whole line of a row: wave
// w takes turns w, w + NW, ... and copies 64 rows of W and the rows of X straight into a ring of
// its own in LDS (DEPTH turns, 8 + 2 MT KiB each, in the tile kernel's order), so that no wave
// waits for another and all of a CU's LDS but the turn in use is on its way from memory. At the end
// the waves' sums meet in LDS and are added in the waves' order. Shares of K go through the
// workspace and are added in order by a second launch, where a product has fewer than half as
// many workgroups as the GPU has CUs.
//
// (Loads straight into the matrix instruction's registers, 64 bytes of 16 rows each, reach 3 TB/s
// where this reaches 5; they are what rows off 16 bytes take.)
#include "launch.hpp"
#include "linear16_finish.hpp"

namespace ll {

using namespace l16;

constexpr int kTurn = 64;     // values of the inner dimension a wave takes at a time
constexpr int kCols = 64;     // columns of a workgroup
constexpr int kPitch = kCols + 4;

// The waves' sums added, and the write-back or the share's sums. The sums are at part[wave][row][column].
template <bool BF16, int MT, int NW>
__device__ __forceinline__ void finish_rows(const L16Params &p, const float *part, const Chunk &c, int m0, int n0, int share)
{
    for (int s = threadIdx.x; s < MT * 16 * 8; s += 64 * NW) {
        const int rl = s / 8, cl = s % 8 * 8, row = m0 + rl, col = n0 + cl, n = p.N - col;
        const bool live = row < c.end && n > 0;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = 0.0f;
#pragma unroll
        for (int k = 0; k < NW; ++k) {
            const f32x4 lo = *reinterpret_cast<const f32x4 *>(&part[(k * MT * 16 + rl) * kPitch + cl]);
            const f32x4 hi = *reinterpret_cast<const f32x4 *>(&part[(k * MT * 16 + rl) * kPitch + cl + 4]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[e] += lo[e], v[4 + e] += hi[e];
        }
        if (p.shares > 1) {
            if (live)
                store_row<LL_TYPE_F32, 8>(p.ws + ((int64_t)share * p.M + row) * p.N + col, n, v);
            continue;
        }
        float bias[8], r[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            r[e] = 0.0f;
        load_row<LL_TYPE_F32, 8>(p.bias + (int64_t)c.group * p.N + col, p.bias != nullptr ? n : 0, bias);
        if (p.R != nullptr)
            load8<BF16>(p.ctype, p.R, (int64_t)row * p.ldr + col, live ? n : 0, r);
        finish_fwd<BF16>(p, v, bias, r, row, col, n, live);
    }
}

// The shares of K added in order, and the write-back: 16 rows by 64 columns a workgroup.
template <bool BF16>
__global__ void __launch_bounds__(128) l16_join_kernel(L16Params p, int tiles_n)
{
    Chunk c{};
    const int id = blockIdx.x / tiles_n;
    if (id >= find_chunk(p.groups, p.M, 16, id, c))
        return;
    const int row = c.begin + c.index * 16 + (int)threadIdx.x / 8;
    const int col = (int)(blockIdx.x % tiles_n) * kCols + (int)threadIdx.x % 8 * 8, n = p.N - col;
    const bool live = row < c.end && n > 0;
    float v[8], bias[8], r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        v[e] = r[e] = 0.0f;
    load_row<LL_TYPE_F32, 8>(p.bias + (int64_t)c.group * p.N + col, p.bias != nullptr ? n : 0, bias);
    if (p.R != nullptr)
        load8<BF16>(p.ctype, p.R, (int64_t)row * p.ldr + col, live ? n : 0, r);
#pragma unroll 4
    for (int s = 0; s < p.shares; ++s) {
        float u[8];
        load_row<LL_TYPE_F32, 8>(p.ws + ((int64_t)s * p.M + row) * p.N + col, live ? n : 0, u);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] += u[e];
    }
    finish_fwd<BF16>(p, v, bias, r, row, col, n, live);
}

template <bool BF16, int MT, int NW, int DEPTH>
__global__ void __launch_bounds__(64 * NW) l16_rows_kernel(L16Params p, int tiles_n)
{
    constexpr int PT = 8 + 2 * MT;            // copies of a turn, 1 KiB each: eight rows of 128 bytes
    constexpr int TURN = PT * 512;            // its values
    static_assert(NW * DEPTH * TURN * 2 <= 160 * 1024 && (DEPTH - 1) * PT <= 63, "the rings fit the LDS, the copies the counter");
    static_assert(NW * MT * 16 * kPitch * 4 <= NW * DEPTH * TURN * 2, "the waves' sums fit the rings");
    __shared__ __attribute__((aligned(1024))) uint16_t ring[NW][DEPTH][TURN];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int share = blockIdx.y;
    Chunk c{};
    const int id = blockIdx.x / tiles_n;
    if (id >= find_chunk(p.groups, p.M, MT * 16, id, c))
        return;
    const int m0 = c.begin + c.index * MT * 16, n0 = (int)(blockIdx.x % tiles_n) * kCols;

    // this share's turns, and this wave's among them: t0, t0 + NW, ...
    const int all = cdiv(p.K, kTurn), each = cdiv(all, p.shares);
    const int t_end = min(all, (share + 1) * each), t0 = share * each + wave;
    const int turns = cdiv(each, NW);   // the same in every wave; past the end zeros come
    const uint16_t *w = static_cast<const uint16_t *>(p.B) + c.group * p.stride_b + (int64_t)n0 * p.ldb;
    const uint16_t *x = p.A + (int64_t)m0 * p.lda;
    const int wrows = min(p.N - n0, kCols), xrows = min(c.end - m0, MT * 16);
    // copy j: rows 8 j + lane / 8; pieces of 16 bytes XORed by (row / 2) % 8, which for eight rows
    // is one of two orders
    const int r8 = lane >> 3;
    int piece[2];
    uint32_t woff[2], xoff[2];
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        piece[v] = ((lane & 7) ^ rows_swz(8 * v + r8)) * 8;
        woff[v] = (uint32_t)(8 * v + r8) * (uint32_t)(2 * p.ldb) + 2 * piece[v];
        xoff[v] = (uint32_t)(8 * v + r8) * (uint32_t)(2 * p.lda) + 2 * piece[v];
    }
    const uint32_t base = lds_addr(&ring[wave][0][0]);
    auto copy = [&](int slot, int i) __attribute__((always_inline)) {
        const int t = t0 + i * NW, left = t < t_end ? min(p.K - t * kTurn, kTurn) : 0;
        const int64_t k0 = (int64_t)t * kTurn;
        const uint64_t wat = (uint64_t)(w + k0), xat = (uint64_t)(x + k0);
        const u32x4 wbuf = {(uint32_t)wat, (uint32_t)(wat >> 32), left > 0 ? (uint32_t)(wrows - 1) * (uint32_t)(2 * p.ldb) + 2 * left : 0u, 0x00020000u};
        const u32x4 xbuf = {(uint32_t)xat, (uint32_t)(xat >> 32), left > 0 ? (uint32_t)(xrows - 1) * (uint32_t)(2 * p.lda) + 2 * left : 0u, 0x00020000u};
        uint32_t wo[2], xo[2];
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            wo[v] = piece[v] < left ? woff[v] : kPastEnd;
            xo[v] = piece[v] < left ? xoff[v] : kPastEnd;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            lds_buffer_16(wbuf, wo[j & 1] + (j >> 1) * 16 * (uint32_t)(2 * p.ldb), base + (slot * PT + j) * 1024);
#pragma unroll
        for (int j = 0; j < 2 * MT; ++j)
            lds_buffer_16(xbuf, xo[j & 1] + (j >> 1) * 16 * (uint32_t)(2 * p.lda), base + (slot * PT + 8 + j) * 1024);
    };
    f32x4 acc[MT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
        copy(d, d);
    const int r16 = lane & 15, grp = lane >> 4;
    int slot = 0;
#pragma unroll 1
    for (int i = 0; i < turns; ++i) {
        __builtin_amdgcn_s_waitcnt(LL_VMCNT((DEPTH - 1) * PT));   // this turn's copies have landed
        asm volatile("" ::: "memory");
        const uint16_t *at = &ring[wave][0][0] + slot * TURN;
        f16x8 fw[2][4], fx[2][MT];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                fw[s][j] = *reinterpret_cast<const f16x8 *>(at + (16 * j + r16) * 64 + ((4 * s + grp) ^ rows_swz(r16)) * 8);
#pragma unroll
            for (int m = 0; m < MT; ++m)
                fx[s][m] = *reinterpret_cast<const f16x8 *>(at + (64 + 16 * m + r16) * 64 + ((4 * s + grp) ^ rows_swz(r16)) * 8);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");        // read: the slot may be filled again
        copy(slot, i + DEPTH);
        slot = slot == DEPTH - 1 ? 0 : slot + 1;
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[m][j] = mma<BF16>(fw[s][j], fx[s][m], acc[m][j]);
    }
    __builtin_amdgcn_s_waitcnt(LL_VMCNT(0));   // (the zeros past the last turn are on their way into the rings)
    __syncthreads();
    float *part = reinterpret_cast<float *>(&ring[0][0][0]);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *reinterpret_cast<f32x4 *>(&part[(wave * MT * 16 + 16 * m + r16) * kPitch + 16 * j + 4 * grp]) = acc[m][j];
    __syncthreads();
    finish_rows<BF16, MT, NW>(p, part, c, m0, n0, share);
}

// Rows off 16 bytes: operands straight into the matrix instruction's registers, 16 bytes a load on
// any four; what crosses a row's end value by value. With rows off four bytes (ODD) the five
// words that hold the eight values are read (the halves outside are of words inside) and cut
// where they are used, not where they are loaded, so that the loads stay in flight. 16x11008x4096:
// 67 us by loads off four bytes, 32 so; on four bytes 32 so, 26 without the fifth word.
template <bool ODD>
struct Words {
    u32x4 v;
    uint32_t last;
};
template <>
struct Words<false> {
    u32x4 v;
};

template <bool ODD>
__device__ __forceinline__ Words<ODD> load8_at(const uint16_t *row, int64_t k, int K)
{
    const uint32_t off = ODD ? (uint32_t)(uintptr_t)row & 2u : 0u;
    Words<ODD> r;
    if (k + 8 <= K) {
        const char *at = reinterpret_cast<const char *>(row + k) - off;
        r.v = load16<u32x4>(at);
        if constexpr (ODD)
            r.last = *reinterpret_cast<const uint32_t *>(at + (off != 0 ? 16 : 12));
    } else {
        u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (k + e < K)
                v[e / 2] |= (uint32_t)row[k + e] << (16 * (e % 2));
        r.v = off == 0 ? v : u32x4{v[0] << 16, v[0] >> 16 | v[1] << 16, v[1] >> 16 | v[2] << 16, v[2] >> 16 | v[3] << 16};
        if constexpr (ODD)
            r.last = v[3] >> 16;
    }
    return r;
}

template <bool ODD>
__device__ __forceinline__ f16x8 cut8(const Words<ODD> &r, const uint16_t *row)
{
    if constexpr (ODD) {
        const uint32_t off = (uint32_t)(uintptr_t)row & 2u;
        return __builtin_bit_cast(f16x8, u32x4{__builtin_amdgcn_alignbyte(r.v[1], r.v[0], off), __builtin_amdgcn_alignbyte(r.v[2], r.v[1], off),
                                               __builtin_amdgcn_alignbyte(r.v[3], r.v[2], off), __builtin_amdgcn_alignbyte(r.last, r.v[3], off)});
    } else {
        return __builtin_bit_cast(f16x8, r.v);
    }
}

template <bool BF16, int MT, int NW, bool ODD>
__global__ void __launch_bounds__(64 * NW) l16_rows_any_kernel(L16Params p, int tiles_n)
{
    constexpr int DEPTH = 2;
    __shared__ float part[NW * MT * 16 * kPitch];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int share = blockIdx.y;
    Chunk c{};
    const int id = blockIdx.x / tiles_n;
    if (id >= find_chunk(p.groups, p.M, MT * 16, id, c))
        return;
    const int m0 = c.begin + c.index * MT * 16, n0 = (int)(blockIdx.x % tiles_n) * kCols;
    const int grp = lane >> 4, r16 = lane & 15;
    const int all = cdiv(p.K, kTurn), each = cdiv(all, p.shares);
    const int t_end = min(all, (share + 1) * each), t0 = share * each + wave, turns = cdiv(each, NW);
    const uint16_t *w = static_cast<const uint16_t *>(p.B) + c.group * p.stride_b;
    const uint16_t *wrow[4], *xrow[MT];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        wrow[j] = w + (int64_t)min(n0 + 16 * j + r16, p.N - 1) * p.ldb;
#pragma unroll
    for (int i = 0; i < MT; ++i)
        xrow[i] = p.A + (int64_t)min(m0 + 16 * i + r16, c.end - 1) * p.lda;
    f32x4 acc[MT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    Words<ODD> wv[DEPTH][2][4], xv[DEPTH][2][MT];
    auto fetch = [&](int i, Words<ODD> (&wd)[2][4], Words<ODD> (&xd)[2][MT]) __attribute__((always_inline)) {
        const int t = t0 + i * NW, end = t < t_end ? p.K : 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t k = (int64_t)t * kTurn + 32 * h + 8 * grp;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                wd[h][j] = load8_at<ODD>(wrow[j], k, end);
#pragma unroll
            for (int m = 0; m < MT; ++m)
                xd[h][m] = load8_at<ODD>(xrow[m], k, end);
        }
    };
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
        fetch(d, wv[d], xv[d]);
    for (int i = 0; i < turns; i += DEPTH) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {   // (past the last turn: zeros)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                f16x8 wc[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    wc[j] = cut8(wv[d][h][j], wrow[j]);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const f16x8 xc = cut8(xv[d][h][m], xrow[m]);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        acc[m][j] = mma<BF16>(wc[j], xc, acc[m][j]);
                }
            }
            fetch(i + d + DEPTH, wv[d], xv[d]);
        }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *reinterpret_cast<f32x4 *>(&part[(wave * MT * 16 + 16 * m + r16) * kPitch + 16 * j + 4 * grp]) = acc[m][j];
    __syncthreads();
    finish_rows<BF16, MT, NW>(p, part, c, m0, n0, share);
}

// ---- which of them, and in how many shares ------------------------------------------

// Tiles of 16 rows a workgroup has: those of a group of average length, up to four. 11008 x 4096 from
// memory in one, two and four tiles: 16 rows 21.7, 21.9, 23.5 us; 17 rows 31.8, 21.9, 23.4; 32 rows 32.5,
// 23.2, 24.4; 33 rows 39.4, 33.0, 24.6. 16 groups of 4096 x 2048: 16 rows each 66.4, 66.5, 68.5; 17 rows 71.3,
// 67.4, 69.4; 32 rows 75.2, 69.2, 70.7; 33 rows 91.9, 76.5, 71.5. (A small weight is read again from the caches:
// 4096 x 4096, 33 rows 16.6, 14.6, 16.8.)
static int row_tiles(int M, int groups)
{
    const int64_t each = ((int64_t)M + groups - 1) / groups;
    return each <= 16 ? 1 : each <= 32 ? 2 : 4;
}

// Up to 64 rows a group on average; in the tile kernel (with its shares) and here: 11008 x 4096, 64 rows 32.9
// and 27.8 us, 65 rows 33.2 and 36.0; 16 groups of 4096 x 2048, 64 rows each 74.8 and 75.8, 65 rows 75.0 and
// 89.1; 4096 x 4096, 64 rows 18.2 and 18.5, 65 rows 18.5 and 17.2.
bool l16_takes_rows(int M, int groups) { return groups > 0 && ((int64_t)M + groups - 1) / groups <= 64; }

static int64_t row_chunks(int M, int groups, int rows) { return (int64_t)M / rows + (groups < M ? groups : M); }

// Shares of K with a workspace: as many as fill the CUs once, with eight turns at least to a
// wave; none where the workgroups fill half of them by themselves.
int l16_row_shares(int M, int N, int K, int groups, int cus)
{
    if (M == 0 || N == 0 || !l16_takes_rows(M, groups))
        return 1;
    const int64_t work = (int64_t)cdiv(N, kCols) * (groups < M ? groups : M);
    const int64_t most = K / (8 * 4 * kTurn), fill = cus / work;
    const int64_t s = fill < most ? fill : most;
    return s < 2 ? 1 : s < 16 ? (int)s : 16;
}

hipError_t launch_l16_join(bool bf16, const L16Params &p, hipStream_t s)
{
    const int tiles_n = cdiv(p.N, kCols);
    const int64_t grid = (p.groups.offsets == nullptr ? cdiv(p.M, 16) : row_chunks(p.M, p.groups.n, 16)) * tiles_n;
    if (grid > max_grid_x(128))
        return hipErrorInvalidValue;
    if (bf16)
        hipLaunchKernelGGL(l16_join_kernel<true>, dim3((unsigned)grid), dim3(128), 0, s, p, tiles_n);
    else
        hipLaunchKernelGGL(l16_join_kernel<false>, dim3((unsigned)grid), dim3(128), 0, s, p, tiles_n);
    return hipGetLastError();
}

template <bool BF16, int MT, int NW>
static hipError_t launch_nw(const L16Params &p, bool vec, int64_t grid, hipStream_t s)
{
    const int tiles_n = cdiv(p.N, kCols);
    if (grid > max_grid_x(64 * NW))
        return hipErrorInvalidValue;
    const dim3 d((unsigned)grid, (unsigned)p.shares), b(64 * NW);
    constexpr int DEPTH = MT == 1 ? 4 : MT == 2 ? 3 : 2;
    if (vec)
        hipLaunchKernelGGL((l16_rows_kernel<BF16, MT, NW, DEPTH>), d, b, 0, s, p, tiles_n);
    else if ((reinterpret_cast<uintptr_t>(p.A) | reinterpret_cast<uintptr_t>(p.B) | 2 * (uintptr_t)(p.lda | p.ldb | p.stride_b)) & 2)
        hipLaunchKernelGGL((l16_rows_any_kernel<BF16, MT, NW, true>), d, b, 0, s, p, tiles_n);
    else
        hipLaunchKernelGGL((l16_rows_any_kernel<BF16, MT, NW, false>), d, b, 0, s, p, tiles_n);
    return p.shares > 1 ? launch_l16_join(BF16, p, s) : hipGetLastError();
}

// Four waves, one workgroup a CU, where the CUs are not filled; else two waves and two workgroups,
// one of which reads on while the other begins or ends.
template <bool BF16, int MT>
static hipError_t launch_mt(const L16Params &p, bool vec, int cus, hipStream_t s)
{
    const int64_t grid = (p.groups.offsets == nullptr ? cdiv(p.M, MT * 16) : row_chunks(p.M, p.groups.n, MT * 16)) * cdiv(p.N, kCols);
    return grid * p.shares <= cus ? launch_nw<BF16, MT, 4>(p, vec, grid, s) : launch_nw<BF16, MT, 2>(p, vec, grid, s);
}

hipError_t launch_l16_rows(bool bf16, const L16Params &p, bool vec, int cus, hipStream_t s)
{
    const int mt = row_tiles(p.M, p.groups.n);
    if (mt == 1)
        return bf16 ? launch_mt<true, 1>(p, vec, cus, s) : launch_mt<false, 1>(p, vec, cus, s);
    if (mt == 2)
        return bf16 ? launch_mt<true, 2>(p, vec, cus, s) : launch_mt<false, 2>(p, vec, cus, s);
    return bf16 ? launch_mt<true, 4>(p, vec, cus, s) : launch_mt<false, 4>(p, vec, cus, s);
}

}  // namespace ll
