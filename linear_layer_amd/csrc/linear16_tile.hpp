// The tile kernel of the 16-bit layer and its gradients: forward, input gradient and
// weight gradient, dense or by groups of rows.
//
// A workgroup computes BM x BM of C on v_mfma_f32_16x16x32 with FP32 sums, over stages of
// 64 of the contracted axis in a ring of two LDS buffers. An operand lies in memory in one
// of two ways:
//   ROWS   the contracted axis is contiguous (X and W of the forward product, dZ of the
//          input gradient): BM rows of 128 bytes a stage, their 16-byte chunks XORed by
//          (row / 2) % 8, read with 128-bit LDS reads;
//   COLS   the other axis is (W of the input gradient, dZ and X of the weight gradient): 64
//          rows of 2 * BM bytes a stage, 32-byte units XORed by 2 * (k % 4) + (k / 8) % 2,
//          read with ds_read_b64_tr_b16, which hands each lane four values of one column;
//   COLS8  as COLS, from E4M3 codes and scales: 16 codes a load into registers, decoded and
//          stored as the 32-byte unit that they are in 16 bits. Decoding on the way into LDS
//          is done once a workgroup; after it, by every wave that reads the stage.
// ROWS and COLS on 16 bytes are copied straight into LDS (16 bytes a lane, lanes outside the
// matrix from a chunk of zeros, so that a wave has a known number of copies in flight). Rows
// off 16 bytes go through registers (DMA false), 16 bytes a load at any alignment, the chunk
// that crosses the row's end value by value.
//
// The MFMA takes the operand of C's columns first, so a lane gets four neighbouring columns
// of a row; the write-back turns them around in LDS to eight a lane, 128 bytes of a row (16
// bits) in one store instruction, which is also the order that R and bias are read in and
// in which four lanes hold one block of 32 of Z's 8 bits.
#pragma once

#include "launch.hpp"
#include "linear16.hpp"

namespace ll {
namespace l16 {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

enum Side : int { ROWS = 0, COLS = 1, COLS8 = 2 };

template <bool BF16>
__device__ __forceinline__ f32x4 mma(const f16x8 &a, const f16x8 &b, const f32x4 &c)
{
    if constexpr (BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                       0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

template <bool BF16> constexpr int kType16 = BF16 ? LL_TYPE_BF16 : LL_TYPE_F16;

// Waves, and the block of C that each has: 256 x 256 as 2 x 4 waves of 128 x 64 (two a
// SIMD), 128 x 128 as 2 x 2 of 64 x 64 (two workgroups a CU).
template <int BM> struct Cfg {
    static constexpr int WGM = 2, WGN = BM == 256 ? 4 : 2, NW = WGM * WGN, NT = 64 * NW;
    static constexpr int BK = 64, STEPS = 2;
    static constexpr int WTM = BM / WGM, WTN = BM / WGN, FM = WTM / 16, FN = WTN / 16;
    static constexpr int STAGE = BM * BK;                   // values of an operand's stage
    static constexpr int COPIES = STAGE * 2 / 1024 / NW;    // KiB copies a wave, operand and stage
};

// 16-byte chunk c of row `row` of a ROWS stage, and unit u of k-row k of a COLS stage.
__device__ __forceinline__ int rows_swz(int row) { return (row >> 1) & 7; }
__device__ __forceinline__ int cols_swz(int k) { return 2 * (k & 3) + ((k >> 3) & 1); }

// One operand's source: `lim` rows or columns of it from `o0` on belong to the tile (more
// may be asked for), `klen` of the contracted axis.
template <bool BF16, int BM, int SIDE, bool DMA>
struct Operand {
    using C = Cfg<BM>;
    // registers of a stage on its way: 16-byte chunks a thread
    static constexpr int REGS = SIDE == COLS8 ? BM * C::BK / 16 / C::NT : DMA ? 1 : C::STAGE * 2 / 16 / C::NT;
    const uint16_t *src;        // the tile's first row (ROWS) or column (COLS), k = 0
    const uint8_t *src8, *scales;
    int64_t ld, lds;
    int lim, klen, col0;
    u32x4 reg[REGS];
    uint32_t sc[REGS];

    // Copy j of this wave of the stage at k0 into the stage at LDS address `base`.
    __device__ __forceinline__ void copy(uint32_t base, int k0, int j, int wave, int lane) const
    {
        const uint16_t *in;
        bool ok;
        if constexpr (SIDE == ROWS) {
            const int row = (wave * C::COPIES + j) * 8 + lane / 8, ch = (lane & 7) ^ rows_swz(row);
            in = src + (int64_t)row * ld + k0 + ch * 8;
            ok = row < lim && k0 + ch * 8 < klen;
        } else {
            const int off = (wave * C::COPIES + j) * 1024 + 16 * lane;
            const int k = off / (2 * BM), u2 = off % (2 * BM) / 16;
            const int col = ((u2 >> 1) ^ cols_swz(k)) * 16 + (u2 & 1) * 8;
            in = src + (int64_t)(k0 + k) * ld + col;
            ok = k0 + k < klen && col < lim;
        }
        lds_dma_16(ok ? in : zero_chunk<uint16_t>(), base + (wave * C::COPIES + j) * 1024);
    }

    // Through registers: every load of the stage at k0, then (`put`) into the stage.
    __device__ __forceinline__ void fetch(int k0, int tid)
    {
#pragma unroll
        for (int i = 0; i < REGS; ++i) {
            reg[i] = u32x4{0u, 0u, 0u, 0u};
            const int c = i * C::NT + tid;
            if constexpr (SIDE == COLS8) {
                const int k = c / (BM / 16), col = c % (BM / 16) * 16;
                sc[i] = 0;
                if (k0 + k < klen && col < lim) {
                    const uint8_t *p = src8 + (int64_t)(k0 + k) * ld + col;
                    sc[i] = scales[(int64_t)(k0 + k) * lds + ((col0 + col) >> 5)];
                    if (col + 16 <= lim) {
                        reg[i] = load16<u32x4>(p);
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if (col + e < lim)
                                reg[i][e / 4] |= (uint32_t)p[e] << (8 * (e % 4));
                    }
                }
            } else {
                int n;
                const uint16_t *p;
                if constexpr (SIDE == ROWS) {
                    const int row = c / 8, k = k0 + c % 8 * 8;
                    n = row < lim ? klen - k : 0;
                    p = src + (int64_t)row * ld + k;
                } else {
                    const int k = c / (BM / 8), col = c % (BM / 8) * 8;
                    n = k0 + k < klen ? lim - col : 0;
                    p = src + (int64_t)(k0 + k) * ld + col;
                }
                if (n >= 8) {
                    reg[i] = load16<u32x4>(p);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (e < n)
                            reg[i][e / 2] |= (uint32_t)p[e] << (16 * (e % 2));
                }
            }
        }
    }
    __device__ __forceinline__ void put(uint16_t *stage, int tid) const
    {
#pragma unroll
        for (int i = 0; i < REGS; ++i) {
            const int c = i * C::NT + tid;
            if constexpr (SIDE == COLS8) {
                const int k = c / (BM / 16), u = c % (BM / 16) ^ cols_swz(k);
                u32x4 w[2];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float v[4];
                    mx8_decode4(reg[i][q], sc[i], v);
                    if constexpr (!BF16) {
                        // a value that rounding to 8 bits carried past binary16's range
                        // (65504 becomes 65536) is its largest
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            v[e] = __builtin_fabsf(v[e]) > 65504.0f ? __builtin_copysignf(65504.0f, v[e]) : v[e];
                    }
                    w[q / 2][2 * (q & 1)] = (uint32_t)from_f32<kType16<BF16>>(v[0]) | (uint32_t)from_f32<kType16<BF16>>(v[1]) << 16;
                    w[q / 2][2 * (q & 1) + 1] = (uint32_t)from_f32<kType16<BF16>>(v[2]) | (uint32_t)from_f32<kType16<BF16>>(v[3]) << 16;
                }
                u32x4 *dst = reinterpret_cast<u32x4 *>(stage + k * BM + u * 16);
                dst[0] = w[0];
                dst[1] = w[1];
            } else if constexpr (SIDE == ROWS) {
                const int row = c / 8, ch = (c & 7) ^ rows_swz(row);
                *reinterpret_cast<u32x4 *>(stage + row * 64 + ch * 8) = reg[i];
            } else {
                const int k = c / (BM / 8), u2 = c % (BM / 8);
                const int u = (u2 >> 1) ^ cols_swz(k);
                *reinterpret_cast<u32x4 *>(stage + k * BM + u * 16 + (u2 & 1) * 8) = reg[i];
            }
        }
    }

    // Block f (16 of the tile's rows or columns from o on) of k-step s: k = 32 s + 8 (lane /
    // 16) .. + 7 of row or column lane % 16.
    __device__ __forceinline__ static f16x8 read(const uint16_t *stage, int o, int s, int lane)
    {
        const int grp = lane >> 4, j = lane & 15;
        if constexpr (SIDE == ROWS) {
            const int row = o + j, c = (4 * s + grp) ^ rows_swz(row);
            return *reinterpret_cast<const f16x8 *>(stage + row * 64 + c * 8);
        } else {
            s16x4 v[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int k = 32 * s + 8 * grp + 4 * e + (j >> 2), n = o + 4 * (j & 3);
                const int at = k * BM + (((n >> 4) ^ cols_swz(k)) << 4) + (n & 15);
                v[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (__attribute__((address_space(3))) s16x4 *)(lds_addr(stage + at)));
            }
            return __builtin_bit_cast(f16x8, (short __attribute__((ext_vector_type(8)))){
                v[0][0], v[0][1], v[0][2], v[0][3], v[1][0], v[1][1], v[1][2], v[1][3]});
        }
    }
};

// Eight sums of row `row`, columns col .. col + 7, to C with everything the forward product's
// write-back does. `n`: how many of them are inside C (at least 1); group g's bias.
template <bool BF16>
__device__ __forceinline__ void finish_fwd(const L16Params &p, float (&v)[8], const float (&bias)[8], int64_t row, int col,
                                           int n, bool live)
{
    constexpr int T = kType16<BF16>;
    float r[8];
    if (live && p.R != nullptr) {
        if (p.ctype == LL_TYPE_F32)
            load_row<LL_TYPE_F32, 8>(static_cast<const float *>(p.R) + row * p.ldr + col, n, r);
        else
            load_row<T, 8>(static_cast<const uint16_t *>(p.R) + row * p.ldr + col, n, r);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            r[e] = 0.0f;
    }
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
        store_row<T, 8>(p.Z + row * p.ldz + col, n, v);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        v[e] = activate(v[e], p.act) + r[e];
    if (p.ctype == LL_TYPE_F32)
        store_row<LL_TYPE_F32, 8>(static_cast<float *>(p.C) + row * p.ldc + col, n, v);
    else
        store_row<T, 8>(static_cast<uint16_t *>(p.C) + row * p.ldc + col, n, v);
}

// Eight sums to C, with beta times what is there (the gradients).
template <bool BF16>
__device__ __forceinline__ void finish_grad(const L16Params &p, float (&v)[8], int64_t at, int n)
{
    constexpr int T = kType16<BF16>;
    float c[8];
    if (p.ctype == LL_TYPE_F32) {
        float *dst = static_cast<float *>(p.C) + at;
        if (p.beta != 0.0f) {
            load_row<LL_TYPE_F32, 8>(dst, n, c);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = __builtin_fmaf(p.beta, c[e], v[e]);
        }
        store_row<LL_TYPE_F32, 8>(dst, n, v);
    } else {
        uint16_t *dst = static_cast<uint16_t *>(p.C) + at;
        if (p.beta != 0.0f) {
            load_row<T, 8>(dst, n, c);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = __builtin_fmaf(p.beta, c[e], v[e]);
        }
        store_row<T, 8>(dst, n, v);
    }
}

// Tile `id` of tiles_m x tiles_n in groups of four rows of tiles, column by column, so that
// the tiles an XCD has at a time share their operands in its L2.
__device__ __forceinline__ void tile_at(int id, int tiles_m, int tiles_n, int &tm, int &tn)
{
    constexpr int GROUP = 4;
    const int per = GROUP * tiles_n, g = id / per, first = g * GROUP;
    const int rows = min(tiles_m - first, GROUP), within = id - g * per;
    tm = first + within % rows;
    tn = within / rows;
}

template <int OP, bool BF16, int BM, int SA, int SB, bool DMA>
__global__ void __launch_bounds__(Cfg<BM>::NT) __attribute__((amdgpu_waves_per_eu(2, 2))) l16_tile_kernel(L16Params p)
{
    using C = Cfg<BM>;
    constexpr bool DMA_A = DMA, DMA_B = DMA && SB != COLS8;
    constexpr int PITCH = C::WTN + 4;   // floats of a row of the write-back's LDS (16 rows a wave)
    static_assert(C::NW * 16 * PITCH * 4 <= 4 * C::STAGE * 2, "the write-back's rows fit the ring");
    __shared__ __attribute__((aligned(1024))) uint16_t ring[2][2][C::STAGE];   // [operand][buffer]

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave / C::WGN, wn = wave % C::WGN;

    // the tile: C's rows [m0, m_end) and columns from n0, contracted range [k_begin, k_begin + klen)
    int g = 0, m0, m_end, n0, k_begin = 0, klen = p.K;
    int64_t c_off = 0;
    if constexpr (OP == L16_DW) {
        const int per = p.tiles_m * p.tiles_n, total = per * p.groups.n;
        const int id = block_index(blockIdx.x, total);
        g = id / per;
        int tm, tn, end;
        tile_at(id - g * per, p.tiles_m, p.tiles_n, tm, tn);
        group_rows(p.groups, p.K, g, k_begin, end);
        klen = end - k_begin;
        m0 = tm * BM;
        m_end = p.M;
        n0 = tn * BM;
        c_off = (int64_t)g * p.stride_c;
    } else {
        // rows of tiles of all groups; workgroups past the last have nothing to do
        Chunk c{};
        const int rows = find_chunk(p.groups, p.M, BM, -1, c), total = rows * p.tiles_n;
        if ((int)blockIdx.x >= total)
            return;
        const int id = block_index(blockIdx.x, total);
        find_chunk(p.groups, p.M, BM, id / p.tiles_n, c);
        int tm, tn;
        tile_at(id - c.group_first * p.tiles_n, cdiv(c.end - c.begin, BM), p.tiles_n, tm, tn);
        g = c.group;
        m0 = c.begin + tm * BM;
        m_end = c.end;
        n0 = tn * BM;
    }

    Operand<BF16, BM, SA, DMA_A> a;
    Operand<BF16, BM, SB, DMA_B> b;
    a.ld = p.lda;
    a.lim = m_end - m0;
    a.klen = b.klen = klen;
    a.src = SA == ROWS ? p.A + (int64_t)m0 * p.lda : p.A + (int64_t)k_begin * p.lda + m0;
    b.ld = p.ldb;
    b.lim = p.N - n0;
    b.col0 = n0;
    if constexpr (SB == COLS8) {
        b.src8 = static_cast<const uint8_t *>(p.B) + (int64_t)k_begin * p.ldb + n0;
        b.scales = p.BS + (int64_t)k_begin * p.ldbs;
        b.lds = p.ldbs;
    } else {
        const uint16_t *w = static_cast<const uint16_t *>(p.B) + (OP == L16_DW ? 0 : (int64_t)g * p.stride_b);
        b.src = SB == ROWS ? w + (int64_t)n0 * p.ldb : w + (int64_t)k_begin * p.ldb + n0;
    }

    f32x4 acc[C::FM][C::FN];
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
            acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    const uint32_t base_a = lds_addr(&ring[0][0][0]), base_b = lds_addr(&ring[1][0][0]);
    constexpr uint32_t STAGE_BYTES = C::STAGE * 2;
    auto read_step = [&](int buf, int s, f16x8 (&fa)[C::FM], f16x8 (&fb)[C::FN]) {
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
            fa[i] = a.read(ring[0][buf], wm * C::WTM + 16 * i, s, lane);
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
            fb[j] = b.read(ring[1][buf], wn * C::WTN + 16 * j, s, lane);
    };
    // Rows of blocks in alternating column order: neighbouring MFMAs share an operand, and
    // the chip, power-limited on 16-bit products, keeps a higher clock.
    auto mfma_row = [&](int i, const f16x8 (&fa)[C::FM], const f16x8 (&fb)[C::FN]) {
#pragma unroll
        for (int jj = 0; jj < C::FN; ++jj) {
            const int j = (i & 1) ? C::FN - 1 - jj : jj;
            acc[i][j] = mma<BF16>(fb[j], fa[i], acc[i][j]);
        }
    };

    const int nk = cdiv(klen, C::BK);
    f16x8 fa[2][C::FM], fb[2][C::FN];
    if constexpr (DMA_A && DMA_B) {
        // Two stages of copies in flight. The barrier of a stage comes before its last step,
        // whose operands are then in registers: it publishes the next stage and frees this
        // one's buffer, which is refilled while the last step's MFMAs run.
        constexpr int PER = 2 * C::COPIES;
        static_assert(PER <= 63, "vmcnt range");
        auto copy = [&](int buf, int k0, int c) {
            if (c < C::COPIES)
                a.copy(base_a + buf * STAGE_BYTES, k0, c, wave, lane);
            else
                b.copy(base_b + buf * STAGE_BYTES, k0, c - C::COPIES, wave, lane);
        };
        for (int st = 0; st < 2; ++st)
            if (st < nk) {
#pragma unroll
                for (int c = 0; c < PER; ++c)
                    copy(st, st * C::BK, c);
            }
        if (nk > 1)
            __builtin_amdgcn_s_waitcnt(LL_VMCNT(PER));
        else
            __builtin_amdgcn_s_waitcnt(LL_VMCNT(0));
        __syncthreads();
        read_step(0, 0, fa[0], fb[0]);
        for (int kt = 0; kt < nk; ++kt) {
            const int buf = kt & 1;
            read_step(buf, 1, fa[1], fb[1]);
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int i = 0; i < C::FM; ++i)
                mfma_row(i, fa[0], fb[0]);
            __builtin_amdgcn_s_setprio(0);
            if (kt + 1 < nk) {
                __builtin_amdgcn_s_waitcnt(LL_VMCNT(0));   // stage kt + 1 has landed
                __syncthreads();
            }
            const bool refill = kt + 2 < nk;
            // first operands of stage kt + 1 (after the last stage: stale, unused)
            read_step(buf ^ 1, 0, fa[0], fb[0]);
            constexpr int CROWS = 2, G = PER / CROWS;   // copies after each of the first rows of MFMAs
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int i = 0; i < C::FM; ++i) {
                mfma_row(i, fa[1], fb[1]);
                if (refill && i < CROWS) {
#pragma unroll
                    for (int c = 0; c < G; ++c)
                        copy(buf, (kt + 2) * C::BK, i * G + c);
                }
            }
            __builtin_amdgcn_s_setprio(0);
        }
    } else {
        // An operand through registers: the next stage's loads are in flight during this one's
        // MFMAs and are stored into the other buffer after them.
        auto begin = [&](int buf, int k0) {
            if constexpr (DMA_A) {
#pragma unroll
                for (int c = 0; c < C::COPIES; ++c)
                    a.copy(base_a + buf * STAGE_BYTES, k0, c, wave, lane);
            } else {
                a.fetch(k0, tid);
            }
            if constexpr (DMA_B) {
#pragma unroll
                for (int c = 0; c < C::COPIES; ++c)
                    b.copy(base_b + buf * STAGE_BYTES, k0, c, wave, lane);
            } else {
                b.fetch(k0, tid);
            }
        };
        auto end = [&](int buf) {
            if constexpr (!DMA_A)
                a.put(ring[0][buf], tid);
            if constexpr (!DMA_B)
                b.put(ring[1][buf], tid);
            __builtin_amdgcn_s_waitcnt(LL_VMCNT(0));
            __syncthreads();
        };
        if (nk > 0) {
            begin(0, 0);
            end(0);
        }
        for (int kt = 0; kt < nk; ++kt) {
            const int buf = kt & 1;
            if (kt + 1 < nk)
                begin(buf ^ 1, (kt + 1) * C::BK);
#pragma unroll
            for (int s = 0; s < C::STEPS; ++s) {
                read_step(buf, s, fa[0], fb[0]);
                __builtin_amdgcn_s_setprio(1);
#pragma unroll
                for (int i = 0; i < C::FM; ++i)
                    mfma_row(i, fa[0], fb[0]);
                __builtin_amdgcn_s_setprio(0);
            }
            if (kt + 1 < nk)
                end(buf ^ 1);
        }
    }

    // The write-back, 16 rows of the wave's block at a time through its own part of the ring.
    __syncthreads();   // the ring is read no more
    float *turn = reinterpret_cast<float *>(&ring[0][0][0]) + wave * 16 * PITCH;
    const int rl = lane >> 3, cl = (lane & 7) * 8;
    const int col = n0 + wn * C::WTN + cl, n = p.N - col;
    static_assert(C::WTN == 64, "eight lanes a row");
    float bias[8];
    if constexpr (OP == L16_FWD)
        load_row<LL_TYPE_F32, 8>(p.bias + (int64_t)g * p.N + col, p.bias != nullptr ? n : 0, bias);
#pragma unroll
    for (int i = 0; i < C::FM; ++i) {
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
            *reinterpret_cast<f32x4 *>(turn + (lane & 15) * PITCH + 16 * j + 4 * (lane >> 4)) = acc[i][j];
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // (the wave's own rows: no barrier)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int row = m0 + wm * C::WTM + 16 * i + 8 * h + rl;
            float v[8];
            const f32x4 lo = *reinterpret_cast<const f32x4 *>(turn + (8 * h + rl) * PITCH + cl);
            const f32x4 hi = *reinterpret_cast<const f32x4 *>(turn + (8 * h + rl) * PITCH + cl + 4);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[e] = lo[e], v[4 + e] = hi[e];
            const bool live = row < m_end && n > 0;
            if constexpr (OP == L16_FWD) {
                finish_fwd<BF16>(p, v, bias, row, col, n, live);
            } else {
                if (live)
                    finish_grad<BF16>(p, v, c_off + (int64_t)row * p.ldc + col, n);
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
}

// ---- launches -------------------------------------------------------------------

// Whether so many tiles of 256 x 256 (one a CU) take less time than so many of 128 x 128 (two
// a CU, 0.88 of the large ones' rate).
inline bool prefer_256(int64_t t256, int64_t t128, int cus)
{
    const double large = (double)((t256 + cus - 1) / cus), small = (double)((t128 + 2 * cus - 1) / (2 * cus));
    return large <= small * 0.5 / 0.88;
}

// The products whose groups are of C's rows.
template <int OP, bool BF16, int BM, int SB, bool DMA>
hipError_t launch_rows_bm(L16Params p, hipStream_t s)
{
    p.tiles_n = cdiv(p.N, BM);
    // every group may end inside a tile
    const int64_t rows = p.groups.offsets == nullptr ? cdiv(p.M, BM)
                                                     : (int64_t)(p.M / BM) + (p.groups.n < p.M ? p.groups.n : p.M);
    const int64_t tiles = rows * p.tiles_n;
    if (tiles > max_grid_x(Cfg<BM>::NT))
        return hipErrorInvalidValue;
    hipLaunchKernelGGL((l16_tile_kernel<OP, BF16, BM, ROWS, SB, DMA>), dim3((unsigned)tiles), dim3(Cfg<BM>::NT), 0, s, p);
    return hipGetLastError();
}

template <int OP, bool BF16, int SB>
hipError_t launch_rows(const L16Params &p, bool vec, int cus, hipStream_t s)
{
    if (!vec)
        return launch_rows_bm<OP, BF16, 128, SB, false>(p, s);
    // rows of tiles, the groups taken as equally long
    const int g = p.groups.n < p.M ? p.groups.n : p.M, each = cdiv(p.M, g);
    return prefer_256((int64_t)g * cdiv(each, 256) * cdiv(p.N, 256), (int64_t)g * cdiv(each, 128) * cdiv(p.N, 128), cus)
               ? launch_rows_bm<OP, BF16, 256, SB, true>(p, s)
               : launch_rows_bm<OP, BF16, 128, SB, true>(p, s);
}

}  // namespace l16
}  // namespace ll
