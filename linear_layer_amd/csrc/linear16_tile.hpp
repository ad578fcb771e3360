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
// ROWS and COLS on 16 bytes are copied straight into LDS by buffer loads (16 bytes a lane)
// whose descriptor ends with the tile's last row and the contracted range, so that what lies
// past them arrives as zeros without a test; only where a stage crosses the range's end inside
// the rows do lanes take an offset past the descriptor. Rows off 16 bytes go through registers
// (DMA false), 16 bytes a load at any alignment, the chunk that crosses the row's end value
// by value.
//
// The MFMA takes the operand of C's columns first, so a lane gets four neighbouring columns
// of a row; the write-back turns them around in LDS to eight a lane, 128 bytes of a row (16
// bits) in one store instruction, which is also the order that R and bias are read in and
// in which four lanes hold one block of 32 of Z's 8 bits.
#pragma once

#include <type_traits>
#include <utility>

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

// buffer_load_dwordx4 into LDS: this lane's 16 bytes at byte `off` of the buffer go to LDS
// byte lds_base + 16 * lane, zeros where they lie past its end. Inline assembly, so that the
// compiler does not take it for an LDS store that every barrier must wait for; the caller
// counts the copies itself before the barrier that publishes them. The compiler's hazard
// checks do not look inside: a scalar that a vector instruction wrote (v_readfirstlane) may be
// read by a load five wait states later, M0 one after its write.
__device__ __forceinline__ void lds_buffer_16(const u32x4 &buffer, uint32_t off, uint32_t lds_base)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(lds_base), "v"(off), "s"(buffer)
                 : "memory", "m0");
}
constexpr uint32_t kPastEnd = 0x80000000u;   // past the end of every buffer here: 256 rows of less than 2^21 values

typedef const __attribute__((address_space(3))) f16x8 *LdsF16x8;
typedef __attribute__((address_space(3))) s16x4 *LdsS16x4;

// One operand's source: `lim` rows or columns of it from the tile's first on exist (more
// may be asked for), `klen` of the contracted axis.
template <bool BF16, int BM, int SIDE, bool DMA>
struct Operand {
    using C = Cfg<BM>;
    // registers of a stage on its way: 16-byte chunks a thread
    static constexpr int REGS = SIDE == COLS8 ? BM * C::BK / 16 / C::NT : DMA ? 1 : C::STAGE * 2 / 16 / C::NT;
    static constexpr int KROWS = 512 / BM;   // k-rows of a copy (COLS)
    const uint16_t *src;        // the tile's first row (ROWS) or column (COLS), k = 0
    const uint8_t *src8, *scales;
    int64_t ld, lds;
    int lim, klen, col0;
    uint32_t off[2];            // a lane's offset in a copy: two swizzles take turns
    u32x4 reg[REGS];
    uint32_t sc[REGS];

    // Copy j of a wave fills KiB wave * COPIES + j of a stage: 8 rows of 128 bytes, or KROWS
    // k-rows of 2 * BM bytes.
    __device__ __forceinline__ void start(int wave, int lane)
    {
        static_assert(C::COPIES == 4, "the copies' swizzles");
        if constexpr (DMA && SIDE == ROWS) {
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const int row = (wave * C::COPIES + v) * 8 + lane / 8;
                off[v] = (uint32_t)row * (uint32_t)(2 * ld) + (((lane & 7) ^ rows_swz(row)) << 4);
            }
        } else if constexpr (DMA) {
            constexpr int LPR = 64 / KROWS;   // lanes of a k-row
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const int k = (wave * C::COPIES + v * (BM == 256 ? 1 : 2)) * KROWS + lane / LPR, u2 = lane % LPR;
                off[v] = (uint32_t)k * (uint32_t)(2 * ld) + ((((u2 >> 1) ^ cols_swz(k)) << 5) | ((u2 & 1) << 4));
            }
        }
    }
    // The buffer of the stage at k0.
    __device__ __forceinline__ u32x4 buffer(int k0) const
    {
        const int left = min(klen - k0, C::BK), n = min(lim, BM);
        const uint64_t at = (uint64_t)(SIDE == ROWS ? src + k0 : src + (int64_t)k0 * ld);
        const uint32_t bytes = SIDE == ROWS ? (uint32_t)(n - 1) * (uint32_t)(2 * ld) + 2 * left
                                            : (uint32_t)(left - 1) * (uint32_t)(2 * ld) + 2 * n;
        return u32x4{(uint32_t)at, (uint32_t)(at >> 32) & 0xffffu, bytes, 0x00020000u};
    }
    // Copy j of this wave of that stage to the stage at LDS address `base`.
    template <int J>
    __device__ __forceinline__ void copy(const u32x4 &buf, uint32_t base, int k0, int wave, int lane) const
    {
        constexpr int v = SIDE == ROWS || BM == 256 ? J & 1 : J >> 1;
        constexpr int r = SIDE == ROWS ? (J & 2) * 8 : BM == 256 ? (J & 2) * KROWS : (J & 1) * KROWS;   // rows past the swizzle's first copy
        uint32_t o = off[v] + r * (uint32_t)(2 * ld);
        if constexpr (SIDE == ROWS) {
            const int row = (wave * C::COPIES + v) * 8 + lane / 8;
            if (k0 + ((lane & 7) ^ rows_swz(row)) * 8 >= klen)
                o = kPastEnd;
        }
        lds_buffer_16(buf, o, base + (wave * C::COPIES + J) * 1024);
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

    // A lane's part of an operand read: k = 32 s + 8 (lane / 16) .. + 7 of row or column
    // lane % 16 of the blocks from the wave's first, o, on.
    __device__ __forceinline__ static uint32_t lane_addr(int o, int lane)
    {
        const int grp = lane >> 4, j = lane & 15;
        if constexpr (SIDE == ROWS)
            return (uint32_t)((o + j) * 128 + ((grp ^ rows_swz(j)) << 4));
        else   // (lanes 4 j' .. + 3 of 16 point at the four 8-byte pieces of k-row j')
            return (uint32_t)((8 * grp + (j >> 2)) * 2 * BM + (((o >> 4) ^ cols_swz(8 * grp + (j >> 2))) << 5) + 8 * (j & 3));
    }
    // Block i of k-step s, `at` being the stage's LDS address plus lane_addr.
    __device__ __forceinline__ static f16x8 read(uint32_t at, int i, int s)
    {
        if constexpr (SIDE == ROWS) {
            return *(LdsF16x8)(uintptr_t)((at ^ (64u * s)) + 2048u * i);
        } else {
            const uint32_t a = (at ^ (32u * i)) + 64u * BM * s;
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsS16x4)(uintptr_t)a);
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsS16x4)(uintptr_t)(a + 8u * BM));
            return __builtin_bit_cast(f16x8, (short __attribute__((ext_vector_type(8)))){lo[0], lo[1], lo[2], lo[3], hi[0],
                                                                                         hi[1], hi[2], hi[3]});
        }
    }
};

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
    activate8(v, p.act);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        v[e] += r[e];
    store8<BF16>(p.ctype, p.C, row * p.ldc + col, n, v);
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
    constexpr int PITCH = C::WTN + 4;   // floats of a row of the write-back's LDS (64 rows a wave)
    constexpr int TURN_BYTES = C::NW * 64 * PITCH * 4, RING_BYTES = 4 * C::STAGE * 2;
    __shared__ __attribute__((aligned(1024))) uint8_t lds_bytes[TURN_BYTES > RING_BYTES ? TURN_BYTES : RING_BYTES];
    uint16_t (*ring)[2][C::STAGE] = reinterpret_cast<uint16_t (*)[2][C::STAGE]>(lds_bytes);   // [operand][buffer]

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

    a.start(wave, lane);
    b.start(wave, lane);
    const uint32_t base_a = lds_addr(&ring[0][0][0]), base_b = lds_addr(&ring[1][0][0]);
    constexpr uint32_t STAGE_BYTES = C::STAGE * 2;
    uint32_t at_a = base_a + a.lane_addr(wm * C::WTM, lane), at_b = base_b + b.lane_addr(wn * C::WTN, lane);
    auto read_step = [&](int buf, int s, f16x8 (&fa)[C::FM], f16x8 (&fb)[C::FN]) __attribute__((always_inline)) {
        const uint32_t xa = at_a + buf * STAGE_BYTES, xb = at_b + buf * STAGE_BYTES;
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
            fb[j] = b.read(xb, j, s);
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
            fa[i] = a.read(xa, i, s);
    };
    // Rows of blocks in alternating column order: neighbouring MFMAs share an operand, and
    // the chip, power-limited on 16-bit products, keeps a higher clock.
    auto mfma_row = [&](int i, const f16x8 (&fa)[C::FM], const f16x8 (&fb)[C::FN]) __attribute__((always_inline)) {
#pragma unroll
        for (int jj = 0; jj < C::FN; ++jj) {
            const int j = (i & 1) ? C::FN - 1 - jj : jj;
            acc[i][j] = mma<BF16>(fb[j], fa[i], acc[i][j]);
        }
    };
    // The products issued so far stay before this point: left alone, the compiler moves them
    // behind the barrier and keeps their operands alive.
    auto pin = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
#pragma unroll
            for (int j = 0; j < C::FN; ++j)
                asm volatile("" : "+v"(acc[i][j]));
    };

    // Stages go through two buffers and two sets of operand registers. A step's operands are
    // read while the step before multiplies. The stage's barrier stands before its last
    // step, whose operands are then in registers: it publishes the next stage and frees this
    // one's buffer, which is refilled while the last step multiplies. Operands that pass
    // through registers are stored into the next buffer just before the barrier, a stage
    // after their loads.
    const int nk = cdiv(klen, C::BK);
    constexpr int PER = (DMA_A ? C::COPIES : 0) + (DMA_B ? C::COPIES : 0);
    u32x4 buf_a, buf_b;
    auto copies = [&](int buf, int k0, auto first, auto count) __attribute__((always_inline)) {
        static_for<decltype(count)::value>([&](auto cc) __attribute__((always_inline)) {
            constexpr int c = decltype(first)::value + decltype(cc)::value;
            if constexpr (DMA_A && c < C::COPIES)
                a.template copy<c>(buf_a, base_a + buf * STAGE_BYTES, k0, wave, lane);
            else
                b.template copy<c - (DMA_A ? C::COPIES : 0)>(buf_b, base_b + buf * STAGE_BYTES, k0, wave, lane);
        });
    };
    auto aim = [&](int k0) __attribute__((always_inline)) {
        if constexpr (DMA_A)
            buf_a = a.buffer(k0);
        if constexpr (DMA_B)
            buf_b = b.buffer(k0);
    };
    auto fetch = [&](int k0) __attribute__((always_inline)) {
        if constexpr (!DMA_A)
            a.fetch(k0, tid);
        if constexpr (!DMA_B)
            b.fetch(k0, tid);
    };
    auto put = [&](int buf) __attribute__((always_inline)) {
        if constexpr (!DMA_A)
            a.put(ring[0][buf], tid);
        if constexpr (!DMA_B)
            b.put(ring[1][buf], tid);
    };
    constexpr std::integral_constant<int, 0> none{};
    constexpr std::integral_constant<int, PER> all{};
    if (nk > 0) {
        aim(0);
        copies(0, 0, none, all);
        fetch(0);
        put(0);
        if (nk > 1) {
            aim(C::BK);
            copies(1, C::BK, none, all);
            fetch(C::BK);
        }
        if (DMA_A && DMA_B && nk > 1)
            __builtin_amdgcn_s_waitcnt(LL_VMCNT(PER));
        else
            __builtin_amdgcn_s_waitcnt(LL_VMCNT(0));
    }
    __syncthreads();
    f16x8 fa[2][C::FM], fb[2][C::FN];
    read_step(0, 0, fa[0], fb[0]);
    auto body = [&](auto more, int kt) __attribute__((always_inline)) {
        constexpr bool REFILL = decltype(more)::value;   // there is a stage kt + 2
        const int buf = kt & 1;
        asm volatile("" : "+v"(at_a), "+v"(at_b));   // (the blocks' addresses are made anew, not kept in registers)
        read_step(buf, 1, fa[1], fb[1]);
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
            mfma_row(i, fa[0], fb[0]);
        __builtin_amdgcn_s_setprio(0);
        pin();
        if (REFILL || kt + 1 < nk) {
            put(buf ^ 1);
            __builtin_amdgcn_s_waitcnt(LL_VMCNT(0));   // stage kt + 1 has landed
        }
        __syncthreads();
        if (REFILL || kt + 1 < nk)
            read_step(buf ^ 1, 0, fa[0], fb[0]);
        const int k0 = (kt + 2) * C::BK;
        if constexpr (REFILL) {
            aim(k0);
            fetch(k0);
        }
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(1);
        // the copies follow the first rows of products, not one burst that the matrix cores
        // would wait through
        constexpr int CROWS = 2, G = (PER + CROWS - 1) / CROWS;
        static_for<C::FM>([&](auto ii) __attribute__((always_inline)) {
            constexpr int i = decltype(ii)::value;
            mfma_row(i, fa[1], fb[1]);
            if constexpr (REFILL && PER > 0 && i < CROWS) {
                __builtin_amdgcn_sched_barrier(0);
                copies(buf, k0, std::integral_constant<int, i * G>{}, std::integral_constant<int, G>{});
                __builtin_amdgcn_sched_barrier(0);
            }
        });
        __builtin_amdgcn_s_setprio(0);
        pin();
    };
    int kt = 0;
    for (; kt + 2 < nk; ++kt)
        body(std::true_type{}, kt);
    for (; kt < nk; ++kt)
        body(std::false_type{}, kt);

    // The write-back, 64 rows of the wave's block at a time through its own part of the
    // LDS, then eight rows a turn of a loop. (All of it unrolled is more code than the
    // instruction cache holds: 2.3 ms where this takes 0.2.) The next turn's R, or C for beta, is
    // on its way during a turn.
    __syncthreads();   // the ring is read no more
    float *turn = reinterpret_cast<float *>(lds_bytes) + wave * 64 * PITCH;
    const int rl = lane >> 3, cl = (lane & 7) * 8;
    const int col = n0 + wn * C::WTN + cl, n = p.N - col;
    static_assert(C::WTN == 64 && C::WTM % 64 == 0, "eight lanes a row");
    const void *more = OP == L16_FWD ? p.R : p.beta != 0.0f ? p.C : nullptr;
    const int64_t more_ld = OP == L16_FWD ? p.ldr : p.ldc;
    float bias[8];
    if constexpr (OP == L16_FWD)
        load_row<LL_TYPE_F32, 8>(p.bias + (int64_t)g * p.N + col, p.bias != nullptr ? n : 0, bias);
    static_for<C::WTM / 64>([&](auto hh) __attribute__((always_inline)) {
        constexpr int half = decltype(hh)::value;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < C::FN; ++j)
                *reinterpret_cast<f32x4 *>(turn + (16 * i + (lane & 15)) * PITCH + 16 * j + 4 * (lane >> 4)) = acc[4 * half + i][j];
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // (the wave's own rows: no barrier)
        const int row0 = m0 + wm * C::WTM + 64 * half + rl;
        float next[8];
        load8<BF16>(p.ctype, more, c_off + (int64_t)row0 * more_ld + col, more != nullptr && row0 < m_end ? n : 0, next);
#pragma unroll 1
        for (int q = 0; q < 8; ++q) {
            const int row = row0 + 8 * q;
            float v[8], r[8];
            const f32x4 lo = *reinterpret_cast<const f32x4 *>(turn + (8 * q + rl) * PITCH + cl);
            const f32x4 hi = *reinterpret_cast<const f32x4 *>(turn + (8 * q + rl) * PITCH + cl + 4);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[e] = lo[e], v[4 + e] = hi[e];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                r[e] = next[e];
            load8<BF16>(p.ctype, more, c_off + (int64_t)(row + 8) * more_ld + col,
                        more != nullptr && q < 7 && row + 8 < m_end ? n : 0, next);
            const bool live = row < m_end && n > 0;
            if constexpr (OP == L16_FWD) {
                finish_fwd<BF16>(p, v, bias, r, row, col, n, live);
            } else if (live) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = __builtin_fmaf(p.beta, r[e], v[e]);   // (r is 0 where beta is)
                store8<BF16>(p.ctype, p.C, c_off + (int64_t)row * p.ldc + col, n, v);
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    });
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
