// The tile kernel of the 16-bit layer and its gradients: forward, input gradient and
// weight gradient, dense or by groups of rows.
//
// A workgroup computes BM x BN of C on v_mfma_f32_16x16x32 with FP32 sums, over stages of
// 64 of the contracted axis in rings of two or three LDS buffers, one for each operand. An operand
// lies in memory in one of three ways:
//   ROWS   the contracted axis is contiguous (X and W of the forward product, dZ of the
//          input gradient): BM rows of 128 bytes a stage, their 16-byte chunks XORed by
//          (row / 2) % 8, read with 128-bit LDS reads;
//   COLS   the other axis is (W of the input gradient, dZ and X of the weight gradient): 64
//          rows of 2 * BM bytes a stage, 32-byte units XORed by 2 * (k % 4) + (k / 8) % 2,
//          read with ds_read_b64_tr_b16, which hands each lane four values of one column;
//   COLS8  as COLS, from E4M3 codes and scales: 16 codes a load into registers, decoded and
//          stored as the 32-byte unit that they are in 16 bits. Decoding on the way into LDS
//          is done once a workgroup; after it, by every wave that reads the stage.
// ROWS and COLS on 16 bytes (VEC) are copied straight into LDS by buffer loads, 16 bytes a
// lane, whose descriptor ends with the tile's last row and the contracted range: what lies
// past them arrives as zeros without a test, and only where a stage crosses the range's end
// inside the rows do lanes take an offset past the descriptor. Rows off 16 bytes and COLS8
// go through registers, loaded a whole stage before they are stored into LDS: 16 bytes a load
// at any alignment, the chunk that crosses the row's end value by value.
//
// The MFMA takes the operand of C's columns first, so a lane gets four neighbouring columns
// of a row; the write-back turns them around in LDS to eight a lane, 128 bytes of a row (16
// bits) in one store instruction, which is also the order that R and bias are read in and
// in which four lanes hold one block of 32 of Z's 8 bits.
//
// Products of many whole rounds of large tiles are bound by the matrix cores and the power they may
// draw; others by rounds that do not fill and by tiles' first loads and write-backs, which nothing
// covers (matrix cores busy 32 to 55 % of the cycles). bfloat16 8192^3
// takes 0.76 to 0.82 ms forward (1.34 to 1.46 PFLOP/s), 0.77 for dX (1.43), 0.79 to 0.83 for dW (1.32 to 1.39) and
// 0.85 to 0.89 with X in 8 bits (1.24 to 1.29), where the library's forward product on the same
// inputs reaches 1.61 and its product on other than rows 1.38. What else was measured there:
// operands through registers instead of copies 1.23 to 1.33 PFLOP/s, eight waves of 128 x 64
// instead of four of 128 x 128 1.33, workgroups set apart over K no gain.
#pragma once

#include "launch.hpp"
#include "linear16_finish.hpp"

namespace ll {
namespace l16 {

enum Side : int { ROWS = 0, COLS = 1, COLS8 = 2 };

// c += a * b with c in accumulation registers. One wave a SIMD has 256 of them beside its 256
// vector registers; left to the compiler, sums wander between the two (500 moves a stage).
// It takes the statement for any other instruction, so nothing may read or write c
// close to it but the next of these: see settle().
template <bool BF16>
__device__ __forceinline__ void mma_acc(const f16x8 &a, const f16x8 &b, f32x4 &c)
{
    if constexpr (BF16)
        asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
    else
        asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
}
// The wait between mma_acc and what else reads its sums (18 wait states at most), and between what
// wrote them and the first mma_acc. The empty statements before and after it take the sums and give them
// on, so that the compiler can move none of their writes behind it and none of their reads ahead of it.
template <int FM, int FN>
__device__ __forceinline__ void settle(f32x4 (&acc)[FM][FN])
{
    const auto tie = [&acc]() __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
                asm volatile("" : "+a"(acc[i][j]));
    };
    tie();
    asm volatile("s_nop 15\n\ts_nop 7" ::: "memory");
    tie();
}

// A workgroup: 2 x 2 waves, each with a quarter of its tile; stages of two steps of the MFMA.
struct Block {
    static constexpr int NW = 4, NT = 64 * NW, BK = 64;
};

typedef const __attribute__((address_space(3))) f16x8 *LdsF16x8;
typedef __attribute__((address_space(3))) s16x4 *LdsS16x4;

// One operand's source: `lim` rows or columns of it from the tile's first on exist (more
// may be asked for), `klen` of the contracted axis.
template <bool BF16, int BM, int SIDE, bool VEC>
struct Operand {
    using C = Block;
    static constexpr bool DMA = VEC && SIDE != COLS8;
    static constexpr int STAGE = BM * C::BK;                     // values of a stage
    static constexpr int PIECES = SIDE == COLS8 ? BM / 64 : BM / 32;   // 16-byte pieces of memory a thread and stage
    static constexpr int KROWS = 512 / BM;   // k-rows of 1 KiB of a COLS stage
    const uint16_t *src;        // the tile's first row (ROWS) or column (COLS), k = 0
    const uint8_t *src8, *scales;
    int64_t ld, lds;
    int lim, klen, col0;
    __amdgpu_buffer_rsrc_t codes, scale_bytes;   // (COLS8)
    uint32_t off[2], cur[2];    // offset of piece 0, and of piece 1 where its swizzle is another; in the stage aimed at
    u32x4 buf;
    u32x4 reg[DMA ? 1 : PIECES];
    uint32_t sc[SIDE == COLS8 ? PIECES : 1];

    // Piece j of a thread fills 16-byte slot (j * NW + wave) * 64 + lane of a stage: a wave fills 8
    // rows of 128 bytes, or KROWS k-rows of 2 * BM. The swizzles repeat every 16 rows,
    // which is one piece of each wave or two.
    static constexpr int STRIDE = C::NW * (SIDE == ROWS ? 8 : KROWS);   // rows from a piece to the next
    static constexpr int SETS = STRIDE % 16 == 0 ? 1 : 2;
    static_assert(STRIDE * SETS % 16 == 0, "the pieces' swizzles");
    // Row, and value within the row, of slot s.
    __device__ __forceinline__ static int slot_row(int s) { return SIDE == ROWS ? s / 8 : s / (BM / 8); }
    __device__ __forceinline__ static int slot_col(int s)
    {
        if constexpr (SIDE == ROWS) {
            return ((s & 7) ^ rows_swz(s / 8)) * 8;
        } else {
            const int u2 = s % (BM / 8);
            return ((u2 >> 1) ^ cols_swz(s / (BM / 8))) * 16 + (u2 & 1) * 8;
        }
    }
    __device__ __forceinline__ void start(int tid)
    {
        if constexpr (DMA) {
#pragma unroll
            for (int v = 0; v < SETS; ++v) {
                const int s = v * C::NT + tid;
                off[v] = (uint32_t)slot_row(s) * (uint32_t)(2 * ld) + 2 * slot_col(s);
            }
        } else if constexpr (VEC && SIDE == COLS8) {   // of codes, and of scales
            const int k = tid / (BM / 16), col = tid % (BM / 16) * 16;
            off[0] = (uint32_t)k * (uint32_t)ld + col;
            off[1] = (uint32_t)k * (uint32_t)lds + ((col0 + col) >> 5);
        }
    }
    // The pieces loaded from now on are of the stage at k0 (past the range: zeros).
    __device__ __forceinline__ void aim(int k0, int tid)
    {
        if constexpr (DMA) {
            const int left = min(klen - k0, C::BK), n = min(lim, BM);
            const int bytes = left <= 0 ? 0 : SIDE == ROWS ? (n - 1) * (int)(2 * ld) + 2 * left : (left - 1) * (int)(2 * ld) + 2 * n;
            const uint16_t *at = SIDE == ROWS ? src + k0 : src + (int64_t)k0 * ld;
            buf = u32x4{(uint32_t)(uint64_t)at, (uint32_t)((uint64_t)at >> 32), (uint32_t)bytes, 0x00020000u};   // (addresses have 48 bits)
#pragma unroll
            for (int v = 0; v < SETS; ++v)
                cur[v] = SIDE == ROWS && slot_col(v * C::NT + tid) >= left ? kPastEnd : off[v];
        } else if constexpr (VEC && SIDE == COLS8) {
            // Codes past a row's end are the next row's, or padding: of columns that are not stored. A load is
            // checked word by word, and a word that is partly past the buffer's end arrives as zero, so the
            // last row ends with its last column's word (rows are whole words: it has no other row's bytes).
            const int left = min(klen - k0, C::BK), n = min(lim, BM);
            const int last = (col0 + n - 1) >> 5;   // scale of the last column
            codes = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(src8 + (int64_t)k0 * ld), 0,
                                                      left <= 0 ? 0 : (left - 1) * (int)ld + ((n + 3) & ~3), 0x00020000);
            scale_bytes = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(scales + (int64_t)k0 * lds), 0,
                                                            left <= 0 ? 0 : (left - 1) * (int)lds + last + 1, 0x00020000);
        }
    }
    // Copy J of this wave of the stage aimed at to the stage at LDS address `base`.
    template <int J>
    __device__ __forceinline__ void copy(uint32_t base, int wave) const
    {
        constexpr int v = J % SETS;
        lds_buffer_16(buf, cur[v] + (J - v) * STRIDE * (uint32_t)(2 * ld), base + (J * C::NW + wave) * 1024);
    }
    // The same through registers: its load, and a stage later its store.
    template <int J>
    __device__ __forceinline__ void load(int k0, int tid)
    {
        if constexpr (SIDE == COLS8 && VEC) {
            constexpr int STEP = J * (C::NT / (BM / 16));   // k-rows from piece 0's
            reg[J] = __builtin_amdgcn_raw_buffer_load_b128(codes, off[0] + STEP * (uint32_t)ld, 0, 0);
            sc[J] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(scale_bytes, off[1] + STEP * (uint32_t)lds, 0, 0);
        } else if constexpr (SIDE == COLS8) {
            reg[J] = u32x4{0u, 0u, 0u, 0u};
            sc[J] = 0;
            const int c = J * C::NT + tid, k = k0 + c / (BM / 16), col = c % (BM / 16) * 16;
            if (k < klen && col < lim) {
                const uint8_t *p = src8 + (int64_t)k * ld + col;
                sc[J] = scales[(int64_t)k * lds + ((col0 + col) >> 5)];
                if (col + 16 <= lim) {
                    reg[J] = load16<u32x4>(p);
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (col + e < lim)
                            reg[J][e / 4] |= (uint32_t)p[e] << (8 * (e % 4));
                }
            }
        } else {
            reg[J] = u32x4{0u, 0u, 0u, 0u};
            const int s = J * C::NT + tid, row = slot_row(s), col = slot_col(s);
            const int n = SIDE == ROWS ? (row < lim ? klen - k0 - col : 0) : (k0 + row < klen ? lim - col : 0);
            const uint16_t *p = SIDE == ROWS ? src + (int64_t)row * ld + k0 + col : src + (int64_t)(k0 + row) * ld + col;
            if (n >= 8) {
                reg[J] = load16<u32x4>(p);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e < n)
                        reg[J][e / 2] |= (uint32_t)p[e] << (16 * (e % 2));
            }
        }
    }
    // (COLS8: half H of it, eight codes.)
    template <int J, int H = 0>
    __device__ __forceinline__ void store(uint16_t *stage, int tid) const
    {
        if constexpr (SIDE == COLS8) {
            const int c = J * C::NT + tid, k = c / (BM / 16), u = c % (BM / 16) ^ cols_swz(k);
            uint32_t w[4];
            mx8_decode4<BF16>(reg[J][2 * H], sc[J], w[0], w[1]);
            mx8_decode4<BF16>(reg[J][2 * H + 1], sc[J], w[2], w[3]);
            *reinterpret_cast<u32x4 *>(stage + k * BM + u * 16 + 8 * H) = u32x4{w[0], w[1], w[2], w[3]};
        } else {
            *reinterpret_cast<u32x4 *>(stage + (J * C::NT + tid) * 8) = reg[J];
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
    // The stage's LDS address plus lane_addr, for k-step s.
    __device__ __forceinline__ static uint32_t step_addr(uint32_t at, int s) { return SIDE == ROWS ? at ^ (64u * s) : at + 64u * BM * s; }
    // Block i, `at` being its step's address.
    __device__ __forceinline__ static f16x8 read(uint32_t at, int i)
    {
        if constexpr (SIDE == ROWS) {
            return *(LdsF16x8)(uintptr_t)(at + 2048u * i);
        } else {
            const uint32_t a = at ^ (32u * i);
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsS16x4)(uintptr_t)a);
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsS16x4)(uintptr_t)(a + 8u * BM));
            return __builtin_bit_cast(f16x8, (short __attribute__((ext_vector_type(8)))){lo[0], lo[1], lo[2], lo[3], hi[0],
                                                                                         hi[1], hi[2], hi[3]});
        }
    }
};

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

// A tile: C's rows m0 .. m_end - 1 (at most BM of them) and columns from n0 on, over klen of the
// contracted axis from k_begin on, for group g.
struct Job {
    int g, m0, m_end, n0, k_begin, klen;
    int64_t c_off;
    float *part;    // where a share's sums go instead (M x N), or null
};

// LDS of a tile: the rings, or the write-back's 64 rows of each wave.
constexpr int kPitch = 64 + 4;   // floats of one of them
template <int BM, int BN, int NA, int NB>
constexpr int tile_lds()
{
    constexpr int ring = (NA * BM + NB * BN) * Block::BK * 2, turn = Block::NW * 64 * kPitch * 4;
    return ring > turn ? ring : turn;
}

// Computes one. WPE: waves a SIMD, one (sums in accumulation registers) or two. NA, NB: buffers of
// the operands' stages, two or (of those copied straight into LDS) three.
template <int OP, bool BF16, int BM, int BN, int WPE, int NA, int NB, int SA, int SB, bool VEC>
__device__ __forceinline__ void l16_tile(const L16Params &p, const Job &job, uint8_t *lds_bytes)
{
    using C = Block;
    constexpr int WTM = BM / 2, WTN = BN / 2, FM = WTM / 16, FN = WTN / 16;   // a wave's block of C
    constexpr int PITCH = kPitch;
    uint16_t (*ring_a)[BM * C::BK] = reinterpret_cast<uint16_t (*)[BM * C::BK]>(lds_bytes);
    uint16_t (*ring_b)[BN * C::BK] = reinterpret_cast<uint16_t (*)[BN * C::BK]>(ring_a + NA);

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave / 2, wn = wave % 2;
    const int g = job.g, m0 = job.m0, m_end = job.m_end, n0 = job.n0, k_begin = job.k_begin, klen = job.klen;
    const int64_t c_off = job.c_off;

    Operand<BF16, BM, SA, VEC> a;
    Operand<BF16, BN, SB, VEC> b;
    a.ld = p.lda;
    a.lim = m_end - m0;
    a.klen = b.klen = klen;
    a.src = SA == ROWS ? p.A + (int64_t)m0 * p.lda + k_begin : p.A + (int64_t)k_begin * p.lda + m0;
    b.ld = p.ldb;
    b.lim = p.N - n0;
    b.col0 = n0;
    if constexpr (SB == COLS8) {
        b.src8 = static_cast<const uint8_t *>(p.B) + (int64_t)k_begin * p.ldb + n0;
        b.scales = p.BS + (int64_t)k_begin * p.ldbs;
        b.lds = p.ldbs;
    } else {
        const uint16_t *w = static_cast<const uint16_t *>(p.B) + (OP == L16_DW ? 0 : (int64_t)g * p.stride_b);
        b.src = SB == ROWS ? w + (int64_t)n0 * p.ldb + k_begin : w + (int64_t)k_begin * p.ldb + n0;
    }

    f32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    a.start(tid);
    b.start(tid);
    const uint32_t base_a = lds_addr(ring_a), base_b = lds_addr(ring_b);
    constexpr uint32_t A_BYTES = BM * C::BK * 2, B_BYTES = BN * C::BK * 2;   // of a stage
    uint32_t at_a = base_a + a.lane_addr(wm * WTM, lane), at_b = base_b + b.lane_addr(wn * WTN, lane);
    // Step s of the stage in buffer buf: where its operands are read. (Opaque to the compiler, so
    // that the blocks are at constant offsets from it and nothing about it is kept in registers
    // over the loop.)
    auto step = [&](int bufa, int bufb, int s, uint32_t &xa, uint32_t &xb) __attribute__((always_inline)) {
        xa = a.step_addr(at_a + bufa * A_BYTES, s);
        xb = b.step_addr(at_b + bufb * B_BYTES, s);
        asm volatile("" : "+v"(xa), "+v"(xb));
    };
    // A stage is two steps. While a step multiplies, the next step's operands are read: its
    // blocks of B into a second set of registers, in the first rows, as the next step's first
    // row needs all of them; a block of A into the registers that a row of products has done
    // with (the last one at the step's own start). The barrier stands after the first rows of
    // a stage's last step, when every operand of the stage is in registers: it publishes the
    // next stage and frees this one's buffers. Then come the copies, in the first half of the
    // rows up to the next barrier: with two buffers those of the stage after next, which have
    // the rest of that time to land in, with three those of the stage after that, which have a
    // whole stage more. (256 x 256 fills the LDS with two of A's and three of B's, which are
    // weights, mostly, and from memory; 2048 x 11008 x 4096 from memory 226 us with two for both.)
    // Pieces through registers go in any row, each followed by the load of its successor (those
    // of COLS8, which are fewer, in the first half too: a wait for copies is one for them).
    // Past the range's end come zeros, and are not used.
    //
    // A wave issues an instruction every four cycles and an MFMA occupies the matrix core for
    // sixteen, so what stands between two MFMAs costs nothing up to three instructions; one
    // wave a SIMD has no other to fill a longer gap. Hence the operations are dealt out
    // singly among a row's MFMAs.
    constexpr int F = FM, ROWS2 = 2 * F;          // rows of products of a step, of a stage
    constexpr int BR = F == 8 ? 2 : 1;            // rows of the last step before the barrier
    constexpr int AFTER = F - BR;                 // and after it
    constexpr int PB = 2 * FN / FM;               // of B's blocks, and copies, a row of half the rows
    using OpA = decltype(a);
    using OpB = decltype(b);
    static_assert(FN % (FM / 2) == 0 && (VEC || (FM == FN && NA == 2 && NB == 2)), "the operations' rows");
    static_assert((NA == 2 || OpA::DMA) && (NB == 2 || OpB::DMA), "through registers there are two buffers");
    // The operations of row w after a barrier, A's and then B's.
    struct Window {
        static constexpr int a(int w) { return OpA::DMA ? (w < F / 2 ? 2 : 0) : w % 2 == 0 ? 2 : 0; }
        static constexpr int b(int w)
        {
            if (OpB::DMA)
                return w >= F / 2 && w < F ? PB : 0;
            if (SB == COLS8 && w >= F)
                return 0;
            return (SB == COLS8 && OpB::PIECES == F) || w % 2 == 1 ? (SB == COLS8 ? 3 : 2) : 0;
        }
        static constexpr int b_piece(int w) { return SB == COLS8 && OpB::PIECES == F ? w : w / 2; }
        static constexpr int n(int w) { return a(w) + b(w); }
    };
    // Operation o of them: into buffers bufa and bufb; the stage that registers are loaded with
    // begins at k0.
    auto window = [&](auto ww, auto oo, int bufa, int bufb, int k0) __attribute__((always_inline)) {
        constexpr int w = decltype(ww)::value, o = decltype(oo)::value, q = o - Window::a(w);
        if constexpr (q < 0) {
            if constexpr (OpA::DMA)
                a.template copy<2 * w + o>(base_a + bufa * A_BYTES, wave);
            else if constexpr (o == 0)
                a.template store<w / 2>(ring_a[bufa], tid);
            else
                a.template load<w / 2>(k0, tid);
        } else {
            if constexpr (OpB::DMA)
                b.template copy<(w - F / 2) * PB + q>(base_b + bufb * B_BYTES, wave);
            else if constexpr (q + 1 < Window::b(w))
                b.template store<Window::b_piece(w), q>(ring_b[bufb], tid);
            else
                b.template load<Window::b_piece(w)>(k0, tid);
        }
    };
    // All of rows first .. first + count - 1's, at once.
    auto windows = [&](auto first, auto count, int bufa, int bufb, int k0) __attribute__((always_inline)) {
        static_for<decltype(count)::value>([&](auto i) __attribute__((always_inline)) {
            constexpr int w = decltype(first)::value + decltype(i)::value;
            static_for<Window::n(w)>([&](auto o) __attribute__((always_inline)) { window(std::integral_constant<int, w>{}, o, bufa, bufb, k0); });
        });
    };
    const int nk = cdiv(klen, C::BK);
    if constexpr (!OpA::DMA)
        static_for<OpA::PIECES>([&](auto j) __attribute__((always_inline)) { a.template load<decltype(j)::value>(0, tid); });
    constexpr int AHEAD = OpB::DMA ? 0 : 1;   // stages that registers are ahead of copies
    b.aim(0, tid);
    if constexpr (!OpB::DMA)
        static_for<OpB::PIECES>([&](auto j) __attribute__((always_inline)) { b.template load<decltype(j)::value>(0, tid); });
    // stage 0, and what the rows after a barrier before it would have begun: copies in the order of
    // their need
    a.aim(0, tid);
    b.aim(AHEAD * C::BK, tid);
    windows(std::integral_constant<int, 0>{}, std::integral_constant<int, ROWS2>{}, 0, 0, C::BK);
    a.aim(C::BK, tid);
    b.aim((1 + AHEAD) * C::BK, tid);
    if constexpr (NA == 3) {
        static_for<OpA::PIECES>([&](auto j) __attribute__((always_inline)) { a.template copy<decltype(j)::value>(base_a + A_BYTES, wave); });
        a.aim(2 * C::BK, tid);
    }
    if constexpr (NB == 3) {
        static_for<OpB::PIECES>([&](auto j) __attribute__((always_inline)) { b.template copy<decltype(j)::value>(base_b + B_BYTES, wave); });
        b.aim(2 * C::BK, tid);
    }
    windows(std::integral_constant<int, 0>{}, std::integral_constant<int, AFTER>{}, NA - 1, NB - 1, 2 * C::BK);
    // copies that may be on their way: at a barrier those past the next stage, in front of the first
    // stage those past it
    constexpr int LATER = (NA - 2) * OpA::PIECES + (NB - 2) * OpB::PIECES;
    constexpr int BEGUN = LATER + OpA::PIECES + (AFTER - F / 2) * PB;
    static_assert(BEGUN <= 63, "the counter's range");
    if constexpr (OpA::DMA && OpB::DMA)
        __builtin_amdgcn_s_waitcnt(LL_VMCNT(BEGUN));
    else if constexpr (OpA::DMA || OpB::DMA)
        __builtin_amdgcn_s_waitcnt(LL_VMCNT(0));
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    f16x8 fa[FM], fb[2][FN];
    {
        uint32_t xa, xb;
        step(0, 0, 0, xa, xb);
#pragma unroll
        for (int i = 0; i + 1 < FM; ++i)
            fa[i] = a.read(xa, i);
#pragma unroll
        for (int j = 0; j < FN; ++j)
            fb[0][j] = b.read(xb, j);
    }
    // Row i of the products on step s's operands, with op(0), .., op(n - 1) dealt out among its
    // MFMAs. Rows alternate in column order: neighbouring MFMAs share an operand, and the
    // chip, power-limited on 16-bit products, keeps a higher clock.
    auto row = [&](auto ii, const f16x8 (&b_)[FN], auto count, auto op) __attribute__((always_inline)) {
        constexpr int i = decltype(ii)::value, n = decltype(count)::value;
        static_for<FN>([&](auto jj) __attribute__((always_inline)) {
            constexpr int q = decltype(jj)::value, j = (i & 1) ? FN - 1 - q : q;
            if constexpr (WPE == 1)
                mma_acc<BF16>(b_[j], fa[i], acc[i][j]);
            else
                acc[i][j] = mma<BF16>(b_[j], fa[i], acc[i][j]);
            __builtin_amdgcn_sched_barrier(0);
            constexpr int lo = q * n / FN, hi = (q + 1) * n / FN;
            static_for<hi - lo>([&](auto k) __attribute__((always_inline)) { op(std::integral_constant<int, lo + decltype(k)::value>{}); });
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    if constexpr (WPE == 1)
        settle(acc);
    // the buffers of stages kt, kt + 1, and of the last one that is on its way
    int bufa = 0, nexta = 1, lasta = NA - 1, bufb = 0, nextb = 1, lastb = NB - 1;
    for (int kt = 0; kt < nk; ++kt) {
        uint32_t xa0, xa1, xb1, unused;
        step(bufa, bufb, 0, xa0, unused);
        step(bufa, bufb, 1, xa1, xb1);
        __builtin_amdgcn_s_setprio(1);
        static_for<F>([&](auto ii) __attribute__((always_inline)) {
            // blocks of B in the first rows, and one of A; the last rows have the operations
            // of those before the barrier too
            constexpr int i = decltype(ii)::value, nb = 2 * i < F ? PB : 0, w = AFTER + i, w2 = w + BR;
            constexpr int n = Window::n(w), n2 = i >= F - BR ? Window::n(w2) : 0;
            row(ii, fb[0], std::integral_constant<int, nb + 1 + n + n2>{}, [&](auto k) __attribute__((always_inline)) {
                constexpr int o = decltype(k)::value, q = o - nb - 1;
                if constexpr (o < nb) {
                    fb[1][PB * i + o] = b.read(xb1, PB * i + o);
                } else if constexpr (q < 0) {
                    if constexpr (i == 0)
                        fa[F - 1] = a.read(xa0, F - 1);
                    else
                        fa[i - 1] = a.read(xa1, i - 1);
                } else if constexpr (q < n) {
                    window(std::integral_constant<int, w>{}, std::integral_constant<int, q>{}, lasta, lastb, (kt + 2) * C::BK);
                } else {
                    window(std::integral_constant<int, w2>{}, std::integral_constant<int, q - n>{}, lasta, lastb, (kt + 2) * C::BK);
                }
            });
        });
        uint32_t xan, xbn;
        static_for<F>([&](auto ii) __attribute__((always_inline)) {
            constexpr int i = decltype(ii)::value, after = i - BR;   // rows since the barrier
            if constexpr (after == 0) {
                // stage kt + 1 has landed
                if constexpr (OpA::DMA && OpB::DMA)
                    __builtin_amdgcn_s_waitcnt(LL_VMCNT(LATER));
                else if constexpr (OpA::DMA || OpB::DMA)
                    __builtin_amdgcn_s_waitcnt(LL_VMCNT(0));
                asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            }
            if constexpr (after < 0) {
                row(ii, fb[1], std::integral_constant<int, 4>{}, [&](auto k) __attribute__((always_inline)) {
                    constexpr int o = decltype(k)::value;
                    if constexpr (i == 0 && o == 0)
                        fa[F - 1] = a.read(xa1, F - 1);
                    else if constexpr (i == 0 && o == 1)
                        step(nexta, nextb, 0, xan, xbn);
                    else if constexpr (i == BR - 1 && o == 2)
                        a.aim((kt + NA) * C::BK, tid);
                    else if constexpr (i == BR - 1 && o == 3)
                        b.aim((kt + NB + AHEAD) * C::BK, tid);
                });
            } else {
                // (after the last stage what is read here is of no use)
                constexpr int nb = 2 * after < F ? PB : 0, na = after < BR - 1 ? 2 : 1;   // (a block of A of the rows before the barrier)
                row(ii, fb[1], std::integral_constant<int, nb + na + Window::n(after)>{}, [&](auto k) __attribute__((always_inline)) {
                    constexpr int o = decltype(k)::value, q = o - nb - na;
                    if constexpr (o < nb)
                        fb[0][PB * after + o] = b.read(xbn, PB * after + o);
                    else if constexpr (o == nb)
                        fa[i - 1] = a.read(xan, i - 1);
                    else if constexpr (q < 0)
                        fa[after] = a.read(xan, after);
                    else
                        window(std::integral_constant<int, after>{}, std::integral_constant<int, q>{}, bufa, bufb, (kt + 3) * C::BK);
                });
            }
        });
        __builtin_amdgcn_s_setprio(0);
        const int donea = bufa, doneb = bufb;
        bufa = nexta, bufb = nextb;
        nexta = NA == 3 ? lasta : donea, nextb = NB == 3 ? lastb : doneb;
        lasta = NA == 3 ? donea : nexta, lastb = NB == 3 ? doneb : nextb;
    }
    if constexpr (WPE == 1)
        settle(acc);

    // The write-back, 64 x 64 of the wave's block at a time through its own part of the LDS,
    // a quarter of those rows a turn of a loop: what depends on the quarter is its stores
    // into LDS alone, and the rest is code once. (All of it unrolled is more than the
    // instruction cache holds, 2.3 ms for a product that takes 0.2; eight rows at a time one
    // after the other, with a wait for each, took 37 us a tile of 256 x 256.)
    __builtin_amdgcn_s_waitcnt(LL_VMCNT(0));   // (the zeros past the last stage are on their way into the ring)
    __syncthreads();                           // nobody reads the ring any more
    float *turn = reinterpret_cast<float *>(lds_bytes) + wave * 64 * PITCH;
    const int rl = lane >> 3, cl = (lane & 7) * 8;
    const void *more = job.part != nullptr ? nullptr : OP == L16_FWD ? p.R : p.beta != 0.0f ? p.C : nullptr;
    const int64_t more_ld = OP == L16_FWD ? p.ldr : p.ldc;
    constexpr int QN = WTN / 64, QUARTERS = WTM / 64 * QN;
#pragma unroll 1
    for (int quarter = 0; quarter < QUARTERS; ++quarter) {
        static_for<QUARTERS>([&](auto qq) __attribute__((always_inline)) {
            constexpr int Q = decltype(qq)::value;
            if (quarter == Q) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        *reinterpret_cast<f32x4 *>(turn + (16 * i + (lane & 15)) * PITCH + 16 * j + 4 * (lane >> 4)) =
                            acc[4 * (Q / QN) + i][4 * (Q % QN) + j];
                asm volatile("; quarter %0" ::"n"(Q) : "memory");   // (merged branches would index acc, in memory)
            }
        });
        const int col = n0 + wn * WTN + 64 * (quarter % QN) + cl, n = p.N - col;
        const int row0 = m0 + wm * WTM + 64 * (quarter / QN) + rl;
        float bias[8];
        if constexpr (OP == L16_FWD)
            load_row<LL_TYPE_F32, 8>(p.bias + (int64_t)g * p.N + col, p.bias != nullptr ? n : 0, bias);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // (the wave's own rows: no barrier)
        // U eight-row groups from row 8 q of the 64 on
        auto rows = [&](auto whole, auto uu, int q) __attribute__((always_inline)) {
            constexpr bool WHOLE = decltype(whole)::value;   // all of them inside C
            constexpr int U = decltype(uu)::value;
            float v[U][8], r[U][8];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int row = row0 + 8 * (q + u);
                if (more != nullptr) {
                    load8<BF16>(p.ctype, more, c_off + (int64_t)row * more_ld + col, WHOLE ? 8 : row < m_end ? n : 0, r[u]);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        r[u][e] = 0.0f;
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const f32x4 lo = *reinterpret_cast<const f32x4 *>(turn + (8 * (q + u) + rl) * PITCH + cl);
                const f32x4 hi = *reinterpret_cast<const f32x4 *>(turn + (8 * (q + u) + rl) * PITCH + cl + 4);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[u][e] = lo[e], v[u][4 + e] = hi[e];
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int row = row0 + 8 * (q + u);
                const bool live = WHOLE || (row < m_end && n > 0);
                if (OP != L16_DW && job.part != nullptr) {
                    if (live)
                        store_row<LL_TYPE_F32, 8>(job.part + (int64_t)row * p.N + col, WHOLE ? 8 : n, v[u]);
                } else if constexpr (OP == L16_FWD) {
                    finish_fwd<BF16>(p, v[u], bias, r[u], row, col, WHOLE ? 8 : n, live);
                } else if (live) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[u][e] = __builtin_fmaf(p.beta, r[u][e], v[u][e]);   // (r is 0 where beta is)
                    store8<BF16>(p.ctype, p.C, c_off + (int64_t)row * p.ldc + col, WHOLE ? 8 : n, v[u]);
                }
            }
        };
        // 32 rows at a time where all of them and the 64 columns exist, else eight
        const int first = m0 + wm * WTM + 64 * (quarter / QN);   // of the 64
        const bool whole_cols = n0 + wn * WTN + 64 * (quarter % QN) + 64 <= p.N;
#pragma unroll 1
        for (int q = 0; q < 8 && first + 8 * q < m_end;) {
            if (whole_cols && first + 8 * q + 32 <= m_end) {
                rows(std::true_type{}, std::integral_constant<int, 4>{}, q);
                q += 4;
            } else {
                rows(std::false_type{}, std::integral_constant<int, 1>{}, q);
                ++q;
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
}

// ---- kernels -----------------------------------------------------------------------

// One 128 x 128 tile a workgroup, two workgroups a CU: products that do not fill the CUs with
// larger ones, and rows off 16 bytes. With shares (of those whose groups are of C's rows) a
// workgroup has a part of K, and launch_l16_join adds the parts (dX of 16 x 11008 x 4096 82 us
// whole, 24 in shares).
template <int OP, bool BF16, int SA, int SB, bool VEC>
__global__ void __launch_bounds__(Block::NT) __attribute__((amdgpu_waves_per_eu(2, 2))) l16_small_kernel(L16Params p)
{
    constexpr int BM = 128, NB = Operand<BF16, BM, SB, VEC>::DMA ? 3 : 2;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[tile_lds<BM, BM, 2, NB>()];
    Job job{0, 0, p.M, 0, 0, p.K, 0, nullptr};
    int tm, tn;
    if constexpr (OP == L16_DW) {
        const int per = p.tiles_m * p.tiles_n, id = block_index(blockIdx.x, per * p.groups.n);
        job.g = id / per;
        tile_at(id - job.g * per, p.tiles_m, p.tiles_n, tm, tn);
        group_rows(p.groups, p.K, job.g, job.k_begin, job.klen);
        job.klen -= job.k_begin;
        job.m0 = tm * BM;
        job.c_off = (int64_t)job.g * p.stride_c;
    } else {
        // rows of tiles of all groups; workgroups past the last have nothing to do
        Chunk c{};
        const int total = find_chunk(p.groups, p.M, BM, -1, c) * p.tiles_n;
        if ((int)blockIdx.x >= total)
            return;
        const int id = block_index(blockIdx.x, total);
        find_chunk(p.groups, p.M, BM, id / p.tiles_n, c);
        tile_at(id - c.group_first * p.tiles_n, cdiv(c.end - c.begin, BM), p.tiles_n, tm, tn);
        job.g = c.group;
        job.m0 = c.begin + tm * BM;
        job.m_end = c.end;
        if (p.shares > 1) {   // this one's whole stages of K, which may be none
            const int each = cdiv(cdiv(p.K, Block::BK), p.shares) * Block::BK;
            job.k_begin = min(p.K, (int)blockIdx.y * each);
            job.klen = min(p.K - job.k_begin, each);
            job.part = p.ws + (int64_t)blockIdx.y * p.M * p.N;
        }
    }
    job.n0 = tn * BM;
    l16_tile<OP, BF16, BM, BM, 2, 2, NB, SA, SB, VEC>(p, job, lds);
}

// What is left after the rounds in which every CU has a 256 x 256 tile, in tiles of 256 x 256, of
// 128 x 256 or of 128 x 128, whichever takes the fewest rounds' time: measured, a round of the
// smaller ones takes 0.58 and 0.41 of a round of the large. `large` of them are left, and `halves`
// pieces of 128 x 256 beside them.
__host__ __device__ inline int piece_split(int64_t large, int64_t halves, int cus, float &cost)
{
    const auto rounds = [cus](int64_t n) { return (float)((n + cus - 1) / cus); };
    const float c1 = rounds(large) + 0.58f * rounds(halves), c2 = 0.58f * rounds(2 * large + halves),
                c4 = 0.41f * rounds(4 * large + 2 * halves);
    cost = c1 <= c2 && c1 <= c4 ? c1 : c2 <= c4 ? c2 : c4;
    return c1 <= c2 && c1 <= c4 ? 1 : c2 <= c4 ? 2 : 4;
}

// Tiles of 256 x 256, one a CU, as many workgroups as there are CUs, each of which takes every
// gridDim.x-th tile. A group's last rows are a tile of 128 rows where no more are left, and what
// does not fill a round is cut up (piece_split).
template <int OP, bool BF16, int SA, int SB>
__global__ void __launch_bounds__(Block::NT) __attribute__((amdgpu_waves_per_eu(1, 1))) l16_large_kernel(L16Params p)
{
    constexpr bool DMA_B = Operand<BF16, 256, SB, true>::DMA;
    constexpr int NB = DMA_B ? 3 : 2;
    constexpr int large = tile_lds<256, 256, 2, NB>(), half = tile_lds<128, 256, 3, NB>();
    __shared__ __attribute__((aligned(1024))) uint8_t lds[large > half ? large : half];
    const int cus = (int)gridDim.x;
    const auto count_large = [](int rows) { return (rows + 127) / 256; };
    const auto count_half = [](int rows) { return (rows & 255) != 0 && (rows & 255) <= 128 ? 1 : 0; };
    int n_large, n_half = 0;
    if constexpr (OP == L16_DW) {
        n_large = p.tiles_m * p.tiles_n * p.groups.n;
    } else {
        Chunk c{};
        n_large = find_chunk_by(p.groups, p.M, count_large, -1, c) * p.tiles_n;
        n_half = find_chunk_by(p.groups, p.M, count_half, -1, c) * p.tiles_n;
    }
    float cost;
    const int left = n_large % cus, split = piece_split(left, n_half, cus, cost);
    const int whole = split == 1 ? n_large : n_large - left;   // in one piece
    const int pieces = (split == 1 ? n_half : 2 * left + n_half) * (split == 4 ? 2 : 1), total = whole + pieces;
    for (int round = 0; round < total; round += cus) {
        const int here = min(cus, total - round);
        if ((int)blockIdx.x >= here)
            break;
        // (another part of each round for a CU: groups' lengths, which weight gradients run over,
        // even out; an XCD's tiles stay together)
        const int id = round + (block_index(blockIdx.x, here) + round / cus * (3 * cus / 8)) % here;
        // the tile, and for a piece its half (of the rows) and quarter (of the columns)
        const int piece = id - whole, q = split == 4 ? piece / 2 : piece, cut = split == 1 ? 0 : 2 * left;
        const int tile = piece < 0 ? id : q < cut ? whole + q / 2 : -1;
        Job job{0, 0, p.M, 0, 0, p.K, 0, nullptr};
        int tm = 0, tn = 0;
        if constexpr (OP == L16_DW) {
            const int per = p.tiles_m * p.tiles_n;
            job.g = tile / per;
            tile_at(tile - job.g * per, p.tiles_m, p.tiles_n, tm, tn);
            group_rows(p.groups, p.K, job.g, job.k_begin, job.klen);
            job.klen -= job.k_begin;
            job.c_off = (int64_t)job.g * p.stride_c;
            job.m0 = tm * 256;
        } else {
            Chunk c{};
            if (tile >= 0) {
                find_chunk_by(p.groups, p.M, count_large, tile / p.tiles_n, c);
                tile_at(tile - c.group_first * p.tiles_n, count_large(c.end - c.begin), p.tiles_n, tm, tn);
                job.m0 = c.begin + tm * 256;
            } else {
                find_chunk_by(p.groups, p.M, count_half, (q - cut) / p.tiles_n, c);
                tn = (q - cut) % p.tiles_n;
                job.m0 = c.end - ((c.end - c.begin) & 255);
            }
            job.g = c.group;
            job.m_end = c.end;
        }
        job.n0 = tn * 256;
        if (piece >= 0) {
            if (tile >= 0)
                job.m0 += 128 * (q & 1);
            if (split == 4)
                job.n0 += 128 * (piece & 1);
            if (job.m0 >= job.m_end || job.n0 >= p.N)
                continue;
        }
        // nobody reads the tile before this one's rows in LDS any more (its stores may be on their way)
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (piece < 0)
            l16_tile<OP, BF16, 256, 256, 1, 2, NB, SA, SB, true>(p, job, lds);
        else if (split != 4)
            l16_tile<OP, BF16, 128, 256, 1, 3, NB, SA, SB, true>(p, job, lds);
        else
            l16_tile<OP, BF16, 128, 128, 1, 3, NB, SA, SB, true>(p, job, lds);
    }
}

// ---- launches -----------------------------------------------------------------------

// Whether large tiles take less time: n_large and n_half of them and of their halves, against
// n_small of 128 x 128. Two small ones a CU take 0.62 of a large one's time; beside its stages
// a tile costs five of them, and the first large one four more, which no other workgroup covers.
// (Measured, large against small: 4096 x 4096 x 512 33 and 28 us, 2048 x 11008 x 4096 220 and 239,
// 16 weights' gradients of 4096 x 2048 over 512 rows each 219 and 325.)
inline bool prefer_large(int64_t n_large, int64_t n_half, int64_t n_small, int k, int cus)
{
    float rest;
    piece_split(n_large % cus, n_half, cus, rest);
    const float stages = (float)cdiv(k, Block::BK) + 5.0f;
    return ((float)(n_large / cus) + rest) * stages + 4.0f <= (float)((n_small + 2 * cus - 1) / (2 * cus)) * 0.62f * stages;
}

// The same of a product: rows of C by groups (taken as equally long), or groups of the contracted rows.
inline bool rows_prefer_large(int M, int N, int K, int groups, int cus)
{
    const int g = groups < M ? groups : M, each = cdiv(M, g), tn = cdiv(N, 256), last = each & 255;
    return ((int64_t)(M / 256) + g) * tn < (1 << 29) &&   // (tiles are counted in 32 bits)
           prefer_large((int64_t)g * ((each + 127) / 256) * tn, last != 0 && last <= 128 ? (int64_t)g * tn : 0,
                        (int64_t)g * cdiv(each, 128) * cdiv(N, 128), K, cus);
}
inline bool weight_prefers_large(int M, int N, int rows, int groups, int cus)
{
    const int64_t n_large = (int64_t)groups * cdiv(M, 256) * cdiv(N, 256);
    return n_large < (1 << 29) &&
           prefer_large(n_large, 0, (int64_t)groups * cdiv(M, 128) * cdiv(N, 128), rows > groups ? cdiv(rows, groups) : 1, cus);
}

// In how many shares of K such a product takes the least time, by the same measure: a share is
// eight stages at least, and the join costs four stages' time and the sums' way through memory
// (1.4 us a stage, 5 bytes a ps). Whole and shared: 16 x 1024 over 4096 12.9 and 12.5 us, 130 x 72
// over 1000 14.8 and 13.2, 512 x 4096 over 4096 38 and 34, 129 x 128 over 16384 120 and 19; whole by the
// rule at 1024 x 4096 over 4096 and 512 x 4096 over 1024.
inline int rows_shares(int M, int N, int K, int groups, int cus)
{
    const int g = groups < M ? groups : M;
    const int64_t tiles = (int64_t)g * cdiv(cdiv(M, g), 128) * cdiv(N, 128);
    const int stages = cdiv(K, Block::BK);
    int64_t s = 2 * cus / tiles;
    s = s < stages / 8 ? s : stages / 8;
    s = s < 16 ? s : 16;
    if (s < 2)
        return 1;
    const float bytes = 8.0f * (float)s * (float)M * (float)N;
    const float shared = 0.62f * ((float)cdiv(stages, (int)s) + 5.0f) + 4.0f + bytes * (1e-6f / 5.0f / 1.4f);
    const int each = cdiv(M, g), tn = cdiv(N, 256), last = each & 255;
    float rest;
    piece_split((int64_t)g * ((each + 127) / 256) * tn, last != 0 && last <= 128 ? (int64_t)g * tn : 0, cus, rest);
    const float large = rest * ((float)stages + 5.0f) + 4.0f, small = 0.62f * ((float)stages + 5.0f);
    return shared < large && shared < small ? (int)s : 1;
}

template <int OP, bool BF16, int SA, int SB>
hipError_t launch_large(L16Params p, int cus, hipStream_t s)
{
    p.tiles_m = cdiv(p.M, 256);
    p.tiles_n = cdiv(p.N, 256);
    hipLaunchKernelGGL((l16_large_kernel<OP, BF16, SA, SB>), dim3((unsigned)cus), dim3(Block::NT), 0, s, p);
    return hipGetLastError();
}

template <int OP, bool BF16, int SA, int SB, bool VEC>
hipError_t launch_small(L16Params p, int64_t rows, hipStream_t s)
{
    p.tiles_m = cdiv(p.M, 128);
    p.tiles_n = cdiv(p.N, 128);
    const int64_t tiles = rows * p.tiles_n;
    if (tiles > max_grid_x(Block::NT))
        return hipErrorInvalidValue;
    hipLaunchKernelGGL((l16_small_kernel<OP, BF16, SA, SB, VEC>), dim3((unsigned)tiles, (unsigned)(OP == L16_DW ? 1 : p.shares)),
                       dim3(Block::NT), 0, s, p);
    return OP != L16_DW && p.shares > 1 ? launch_l16_join(BF16, p, s) : hipGetLastError();
}

// The products whose groups are of C's rows. (Every group may end inside a tile.)
template <int OP, bool BF16, int SB>
hipError_t launch_rows(const L16Params &p, bool vec, int cus, hipStream_t s)
{
    const int g = p.groups.n < p.M ? p.groups.n : p.M;
    const int64_t rows = p.groups.offsets == nullptr ? cdiv(p.M, 128) : (int64_t)(p.M / 128) + g;
    if (!vec)
        return launch_small<OP, BF16, ROWS, SB, false>(p, rows, s);
    if (p.shares == 1 && rows_prefer_large(p.M, p.N, p.K, p.groups.n, cus))
        return launch_large<OP, BF16, ROWS, SB>(p, cus, s);
    return launch_small<OP, BF16, ROWS, SB, true>(p, rows, s);
}

}  // namespace l16
}  // namespace ll
