// Tile kernel of the products with a 4-bit microscaled operand (the operands'
// layout in the matrix instructions: gemm_mx4.hip).
//
// A workgroup computes a BM x BN tile of C, eight waves (256 x 256, one to a CU) or
// four (128 x 128, two to a CU), a wave's share in 16 x 16 blocks. Codes and 16-bit
// values go from memory straight into a ring of LDS stages (global_load_lds, rows of
// 128 bytes where the operand allows, 16-byte pieces XOR-swizzled so that 16 lanes
// read 16 different bank groups); operands that are not 16-byte aligned go through
// registers into the same stages. A stage is two steps of the matrix instruction
// (256 values of K in 4 bits, 64 with 16-bit A); a step's operands are read while the
// step before multiplies, and 16-bit A finds B decoded in registers.
//
// Scales are single bytes, 32 values apart: loaded stage by stage they cost as many
// requests as the codes. They come in panels of 16 a row instead, turned around in
// registers so that one LDS read gives a lane the scales of all its rows, which the
// instruction picks by byte.
//
// What bounds it: with both operands in 4 bits the rate at which L2 fills the CUs.
// 8192 x 8192 x K takes 48 us and 32.8 for every 1024 of K (512: 64, 2048: 109, 8192: 311, 3.5
// PFLOP/s; on inputs that change from pass to pass 336 to 341): 2.05 us a stage of 256 x 256,
// 64 KiB, 32 bytes a ns and CU, with the matrix cores busy 40 % of the time; a third
// stage, 128 x 256 tiles in three stages or twice as many workgroups were no faster. The
// 48 us are C's 268 MB, which one workgroup a CU does not write behind another tile's
// stages; they leave in whole rows of 256 bytes through LDS (in the instruction's 64-byte
// pieces 30 us more). A workgroup that fetches its next tile meanwhile has not been
// tried. LDS bank conflicts are 96 cycles a stage and 1024 an epilogue, 2.5 % of a tile's
// time. With bfloat16 A the matrix cores' power limit: 8192^3 773 us, 1.42 PFLOP/s, 2047 x
// 11008 x 4096 153 to 158 us.
#include "linear_layer.h"
#include "gemm_mx4.hpp"

#include <type_traits>
#include <utility>

namespace ll {

template <int... I, class F>
__device__ __forceinline__ void static_for_(std::integer_sequence<int, I...>, F f)
{
    (f(std::integral_constant<int, I>{}), ...);
}
// f(0), .., f(N - 1) with constants for arguments (an instruction's immediate
// cannot be a loop's variable).
template <int N, class F>
__device__ __forceinline__ void static_for(F f)
{
    static_for_(std::make_integer_sequence<int, N>{}, f);
}

// global_load_lds_dwordx4 from a scalar base and a lane's offset: this lane's 16
// bytes go to LDS byte lds_base + 16 * lane. As in common.hpp the caller counts
// the copies itself.
__device__ __forceinline__ void lds_dma_16(const uint8_t *base, uint32_t off, uint32_t lds_base)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(lds_base), "v"(off), "s"(base)
                 : "memory", "m0");
}

// Bytes of LDS a tile takes: the ring's stages and two panels of scales.
template <int A>
constexpr int tile_lds(int BM, int BN, int steps, int nbuf)
{
    const int bk = steps * (A == MXA_MX4 ? 128 : 32);
    return nbuf * (BM * (A == MXA_MX4 ? bk / 2 : bk * 2) + BN * bk / 2) + 2 * 16 * ((A == MXA_MX4 ? BM : 0) + BN);
}

// The BM x BN block of C from row m0 and column n0 on, by WGM x WGN waves. For
// 16-bit A it returns false, with nothing stored, where a scale is past what A's
// type can take (of bfloat16: the far ones).
template <int A, int BM, int BN, int STEPS, int NBUF, int WGM, int WGN, bool DMA>
__device__ __forceinline__ bool mx4_tile(const MxParams &p, int64_t m0, int64_t n0, uint8_t *raw)
{
    constexpr bool MX = A == MXA_MX4;
    constexpr int NW = WGM * WGN, NT = 64 * NW;
    constexpr int SK = MX ? 128 : 32, BK = STEPS * SK;     // k-values of a step, of a stage
    constexpr int AR = MX ? BK / 2 : 2 * BK, BR = BK / 2;  // bytes of a row in a stage
    constexpr int ACPR = AR / 16, BCPR = BR / 16;          // its 16-byte chunks
    constexpr int NB = BK / kMxBlock;                      // its scales
    constexpr int WTM = BM / WGM, WTN = BN / WGN, FM = WTM / 16, FN = WTN / 16;
    constexpr int A_STAGE = BM * AR, B_STAGE = BN * BR;
    constexpr int PS = 16 / NB;                            // stages of a panel of 16 scales a row
    constexpr int SA_PANEL = MX ? BM * 16 : 0, SB_PANEL = BN * 16;
    constexpr int COPIES_A = A_STAGE / 1024 / NW, COPIES_B = B_STAGE / 1024 / NW;   // of 1 KiB, a wave's
    constexpr int COPIES = COPIES_A + COPIES_B;
    constexpr int ARPC = 1024 / AR, BRPC = 1024 / BR;      // rows of a copy
    constexpr int CHUNKS = (A_STAGE + B_STAGE) / 16 / NT;  // of 16 bytes, a thread's
    constexpr int SROWS = (MX ? BM : 0) + BN;              // rows of scales
    static_assert(COPIES_A * 1024 * NW == A_STAGE && COPIES_B * 1024 * NW == B_STAGE, "whole copies");
    static_assert((COPIES_A * ARPC) % 16 == 0 && (COPIES_B * BRPC) % 16 == 0, "the swizzles repeat every 16 rows");
    static_assert(PS * NB == 16 && PS >= 2, "whole panels");
    static_assert(STEPS % 2 == 0, "a stage leaves the register sets as it found them");
    static_assert(NBUF == 2 || DMA, "chunks through registers take two stages");
    static_assert(DMA || (A_STAGE / 16) % NT == 0, "a thread's chunk is A's or B's for the whole workgroup");
    typedef typename std::conditional<MX, u32x4, uint32_t>::type BFrag;   // a block, or 8 of its values

    struct Lds {
        uint8_t a[NBUF][A_STAGE], b[NBUF][B_STAGE], s[2][SA_PANEL + SB_PANEL];
    };
    static_assert(sizeof(Lds) == tile_lds<A>(BM, BN, STEPS, NBUF), "as the kernel allots it");
    Lds &lds = *reinterpret_cast<Lds *>(raw);
    auto &As = lds.a;
    auto &Bs = lds.b;
    auto &Ss = lds.s;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WGN, wn = wave % WGN;
    const int g = lane >> 4, r16 = lane & 15;
    const int K = p.K;
    // The tile's first rows of A and B. With copies the last tile starts early
    // enough to be whole (M >= BM, N >= BN); the rows and columns that its
    // neighbour computes too are not stored.
    const int64_t ma = DMA && m0 + BM > p.M ? p.M - BM : m0, nb = DMA && n0 + BN > p.N ? p.N - BN : n0;
    const int mleft = (int)(p.M - ma < BM ? p.M - ma : BM), nleft = (int)(p.N - nb < BN ? p.N - nb : BN);
    const int nblk = (K - 1) / kMxBlock + 1;
    const int nk = K / BK;   // whole stages: at least one
    const uint8_t *abase = p.A + ma * p.lda, *bbase = p.B + nb * p.ldb;
    const uint8_t *sabase = MX ? p.SA + ma * p.ldsa : nullptr, *sbbase = p.SB + nb * p.ldsb;

    // ---- copies: copy j of this wave covers the RPC rows from
    // (wave * COPIES + j) * RPC on; lane l fills row l / CPR, slot l % CPR with
    // the chunk that the swizzle puts there. Addresses are a scalar base and a
    // lane's 32-bit offset.
    constexpr int NV = AR == 128 ? 2 : 1, NVB = BR == 128 ? 2 : 1;   // rows of 128 bytes: eight a copy, so two swizzles
    static_assert(AR <= 128 && BR <= 128, "a copy's rows take one of two swizzles");
    uint32_t aoff[NV], boff[NVB];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int ch = (lane % ACPR) ^ swz<AR>(v * ARPC + lane / ACPR);
        aoff[v] = (uint32_t)(lane / ACPR) * (uint32_t)p.lda + ch * 16;
    }
#pragma unroll
    for (int v = 0; v < NVB; ++v) {
        const int ch = (lane % BCPR) ^ swz<BR>(v * BRPC + lane / BCPR);
        boff[v] = (uint32_t)(lane / BCPR) * (uint32_t)p.ldb + ch * 16;
    }
    const uint32_t as_base = lds_addr(&As[0][0]), bs_base = lds_addr(&Bs[0][0]);
    const int arow = wave * (COPIES_A * ARPC), brow = wave * (COPIES_B * BRPC);   // of copy 0
    const uint8_t *anext = abase + arow * p.lda, *bnext = bbase + brow * p.ldb, *src = nullptr;   // of the next stage
    const int64_t astep = ARPC * p.lda, bstep = BRPC * p.ldb;
    // Copies 0 .. COPIES - 1 of a stage, in turn.
    auto copy = [&](int buf, auto cc) __attribute__((always_inline)) {
        constexpr int c = decltype(cc)::value, j = c - COPIES_A;
        if constexpr (c < COPIES_A) {
            src = c == 0 ? anext : src + astep;
            lds_dma_16(src, aoff[c & (NV - 1)], as_base + buf * A_STAGE + (arow + c * ARPC) * AR);
        } else {
            src = j == 0 ? bnext : src + bstep;
            lds_dma_16(src, boff[j & (NVB - 1)], bs_base + buf * B_STAGE + (brow + j * BRPC) * BR);
        }
        asm volatile("" : "+s"(src));   // (a running sum: the compiler would keep each copy's base in registers)
        if constexpr (c == COPIES - 1)
            anext += AR, bnext += BR;
    };

    // ---- the same through registers, at any alignment: chunk c of this thread
    u32x4 held[DMA ? 1 : CHUNKS];
    auto load_chunks = [&](int kt) __attribute__((always_inline)) {
#pragma unroll
        for (int c = 0; c < (DMA ? 0 : CHUNKS); ++c) {
            int i = c * NT + tid;
            if (c * NT < A_STAGE / 16) {
                const int row = i / ACPR, ch = i % ACPR;
                const uint8_t *src = abase + (row < mleft ? row : mleft - 1) * p.lda;
                held[c] = MX ? load_block<true>(src, (int64_t)kt * NB + ch, K)
                             : load_halves<true>(src, (int64_t)kt * BK + ch * 8, K);
            } else {
                i -= A_STAGE / 16;
                const int row = i / BCPR, ch = i % BCPR;
                held[c] = load_block<true>(bbase + (row < nleft ? row : nleft - 1) * p.ldb, (int64_t)kt * NB + ch, K);
            }
        }
    };
    auto store_chunks = [&](int buf) __attribute__((always_inline)) {
#pragma unroll
        for (int c = 0; c < (DMA ? 0 : CHUNKS); ++c) {
            int i = c * NT + tid;
            if (c * NT < A_STAGE / 16) {
                const int row = i / ACPR, ch = i % ACPR;
                *reinterpret_cast<u32x4 *>(&As[buf][row * AR + (ch ^ swz<AR>(row)) * 16]) = held[c];
            } else {
                i -= A_STAGE / 16;
                const int row = i / BCPR, ch = i % BCPR;
                *reinterpret_cast<u32x4 *>(&Bs[buf][row * BR + (ch ^ swz<BR>(row)) * 16]) = held[c];
            }
        }
    };

    // ---- scales: through registers, at any alignment, in panels of 16 a row
    // (PS stages), two panels in LDS. A wave takes 64 rows: lane l the rows
    // l / 4 + 16 i and their blocks 4 (l % 4) .. +3, and turns these 4 x 4 bytes
    // around, so that a lane of the products finds the scales of its rows 16
    // apart side by side: [wave row][block][row % 16][row / 16].
    static_assert((!MX || WTM % 64 == 0) && WTN % 64 == 0 && SROWS <= NT,
                  "a wave's rows of scales are one operand's and one wave row's");
    const bool s_any = wave * 64 < SROWS, s_is_a = MX && wave * 64 < BM;
    const int s_row = s_is_a ? wave * 64 : wave * 64 - (SROWS - BN);
    const uint8_t *s_base = s_is_a ? sabase + s_row * p.ldsa : sbbase + s_row * p.ldsb;
    const int64_t s_ld = s_is_a ? p.ldsa : p.ldsb;
    const uint32_t s_off = (uint32_t)(lane >> 2) * (uint32_t)s_ld + (lane & 3) * 4;
    u32x4 sheld = {0u, 0u, 0u, 0u};
    bool wide = false;   // this thread saw a scale that binary16 cannot take
    auto load_panel = [&](int b0) __attribute__((always_inline)) {
        if (!s_any)
            return;
        const uint8_t *from = s_base + min(b0, nblk - 16);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t v;
            if constexpr (DMA) {
                __builtin_memcpy(&v, from + 16 * j * s_ld + s_off, 4);
            } else {
                const int r = min((lane >> 2) + 16 * j, (s_is_a ? mleft : nleft) - 1 - s_row);
                __builtin_memcpy(&v, from + r * s_ld + (lane & 3) * 4, 4);
            }
            sheld[j] = v;
        }
    };
    int origin = 0, panel = 1;   // the current panel's first block (the last one ends with the row: K >= 512), its buffer
    auto store_panel = [&](int b0) __attribute__((always_inline)) {
        origin = min(b0, nblk - 16);
        panel ^= 1;
        if (!s_any)
            return;
        const u32x4 v = sheld;
        if constexpr (A == MXA_F16)
#pragma unroll
            for (int j = 0; j < 16; ++j)
                wide |= !f16_scale_ok(v[j / 4] >> (8 * (j % 4)) & 0xffu);
        const uint32_t lo01 = __builtin_amdgcn_perm(v[1], v[0], 0x05010400u), hi01 = __builtin_amdgcn_perm(v[1], v[0], 0x07030602u);
        const uint32_t lo23 = __builtin_amdgcn_perm(v[3], v[2], 0x05010400u), hi23 = __builtin_amdgcn_perm(v[3], v[2], 0x07030602u);
        const u32x4 w = {__builtin_amdgcn_perm(lo23, lo01, 0x05040100u), __builtin_amdgcn_perm(lo23, lo01, 0x07060302u),
                         __builtin_amdgcn_perm(hi23, hi01, 0x05040100u), __builtin_amdgcn_perm(hi23, hi01, 0x07060302u)};
        auto put = [&](uint8_t *dst, auto wt) __attribute__((always_inline)) {
            constexpr int WT = decltype(wt)::value, F = WT / 16;
            dst += ((s_row / WT * 16 + 4 * (lane & 3)) * 16 + (lane >> 2)) * F + s_row % WT / 16;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<uint32_t *>(dst + j * 16 * F) = w[j];
        };
        if (s_is_a)
            put(Ss[panel], std::integral_constant<int, WTM>{});
        else
            put(Ss[panel] + SA_PANEL, std::integral_constant<int, WTN>{});
    };

    // ---- operands of a step
    struct Ops {
        u32x4 a[FM];
        BFrag b[FN];
        uint32_t sa[MX ? (FM + 3) / 4 : 1], sb[(FN + 3) / 4];
    };
    // (rows 16 apart have the same swizzle)
    const int sa_lane = ((wm * 16 + g) * 16 + r16) * FM;
    const int sb_lane = SA_PANEL + ((wn * 16 + (MX ? g : 0)) * 16 + r16) * FN;
    const int a_row = (wm * WTM + r16) * AR, b_row = (wn * WTN + r16) * BR;
    auto read_ops = [&](int buf, int kt, auto ss, Ops &o) __attribute__((always_inline)) {
        constexpr int s = decltype(ss)::value;
        const int blk = kt * NB + s * (SK / kMxBlock) - origin;   // of the panel's 16
        if constexpr (MX)
            __builtin_memcpy(o.sa, __builtin_assume_aligned(&Ss[panel][sa_lane + blk * 16 * FM], FM), FM);
        __builtin_memcpy(o.sb, __builtin_assume_aligned(&Ss[panel][sb_lane + blk * 16 * FN], FN), FN);
        const int bc = MX ? ((4 * s + g) ^ swz<BR>(r16)) * 16 : (s ^ swz<BR>(r16)) * 16 + g * 4;
#pragma unroll
        for (int f = 0; f < FN; ++f)
            o.b[f] = *reinterpret_cast<const BFrag *>(&Bs[buf][b_row + bc + f * 16 * BR]);
        const int ac = ((4 * s + g) ^ swz<AR>(r16)) * 16;
#pragma unroll
        for (int f = 0; f < FM; ++f)
            o.a[f] = *reinterpret_cast<const u32x4 *>(&As[buf][a_row + ac + f * 16 * AR]);
    };

    f32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    // The products of a step; `between` is called after each of the FN columns of
    // blocks. B stands first in the instruction, so that a lane gets one row
    // of C and four neighbouring columns of it.
    auto multiply = [&](const Ops &o, auto between) __attribute__((always_inline)) {
        if constexpr (MX) {
            static_for<FN>([&](auto nn) __attribute__((always_inline)) {
                constexpr int n = decltype(nn)::value;
                static_for<FM>([&](auto mm) __attribute__((always_inline)) {
                    constexpr int m = (n & 1) ? FM - 1 - decltype(mm)::value : decltype(mm)::value;
                    acc[m][n] = mma_mx4<n & 3, m & 3>(o.b[n], o.a[m], acc[m][n], (int)o.sb[n / 4], (int)o.sa[m / 4]);
                });
                between(nn);
            });
        } else {
            auto scale = [&](int n) __attribute__((always_inline)) { return __builtin_bit_cast(float, (o.sb[n / 4] >> (8 * (n & 3)) & 0xffu) << 23); };
            static_for<FN>([&](auto nn) __attribute__((always_inline)) {
                constexpr int n = decltype(nn)::value;
                const u32x4 b = decode8<A == MXA_BF16>(o.b[n], scale(n));
#pragma unroll
                for (int i = 0; i < FM; ++i) {
                    const int m = (n & 1) ? FM - 1 - i : i;
                    acc[m][n] = A == MXA_BF16 ? mma_bf16(b, o.a[m], acc[m][n]) : mma_f16(b, o.a[m], acc[m][n]);
                }
                between(nn);
            });
        }
    };

    // The products issued so far stay before this point: left alone, the compiler
    // moves them behind the barrier and keeps their operands alive.
    auto pin = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int m = 0; m < FM; ++m)
#pragma unroll
            for (int n = 0; n < FN; ++n)
                asm volatile("" : "+v"(acc[m][n]));
    };

    // ---- pipeline: a ring of NBUF stages and two register sets. A step's
    // operands are read while the previous step's products run. The stage's
    // barrier stands before its last step, whose operands are then in
    // registers: it publishes stage kt + 1 and frees stage kt's buffer, which is
    // refilled at once with stage kt + NBUF.
    auto fetch = [&](int buf) __attribute__((always_inline)) {
        static_for<COPIES>([&](auto c) __attribute__((always_inline)) { copy(buf, c); });
    };
    // Stage kt has landed: the copies of at most NBUF - 2 later ones are in flight.
    auto wait_stage = [&](int kt) __attribute__((always_inline)) {
        if (NBUF > 2 && kt + NBUF - 2 < nk)
            __builtin_amdgcn_s_waitcnt(LL_VMCNT((NBUF - 2) * COPIES));
        else
            __builtin_amdgcn_s_waitcnt(LL_VMCNT(0));
    };
    Ops ops[2];
    load_panel(0);
    if constexpr (DMA) {   // (the compiler's wait for the panel is one for these copies too)
#pragma unroll
        for (int st = 0; st < NBUF; ++st)
            if (st < nk)
                fetch(st);
    } else {
        load_chunks(0);
        store_chunks(0);
        if (nk > 1)
            load_chunks(1);
    }
    store_panel(0);
    __builtin_amdgcn_s_waitcnt(LL_VMCNT(0));
    __syncthreads();
    read_ops(0, 0, std::integral_constant<int, 0>{}, ops[0]);
    int buf = 0;
    // The refill's copies follow the first columns of products, so that the matrix
    // cores do not wait through one burst of them.
    constexpr int CCOLS = FN < 2 ? 1 : 2;
    auto body = [&](auto more, int kt) __attribute__((always_inline)) {
        constexpr bool REFILL = decltype(more)::value;   // there is a stage kt + NBUF
        const int next = buf == NBUF - 1 ? 0 : buf + 1;
        static_for<STEPS - 1>([&](auto ss) __attribute__((always_inline)) {
            constexpr int s = decltype(ss)::value;
            read_ops(buf, kt, std::integral_constant<int, s + 1>{}, ops[(s + 1) & 1]);
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_setprio(1);
            multiply(ops[s & 1], [](auto) {});
            __builtin_amdgcn_s_setprio(0);
            pin();
        });
        if (REFILL || kt + 1 < nk) {
            if constexpr (DMA)
                wait_stage(kt + 1);
            else
                store_chunks(next);
            if ((kt + 1) % PS == 0)
                store_panel((kt + 1) * NB);
        }
        __syncthreads();
        if (REFILL || kt + 1 < nk)
            read_ops(next, kt + 1, std::integral_constant<int, 0>{}, ops[0]);
        if ((kt + 2) % PS == 0 && (REFILL || kt + 2 < nk))
            load_panel((kt + 2) * NB);
        if constexpr (REFILL && !DMA)
            load_chunks(kt + NBUF);
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(1);
        multiply(ops[1], [&](auto nn) __attribute__((always_inline)) {
            constexpr int n = decltype(nn)::value, PER = (COPIES + CCOLS - 1) / CCOLS;
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (REFILL && DMA && n < CCOLS)
                static_for<PER>([&](auto c) __attribute__((always_inline)) {
                    constexpr int i = n * PER + decltype(c)::value;
                    if constexpr (i < COPIES)
                        copy(buf, std::integral_constant<int, i>{});
                });
            __builtin_amdgcn_sched_barrier(0);
        });
        __builtin_amdgcn_s_setprio(0);
        pin();
        buf = next;
    };
    constexpr std::true_type refill{};
    constexpr std::false_type drain{};
    int kt = 0;
    for (; kt + NBUF < nk; ++kt)
        body(refill, kt);
    for (; kt < nk; ++kt)
        body(drain, kt);

    // ---- what K leaves past the whole stages: operands straight into registers
    for (int64_t blk0 = (int64_t)nk * NB; blk0 < nblk; blk0 += SK / kMxBlock) {
        Ops &o = ops[0];
        const int64_t blk = blk0 + (MX ? g : 0);
#pragma unroll
        for (int i = 0; i < (FN + 3) / 4; ++i)
            o.sb[i] = 0;
#pragma unroll
        for (int f = 0; f < FN; ++f) {
            const int row = min(wn * WTN + f * 16 + r16, nleft - 1);
            const u32x4 v = load_block<true>(bbase + row * p.ldb, blk, K);
            if constexpr (MX)
                o.b[f] = v;
            else
                o.b[f] = g < 2 ? (g == 0 ? v[0] : v[1]) : (g == 2 ? v[2] : v[3]);
            o.sb[f / 4] |= (blk < nblk ? (uint32_t)sbbase[row * p.ldsb + blk] : 127u) << (8 * (f % 4));
        }
        if constexpr (MX) {
#pragma unroll
            for (int i = 0; i < (FM + 3) / 4; ++i)
                o.sa[i] = 0;
        }
#pragma unroll
        for (int f = 0; f < FM; ++f) {
            const int row = min(wm * WTM + f * 16 + r16, mleft - 1);
            if constexpr (MX) {
                o.a[f] = load_block<true>(abase + row * p.lda, blk, K);
                o.sa[f / 4] |= (blk < nblk ? (uint32_t)sabase[row * p.ldsa + blk] : 127u) << (8 * (f % 4));
            } else {
                o.a[f] = load_halves<true>(abase + row * p.lda, blk0 * kMxBlock + 8 * g, K);
            }
        }
        if constexpr (A == MXA_F16)
#pragma unroll
            for (int f = 0; f < FN; ++f)
                wide |= !f16_scale_ok(o.sb[f / 4] >> (8 * (f % 4)) & 0xffu);
        multiply(o, [](auto) {});
    }
    if constexpr (A == MXA_BF16) {
        static_assert(WTN == 64, "a lane to each of the wave's rows of B");
        if (__builtin_expect(__any(!all_finite(acc)), 0)) {
            const uint8_t *row = sbbase + min(wn * WTN + lane, nleft - 1) * p.ldsb;
            bool nan = false;   // (a row with a NaN block is NaN in any case)
#pragma unroll 1
            for (int blk = 0; blk < nblk; ++blk) {
                wide |= far_scale(row[blk]);
                nan |= row[blk] == 255;
            }
            wide &= !nan;
        }
    }
    if (!MX && __syncthreads_or(wide))
        return false;

    // ---- epilogue: lane l has row l % 16 and columns 4 * (l / 16) .. +3 of a
    // block, 64 bytes of a row of C in four lanes. Through LDS, 32 rows at a
    // time, a wave stores whole 256-byte rows instead. (Nobody reads the stages
    // any more: every wave has passed the last stage's barrier with its operands
    // in registers.)
    static_assert(WTN == 64 && FM % 2 == 0, "16 lanes store a row of a wave's tile");
    constexpr int LDC = WTN + 4;   // floats: rows four banks apart
    static_assert(NW * 32 * LDC * 4 <= sizeof(Lds), "the waves' rows fit the stages");
    float *mine = reinterpret_cast<float *>(&lds) + wave * (32 * LDC);
    const int64_t n = nb + wn * WTN + 4 * r16;
    const bool plain = p.beta == 0.0f && ma == m0 && nb == n0 && mleft == BM && nleft == BN;
#pragma unroll
    for (int i = 0; i < FM; i += 2) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < FN; ++j)
                *reinterpret_cast<f32x4 *>(&mine[(16 * h + r16) * LDC + 16 * j + 4 * g]) = acc[i + h][j];
        float *dst = p.C + (ma + wm * WTM + 16 * i + g) * p.ldc + n;
        const float *from = &mine[g * LDC + 4 * r16];
        if (plain) {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                f32x4 v = *reinterpret_cast<const f32x4 *>(from + 4 * q * LDC);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] *= p.alpha;
                __builtin_memcpy(dst + 4 * q * p.ldc, &v, 16);
            }
        } else {
#pragma unroll 1
            for (int q = 0; q < 8; ++q) {
                const int64_t m = ma + wm * WTM + 16 * i + 4 * q + g;
                if (m >= m0 && m < p.M)
                    finish4(p, *reinterpret_cast<const f32x4 *>(from + 4 * q * LDC), dst + 4 * q * p.ldc, n0 - n, p.N - n);
            }
        }
    }
    return true;
}

// 16-bit A against scales past its range: through the bfloat16 instruction, binary16
// values in two parts, and a block's products apart from the sum where a scale is far. A
// wave takes its rows 32 at a time (few registers, so that the path above keeps them),
// operands straight from memory.
template <int A, int BM, int BN, int WGM, int WGN>
__device__ __forceinline__ void mx4_tile_wide(const MxParams &p, int64_t m0, int64_t n0)
{
    constexpr int FM = 2, FN = BN / WGN / 16;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 4, r16 = lane & 15;
    const int64_t n = n0 + wave % WGN * (BN / WGN);
    const int nblk = (p.K - 1) / kMxBlock + 1;
#pragma unroll 1
    for (int i = 0; i < BM / WGM / 32; ++i) {
        const int64_t m = m0 + wave / WGN * (BM / WGM) + i * 32;
        f32x4 acc[FM][FN];
#pragma unroll
        for (int a = 0; a < FM; ++a)
#pragma unroll
            for (int b = 0; b < FN; ++b)
                acc[a][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
        for (int blk = 0; blk < nblk; ++blk) {
            u32x4 hi[FM], lo[FM];
#pragma unroll
            for (int a = 0; a < FM; ++a) {
                const int64_t row = m + 16 * a + r16 < p.M ? m + 16 * a + r16 : p.M - 1;
                hi[a] = load_halves<true>(p.A + row * p.lda, (int64_t)blk * kMxBlock + 8 * g, p.K);
                if constexpr (A == MXA_F16)
                    split8(hi[a], hi[a], lo[a]);
            }
            auto product = [&](const u32x4 &d, int a, f32x4 c) __attribute__((always_inline)) {
                if constexpr (A == MXA_F16)
                    c = mma_bf16(d, lo[a], c);
                return mma_bf16(d, hi[a], c);
            };
#pragma unroll
            for (int b = 0; b < FN; ++b) {
                const int64_t row = n + 16 * b + r16 < p.N ? n + 16 * b + r16 : p.N - 1;
                const u32x4 v = load_block<true>(p.B + row * p.ldb, blk, p.K);
                const uint32_t q = g < 2 ? (g == 0 ? v[0] : v[1]) : (g == 2 ? v[2] : v[3]);
                const uint32_t s = p.SB[row * p.ldsb + blk];
                const u32x4 d = decode8<true>(q, near_part(s));
                if (__any(far_scale(s))) {
                    float up[4];   // of this lane's four columns of C, rows 4 g .. +3 of B's 16
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        up[r] = __shfl(far_part(s), 4 * g + r);
#pragma unroll
                    for (int a = 0; a < FM; ++a) {
                        const f32x4 c = product(d, a, f32x4{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            acc[a][b][r] = __builtin_fmaf(c[r], up[r], acc[a][b][r]);
                    }
                } else {
#pragma unroll
                    for (int a = 0; a < FM; ++a)
                        acc[a][b] = product(d, a, acc[a][b]);
                }
            }
        }
#pragma unroll
        for (int a = 0; a < FM; ++a) {
            const int64_t row = m + 16 * a + r16;
            if (row >= p.M)
                continue;
#pragma unroll
            for (int b = 0; b < FN; ++b) {
                const int64_t col = n + 16 * b + 4 * g;
                finish4(p, acc[a][b], p.C + row * p.ldc + col, 0, p.N - col);
            }
        }
    }
}

template <int A, int BM, int BN, int NBUF, int WGM, int WGN, bool DMA>
__device__ __forceinline__ void mx4_tile_any(const MxParams &p, int64_t m0, int64_t n0, uint8_t *raw)
{
    const bool done = mx4_tile<A, BM, BN, 2, NBUF, WGM, WGN, DMA>(p, m0, n0, raw);
    if constexpr (A != MXA_MX4)
        if (!done)
            mx4_tile_wide<A, BM, BN, WGM, WGN>(p, m0, n0);
}

// One workgroup a tile, in an order that keeps an XCD's tiles together. The last
// p.halved tiles (SPLIT) are done in two halves by two workgroups, so that a last
// round with few tiles takes half as long.
template <int A, int BM, int BN, int NBUF, int WGM, int WGN, bool SPLIT, bool DMA>
__global__ void __launch_bounds__(64 * WGM * WGN) __attribute__((amdgpu_waves_per_eu(2, 2)))
gemm_mx4_tile_kernel(MxParams p)
{
    __shared__ __attribute__((aligned(1024))) uint8_t raw[tile_lds<A>(BM, BN, 2, NBUF)];
    const int wholes = (int)gridDim.x - 2 * p.halved, b = (int)blockIdx.x;
    int tm, tn;
    if (!SPLIT || b < wholes) {
        mx_tile_of(p, block_index(b, wholes), tm, tn);
        mx4_tile_any<A, BM, BN, NBUF, WGM, WGN, DMA>(p, (int64_t)tm * BM, (int64_t)tn * BN, raw);
    } else if constexpr (SPLIT) {
        const int id = block_index(b - wholes, 2 * p.halved);
        mx_tile_of(p, wholes + id / 2, tm, tn);
        const int64_t m0 = (int64_t)tm * BM + (id & 1) * (BM / 2);
        if (m0 < p.M)
            mx4_tile_any<A, BM / 2, BN, NBUF, WGM, WGN, DMA>(p, m0, (int64_t)tn * BN, raw);
    }
}

template <int A, int BM, int BN, int NBUF, int WGM, int WGN, bool SPLIT, bool DMA>
static hipError_t launch_tile(MxParams p, int cus, hipStream_t s)
{
    p.tiles_m = cdiv(p.M, BM);
    p.tiles_n = cdiv(p.N, BN);
    const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
    if (tiles > max_grid_x(64 * WGM * WGN) / 2)
        return hipErrorInvalidValue;
    const int64_t last = tiles % cus;   // tiles of the last round
    p.halved = SPLIT && 2 * last <= cus ? (int)last : 0;
    hipLaunchKernelGGL((gemm_mx4_tile_kernel<A, BM, BN, NBUF, WGM, WGN, SPLIT, DMA>), dim3((unsigned)(tiles + p.halved)),
                       dim3(64 * WGM * WGN), 0, s, p);
    return hipGetLastError();
}

template <int A>
static hipError_t tile_a(const MxParams &p, int tile, bool dma, int cus, hipStream_t s)
{
    constexpr int NBUF = A == MXA_MX4 ? 2 : 3;
    if (!dma)
        return launch_tile<A, 128, 128, 2, 2, 2, false, false>(p, cus, s);
    if (tile == MX_TILE_256)
        return launch_tile<A, 256, 256, NBUF, 2, 4, true, true>(p, cus, s);
    return launch_tile<A, 128, 128, NBUF, 2, 2, false, true>(p, cus, s);
}

hipError_t launch_gemm_mx4_tile(MxParams p, int a, int tile, bool dma, int cus, hipStream_t s)
{
    p.group_m = 8;
    if (a == MXA_MX4)
        return tile_a<MXA_MX4>(p, tile, dma, cus, s);
    if (a == MXA_F16)
        return tile_a<MXA_F16>(p, tile, dma, cus, s);
    return tile_a<MXA_BF16>(p, tile, dma, cus, s);
}

}  // namespace ll
