// The 16-bit layer's weight gradient. Its contracted axis, the rows, is not shared out over
// workgroups: a result of few tiles leaves CUs without work however long the rows are (bfloat16,
// results in FP32: 8192 rows to 64 x 64 69 us, to 512 x 512 70, to 1024 x 1024 71, to 2048 x 2048 79; X in 8
// bits 512 x 512 97; 65536 rows to 512 x 512 546).
#include "linear16_tile.hpp"

namespace ll {

using namespace l16;

template <bool BF16, int SB>
static hipError_t launch_dw(const L16Params &p, bool vec, int cus, hipStream_t s)
{
    const int64_t rows = (int64_t)p.groups.n * cdiv(p.M, 128);
    if (!vec)
        return launch_small<L16_DW, BF16, COLS, SB, false>(p, rows, s);
    if (weight_prefers_large(p.M, p.N, p.K, p.groups.n, cus))
        return launch_large<L16_DW, BF16, COLS, SB>(p, cus, s);
    return launch_small<L16_DW, BF16, COLS, SB, true>(p, rows, s);
}

hipError_t launch_l16_dw(bool bf16, L16Params p, bool vec, int cus, hipStream_t s)
{
    if (p.BS != nullptr)
        return bf16 ? launch_dw<true, COLS8>(p, vec, cus, s) : launch_dw<false, COLS8>(p, vec, cus, s);
    return bf16 ? launch_dw<true, COLS>(p, vec, cus, s) : launch_dw<false, COLS>(p, vec, cus, s);
}

int l16_shares(int op, int M, int N, int K, int groups, int cus)
{
    if (op == L16_DW || M == 0 || N == 0 || K == 0 || groups == 0)
        return 1;
    if (op == L16_DX)
        return rows_shares(M, K, N, groups, cus);
    return l16_takes_rows(M, groups) ? l16_row_shares(M, N, K, groups, cus) : rows_shares(M, N, K, groups, cus);
}

const char *l16_kernel_name(int op, int M, int N, int K, int groups, bool vec, int cus)
{
    if (op == L16_FWD && l16_takes_rows(M, groups))
        return vec ? "rows" : "rows_any";
    if (!vec)
        return "small_any";
    const bool large = op == L16_DW ? weight_prefers_large(N, K, M, groups, cus)
                                    : op == L16_DX ? rows_prefer_large(M, K, N, groups, cus)
                                                   : rows_prefer_large(M, N, K, groups, cus);
    return large ? "large" : "small";
}

}  // namespace ll
