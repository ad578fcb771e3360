// The 16-bit layer's weight gradient.
#include "linear16_tile.hpp"

namespace ll {

using namespace l16;

template <bool BF16, int SB>
static hipError_t launch_dw(const L16Params &p, bool vec, int cus, hipStream_t s)
{
    const int64_t n = p.groups.n, rows = n * cdiv(p.M, 128);
    if (!vec)
        return launch_small<L16_DW, BF16, COLS, SB, false>(p, rows, s);
    const int64_t n_large = n * cdiv(p.M, 256) * cdiv(p.N, 256);
    const int each = p.K > n ? cdiv(p.K, (int)n) : 1;   // rows of a group
    if (n_large < (1 << 29) && prefer_large(n_large, 0, rows * cdiv(p.N, 128), each, cus))
        return launch_large<L16_DW, BF16, COLS, SB>(p, cus, s);
    return launch_small<L16_DW, BF16, COLS, SB, true>(p, rows, s);
}

hipError_t launch_l16_dw(bool bf16, L16Params p, bool vec, int cus, hipStream_t s)
{
    if (p.BS != nullptr)
        return bf16 ? launch_dw<true, COLS8>(p, vec, cus, s) : launch_dw<false, COLS8>(p, vec, cus, s);
    return bf16 ? launch_dw<true, COLS>(p, vec, cus, s) : launch_dw<false, COLS>(p, vec, cus, s);
}

}  // namespace ll
