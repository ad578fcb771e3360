// The 16-bit layer's weight gradient.
#include "linear16_tile.hpp"

namespace ll {

using namespace l16;

template <bool BF16, int BM, int SB, bool DMA>
static hipError_t launch_dw(L16Params p, hipStream_t s)
{
    p.tiles_m = cdiv(p.M, BM);
    p.tiles_n = cdiv(p.N, BM);
    const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n * p.groups.n;
    if (tiles > max_grid_x(Cfg<BM>::NT))
        return hipErrorInvalidValue;
    hipLaunchKernelGGL((l16_tile_kernel<L16_DW, BF16, BM, COLS, SB, DMA>), dim3((unsigned)tiles), dim3(Cfg<BM>::NT), 0, s, p);
    return hipGetLastError();
}

template <bool BF16, int SB>
static hipError_t launch_dw_side(const L16Params &p, bool vec, int cus, hipStream_t s)
{
    if (!vec)
        return launch_dw<BF16, 128, SB, false>(p, s);
    return prefer_256((int64_t)p.groups.n * cdiv(p.M, 256) * cdiv(p.N, 256),
                      (int64_t)p.groups.n * cdiv(p.M, 128) * cdiv(p.N, 128), cus)
               ? launch_dw<BF16, 256, SB, true>(p, s)
               : launch_dw<BF16, 128, SB, true>(p, s);
}

hipError_t launch_l16_dw(bool bf16, L16Params p, bool vec, int cus, hipStream_t s)
{
    if (p.BS != nullptr)
        return bf16 ? launch_dw_side<true, COLS8>(p, vec, cus, s) : launch_dw_side<false, COLS8>(p, vec, cus, s);
    return bf16 ? launch_dw_side<true, COLS>(p, vec, cus, s) : launch_dw_side<false, COLS>(p, vec, cus, s);
}

}  // namespace ll
