// The 16-bit layer's input gradient.
#include "linear16_tile.hpp"

namespace ll {

using namespace l16;

hipError_t launch_l16_dx(bool bf16, L16Params p, bool vec, int cus, hipStream_t s)
{
    return bf16 ? launch_rows<L16_DX, true, COLS>(p, vec, cus, s) : launch_rows<L16_DX, false, COLS>(p, vec, cus, s);
}

}  // namespace ll
