// The 16-bit layer's forward product: which kernel it takes.
#include "linear16_tile.hpp"

namespace ll {

using namespace l16;

hipError_t launch_l16_fwd(bool bf16, L16Params p, bool vec, int cus, hipStream_t s)
{
    // few rows to a weight: read it once
    if (l16_takes_rows(p.M, p.groups.n))
        return launch_l16_rows(bf16, p, vec, cus, s);
    return bf16 ? launch_rows<L16_FWD, true, ROWS>(p, vec, cus, s) : launch_rows<L16_FWD, false, ROWS>(p, vec, cus, s);
}

}  // namespace ll
