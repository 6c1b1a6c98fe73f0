// linear_xent_f16.hip -- the products of the cross entropy's logits, fp16.
#include "linear_launch.hpp"

namespace gemm_epi {

hipError_t lin_launch_xent_f16(int epi, int tile, const LinParams &p, int groups, hipStream_t s)
{
    if (epi == LE_XFWD)
        return tile == kLinBig ? lin_launch_one<kLinBig, false, false, LE_XFWD, 0, false>(p, groups, s)
                               : lin_launch_one<kLinSmall, false, false, LE_XFWD, 0, false>(p, groups, s);
    return tile == kLinBig ? lin_launch_one<kLinBig, false, false, LE_XP, 0, false>(p, groups, s)
                           : lin_launch_one<kLinSmall, false, false, LE_XP, 0, false>(p, groups, s);
}

}  // namespace gemm_epi
