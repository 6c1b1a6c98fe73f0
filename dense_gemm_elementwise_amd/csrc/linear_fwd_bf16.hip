// linear_fwd_bf16.hip -- the forward product's other tiles and its split form, bfloat16.
#include "linear_launch.hpp"

namespace gemm_epi {

hipError_t lin_launch_fwd_bf16(int act, int tile, const LinParams &p, int groups, hipStream_t s)
{
    switch (tile) {
    case 1: return lin_launch_act<1, true>(act, p, groups, s);
    case 2: return lin_launch_act<2, true>(act, p, groups, s);
    default: return lin_launch_act<3, true>(act, p, groups, s);
    }
}

hipError_t lin_launch_fwd_split_bf16(const LinParams &p, int groups, hipStream_t s)
{
    return lin_launch_one<kLinSmall, false, false, LE_OUT, 0, true>(p, groups, s);
}

}  // namespace gemm_epi
