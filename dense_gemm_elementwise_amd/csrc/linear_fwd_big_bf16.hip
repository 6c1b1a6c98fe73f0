// linear_fwd_big_bf16.hip -- the forward product's 256 x 256 tile, bfloat16 (a
// translation unit of its own because it takes longest to compile).
#include "linear_launch.hpp"

namespace gemm_epi {

hipError_t lin_launch_fwd_big_bf16(int act, const LinParams &p, int groups, hipStream_t s)
{
    return lin_launch_act<kLinBig, true>(act, p, groups, s);
}

}  // namespace gemm_epi
