// linear_nn_bf16.hip -- the gradients' NN products (dX = dZ W), bfloat16.
#include "linear_launch.hpp"

namespace gemm_epi {

hipError_t lin_launch_nn_bf16(int tile, const LinParams &p, int groups, hipStream_t s)
{
    return lin_launch_out<false, true, true>(tile, p, groups, s);
}

}  // namespace gemm_epi
