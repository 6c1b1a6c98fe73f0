// linear_grad_bf16.hip -- the gradients' products, bfloat16: NN (dX = dZ W) and TN
// (dW = dZ^T X).
#include "linear_launch.hpp"

namespace gemm_epi {

hipError_t lin_launch_nn_bf16(int tile, const LinParams &p, int groups, hipStream_t s)
{
    return lin_launch_out<false, true, true>(tile, p, groups, s);
}

hipError_t lin_launch_tn_bf16(int tile, const LinParams &p, int groups, hipStream_t s)
{
    return lin_launch_out<true, true, true>(tile, p, groups, s);
}

}  // namespace gemm_epi
