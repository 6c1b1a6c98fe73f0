// linear_tn_bf16.hip -- the gradients' TN products (dW = dZ^T X), bfloat16.
#include "linear_launch.hpp"

namespace gemm_epi {

hipError_t lin_launch_tn_bf16(int tile, const LinParams &p, int groups, hipStream_t s)
{
    return lin_launch_out<true, true, true>(tile, p, groups, s);
}

}  // namespace gemm_epi
