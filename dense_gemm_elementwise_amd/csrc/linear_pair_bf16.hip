// linear_pair_bf16.hip -- a gradient's two products in one launch, bfloat16.
#include "linear_launch.hpp"

namespace gemm_epi {

hipError_t lin_launch_pair_bf16(const LinPair &p, int groups, hipStream_t s)
{
    LinPair arg = p;
    void *args[] = {(void *)&arg};
    return hipLaunchKernel((const void *)&lin_grad_pair_kernel<true>, dim3(groups), dim3(256), args, 0, s);
}

}  // namespace gemm_epi
