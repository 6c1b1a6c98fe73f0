// fp8_fwd_bf16.hip -- the 8-bit products with bfloat16 outputs.
#include "fp8_launch.hpp"

namespace gemm_epi {

hipError_t fp8_launch_fwd_bf16(int act, const Fp8Params &p, int groups, hipStream_t s)
{
    return fp8_launch_act<128, 128, true>(act, p, groups, s);
}

hipError_t fp8_launch_out_bf16(const Fp8Params &p, int groups, hipStream_t s)
{
    return fp8_launch_one<128, 128, LE_OUT, 0, true>(p, groups, s);
}

}  // namespace gemm_epi
