// fp8_fwd_f16.hip -- the 8-bit products with fp16 outputs.
#include "fp8_launch.hpp"

namespace gemm_epi {

hipError_t fp8_launch_fwd_f16(int act, const Fp8Params &p, int groups, hipStream_t s)
{
    return fp8_launch_act<128, 128, false>(act, p, groups, s);
}

hipError_t fp8_launch_out_f16(const Fp8Params &p, int groups, hipStream_t s)
{
    return fp8_launch_one<128, 128, LE_OUT, 0, false>(p, groups, s);
}

}  // namespace gemm_epi
