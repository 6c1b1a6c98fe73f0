// fp8_e5m2_bf16.hip -- the products of e5m2 A with bfloat16 outputs.
#include "fp8_launch.hpp"

namespace gemm_epi {

hipError_t fp8_launch_fwd_e5m2_bf16(int act, int tile, const Fp8Params &p, int groups, hipStream_t s)
{
    return fp8_launch_fwd<true, 1>(act, tile, p, groups, s);
}

hipError_t fp8_launch_out_e5m2_bf16(int tile, const Fp8Params &p, int groups, hipStream_t s)
{
    return fp8_launch_out<true, 1>(tile, p, groups, s);
}

hipError_t fp8_launch_pair_e5m2_bf16(int tile, const Fp8Pair &p, hipStream_t s)
{
    return fp8_launch_pair<true, 1>(tile, p, s);
}

}  // namespace gemm_epi
