// fp8_e4m3_f16.hip -- the products of e4m3 A with fp16 outputs.
#include "fp8_launch.hpp"

namespace gemm_epi {

hipError_t fp8_launch_fwd_e4m3_f16(int act, int tile, const Fp8Params &p, int groups, hipStream_t s)
{
    return fp8_launch_fwd<false, 0>(act, tile, p, groups, s);
}

hipError_t fp8_launch_out_e4m3_f16(int tile, const Fp8Params &p, int groups, hipStream_t s)
{
    return fp8_launch_out<false, 0>(tile, p, groups, s);
}

hipError_t fp8_launch_pair_e4m3_f16(int tile, const Fp8Pair &p, hipStream_t s)
{
    return fp8_launch_pair<false, 0>(tile, p, s);
}

}  // namespace gemm_epi
