// fp8_launch.hpp -- the 8-bit products' launch functions, one for each group of
// kernels that a translation unit holds.
#pragma once

#include <hip/hip_runtime.h>

#include "fp8_gemm.hpp"

namespace gemm_epi {

// Launches the forward's kernel (epilogue of linear, or fp32 partial sums for
// split = true), or a gradient's (output alone), on `groups` workgroups.
hipError_t fp8_launch_fwd_f16(int act, const Fp8Params &p, int groups, hipStream_t s);
hipError_t fp8_launch_fwd_bf16(int act, const Fp8Params &p, int groups, hipStream_t s);
hipError_t fp8_launch_out_f16(const Fp8Params &p, int groups, hipStream_t s);
hipError_t fp8_launch_out_bf16(const Fp8Params &p, int groups, hipStream_t s);

template <int BM, int BN, int EPI, int ACT, bool BF>
hipError_t fp8_launch_one(const Fp8Params &p, int groups, hipStream_t stream)
{
    Fp8Params arg = p;
    void *args[] = {(void *)&arg};
    return hipLaunchKernel((const void *)&fp8_gemm_kernel<BM, BN, EPI, ACT, BF>, dim3(groups), dim3(256), args, 0,
                           stream);
}

template <int BM, int BN, bool BF>
hipError_t fp8_launch_act(int act, const Fp8Params &p, int groups, hipStream_t s)
{
    switch (act) {
    case ACT_RELU: return fp8_launch_one<BM, BN, LE_LINEAR, ACT_RELU, BF>(p, groups, s);
    case ACT_GELU: return fp8_launch_one<BM, BN, LE_LINEAR, ACT_GELU, BF>(p, groups, s);
    case ACT_SILU: return fp8_launch_one<BM, BN, LE_LINEAR, ACT_SILU, BF>(p, groups, s);
    default: return fp8_launch_one<BM, BN, LE_LINEAR, ACT_IDENTITY, BF>(p, groups, s);
    }
}

}  // namespace gemm_epi
