// fp8_convert.hpp -- from 32 bits to 8-bit floating point with a power-of-two
// scale for a block of 128 (include/fp8_ops.h).
//
// A block's largest finite magnitude is a = 1.m 2^k; the largest element of the
// format is 1.75 2^t (e4m3: t = 8, e5m2: t = 15), so the smallest power of two
// that holds the block is 2^e, e = k - t, or one more where 1.m > 1.75: adding
// 0x1FFFFF to the bits of a carries into the exponent in exactly those cases.
// Division by 2^e is exact, so an element is rounded once.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gemm_epi {

constexpr int kBlock = 128;

// The exponent of a block's scale; top: t of the format.
__device__ __forceinline__ int block_exponent(float a, int top)
{
    const int k = (int)((__builtin_bit_cast(uint32_t, a) + 0x1FFFFFu) >> 23) - 127 - top;
    return a > 0.0f ? max(k, -127) : 0;
}
__device__ __forceinline__ float pow2f(int e) { return __builtin_bit_cast(float, (uint32_t)(e + 127) << 23); }

// four elements to bytes, the first in the lowest
template <int FMT>
__device__ __forceinline__ uint32_t cvt4(float a, float b, float c, float d)
{
    int r = 0;
    if constexpr (FMT == 0) {
        r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, r, false);
        r = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
    } else {
        r = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, r, false);
        r = __builtin_amdgcn_cvt_pk_bf8_f32(c, d, r, true);
    }
    return (uint32_t)r;
}

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x2 u32x2u __attribute__((aligned(1)));
typedef u32x4 u32x4u __attribute__((aligned(1)));

// |v|, 0 where it is not finite
__device__ __forceinline__ float finite_abs(float v)
{
    const float a = __builtin_fabsf(v);
    return a < __builtin_inff() ? a : 0.0f;
}

}  // namespace gemm_epi
