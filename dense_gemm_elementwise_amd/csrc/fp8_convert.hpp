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

// The same of 16-bit elements, two to a dword, divided by 2^e: one instruction for
// two, the same bits (compared for all 16-bit values and exponents from -126 to 120).
template <int FMT, bool BF>
__device__ __forceinline__ uint32_t cvt4_16(uint32_t ab, uint32_t cd, int e)
{
    if (BF && e == -127) {  // (no normal number; fp16 has no such blocks)
        auto f = [](uint32_t v) { return __builtin_bit_cast(float, v) * 0x1p127f; };
        return cvt4<FMT>(f(ab << 16), f(ab & 0xFFFF0000u), f(cd << 16), f(cd & 0xFFFF0000u));
    }
    typedef short s16x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));
    typedef _Float16 f16x2v __attribute__((ext_vector_type(2)));
    const float scale = pow2f(e);
    s16x2 r = {0, 0};
    if constexpr (BF && FMT == 0) {
        r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2v, ab), scale, false);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2v, cd), scale, true);
    } else if constexpr (BF) {
        r = __builtin_amdgcn_cvt_scalef32_pk_bf8_bf16(r, __builtin_bit_cast(bf16x2v, ab), scale, false);
        r = __builtin_amdgcn_cvt_scalef32_pk_bf8_bf16(r, __builtin_bit_cast(bf16x2v, cd), scale, true);
    } else if constexpr (FMT == 0) {
        r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(r, __builtin_bit_cast(f16x2v, ab), scale, false);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(r, __builtin_bit_cast(f16x2v, cd), scale, true);
    } else {
        r = __builtin_amdgcn_cvt_scalef32_pk_bf8_f16(r, __builtin_bit_cast(f16x2v, ab), scale, false);
        r = __builtin_amdgcn_cvt_scalef32_pk_bf8_f16(r, __builtin_bit_cast(f16x2v, cd), scale, true);
    }
    return __builtin_bit_cast(uint32_t, r);
}

// Magnitudes of 16-bit elements, two to a dword, are ordered as integers.
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b)
{
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}
template <bool BF>
__device__ __forceinline__ bool has_not_finite(uint32_t m)  // a magnitude of the two
{
    constexpr uint32_t INF = BF ? 0x7F80u : 0x7C00u;
    return (m & 0xFFFF) >= INF || (m >> 16) >= INF;
}
template <bool BF>
__device__ __forceinline__ uint32_t finite_u16x2(uint32_t m)  // 0 in place of what is not finite
{
    constexpr uint32_t INF = BF ? 0x7F80u : 0x7C00u;
    return ((m & 0xFFFF) >= INF ? 0 : m & 0xFFFF) | ((m >> 16) >= INF ? 0 : m & 0xFFFF0000u);
}
template <bool BF>
__device__ __forceinline__ float value_u16(uint32_t m)
{
    if constexpr (BF)
        return __builtin_bit_cast(float, m << 16);
    else
        return (float)__builtin_bit_cast(_Float16, (unsigned short)m);
}
template <bool BF>
__device__ __forceinline__ float larger_of(uint32_t m)  // of the two
{
    return value_u16<BF>(max(m & 0xFFFF, m >> 16));
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
