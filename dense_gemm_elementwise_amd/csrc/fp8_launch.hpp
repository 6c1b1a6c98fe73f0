// fp8_launch.hpp -- what the translation units of the 8-bit products share: the
// tiles, and one launch function per format of A, element type and epilogue.
#pragma once

#include <hip/hip_runtime.h>

#include "fp8_gemm.hpp"

namespace gemm_epi {

struct Fp8Tile {
    int bm, bn;
    int depth;  // of the rings, see fp8_gemm.hpp
};
inline constexpr Fp8Tile kFp8Tiles[] = {{256, 256, 0}, {128, 128, 0}, {128, 128, 4}, {128, 256, 3}};
constexpr int kFp8Big = 0, kFp8Small = 1, kFp8Deep = 2, kFp8Wide = 3;  // indices

// Launches the forward's kernel (the epilogue of linear), or the one that writes
// the product alone (gradients and the splits' fp32 partial sums), with tile
// `tile` (an index into kFp8Tiles) on `groups` workgroups.
hipError_t fp8_launch_fwd_e4m3_f16(int act, int tile, const Fp8Params &p, int groups, hipStream_t s);
hipError_t fp8_launch_fwd_e4m3_bf16(int act, int tile, const Fp8Params &p, int groups, hipStream_t s);
hipError_t fp8_launch_fwd_e5m2_f16(int act, int tile, const Fp8Params &p, int groups, hipStream_t s);
hipError_t fp8_launch_fwd_e5m2_bf16(int act, int tile, const Fp8Params &p, int groups, hipStream_t s);
hipError_t fp8_launch_out_e4m3_f16(int tile, const Fp8Params &p, int groups, hipStream_t s);
hipError_t fp8_launch_out_e4m3_bf16(int tile, const Fp8Params &p, int groups, hipStream_t s);
hipError_t fp8_launch_out_e5m2_f16(int tile, const Fp8Params &p, int groups, hipStream_t s);
hipError_t fp8_launch_out_e5m2_bf16(int tile, const Fp8Params &p, int groups, hipStream_t s);

// Two products and the bias's gradient in one launch; tile: any but kFp8Small.
hipError_t fp8_launch_pair_e4m3_f16(int tile, const Fp8Pair &p, hipStream_t s);
hipError_t fp8_launch_pair_e4m3_bf16(int tile, const Fp8Pair &p, hipStream_t s);
hipError_t fp8_launch_pair_e5m2_f16(int tile, const Fp8Pair &p, hipStream_t s);
hipError_t fp8_launch_pair_e5m2_bf16(int tile, const Fp8Pair &p, hipStream_t s);

// Up to 16 rows (fp8_rows.hpp).  Without scales p.X has 16 bits and up to 4 rows.
struct FewRows8;
hipError_t fp8_launch_rows(bool bf, bool e5m2, const FewRows8 &p, hipStream_t s);

template <int T, int EPI, int ACT, bool BF, int FA>
hipError_t fp8_launch_one(const Fp8Params &p, int groups, hipStream_t stream)
{
    constexpr Fp8Tile t = kFp8Tiles[T];
    Fp8Params arg = p;
    void *args[] = {(void *)&arg};
    return hipLaunchKernel((const void *)&fp8_gemm_kernel<t.bm, t.bn, t.depth, EPI, ACT, BF, FA>, dim3(groups), dim3(256), args,
                           0, stream);
}

template <int T, bool BF, int FA>
hipError_t fp8_launch_act(int act, const Fp8Params &p, int groups, hipStream_t s)
{
    switch (act) {
    case ACT_RELU: return fp8_launch_one<T, LE_LINEAR, ACT_RELU, BF, FA>(p, groups, s);
    case ACT_GELU: return fp8_launch_one<T, LE_LINEAR, ACT_GELU, BF, FA>(p, groups, s);
    case ACT_SILU: return fp8_launch_one<T, LE_LINEAR, ACT_SILU, BF, FA>(p, groups, s);
    default: return fp8_launch_one<T, LE_LINEAR, ACT_IDENTITY, BF, FA>(p, groups, s);
    }
}

template <bool BF, int FA>
hipError_t fp8_launch_fwd(int act, int tile, const Fp8Params &p, int groups, hipStream_t s)
{
    switch (tile) {
    case 0: return fp8_launch_act<0, BF, FA>(act, p, groups, s);
    case 1: return fp8_launch_act<1, BF, FA>(act, p, groups, s);
    case 2: return fp8_launch_act<2, BF, FA>(act, p, groups, s);
    default: return fp8_launch_act<3, BF, FA>(act, p, groups, s);
    }
}

template <bool BF, int FA>
hipError_t fp8_launch_out(int tile, const Fp8Params &p, int groups, hipStream_t s)
{
    switch (tile) {
    case 0: return fp8_launch_one<0, LE_OUT, 0, BF, FA>(p, groups, s);
    case 1: return fp8_launch_one<1, LE_OUT, 0, BF, FA>(p, groups, s);
    case 2: return fp8_launch_one<2, LE_OUT, 0, BF, FA>(p, groups, s);
    default: return fp8_launch_one<3, LE_OUT, 0, BF, FA>(p, groups, s);
    }
}

template <int T, bool BF, int FA>
hipError_t fp8_launch_pair_one(const Fp8Pair &p, hipStream_t s)
{
    constexpr Fp8Tile t = kFp8Tiles[T];
    Fp8Pair arg = p;
    void *args[] = {(void *)&arg};
    const int groups = p.groups[0] + p.groups[1] + (p.bias.out ? (p.bias.cols + 255) / 256 : 0);
    return hipLaunchKernel((const void *)&fp8_pair_kernel<t.bm, t.bn, t.depth, BF, FA>, dim3(groups), dim3(256), args, 0, s);
}
template <bool BF, int FA>
hipError_t fp8_launch_pair(int tile, const Fp8Pair &p, hipStream_t s)
{
    switch (tile) {
    case kFp8Big: return fp8_launch_pair_one<kFp8Big, BF, FA>(p, s);
    case kFp8Wide: return fp8_launch_pair_one<kFp8Wide, BF, FA>(p, s);
    default: return fp8_launch_pair_one<kFp8Deep, BF, FA>(p, s);
    }
}

}  // namespace gemm_epi
