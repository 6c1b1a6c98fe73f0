// linear_launch.hpp -- what the translation units of the products share: the
// tiles, and one launch function per group of kernels and element type.
#pragma once

#include <hip/hip_runtime.h>

#include "linear_gemm.hpp"

namespace gemm_epi {

struct LinTile {
    int bm, bn;
};
inline constexpr LinTile kLinTiles[] = {{256, 256}, {128, 256}, {256, 128}, {128, 128}};
constexpr int kLinBig = 0, kLinSmall = 3;  // indices of the square tiles

// Launches the kernel of tile `tile` (an index into kLinTiles) on `groups`
// workgroups.  The forward has every tile for every activation, its split form
// (fp32 partial sums) the small one only; the cross entropy has the square
// tiles; the gradients have every tile.
hipError_t lin_launch_fwd_big_f16(int act, const LinParams &p, int groups, hipStream_t s);
hipError_t lin_launch_fwd_big_bf16(int act, const LinParams &p, int groups, hipStream_t s);
hipError_t lin_launch_fwd_f16(int act, int tile, const LinParams &p, int groups, hipStream_t s);
hipError_t lin_launch_fwd_bf16(int act, int tile, const LinParams &p, int groups, hipStream_t s);
hipError_t lin_launch_fwd_split_f16(const LinParams &p, int groups, hipStream_t s);
hipError_t lin_launch_fwd_split_bf16(const LinParams &p, int groups, hipStream_t s);
hipError_t lin_launch_xent_f16(int epi, int tile, const LinParams &p, int groups, hipStream_t s);
hipError_t lin_launch_xent_bf16(int epi, int tile, const LinParams &p, int groups, hipStream_t s);
hipError_t lin_launch_nn_f16(int tile, const LinParams &p, int groups, hipStream_t s);
hipError_t lin_launch_nn_bf16(int tile, const LinParams &p, int groups, hipStream_t s);
hipError_t lin_launch_pair_f16(const LinPair &p, int groups, hipStream_t s);
hipError_t lin_launch_pair_bf16(const LinPair &p, int groups, hipStream_t s);
hipError_t lin_launch_tn_f16(int tile, const LinParams &p, int groups, hipStream_t s);
hipError_t lin_launch_tn_bf16(int tile, const LinParams &p, int groups, hipStream_t s);

template <int T, bool AKM, bool BKM, int EPI, int ACT, bool BF>
hipError_t lin_launch_one(const LinParams &p, int groups, hipStream_t stream)
{
    constexpr LinTile t = kLinTiles[T];
    LinParams arg = p;
    void *args[] = {(void *)&arg};
    return hipLaunchKernel((const void *)&lin_gemm_kernel<t.bm, t.bn, AKM, BKM, EPI, ACT, BF>, dim3(groups), dim3(256),
                           args, 0, stream);
}

template <int T, bool BF>
hipError_t lin_launch_act(int act, const LinParams &p, int groups, hipStream_t s)
{
    switch (act) {
    case ACT_RELU: return lin_launch_one<T, false, false, LE_LINEAR, ACT_RELU, BF>(p, groups, s);
    case ACT_GELU: return lin_launch_one<T, false, false, LE_LINEAR, ACT_GELU, BF>(p, groups, s);
    case ACT_SILU: return lin_launch_one<T, false, false, LE_LINEAR, ACT_SILU, BF>(p, groups, s);
    default: return lin_launch_one<T, false, false, LE_LINEAR, ACT_IDENTITY, BF>(p, groups, s);
    }
}

template <bool AKM, bool BKM, bool BF>
hipError_t lin_launch_out(int tile, const LinParams &p, int groups, hipStream_t s)
{
    switch (tile) {
    case 0: return lin_launch_one<0, AKM, BKM, LE_OUT, 0, BF>(p, groups, s);
    case 1: return lin_launch_one<1, AKM, BKM, LE_OUT, 0, BF>(p, groups, s);
    case 2: return lin_launch_one<2, AKM, BKM, LE_OUT, 0, BF>(p, groups, s);
    default: return lin_launch_one<3, AKM, BKM, LE_OUT, 0, BF>(p, groups, s);
    }
}

}  // namespace gemm_epi
