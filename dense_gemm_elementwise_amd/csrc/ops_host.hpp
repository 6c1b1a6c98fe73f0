// ops_host.hpp -- what the C entry points of the operators share on the host:
// argument checks, workspace layout, launches, and the small kernels of
// linear_ops.hip that other operators use.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "linear_ops.h"

namespace gemm_epi {

void set_last_hip_error(int e);  // gemm_epi.hip

inline constexpr int kCUs = 256;

inline bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
inline int64_t ceil_div(int64_t v, int64_t m) { return (v + m - 1) / m; }

inline int hip_status(hipError_t e)
{
    if (e == hipSuccess) return GEMM_EPI_OK;
    set_last_hip_error((int)e);
    return GEMM_EPI_ERR_HIP;
}

#define GE_TRY(call)                                  \
    do {                                              \
        const int ge_rc = hip_status(call);           \
        if (ge_rc != GEMM_EPI_OK) return ge_rc;       \
    } while (0)

// (arguments convert to the kernel's own parameter types)
template <typename T>
struct Same {
    using type = T;
};
template <typename... P>
hipError_t launch(void (*kernel)(P...), dim3 grid, dim3 block, hipStream_t s, typename Same<P>::type... a)
{
    void *args[] = {(void *)&a...};
    return hipLaunchKernel((const void *)kernel, grid, block, args, 0, s);
}

// a matrix operand: NULL, alignment and row stride
inline int check_matrix(const void *p, int64_t ld, int64_t cols, uintptr_t es, int null_status)
{
    if (!p) return null_status;
    if (!aligned(p, es)) return GEMM_EPI_ERR_ALIGN;
    if (ld < cols || ld > GE_MAX_COLS) return GEMM_EPI_ERR_SHAPE;
    return GEMM_EPI_OK;
}
#define GE_CHECK(call)                          \
    do {                                        \
        const int ge_rc = (call);               \
        if (ge_rc != GEMM_EPI_OK) return ge_rc; \
    } while (0)

inline int check_dims(int64_t rows, int64_t rows2, int64_t cols)
{
    if (rows < 0 || rows > INT32_MAX - 256 || rows2 < 1 || rows2 > INT32_MAX - 256 || cols < 1 || cols > GE_MAX_COLS)
        return GEMM_EPI_ERR_SHAPE;
    return GEMM_EPI_OK;
}
inline int check_dtype(int64_t dtype) { return dtype == GEMM_EPI_F16 || dtype == GEMM_EPI_BF16 ? GEMM_EPI_OK : GEMM_EPI_ERR_DTYPE; }

// A region of the workspace.
struct Layout {
    int64_t bytes = 0;
    int64_t take(int64_t n)
    {
        const int64_t at = bytes;
        bytes = round_up(bytes + n, 256);
        return at;
    }
};

inline int check_workspace(const void *ws, int64_t have, int64_t need)
{
    if (need == 0) return GEMM_EPI_OK;
    if (!ws || have < need) return GEMM_EPI_ERR_WORKSPACE;
    return aligned(ws, 16) ? GEMM_EPI_OK : GEMM_EPI_ERR_ALIGN;
}

// rows that the 16-byte accesses of the 16-bit products can take
inline bool dma_rows(const void *p, int64_t ld, int64_t cols) { return cols % 8 == 0 && ld % 8 == 0 && aligned(p, 16); }

// a launch holds fewer than 2^32 threads: 2^24 workgroups of 256
inline constexpr int64_t kMaxGroups = (1 << 24) - 1;

// ---- shared kernels (linear_ops.hip) --------------------------------------------
struct SplitSumParams {
    const float *part;  // [splits][M][ldc]
    int splits, lanes, M, N;  // lanes: 1, 4 or 8
    int64_t ldc, c_split;
    const _Float16 *bias, *R;
    _Float16 *D, *Z;
    int64_t ldr, ldd, ldz;
    float *C32;  // LE_OUT: accumulator, rows of ldc
    int acc_in, acc_out;
    const float *alpha;
};
// the sum over a product's splits with linear's epilogue, or into D alone
hipError_t run_split_sum_linear(bool bf, int act, const SplitSumParams &q, hipStream_t s);
hipError_t run_split_sum_out(bool bf, const SplitSumParams &q, hipStream_t s);
// dbias [cols] = sum over parts of partial[part][cols]
hipError_t run_colsum(const float *partial, float *out, int parts, int cols, hipStream_t s);
// zeros in `rows` rows of `bytes` bytes (even), ld_bytes apart
hipError_t run_zero(void *p, int64_t ld_bytes, int64_t rows, int64_t bytes, hipStream_t s);

}  // namespace gemm_epi
