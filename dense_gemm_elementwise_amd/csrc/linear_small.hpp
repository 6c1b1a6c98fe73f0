// linear_small.hpp -- the kernels around the matrix products of
// linear_gemm.hpp: products with few rows, dZ and the bias gradient, the sum
// over splits of the contraction, operand staging, and the row passes of the
// cross entropy.  All are bound by memory or by latency.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "linear_gemm.hpp"
#include "ops_host.hpp"

namespace gemm_epi {

// Workgroups of one row (or one block of columns) each: a launch holds fewer
// than 2^32 threads along x, so past 2^21 rows (1024 threads each at most) the
// rows go on along y.
constexpr int64_t kRowGrid = 1 << 21;
__device__ __forceinline__ int64_t block_row() { return (int64_t)blockIdx.y * kRowGrid + blockIdx.x; }

// ---------------------------------------------------------------------------
// Products with at most 16 rows of X (single tokens, small batches of them):
// bound by reading W once.  No LDS on the way in, 16-byte loads at any
// alignment, and plain loads: non-temporal ones were 15-18% slower.
//   row_dot_kernel: a wave reads one row of W, 1 KB contiguous per load,
//     against the rows of X in fp32 multiply-adds;
//   skinny_kernel: a wave reads 16 rows of W, 64 bytes of each per load,
//     straight into the operand layout of one 16x16x32 MFMA against all rows of
//     X, as fast whatever the rows of X.
// Whole calls with W in HBM, us, row_dot_kernel first: one row of X, bf16,
// 100003 x 4096 (loss) 137 and 161 (6.0 and 5.1 TB/s), 28672 x 8192 82 and 92,
// 8192 x 4096 14.2 and 16.2, 4096 x 11008 23.1 and 21.9; fp16 the same within 15%
// (20.4 and 21.9).  Two rows, where the multiply-adds start to count: fp16, whose
// operands convert inside them, 154 and 162, 93.7 and 93.3, 14.8 and 16.5, 22.6
// and 21.8; bf16, with a shift for each, 169 and 162, 103 and 93, 18.6 and 16.5,
// 30.4 and 21.8.  So row_dot_kernel takes one row, and two of fp16.
// ---------------------------------------------------------------------------
struct SkinnyParams {
    const _Float16 *X, *W;
    int64_t ldx, ldw;
    int M, N, K;
    const _Float16 *bias, *R;
    _Float16 *D, *Z;
    int64_t ldr, ldd, ldz;
    const int64_t *target;
    float *part_max, *part_sum, *tlogit;
    int nparts;
    const XentRow *rows;  // SK_P: row data; D is P, W the piece's first row, v0 its vocabulary index
    int v0;
};

// Joins the four waves' running (maximum, sum) of M rows and leaves them in the
// workgroup's column (`part`) of the partial statistics; red: [2][4][MX].
template <int MX>
__device__ __forceinline__ void xent_part(float *red, int M, float *part_max, float *part_sum, int nparts, int part)
{
    __syncthreads();
    const int tid = threadIdx.x;
    if (tid >= M) return;
    float m = red[tid], s = red[4 * MX + tid];
#pragma unroll
    for (int u = 1; u < 4; u++) softmax_join(m, s, red[u * MX + tid], red[4 * MX + u * MX + tid]);
    const int64_t o = (int64_t)tid * nparts + part;
    part_max[o] = m;
    part_sum[o] = s;
}

// One row of W per wave and turn, rows dealt out over all waves; lane l takes
// columns 8 l + 512 i.  MX: M, 1 or 2.  In the cross entropy a
// wave keeps a running maximum and sum over its rows.
template <bool BF, bool XENT, int ACT, int MX>
__global__ __launch_bounds__(256, 8) void row_dot_kernel(SkinnyParams p)
{
    __shared__ float red[2 * 4 * MX];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    constexpr int U = 4 / MX;  // groups of 512 columns whose loads are in flight together
    const int mine = lane < p.M ? lane : 0;  // lanes 0 .. M-1 finish one row of X each
    const int64_t target = XENT ? p.target[mine] : 0;
    float top = -__builtin_inff(), sum = 0.0f;
    // (unsigned: the step past the last row of a vocabulary near 2^31 leaves int)
    for (uint32_t n = blockIdx.x * 4 + wave; n < (uint32_t)p.N; n += gridDim.x * 4) {
        const _Float16 *w = p.W + (int64_t)n * p.ldw;
        float bias = 0.0f, res = 0.0f;
        if constexpr (!XENT) {
            if (p.bias) bias = ld16<BF>(p.bias[n]);
            if (p.R) res = ld16<BF>(p.R[mine * p.ldr + n]);
        }
        float acc[MX] = {};
        auto add = [&](const half8 &wv, const half8 &xv, int m) {
#pragma unroll
            for (int e = 0; e < 8; e++) acc[m] = __builtin_fmaf(ld16<BF>(wv[e]), ld16<BF>(xv[e]), acc[m]);
        };
        int k = 0;
        for (; k + 512 * U <= p.K; k += 512 * U) {
            half8 wv[U], xv[U][MX];
#pragma unroll
            for (int u = 0; u < U; u++) wv[u] = *(const half8u *)(w + k + u * 512 + lane * 8);
#pragma unroll
            for (int u = 0; u < U; u++)
#pragma unroll
                for (int m = 0; m < MX; m++)
                    xv[u][m] = *(const half8u *)(p.X + min(m, p.M - 1) * p.ldx + k + u * 512 + lane * 8);
#pragma unroll
            for (int u = 0; u < U; u++)
#pragma unroll
                for (int m = 0; m < MX; m++) add(wv[u], xv[u][m], m);
        }
        for (k += lane * 8; k < p.K; k += 512) {
            const half8 wv = load8(w + k, p.K - k);
#pragma unroll
            for (int m = 0; m < MX; m++) add(wv, load8(p.X + min(m, p.M - 1) * p.ldx + k, p.K - k), m);
        }
        float v = 0.0f;  // lane m: row m's sum
#pragma unroll
        for (int m = 0; m < MX; m++) {
            float a = row16_sum(acc[m]);
            a += __shfl_xor(a, 16);
            a += __shfl_xor(a, 32);
            if (lane == m) v = a;
        }
        if constexpr (XENT) {
            if (lane < p.M) {
                softmax_join(top, sum, v, 1.0f);
                if (target == n) p.tlogit[lane] = v;
            }
        } else if (lane < p.M) {
            const float z = v + bias;
            if (p.Z) p.Z[lane * p.ldz + n] = st16<BF>(z);
            p.D[lane * p.ldd + n] = st16<BF>(lin_act<ACT>(z) + res);
        }
    }
    if constexpr (XENT) {
        if (lane < MX) {
            red[wave * MX + lane] = top;
            red[4 * MX + wave * MX + lane] = sum;
        }
        xent_part<MX>(red, p.M, p.part_max, p.part_sum, p.nparts, blockIdx.x);
    }
}

// A wave holds 16 rows of W against all rows of X in one MFMA block; a lane
// reads 16 bytes of a W row per MFMA, 8 MFMAs (512 contiguous bytes a row) per
// group of loads and the next group's loads in flight.  Rows past N or M repeat
// the last one and are never stored.
//   linear: the workgroup's four waves take turns over K for the same 16
//     rows (N / 16 workgroups fill the chip from N = 4096 on), their sums meet
//     in LDS, 256 threads apply the epilogue.
//   cross entropy: the same below a vocabulary of 32768, and past it 16 rows
//     and all of K for every wave (64 columns a workgroup fill the chip); the
//     workgroup leaves the softmax statistics of its columns, or, in the gradient, its part of P (11 rows against 7824 x 2176
//     f16: 12 us; the 128 x 128 tiles take 22).
enum SkinnyMode : int { SK_LINEAR = 0, SK_STATS = 1, SK_P = 2 };
template <bool BF, int MODE, int ACT, bool SPLIT>
__global__ __launch_bounds__(256) void skinny_kernel(SkinnyParams p)
{
    constexpr int U = 8, SPAN = 32 * U;
    constexpr bool XENT = MODE != SK_LINEAR;
    __shared__ float red[SPLIT ? 4 * 256 : 2 * 4 * 16];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int li = lane & 15, lg = lane >> 4;
    const int block = (int)block_row();
    if (block >= (p.N + (SPLIT ? 15 : 63)) / (SPLIT ? 16 : 64)) return;  // (the grid's last row of blocks)
    const int n0 = SPLIT ? block * 16 : block * 64 + wave * 16;
    const _Float16 *w = p.W + (int64_t)min(n0 + li, p.N - 1) * p.ldw + lg * 8;
    const _Float16 *x = p.X + (int64_t)min(li, p.M - 1) * p.ldx + lg * 8;
    const int step = SPLIT ? 4 * SPAN : SPAN;
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    half8 wv[U], xv[U];
    auto fetch = [&](int k0) {
        if (k0 + SPAN <= p.K) {
#pragma unroll
            for (int u = 0; u < U; u++) wv[u] = *(const half8u *)(w + k0 + u * 32);
#pragma unroll
            for (int u = 0; u < U; u++) xv[u] = *(const half8u *)(x + k0 + u * 32);
        } else {
#pragma unroll
            for (int u = 0; u < U; u++) {
                const int n = p.K - (k0 + u * 32 + lg * 8);
                wv[u] = load8(w + k0 + u * 32, n);
                xv[u] = load8(x + k0 + u * 32, n);
            }
        }
    };
    int k0 = SPLIT ? wave * SPAN : 0;
    if (k0 < p.K) fetch(k0);
    while (k0 < p.K) {
        half8 wc[U], xc[U];
#pragma unroll
        for (int u = 0; u < U; u++) {
            wc[u] = wv[u];
            xc[u] = xv[u];
        }
        k0 += step;
        if (k0 < p.K) fetch(k0);
#pragma unroll
        for (int u = 0; u < U; u++) {
            if constexpr (BF)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, wc[u]),
                                                              __builtin_bit_cast(bf16x8, xc[u]), acc, 0, 0, 0);
            else
                acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(wc[u], xc[u], acc, 0, 0, 0);
        }
    }
    // lane (li, lg), register r: row li of X, row 4 lg + r of W
    if constexpr (SPLIT) {
        *(f32x4 *)(red + (wave * 64 + lane) * 4) = acc;
        __syncthreads();
    }
    if constexpr (XENT && SPLIT) {  // the first wave goes on with the sums
        if (wave != 0) return;
        acc = (acc + *(const f32x4 *)(red + (64 + lane) * 4)) +
              (*(const f32x4 *)(red + (128 + lane) * 4) + *(const f32x4 *)(red + (192 + lane) * 4));
    }
    if constexpr (!XENT) {
        const int wr = tid & 15, xr = tid >> 4;  // adjacent threads on adjacent columns of D
        const int at = ((wr >> 2) * 16 + xr) * 4 + (wr & 3);
        const int n = n0 + wr;
        if (xr < p.M && n < p.N) {
            const float s = (red[at] + red[256 + at]) + (red[512 + at] + red[768 + at]);
            const float z = s + (p.bias ? ld16<BF>(p.bias[n]) : 0.0f);
            const float r = p.R ? ld16<BF>(p.R[xr * p.ldr + n]) : 0.0f;
            if (p.Z) p.Z[xr * p.ldz + n] = st16<BF>(z);
            p.D[xr * p.ldd + n] = st16<BF>(lin_act<ACT>(z) + r);
        }
    } else if constexpr (MODE == SK_P) {
        // as in the tiles' epilogue: lane (li, lg) has 4 columns of row li
        const int col = n0 + 4 * lg;
        if (li >= p.M || col >= (p.N + 7) / 8 * 8) return;
        const XentRow row = p.rows[li];
        const float c = row.lse * kLog2e;
        half4 h;
#pragma unroll
        for (int r = 0; r < 4; r++) {
            float pr = exp2_hw(__builtin_fmaf(acc[r], kLog2e, -c));
            if (row.target - p.v0 == col + r) pr -= 1.0f;
            pr *= row.scale;
            h[r] = st16<BF>(row.ignored || col + r >= p.N ? 0.0f : pr);
        }
        *(half4 *)(p.D + li * p.ldd + col) = h;
    } else {
        float m = -__builtin_inff();
        const int64_t t = li < p.M ? p.target[li] : -1;
#pragma unroll
        for (int r = 0; r < 4; r++) {
            const int v = n0 + 4 * lg + r;
            if (v >= p.N) acc[r] = -__builtin_inff();
            if (li < p.M && v < p.N && v == t) p.tlogit[li] = acc[r];
            m = __builtin_fmaxf(m, acc[r]);
        }
        m = __builtin_fmaxf(m, __shfl_xor(m, 16));
        m = __builtin_fmaxf(m, __shfl_xor(m, 32));
        const float ref = m == -__builtin_inff() ? 0.0f : m;
        float s = 0.0f;
#pragma unroll
        for (int r = 0; r < 4; r++) s += exp2_hw((acc[r] - ref) * kLog2e);
        s += __shfl_xor(s, 16);
        s += __shfl_xor(s, 32);
        if constexpr (SPLIT) {
            if (lg == 0 && li < p.M) {
                p.part_max[(int64_t)li * p.nparts + block] = m;
                p.part_sum[(int64_t)li * p.nparts + block] = s;
            }
            return;
        }
        if (lg == 0) {
            red[wave * 16 + li] = m;
            red[64 + wave * 16 + li] = s;
        }
        xent_part<16>(red, p.M, p.part_max, p.part_sum, p.nparts, block);
    }
}

// ---------------------------------------------------------------------------
// Staging: operands whose rows are not 16-byte aligned, or not a multiple of
// 8 elements long, are copied to rows of ldo elements (a multiple of 8), zeros
// past the row's end.  One grid row per tensor.
// ---------------------------------------------------------------------------
struct PadParams {
    const _Float16 *src[2];
    _Float16 *dst[2];
    int64_t lds[2], rows[2];
    int cols, ldo;
};
// tensor v's part of block `block` of `blocks`
__device__ __forceinline__ void pad_rows(const PadParams &p, int v, int block, int blocks)
{
    const int groups = p.ldo / 8;
    const int64_t total = p.rows[v] * groups;
    for (int64_t i = (int64_t)block * 256 + threadIdx.x; i < total; i += (int64_t)blocks * 256) {
        const int64_t r = i / groups;
        const int c = (int)(i - r * groups) * 8;
        *(half8 *)(p.dst[v] + r * p.ldo + c) = load8(p.src[v] + r * p.lds[v] + c, p.cols - c);
    }
}
__global__ __launch_bounds__(256) void pad_rows_kernel(PadParams p)
{
    pad_rows(p, blockIdx.y, blockIdx.x, gridDim.x);
}

// ---------------------------------------------------------------------------
// dZ = dD act'(Z), rounded once to the element type (it is an MFMA operand),
// in rows of ldo elements zero-padded to a multiple of 8 columns, and the
// column sums of the unrounded dZ over each strip of rows.  A block covers 256
// columns x a strip: 32 lanes of 8 columns by 8 rows at a time; one pass over
// dD and Z, bound by their bytes (8192 x 8192: 72 us, 5.6 TB/s).  The blocks past
// dz_blocks stage the products' other operands in the same launch.
// ---------------------------------------------------------------------------
struct DzParams {
    const _Float16 *dD, *Z;
    int64_t ldd, ldz, ldo;
    _Float16 *out;  // NULL: only the sums (identity, dD usable as it is)
    float *partial;  // [strips][N], or NULL
    int M, N, N8, rows_per_strip;
    int cols_blocks, dz_blocks;  // blocks of 256 columns; all blocks of dZ
    PadParams pad;
    int pads;  // tensors to stage
};

template <bool BF, int ACT>
__global__ __launch_bounds__(256) void dz_kernel(DzParams p)
{
    __shared__ float red[8][256 + 8];
    if ((int)blockIdx.x >= p.dz_blocks) {
        for (int v = 0; v < p.pads; v++)
            pad_rows(p.pad, v, (int)blockIdx.x - p.dz_blocks, (int)gridDim.x - p.dz_blocks);
        return;
    }
    const int strip = (int)blockIdx.x / p.cols_blocks, cb = (int)blockIdx.x - strip * p.cols_blocks;
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int c = cb * 256 + tx * 8;
    const int n = p.N - c;  // columns that exist from c on
    // (the strip's length before the end: r0 + rows_per_strip may pass 2^31)
    const int r0 = strip * p.rows_per_strip, r1 = r0 + min(p.M - r0, p.rows_per_strip);
    float sum[8] = {};
    if (c < p.N8) {
        auto one = [&](int m, half8 d, half8 z) {
            half8 o;
#pragma unroll
            for (int e = 0; e < 8; e++) {
                float v = ld16<BF>(d[e]);
                if constexpr (ACT == ACT_RELU)
                    // a mask: an infinity or a NaN that arrives at z <= 0 does not
                    // pass either; a NaN z, which the forward keeps, lets dD pass
                    v = ld16<BF>(z[e]) <= 0.0f ? 0.0f : v;
                else if constexpr (ACT != ACT_IDENTITY)
                    v *= lin_act_grad<ACT>(ld16<BF>(z[e]));
                if (e >= n) v = 0.0f;
                sum[e] += v;
                o[e] = st16<BF>(v);
            }
            if (p.out) *(half8 *)(p.out + (int64_t)m * p.ldo + c) = o;
        };
        int m = r0 + ty;
        for (; m + 24 < r1; m += 32) {  // four rows' loads in flight
            half8 d[4], z[4] = {};
#pragma unroll
            for (int u = 0; u < 4; u++) {
                d[u] = load8(p.dD + (int64_t)(m + 8 * u) * p.ldd + c, n);
                if constexpr (ACT != ACT_IDENTITY) z[u] = load8(p.Z + (int64_t)(m + 8 * u) * p.ldz + c, n);
            }
#pragma unroll
            for (int u = 0; u < 4; u++) one(m + 8 * u, d[u], z[u]);
        }
        for (; m < r1; m += 8) {
            const half8 d = load8(p.dD + (int64_t)m * p.ldd + c, n);
            half8 z = {};
            if constexpr (ACT != ACT_IDENTITY) z = load8(p.Z + (int64_t)m * p.ldz + c, n);
            one(m, d, z);
        }
    }
    if (!p.partial) return;
#pragma unroll
    for (int e = 0; e < 8; e++) red[ty][tx * 8 + e] = sum[e];
    __syncthreads();
    const int col = cb * 256 + threadIdx.x;
    float s = 0.0f;
#pragma unroll
    for (int y = 0; y < 8; y++) s += red[y][threadIdx.x];
    if (col < p.N) p.partial[(int64_t)strip * p.N + col] = s;
}

// The last step of every column sum: out[c] = sum over parts, in a fixed order,
// of partial[part][c].  Grid row 0 and 1 are two sums over all parts; grid rows
// from 2 on are the groups of a third, each over parts of its own.  64 columns
// per block; 16 groups of threads take every 16th part, 8 loads in flight.
struct ColSumParams {
    const float *partial[3];
    float *out[3];  // NULL: not wanted
    int parts[3];
    int ld, cols;
};
__global__ __launch_bounds__(1024) void colsum_kernel(ColSumParams p)
{
    __shared__ float red[16][64];
    const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
    const int c = blockIdx.x * 64 + tx, v = min((int)blockIdx.y, 2), g = (int)blockIdx.y - v;
    if (!p.out[v]) return;
    const int parts = p.parts[v];
    const float *src = p.partial[v] + (int64_t)g * parts * p.ld + c;
    float s = 0.0f;
    if (c < p.cols) {
        int i = ty;
        for (; i + 112 < parts; i += 128) {
            float x[8];
#pragma unroll
            for (int u = 0; u < 8; u++) x[u] = src[(int64_t)(i + 16 * u) * p.ld];
            s += ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
        }
        for (; i < parts; i += 16) s += src[(int64_t)i * p.ld];
    }
    red[ty][tx] = s;
    __syncthreads();
    if (ty == 0 && c < p.cols) {
        s = 0.0f;
#pragma unroll
        for (int u = 0; u < 16; u++) s += red[u][tx];
        p.out[v][(int64_t)g * p.cols + c] = s;
    }
}

// ---------------------------------------------------------------------------
// The sum over the splits of a product's contraction and the epilogue the
// product would have had: 8 columns per thread, or, where there are many
// splits of a small product, per `lanes` adjacent threads that take every
// lanes-th split (3 x 200 over 64 splits: 19 us in one thread each).  The order is
// fixed by the plan.
// ---------------------------------------------------------------------------
template <bool BF, int EPI, int ACT>
__global__ __launch_bounds__(256) void split_sum_kernel(SplitSumParams p)
{
    const int groups = (p.N + 7) / 8;
    const int64_t total = (int64_t)p.M * groups, step = (int64_t)gridDim.x * 256 / p.lanes;
    const int lane = threadIdx.x & (p.lanes - 1);
    float alpha = 1.0f;
    if constexpr (EPI == LE_OUT)
        if (p.alpha) alpha = *p.alpha;
    // (whole groups of lanes stay in the loop together: they exchange sums)
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) / p.lanes; i < total; i += step) {
        const int m = (int)(i / groups), c = (int)(i - (int64_t)m * groups) * 8, n = p.N - c;
        const float *src = p.part + (int64_t)m * p.ldc + c + lane * p.c_split;
        float v[8] = {};
        if (EPI == LE_OUT && p.acc_in && lane == 0) {
            const float *a = p.C32 + (int64_t)m * p.ldc + c;
#pragma unroll
            for (int e = 0; e < 8; e++) v[e] = a[e];
        }
        for (int s = lane; s < p.splits; s += p.lanes, src += p.lanes * p.c_split) {
            const f32x4 a = *(const f32x4 *)src, b = *(const f32x4 *)(src + 4);
#pragma unroll
            for (int e = 0; e < 4; e++) {
                v[e] += a[e];
                v[4 + e] += b[e];
            }
        }
        if (p.lanes > 1) {
#pragma unroll
            for (int e = 0; e < 8; e++) {
                v[e] += __shfl_xor(v[e], 1);
                v[e] += __shfl_xor(v[e], 2);
                if (p.lanes > 4) v[e] += __shfl_xor(v[e], 4);
            }
            if (lane) continue;
        }
        half8 d, z;
        if constexpr (EPI == LE_LINEAR) {
            half8 bias = {}, r = {};
            if (p.bias) bias = load8(p.bias + c, n);
            if (p.R) r = load8(p.R + (int64_t)m * p.ldr + c, n);
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const float t = v[e] + ld16<BF>(bias[e]);
                z[e] = st16<BF>(t);
                d[e] = st16<BF>(lin_act<ACT>(t) + ld16<BF>(r[e]));
            }
            if (p.Z) store8(p.Z + (int64_t)m * p.ldz + c, z, n);
            store8(p.D + (int64_t)m * p.ldd + c, d, n);
        } else if (p.acc_out) {
            float *a = p.C32 + (int64_t)m * p.ldc + c;
            *(f32x4 *)a = f32x4{v[0], v[1], v[2], v[3]};
            *(f32x4 *)(a + 4) = f32x4{v[4], v[5], v[6], v[7]};
        } else {
#pragma unroll
            for (int e = 0; e < 8; e++) d[e] = st16<BF>(v[e] * alpha);
            store8(p.D + (int64_t)m * p.ldd + c, d, n);
        }
    }
}

// Zeros (gradients of an empty batch): a kernel, so that the call records into a HIP graph.
__global__ __launch_bounds__(256) void zero_rows_kernel(char *dst, int64_t ld_bytes, int64_t rows, int64_t halves)
{
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * halves; i += (int64_t)gridDim.x * 256)
        *(uint16_t *)(dst + i / halves * ld_bytes + i % halves * 2) = 0;
}

// ---------------------------------------------------------------------------
// Cross entropy, the row passes.
// ---------------------------------------------------------------------------
// Joins the column tiles' (maximum, sum) pairs of one row per block.
__global__ __launch_bounds__(256) void xent_loss_kernel(int64_t T, const float *part_max, const float *part_sum,
                                                        int nparts, const float *tlogit, const int64_t *target,
                                                        int64_t V, int64_t ignore, float *loss, float *lse)
{
    __shared__ float rm[4], rs[4];
    const int64_t row = block_row();
    if (row >= T) return;
    const float *pm = part_max + row * nparts, *ps = part_sum + row * nparts;
    float m = -__builtin_inff(), s = 0.0f;
    for (int i = threadIdx.x; i < nparts; i += blockDim.x) softmax_join(m, s, pm[i], ps[i]);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const float m2 = __shfl_xor(m, o), s2 = __shfl_xor(s, o);
        softmax_join(m, s, m2, s2);
    }
    if ((threadIdx.x & 63) == 0) {
        rm[threadIdx.x >> 6] = m;
        rs[threadIdx.x >> 6] = s;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int u = 1; u < (int)blockDim.x / 64; u++) softmax_join(m, s, rm[u], rs[u]);
        const float l = m + logf(s);
        const int64_t t = target[row];
        lse[row] = l;
        if (t == ignore)
            loss[row] = 0.0f;
        else if (t < 0 || t >= V)
            loss[row] = __builtin_nanf("");
        else
            loss[row] = l - tlogit[row];
    }
}

// The gradient's row data.  P is stored in 16 bits, and fp16 has no room for
// a probability of 1e-6 times a loss of 1/T.  So the incoming gradients are
// divided by the largest of their magnitudes (fp32) and multiplied by 2^14:
// |P| stays below 2^14 + 1 < 65504 and a probability down to 2^-28 is still a
// normal number.  The products' fp32 sums are multiplied by that magnitude
// times 2^-14 (`alpha`) before their one rounding.  There is one factor for all
// rows, because dW adds them up: in a row whose incoming gradient is r times the
// largest, fp16 keeps all its digits down to a probability of 2^-28 / r, and
// entries below are off by at most 2^-39 of the largest incoming gradient (bf16
// has fp32's range and keeps them).  Dividing by the magnitude
// itself, not by the power of two below it, keeps the entry at the target, near
// -1 in a row of the largest gradient, where 16 bits hold it best: a mean over
// the batch has only such rows, and fp16 gradients of a 333 x 9999 batch came
// out 1.5 times as far from exact with the power of two.  One block; T values
// are read twice.
__global__ __launch_bounds__(1024) void xent_rows_kernel(int T, int64_t V, int64_t ignore, const float *dloss,
                                                         const float *lse, const int64_t *target, XentRow *rows,
                                                         float *alpha)
{
    __shared__ float red[16];
    float top = 0.0f;
    for (int64_t t = threadIdx.x; t < T; t += 1024) {
        const float a = __builtin_fabsf(dloss[t]);
        if (target[t] != ignore && a < __builtin_inff()) top = __builtin_fmaxf(top, a);
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) top = __builtin_fmaxf(top, __shfl_xor(top, o));
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 16; u++) top = __builtin_fmaxf(top, red[u]);
    if (threadIdx.x == 0) *alpha = top * 0x1p-14f;
    const float div = top > 0.0f ? top : 1.0f;
    for (int64_t t = threadIdx.x; t < T; t += 1024) {
        const int64_t c = target[t];
        XentRow r;
        r.lse = lse[t];
        r.ignored = c == ignore;
        r.target = c >= 0 && c < V ? (int)c : -1;
        r.scale = dloss[t] / div * 0x1p14f;
        if (!r.ignored && r.target < 0) r.scale = __builtin_nanf("");
        rows[t] = r;
    }
}

}  // namespace gemm_epi
