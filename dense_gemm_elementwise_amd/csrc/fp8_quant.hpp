// fp8_quant.hpp -- quantisation to 8-bit floating point with a power-of-two
// scale for each block of 128 (include/fp8_ops.h), alone and of the gradient dZ.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8_convert.hpp"
#include "linear_gemm.hpp"
#include "ops_host.hpp"
#include "row_pieces.hpp"

namespace gemm_epi {

// Operands and scales that the products cannot read in place (rows off the
// 16-byte rule, scales off the 4-byte rule): copied to rows of ldo bytes, a
// multiple of 16, of which those from cols on are zeros.  16 bytes a thread and turn.
struct PadBytes {
    const uint8_t *src[4];
    uint8_t *dst[4];
    int64_t lds[4], ldo[4];
    int rows[4], cols[4];
    int n;
};
// thread `at` of `threads`
__device__ __forceinline__ void pad_bytes(const PadBytes &p, int64_t at, int64_t threads)
{
#pragma unroll 1
    for (int v = 0; v < p.n; v++) {
        const uint32_t pieces = (uint32_t)(p.ldo[v] / 16);
        const int64_t total = (int64_t)p.rows[v] * pieces;
        const int cols = p.cols[v];
        for (int64_t i = at; i < total; i += threads) {
            const int64_t r = i / pieces;
            const int c = (int)(i - r * pieces) * 16;
            const char *row = (const char *)p.src[v] + r * p.lds[v];
            i32x4 x;
            if (cols >= 16)
                x = move_down(load_piece<1>(row + min(c, cols - 16)), min(max(c + 16 - cols, 0), 16));
            else
                x = load_piece_short<1>(row + c, cols - c);
            *(i32x4 *)(p.dst[v] + r * p.ldo[v] + c) = x;
        }
    }
}
__global__ __launch_bounds__(256) void pad_bytes_kernel(PadBytes p)
{
    pad_bytes(p, (int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256);
}

struct QuantParams {
    const void *X;
    int64_t ldx;
    int R, C;
    uint8_t *Q, *S, *QT, *ST;
    int64_t ldq, lds, ldqt, ldst;
    // gradient: X is dD; Z and the column sums of dZ over each band of 128 rows
    const void *Z;
    int64_t ldz;
    float *partial;  // [bands][C], or NULL
    int bands;       // of 128 rows; the workgroups past them copy pad's operands
    PadBytes pad;
};

enum QuantSrc : int { QS_F16 = 0, QS_BF16 = 1, QS_F32 = 2 };
constexpr int kNoGrad = -1;

// 8 bytes at any address, the first n of which exist
__device__ __forceinline__ void store_bytes8(uint8_t *p, u32x2 v, int n)
{
    if (n >= 8) {
        *(u32x2u *)p = v;
        return;
    }
#pragma unroll
    for (int e = 0; e < 7; e++)
        if (e < n) p[e] = (uint8_t)(v[e >> 2] >> ((e & 3) * 8));
}

// ---------------------------------------------------------------------------
// One workgroup quantises one 128 x 128 block of X in registers: thread (tx, ty)
// holds rows 4 ty .. + 3 of columns 8 tx .. + 7, so a row's maximum is one over
// 16 adjacent lanes, a column's one over 4 lanes and the 8 waves.  The row-wise bytes
// leave as they are, 128 bytes a row; the transposed ones are turned around in
// LDS, 4 rows of a column (4 bytes) at a time.  Bound by the bytes: 2 in, 1 or 2 out.
// All loads are issued together, at the edge too: a row's last 16 bytes where the
// row ends inside them, moved down (with a branch a row and single elements at
// the edge, 2400 x 3233 of fp16 into both orientations 13.8 us, 12.0 so, 10.0
// with 16-bit elements kept packed; its bytes would take 6.4).
// ---------------------------------------------------------------------------
template <int SRC, bool TILE, bool BOTH, int FMT, int GRAD>
__global__ __launch_bounds__(512) void quant_kernel(QuantParams p)
{
    constexpr int TOP = FMT == 0 ? 8 : 15, RT = 4, WAVES = 8;  // RT: rows a thread
    constexpr bool BF = SRC == QS_BF16;
    constexpr int PITCH = 132;  // bytes of a column in LDS, off the bank stride
    constexpr bool WITH_Z = GRAD > ACT_IDENTITY;
    constexpr bool PACKED = SRC != QS_F32 && GRAD <= ACT_RELU;  // elements stay in 16 bits, two to a dword
    __shared__ __attribute__((aligned(16))) float colmax[WAVES][kBlock];  // (packed: dwords of two columns' magnitudes)
    __shared__ __attribute__((aligned(16))) int colscale[kBlock];
    __shared__ float tilemax[WAVES];
    __shared__ __attribute__((aligned(16))) uint8_t turned[BOTH ? kBlock * PITCH : 8];
    __shared__ float colsum[GRAD >= 0 ? WAVES : 1][kBlock];
    const int tid = threadIdx.x, wave = tid >> 6, tx = tid & 15, ty = tid >> 4;
    // (one axis: an axis of its own for the rows' blocks would end at 65535)
    const int across = (p.C + kBlock - 1) / kBlock, by = (int)blockIdx.x / across, bx = (int)blockIdx.x - by * across;
    const int r0 = by * kBlock, c0 = bx * kBlock;
    const int rows = min(p.R - r0, kBlock), cols = min(p.C - c0, kBlock);
    const int n = cols - tx * 8;  // columns that exist from this thread's on

    if constexpr (GRAD >= 0)
        if ((int)blockIdx.x >= p.bands * across) {
            pad_bytes(p.pad, ((int64_t)blockIdx.x - p.bands * across) * 512 + tid,
                      ((int64_t)gridDim.x - p.bands * across) * 512);
            return;
        }

    float v[RT][8];
    uint32_t d[RT][4];  // packed: columns 2 j and 2 j + 1
    if constexpr (SRC == QS_F32) {
        i32x4 x[RT][2];
#pragma unroll
        for (int i = 0; i < RT; i++) {
            const float *row = (const float *)p.X + (int64_t)(r0 + min(ty * RT + i, rows - 1)) * p.ldx;
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const int c = c0 + tx * 8 + h * 4;
                x[i][h] = p.C >= 4 ? load_piece<4>((const char *)(row + min(c, p.C - 4)))
                                   : load_piece_short<4>((const char *)(row + c), p.C - c);
            }
        }
#pragma unroll
        for (int i = 0; i < RT; i++)
#pragma unroll
            for (int h = 0; h < 2; h++) {
                if (cols < kBlock && p.C >= 4) x[i][h] = move_down(x[i][h], min(max(4 - (n - h * 4), 0), 4) * 4);
                const f32x4 f = __builtin_bit_cast(f32x4, x[i][h]);
#pragma unroll
                for (int e = 0; e < 4; e++) v[i][h * 4 + e] = f[e];
            }
    } else {
        i32x4 x[RT], z[WITH_Z ? RT : 1];
        auto load = [&](i32x4 (&f)[RT], const void *from, int64_t ld) {
            const int c = c0 + tx * 8;
#pragma unroll
            for (int i = 0; i < RT; i++) {
                const _Float16 *row = (const _Float16 *)from + (int64_t)(r0 + min(ty * RT + i, rows - 1)) * ld;
                f[i] = p.C >= 8 ? load_piece<2>((const char *)(row + min(c, p.C - 8)))
                                : load_piece_short<2>((const char *)(row + c), p.C - c);
            }
        };
        load(x, p.X, p.ldx);
        if constexpr (WITH_Z) load(z, p.Z, p.ldz);
        if (cols < kBlock && p.C >= 8) {
            const int miss = min(max(8 - n, 0), 8) * 2;
#pragma unroll
            for (int i = 0; i < RT; i++) {
                x[i] = move_down(x[i], miss);
                if constexpr (WITH_Z) z[i] = move_down(z[i], miss);
            }
        }
#pragma unroll
        for (int i = 0; i < RT; i++) {
            if constexpr (PACKED) {
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    d[i][j] = (uint32_t)x[i][j];
                    if constexpr (GRAD == ACT_RELU) {  // a mask, as in linear_backward: 0 where z <= 0, a NaN of z passes
                        const uint32_t zz = (uint32_t)z[i][j];
                        const float lo = value_u16<BF>(zz & 0xFFFF), hi = value_u16<BF>(zz >> 16);
                        d[i][j] = (lo <= 0.0f ? 0 : d[i][j] & 0xFFFF) | (hi <= 0.0f ? 0 : d[i][j] & 0xFFFF0000u);
                    }
                }
            } else {
                const half8 xv = __builtin_bit_cast(half8, x[i]);
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    v[i][e] = ld16<BF>(xv[e]);
                    // (behind the row's end both are 0, and the slope of 0 is finite)
                    if constexpr (WITH_Z) v[i][e] *= lin_act_grad<GRAD>(ld16<BF>(__builtin_bit_cast(half8, z[i])[e]));
                }
            }
        }
    }
    if (rows < kBlock)  // (the last row stands for those that are not there)
#pragma unroll
        for (int i = 0; i < RT; i++)
            if (ty * RT + i >= rows) {
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    if constexpr (PACKED)
                        d[i][e / 2] = 0;
                    else
                        v[i][e] = 0.0f;
                }
            }

    if constexpr (GRAD >= 0) {
        if (p.partial) {
            float s[8];
#pragma unroll
            for (int e = 0; e < 8; e++) {
                if constexpr (PACKED) {
                    auto f = [&](int i) { return value_u16<BF>(e & 1 ? d[i][e / 2] >> 16 : d[i][e / 2] & 0xFFFF); };
                    s[e] = (f(0) + f(1)) + (f(2) + f(3));
                } else {
                    s[e] = (v[0][e] + v[1][e]) + (v[2][e] + v[3][e]);
                }
                s[e] += __shfl_xor(s[e], 16);
                s[e] += __shfl_xor(s[e], 32);
            }
            if ((tid & 63) < 16) {
#pragma unroll
                for (int e = 0; e < 8; e++) colsum[wave][tx * 8 + e] = s[e];
            }
            __syncthreads();
            if (tid < cols) {
                float sum = 0.0f;
#pragma unroll
                for (int w = 0; w < WAVES; w += 2) sum += colsum[w][tid] + colsum[w + 1][tid];
                p.partial[(int64_t)by * p.C + c0 + tid] = sum;
            }
        }
    }

    // the rows' maxima; where one is infinite, the finite elements' alone
    // (v_max drops a NaN by itself)
    float rm[RT];
    uint32_t size[RT][4];  // packed: magnitudes, 0 for what is not finite
#pragma unroll
    for (int i = 0; i < RT; i++) {
        if constexpr (PACKED) {
#pragma unroll
            for (int j = 0; j < 4; j++) size[i][j] = d[i][j] & 0x7FFF7FFFu;
            uint32_t m = max_u16x2(max_u16x2(size[i][0], size[i][1]), max_u16x2(size[i][2], size[i][3]));
            if (has_not_finite<BF>(m)) {
#pragma unroll
                for (int j = 0; j < 4; j++) size[i][j] = finite_u16x2<BF>(size[i][j]);
                m = max_u16x2(max_u16x2(size[i][0], size[i][1]), max_u16x2(size[i][2], size[i][3]));
            }
            rm[i] = larger_of<BF>(m);
        } else {
            rm[i] = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; e++) rm[i] = __builtin_fmaxf(rm[i], __builtin_fabsf(v[i][e]));
            if (!(rm[i] < __builtin_inff())) {
                rm[i] = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; e++) rm[i] = __builtin_fmaxf(rm[i], finite_abs(v[i][e]));
            }
        }
    }
    int ex[RT];
    if constexpr (TILE) {
        float m = __builtin_fmaxf(__builtin_fmaxf(rm[0], rm[1]), __builtin_fmaxf(rm[2], rm[3]));
        m = row16_max(m);
        m = __builtin_fmaxf(m, __shfl_xor(m, 16));
        m = __builtin_fmaxf(m, __shfl_xor(m, 32));
        if ((tid & 63) == 0) tilemax[wave] = m;
        __syncthreads();
        m = tilemax[0];
#pragma unroll
        for (int w = 1; w < WAVES; w++) m = __builtin_fmaxf(m, tilemax[w]);
        const int e = block_exponent(m, TOP);
#pragma unroll
        for (int i = 0; i < RT; i++) ex[i] = e;
        if (tid == 0) {
            p.S[(int64_t)by * p.lds + bx] = (uint8_t)(e + 127);
            if (BOTH) p.ST[(int64_t)bx * p.ldst + by] = (uint8_t)(e + 127);
        }
    } else {
#pragma unroll
        for (int i = 0; i < RT; i++) ex[i] = block_exponent(row16_max(rm[i]), TOP);
        if (tx == 0) {
#pragma unroll
            for (int i = 0; i < RT; i++)
                if (ty * RT + i < rows)
                    p.S[(int64_t)(r0 + ty * RT + i) * p.lds + bx] = (uint8_t)(ex[i] + 127);
        }
    }
#pragma unroll
    for (int i = 0; i < RT; i++) {
        u32x2 q;
        if constexpr (PACKED) {
            q = u32x2{cvt4_16<FMT, BF>(d[i][0], d[i][1], ex[i]), cvt4_16<FMT, BF>(d[i][2], d[i][3], ex[i])};
        } else {
            const float f = pow2f(-ex[i]);
            q = u32x2{cvt4<FMT>(v[i][0] * f, v[i][1] * f, v[i][2] * f, v[i][3] * f),
                      cvt4<FMT>(v[i][4] * f, v[i][5] * f, v[i][6] * f, v[i][7] * f)};
        }
        if (ty * RT + i < rows) store_bytes8(p.Q + (int64_t)(r0 + ty * RT + i) * p.ldq + c0 + tx * 8, q, n);
    }
    if constexpr (BOTH) {
        int ec[8];
        if constexpr (TILE) {
#pragma unroll
            for (int e = 0; e < 8; e++) ec[e] = ex[0];
        } else {
            if constexpr (PACKED) {
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    uint32_t m = max_u16x2(max_u16x2(size[0][j], size[1][j]), max_u16x2(size[2][j], size[3][j]));
                    m = max_u16x2(m, (uint32_t)__shfl_xor((int)m, 16));
                    m = max_u16x2(m, (uint32_t)__shfl_xor((int)m, 32));
                    if ((tid & 63) < 16) ((uint32_t *)colmax[wave])[tx * 4 + j] = m;
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    float m = 0.0f;
#pragma unroll
                    for (int i = 0; i < RT; i++) m = __builtin_fmaxf(m, __builtin_fabsf(v[i][e]));
                    if (!(m < __builtin_inff())) {
                        m = 0.0f;
#pragma unroll
                        for (int i = 0; i < RT; i++) m = __builtin_fmaxf(m, finite_abs(v[i][e]));
                    }
                    m = __builtin_fmaxf(m, __shfl_xor(m, 16));
                    m = __builtin_fmaxf(m, __shfl_xor(m, 32));
                    if ((tid & 63) < 16) colmax[wave][tx * 8 + e] = m;
                }
            }
            __syncthreads();
            if (tid < kBlock) {  // the column's scale, for all that hold a part of it
                float m;
                if constexpr (PACKED) {
                    uint32_t u = 0;
#pragma unroll
                    for (int w = 0; w < WAVES; w++) u = max(u, (uint32_t)((const unsigned short *)colmax[w])[tid]);
                    m = value_u16<BF>(u);
                } else {
                    m = colmax[0][tid];
#pragma unroll
                    for (int w = 1; w < WAVES; w++) m = __builtin_fmaxf(m, colmax[w][tid]);
                }
                const int e = block_exponent(m, TOP);
                if (tid < cols) p.ST[(int64_t)(c0 + tid) * p.ldst + by] = (uint8_t)(e + 127);
                colscale[tid] = e;
            }
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 8; e++) ec[e] = colscale[tx * 8 + e];
        }
#pragma unroll
        for (int e = 0; e < 8; e++) {
            uint32_t q;
            if constexpr (PACKED) {
                const uint32_t half = e & 1 ? 0x07060302u : 0x05040100u;  // the column's of two dwords
                q = cvt4_16<FMT, BF>(__builtin_amdgcn_perm(d[1][e / 2], d[0][e / 2], half),
                                     __builtin_amdgcn_perm(d[3][e / 2], d[2][e / 2], half), ec[e]);
            } else {
                const float f = pow2f(-ec[e]);
                q = cvt4<FMT>(v[0][e] * f, v[1][e] * f, v[2][e] * f, v[3][e] * f);
            }
            *(uint32_t *)(turned + (tx * 8 + e) * PITCH + ty * RT) = q;
        }
        __syncthreads();
        // 8 threads a column, 16 bytes each
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const int c = i * 64 + (tid >> 3), at = (tid & 7) * 16, m = rows - at;
            const uint32_t *from = (const uint32_t *)(turned + c * PITCH + at);
            const u32x4 w = {from[0], from[1], from[2], from[3]};
            if (c < cols && m > 0) {
                uint8_t *q = p.QT + (int64_t)(c0 + c) * p.ldqt + r0 + at;
                if (m >= 16) {
                    *(u32x4u *)q = w;
                } else {
                    store_bytes8(q, u32x2{w[0], w[1]}, m);
                    if (m > 8) store_bytes8(q + 8, u32x2{w[2], w[3]}, m - 8);
                }
            }
        }
    }
}

}  // namespace gemm_epi
