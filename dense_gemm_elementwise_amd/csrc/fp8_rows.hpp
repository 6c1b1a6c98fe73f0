// fp8_rows.hpp -- gfx950 products of up to 16 rows with 8-bit weights
// (include/fp8_ops.h), epilogue included.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8_convert.hpp"
#include "linear_gemm.hpp"
#include "row_pieces.hpp"

namespace gemm_epi {

constexpr int kFewRows = 16;       // of one MFMA operand
constexpr int kFewRows16Bit = 4;   // of one load of 16-bit rows

struct FewRows8 {
    const void *X;
    const uint8_t *XS, *W, *WS;
    int64_t ldx, ldxs, ldw, ldws;
    int M, N, K, act;
    const _Float16 *bias, *R;
    _Float16 *D, *Z;
    int64_t ldr, ldd, ldz;
};

// ---------------------------------------------------------------------------
// D = act(X W^T + bias) + R for M <= 16.  A workgroup takes 16 rows of W, its
// waves every WAVES-th block of 128 along K, each one MFMA; the waves' sums meet
// in LDS.  X is in 8 bits with scales, or (X8 = false, M <= 4) in 16 bits and
// quantised here as quantize_fp8 does, a block after the other: 60 instructions
// of a wave for 2 KB of W.  XL: the loads that a block of X's rows takes.
// Bound by reading W: one row, 8192 x 4096 6.8 us (4.9 TB/s; quantisation, a
// 128 x 128 tile in splits and their sum, each a launch, took 17); 16 rows in 8 bits 8.4.
// ---------------------------------------------------------------------------
template <bool BF, int FX, bool X8, int XL, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void fp8_few_rows_kernel(FewRows8 p)
{
    constexpr int DEPTH = WAVES == 4 ? 4 : 2, TOP = FX == 0 ? 8 : 15, ROWS = XL * (X8 ? 8 : 4);  // ROWS: loaded ones
    using RW = RowBlocks<1>;
    using RX = RowBlocks<X8 ? 1 : 2>;
    __shared__ __attribute__((aligned(16))) char turned[WAVES][2 * RW::BYTES];
    __shared__ uint8_t xscale[WAVES][kFewRows];
    __shared__ f32x4 red[WAVES][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), li = lane & 15,
              lg = lane >> 4;
    const int n0 = (int)blockIdx.x * 16;
    RW w;
    RX x;
    w.init((const char *)p.W + (int64_t)n0 * p.ldw, p.K, lane,
           [&](int r) { return (uint32_t)(min(r, p.N - 1 - n0) * (int)p.ldw); });
    x.init((const char *)p.X, p.K, lane, [&](int r) { return (uint32_t)(min(r, p.M - 1) * (int)p.ldx) * (X8 ? 1 : 2); });
    const uint8_t *ws = p.WS + (int64_t)(n0 >> 7) * p.ldws;  // (16 rows lie in one tile)
    const uint8_t *xs = X8 ? p.XS + (int64_t)min(li, p.M - 1) * p.ldxs : nullptr;
    struct Block {
        i32x4 w[RW::NL], x[XL];
        uint32_t sw, sx;
    } ring[DEPTH];
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    char *tw = turned[wave], *tx = tw + RW::BYTES;
    auto scales = [&](Block &b, int block) {
        b.sw = ws[block];
        if constexpr (X8) b.sx = xs[block];
    };
    auto fetch = [&](int d, int block) {
        w.load(ring[d].w, block);
        x.load(ring[d].x, block);
        scales(ring[d], block);
    };
    auto use = [&](int d, int finish) {  // finish: the block in which the rows end, or -1
        Block &b = ring[d];
        if (finish >= 0) {
            w.finish(b.w, finish);
            x.finish(b.x, finish);
        }
        RW::put(tw, b.w, lane);
        if constexpr (X8) {
            RX::put(tx, b.x, lane);
        } else {
#pragma unroll
            for (int v = 0; v < XL; v++) {
                const half8 h = __builtin_bit_cast(half8, b.x[v]);
                float f[8], m = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    f[e] = ld16<BF>(h[e]);
                    m = __builtin_fmaxf(m, __builtin_fabsf(f[e]));
                }
                if (!(m < __builtin_inff())) {
                    m = 0.0f;
#pragma unroll
                    for (int e = 0; e < 8; e++) m = __builtin_fmaxf(m, finite_abs(f[e]));
                }
                const int ex = block_exponent(row16_max(m), TOP);
                const float s = pow2f(-ex);
                const u32x2 q = {cvt4<FX>(f[0] * s, f[1] * s, f[2] * s, f[3] * s),
                                 cvt4<FX>(f[4] * s, f[5] * s, f[6] * s, f[7] * s)};
                *(u32x2 *)(tx + RW::at(v * 4 + lg, li >> 1) + (li & 1) * 8) = q;
                if (li == 0) xscale[wave][v * 4 + lg] = (uint8_t)(ex + 127);
            }
        }
        wave_lds_sync();
        // columns 16 lg .. and 64 + 16 lg .. of row li (of X: the rows that were loaded, again)
        auto operand = [&](const char *t, int row) {
            const i32x4 lo = *(const i32x4 *)(t + RW::at(row, lg)), hi = *(const i32x4 *)(t + RW::at(row, 4 + lg));
            return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        };
        const i32x8 a = operand(tx, li & (ROWS - 1)), bw = operand(tw, li);
        const int sx = X8 ? (int)b.sx : (int)xscale[wave][li & (ROWS - 1)];
        acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, bw, acc, FX, 0, 0, sx, 0, (int)b.sw);
        wave_lds_sync();
    };
    if (p.K < kShortRow) {
        if (wave == 0) {
            w.load_short(ring[0].w);
            x.load_short(ring[0].x);
            scales(ring[0], 0);
            use(0, -1);
        }
    } else {
        stream_row_blocks<DEPTH>(wave, WAVES, p.K, (int)blockIdx.x * 5 % max(p.K >> 7, 1), fetch, use);
    }
    red[wave][lane] = acc;  // tokens 4 lg .. of row li
    __syncthreads();
    const int m = tid >> 4, r = tid & 15;
    if (m >= p.M || n0 + r >= p.N) return;
    float v = 0.0f;
#pragma unroll
    for (int u = 0; u < WAVES; u++) v += ((const float *)&red[u][(m >> 2) * 16 + r])[m & 3];
    if (p.bias) v += ld16<BF>(p.bias[n0 + r]);
    if (p.Z) p.Z[m * p.ldz + n0 + r] = st16<BF>(v);
    v = p.act == ACT_RELU   ? lin_act<ACT_RELU>(v)
        : p.act == ACT_GELU ? lin_act<ACT_GELU>(v)
        : p.act == ACT_SILU ? lin_act<ACT_SILU>(v)
                            : v;
    p.D[m * p.ldd + n0 + r] = st16<BF>(p.R ? v + ld16<BF>(p.R[m * p.ldr + n0 + r]) : v);
}

}  // namespace gemm_epi
