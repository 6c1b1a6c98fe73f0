// fp8_gemm.hpp -- gfx950 products of 8-bit matrices with block scales
// (include/fp8_ops.h).
//
// One workgroup of four waves computes one BM x BN tile of
//   C[m][n] = sum over blocks b of 128 along K of sa(m, b) sb(n, b) sum_{k in b} A(m, k) B(n, k),
// both operands K-contiguous, A with a scale for each row and block, B with one
// for each row (shift 0) or each 128 rows (shift 7) and block.  A block is one
// v_mfma_scale_f32_16x16x128_f8f6f4, which applies both scales, so the scales
// cost no arithmetic.  The blocks of the tile and their epilogues are those of
// linear_gemm.hpp: the MFMA operands are swapped, a lane ends with 4 consecutive
// columns of one row.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "linear_gemm.hpp"

namespace gemm_epi {

typedef int i32x8 __attribute__((ext_vector_type(8)));

struct Fp8Params {
    LinParams e;  // the epilogue's part, M, N, the tiles and the split
    const uint8_t *A, *B, *SA, *SB;
    int64_t lda, ldb, ldsa, ldsb;  // bytes: operand rows multiples of 16, scale rows multiples of 4
    int K, shift_b, a_e5m2;
};

// One operand's share of the main loop: R rows of one 128-byte chunk.  Rows lie
// 128 bytes apart in LDS, their 16-byte pieces swizzled as in the 16-bit loops.
template <int R>
struct Fp8Operand {
    static constexpr int TB = R / 32;  // 16-row blocks per wave
    static constexpr int ND = R / 32;  // DMA instructions per wave and chunk (8 rows each)
    static constexpr int BYTES = R * 128;
    const uint8_t *base;
    int64_t ld, bytes;  // bytes: of the tile's rows
    int row, col;       // this lane's row and column of DMA 0
    const char *rd[2];

    __device__ __forceinline__ void init(const uint8_t *ptr, int64_t ld_, int r0, int count, int K, const char *lds,
                                         int lane, int wave, int w)
    {
        ld = ld_;
        base = ptr + (int64_t)r0 * ld;
        bytes = (int64_t)(min(count, R) - 1) * ld + (K + 15) / 16 * 16;
        row = 8 * wave + (lane >> 3);
        col = ((lane & 7) ^ swz_a<8>(row)) * 16;
        const int li = lane & 15, lg = lane >> 4;
        const int lr = w * (R / 2) + li;
#pragma unroll
        for (int kk = 0; kk < 2; kk++) rd[kk] = lds + lr * 128 + (((kk * 4 + lg) ^ swz_a<8>(lr)) * 16);
    }
    __device__ __forceinline__ i32x4 rsrc(int k0) const { return make_rsrc(base + k0, (uint32_t)(bytes - k0)); }
    __device__ __forceinline__ int off(int k0, int K, int q) const
    {
        return k0 + col < K ? (int)((row + 32 * q) * ld + col) : 0x7FFFFFF0;
    }
    __device__ __forceinline__ i32x8 read(int i) const
    {
        const i32x4 lo = *(const i32x4 *)(rd[0] + i * 2048), hi = *(const i32x4 *)(rd[1] + i * 2048);
        return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    }
};

template <int BM, int BN>
struct Fp8Cfg {
    using OA = Fp8Operand<BM>;
    using OB = Fp8Operand<BN>;
    static constexpr int MAIN = OA::BYTES + OB::BYTES, EPI = LinCfg<BM, BN, false, false>::EPI;
    static constexpr int LDS = MAIN > EPI ? MAIN : EPI;
};

template <int BM, int BN, int FA>
__device__ __forceinline__ void mainloop_fp8(f32x4 (&acc)[BM / 32][BN / 32], const Fp8Params &p, int m0, int n0,
                                             int kb, int k_end, char *smem)
{
    using C = Fp8Cfg<BM, BN>;
    using OA = typename C::OA;
    using OB = typename C::OB;
    constexpr int TM = OA::TB, TN = OB::TB;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave >> 1, wn = wave & 1, li = lane & 15;
    const uint32_t lds_w = (uint32_t)__builtin_amdgcn_readfirstlane((int)(lds_addr_of(smem) + wave * 1024));
    OA oa;
    OB ob;
    oa.init(p.A, p.lda, m0, p.e.M - m0, p.K, smem, lane, wave, wm);
    ob.init(p.B, p.ldb, n0, p.e.N - n0, p.K, smem + OA::BYTES, lane, wave, wn);
    for (int k0 = kb; k0 < k_end; k0 += 128) {
        const i32x4 ra = oa.rsrc(k0), rb = ob.rsrc(k0);
#pragma unroll
        for (int q = 0; q < OA::ND; q++) dma16(ra, lds_w + q * 4096, oa.off(k0, p.K, q));
#pragma unroll
        for (int q = 0; q < OB::ND; q++) dma16(rb, lds_w + OA::BYTES + q * 4096, ob.off(k0, p.K, q));
        wait_vmcnt<0>();
        barrier_lds();
        if (p.K - k0 < 128 && (p.K & 15)) {
            // the bytes behind a row's end, in its last 16, may be anything
            const int c = (p.K - k0) >> 4, keep = (p.K - k0) & 15;
            for (int r = tid; r < BM + BN; r += 256) {
                const int lr = r < BM ? r : r - BM;
                i32x4 *at = (i32x4 *)(smem + (r < BM ? 0 : OA::BYTES) + lr * 128 + ((c ^ swz_a<8>(lr)) * 16));
                i32x4 v = *at;
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const int left = keep - 4 * e;
                    v[e] = left >= 4 ? v[e] : left <= 0 ? 0 : v[e] & (int)((1u << (8 * left)) - 1);
                }
                *at = v;
            }
            barrier_lds();
        }
        const int b = k0 >> 7;
        int sa[TM], sb[TN];
#pragma unroll
        for (int i = 0; i < TM; i++) {
            const int m = min(m0 + wm * (BM / 2) + i * 16 + li, p.e.M - 1);
            sa[i] = p.SA[(int64_t)m * p.ldsa + b];
        }
#pragma unroll
        for (int j = 0; j < TN; j++) {
            const int n = min(n0 + wn * (BN / 2) + j * 16 + li, p.e.N - 1) >> p.shift_b;
            sb[j] = p.SB[(int64_t)n * p.ldsb + b];
        }
        i32x8 fa[TM];
#pragma unroll
        for (int i = 0; i < TM; i++) fa[i] = oa.read(i);
#pragma unroll
        for (int j = 0; j < TN; j++) {
            const i32x8 fb = ob.read(j);
#pragma unroll
            for (int i = 0; i < TM; i++)
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb, fa[i], acc[i][j], 0, FA, 0, sb[j], 0,
                                                                             sa[i]);
        }
        barrier_lds();
    }
}

template <int BM, int BN, int EPI, int ACT, bool BF>
__global__ __launch_bounds__(256) void fp8_gemm_kernel(Fp8Params p)
{
    __shared__ __attribute__((aligned(1024))) char smem[Fp8Cfg<BM, BN>::LDS];
    const LinParams &e = p.e;
    const int lid = xcd_logical_id((int)gridDim.x, (int)blockIdx.x);
    const int split = lid / e.num_tiles, t = lid - split * e.num_tiles;
    const int full = e.group_m * e.tiles_n, g = t / full, first = g * e.group_m;
    const int gm = min(e.tiles_m - first, e.group_m), rr = t - g * full;
    const int tm = first + rr % gm, tn = rr / gm;
    const int m0 = tm * BM, n0 = tn * BN;
    const int kb = split * e.k_split, k_end = kb + min(p.K - kb, e.k_split);
    f32x4 acc[BM / 32][BN / 32];
#pragma unroll
    for (int i = 0; i < BM / 32; i++)
#pragma unroll
        for (int j = 0; j < BN / 32; j++) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (p.a_e5m2)
        mainloop_fp8<BM, BN, 1>(acc, p, m0, n0, kb, k_end, smem);
    else
        mainloop_fp8<BM, BN, 0>(acc, p, m0, n0, kb, k_end, smem);
    lin_epilogue<BM, BN, EPI, ACT, BF>(acc, e, m0, n0, tn, split, smem);
}

}  // namespace gemm_epi
