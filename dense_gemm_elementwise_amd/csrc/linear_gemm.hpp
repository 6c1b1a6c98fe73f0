// linear_gemm.hpp -- gfx950 matrix products of the training and serving
// operators (include/linear_ops.h) and the epilogues fused into them.
//
// One workgroup of four waves computes one BM x BN tile of
//   C[m][n] = sum_k A(m, k) B(n, k),      16-bit operands, fp32 accumulation,
// in three layouts of the same product, by how each operand lies in memory:
//   NT  A rows and B rows are both K-contiguous   (D = X W^T: the forward)
//   NN  A K-contiguous, B k-major (k rows of n)   (dX = dZ W)
//   TN  both k-major                              (dW = dZ^T X)
// so that a gradient needs no transposed copy of anything.
//
// Layout in LDS and schedule.  Like the 4-wave tiles of gemm_epi_kernels.hpp,
// each wave owns a (BM/2) x (BN/2) block of 16x16x32 MFMAs held in AGPRs, K
// is walked in steps of 32, and every step's instruction order is fixed by
// hand: the next step's operand reads and the DMAs of a later step sit in
// the gaps between the MFMAs.  Both kinds of operand fill exactly one LDS
// slot of 64 R bytes per step (R = BM or BN):
//   k-major       32 k-rows of R columns, a ring of 4 slots, filled 4 steps
//                 ahead, read with the transposing ds_read_b64_tr_b16;
//   K-contiguous  half the rows (of each wave's share) of a 64-deep chunk, so
//                 that a DMA moves full 128-byte lines, read with
//                 ds_read_b128.  A ring of NH halves, filled NH - 1 steps
//                 ahead: NH = 6 beside a k-major operand (160 KB of LDS in
//                 all at 256 x 256); beside another K-contiguous one 5 each
//                 (160 KB again).
// Chunk c is read in steps 2c-1 and 2c (fragments are read one step early),
// so its halves are free after the barrier at the start of step 2c+1, and
// step t may refill the slot of half t-1 for either ring.  With NH = 5 a
// chunk lands at least two steps before its first read, and NT needs a
// barrier (and a wait) on odd steps only.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_epi_kernels.hpp"

namespace gemm_epi {

enum LinAct : int { ACT_IDENTITY = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_SILU = 3 };

// What the epilogue does with the fp32 tile.
enum LinEpi : int {
    LE_LINEAR = 0,  // Z = acc + bias, D = act(Z) + residual
    LE_OUT = 1,     // [C32 +] acc, into C32 or, times *alpha, into D
    LE_XFWD = 2,    // per row: maximum and sum of exponentials over the tile's columns; the target's logit
    LE_XP = 3,      // P = (exp(acc - lse) - [column == target]) * scale, 16-bit
};

// One row of the cross entropy's gradient: scale is the incoming gradient
// times a power of two (see xent_rows_kernel), 0 with target -1 in ignored rows.
struct XentRow {
    float lse, scale;
    int target, ignored;
};

struct LinParams {
    const _Float16 *A, *B;
    int64_t lda, ldb;    // elements between rows (K-contiguous) or k-rows (k-major)
    int M, N, K;         // output rows and columns; contraction length (K-contiguous operands: a multiple of 8)
    int m_read, n_read;  // columns a k-major A / B may read: M / N rounded up to 8
    int k_rows;          // k-rows a k-major operand has (<= K; the ones past it read as zeros)
    int tiles_m, tiles_n, num_tiles, group_m;
    int k_split;         // contraction length of one split, a multiple of 64 (K rounded up when there is one)
    const _Float16 *bias, *R;
    _Float16 *D, *Z;
    int64_t ldr, ldd, ldz;
    float *C32;            // fp32 output or accumulator, rows of ldc floats (a multiple of 8); split s adds s * c_split
    int64_t ldc, c_split;
    int acc_in, acc_out;   // add C32's values; write to C32 instead of D
    const float *alpha;    // device scalar that D is multiplied by, or NULL
    int vec;               // D, Z and R take 16-byte vectors (host rule: alignment, leading dimensions and N)
    const XentRow *rows;   // LE_XP
    const int64_t *target; // LE_XFWD
    int v0;                // vocabulary index of column 0
    float *part_max, *part_sum;  // LE_XFWD: [M][nparts]
    int nparts;
    float *tlogit;         // LE_XFWD: the target's logit of each row
    int n_store;           // LE_XP: columns written (N rounded up to 8, zeros past N)
};

// Activations of the linear operator.  An epilogue's arithmetic runs while the
// matrix units wait, so these are cheaper forms than those of the epilogue
// kinds (act_gelu, act_silu): at 8192 x 8192 x 2048 gelu went from 301 to 237
// us and silu from 267 to 223, where the product alone takes 210.  Relative
// error: gelu 2.4e-6 from z = -3 on, where the fit decides, 4e-6 at -6, 5.6e-6
// at -11 and 1e-5 at -13, where the exponent z^2 / 4 log2 e, rounded twice,
// does; silu 4e-7 from -3 on, 2e-6 at -40 and 4e-6 at -87.  An output's own
// rounding is 4e-3 (bf16) or 5e-4 (fp16), so nearly all are the correctly
// rounded value, as all of the epilogue kinds' are.
//
// The upper tail Q(|x|) = erfc(|x| / sqrt 2) / 2 of the normal distribution is
// q h h, h = e^(-x^2/4), q a polynomial in 1 / (1 + 0.3 |x|) by
// fit_normal_tail.py.
__device__ __forceinline__ void act_normal_tail(float x, float &q, float &h)
{
#pragma clang fp contract(off)
    const float u = act_rcp(__builtin_fmaf(0.3f, __builtin_fabsf(x), 1.0f));
    float p = -8.459328115e-02f;
    p = __builtin_fmaf(p, u, 2.405729890e-01f);
    p = __builtin_fmaf(p, u, -4.864473268e-02f);
    p = __builtin_fmaf(p, u, 1.647647172e-01f);
    p = __builtin_fmaf(p, u, 1.067044288e-01f);
    p = __builtin_fmaf(p, u, 1.212747246e-01f);
    q = __builtin_fmaf(p, u, -7.979097427e-05f);
    h = __builtin_amdgcn_exp2f((x * (-0.25f * 1.44269504088896341f)) * x);
}

template <int ACT>
__device__ __forceinline__ float lin_act(float z)
{
#pragma clang fp contract(off)
    if constexpr (ACT == ACT_RELU) {
        return z < 0.0f ? 0.0f : z;  // keeps a NaN
    } else if constexpr (ACT == ACT_GELU) {
        // z Phi(z) = max(z, 0) - |z| Q(|z|).  The factor |z| is clamped against
        // infinity times zero; h of a NaN is a NaN.
        float q, h;
        act_normal_tail(z, q, h);
        return __builtin_fmaxf(z, 0.0f) - ((__builtin_fminf(__builtin_fabsf(z), 100.0f) * q) * h) * h;
    } else if constexpr (ACT == ACT_SILU) {
        // z / (1 + e^-z), below zero z e^z / (1 + e^z), e^-|z| = v v
        const float v = __builtin_amdgcn_exp2f(__builtin_fabsf(z) * (-0.5f * 1.44269504088896341f));
        return (z < 0.0f ? (z * v) * v : z) * act_rcp(__builtin_fmaf(v, v, 1.0f));
    } else {
        return z;
    }
}

// act'(z) of gelu and silu.  The clamps only replace values where the derivative
// has long reached 0 or 1 (they keep infinity times zero out); a NaN passes
// through.
template <int ACT>
__device__ __forceinline__ float lin_act_grad(float z)
{
#pragma clang fp contract(off)
    static_assert(ACT == ACT_GELU || ACT == ACT_SILU, "the others have no factor");
    if constexpr (ACT == ACT_GELU) {
        // Phi(z) + z phi(z), phi(z) = e^(-z^2/2) / sqrt(2 pi)
        z = z < -40.0f ? -40.0f : (z > 40.0f ? 40.0f : z);
        float q, h;
        act_normal_tail(z, q, h);
        const float e = h * h;
        const float cdf = z < 0.0f ? q * e : 1.0f - q * e;
        return cdf + z * (0.398942280401432678f * e);
    } else {
        // s (1 + z (1 - s)), s = sigmoid(z), 1 - s = sigmoid(-z)
        z = z < -200.0f ? -200.0f : (z > 200.0f ? 200.0f : z);
        return act_sigmoid(z) * __builtin_fmaf(z, act_sigmoid(-z), 1.0f);
    }
}

// 2^x on the hardware exponential; logits are turned to base 2 with one fma
constexpr float kLog2e = 1.44269504088896341f;
__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

template <int CTRL>
__device__ __forceinline__ float dpp_row(float x)
{
    return __builtin_bit_cast(
        float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xF, 0xF, false));
}
// over the 16 lanes of a DPP row (rotations by 8, 4, 2, 1), every lane gets the result
__device__ __forceinline__ float row16_max(float v)
{
    v = __builtin_fmaxf(v, dpp_row<0x128>(v));
    v = __builtin_fmaxf(v, dpp_row<0x124>(v));
    v = __builtin_fmaxf(v, dpp_row<0x122>(v));
    return __builtin_fmaxf(v, dpp_row<0x121>(v));
}
__device__ __forceinline__ float row16_sum(float v)
{
    v += dpp_row<0x128>(v);
    v += dpp_row<0x124>(v);
    v += dpp_row<0x122>(v);
    return v + dpp_row<0x121>(v);
}

// Joins two (maximum, sum of exponentials) pairs.  A maximum of -infinity
// (nothing, or nothing but -infinity, so far) counts as 0 in the exponent, so
// that no infinity is subtracted from itself.
__device__ __forceinline__ void softmax_join(float &m, float &s, float m2, float s2)
{
    const float top = __builtin_fmaxf(m, m2);
    const float ref = top == -__builtin_inff() ? 0.0f : top;
    s = s * exp2_hw((m - ref) * kLog2e) + s2 * exp2_hw((m2 - ref) * kLog2e);
    m = top;
}

// ---------------------------------------------------------------------------
// One operand of the main loop (R: BM or BN; KM: k-major; NH: ring halves of a
// K-contiguous one).
// ---------------------------------------------------------------------------
template <int R, bool KM, int NH>
struct LinOperand {
    static constexpr int TB = R / 32;            // 16-wide blocks per wave
    static constexpr int ND = R / 64;            // DMA instructions per wave and step
    static constexpr int SLOT = 64 * R;          // bytes
    static constexpr int NSLOT = KM ? 4 : NH;
    static constexpr int LEAD = KM ? 4 : NH - 1;  // steps between a fill and the step that it feeds (KM) / half index
    static constexpr int BYTES = SLOT * NSLOT;
    static constexpr int NR = KM ? 2 * TB : TB;  // LDS reads per wave and step
    static constexpr int CH = R / 8;             // 16-byte chunks per k-row (KM)
    static constexpr uint32_t kParked = 0x7FFFFFF0u;

    // DMA q of a fill moves the same lane's chunk by whole rows (or k-rows), so
    // only the lane's own offset stays in registers: one, or two for the
    // 256-wide k-major operand, whose swizzle alternates with q.
    static constexpr int NV = KM && R == 256 ? 2 : 1;

    const _Float16 *base;  // first element of the tile's rows / columns at k = 0
    int64_t ld;
    int ld2;               // bytes between rows or k-rows
    int64_t row_bytes;     // K-contiguous: bytes of the tile's rows
    int k_rows, kb, k_end, nk;
    int kcol;              // K-contiguous: this lane's column inside a chunk
    uint32_t voff[NV];
    const char *rd[KM ? TB : 2];

    // r0: first row / column of the tile, count: how many exist past it
    // (readable ones); w: this wave's index along the operand
    __device__ __forceinline__ void init(const _Float16 *ptr, int64_t ld_, int r0, int count, int k_rows_, int kb_,
                                         int k_end_, int nk_, const char *lds, int lane, int wave, int w)
    {
        ld = ld_;
        ld2 = (int)ld * 2;
        k_rows = k_rows_;
        kb = kb_;
        k_end = k_end_;
        nk = nk_;
        const int li = lane & 15, lg = lane >> 4;
        if constexpr (KM) {
            base = ptr + r0;
            row_bytes = 0;
            kcol = 0;
#pragma unroll
            for (int q = 0; q < NV; q++) {
                const int lin = (q * 4 + wave) * 64 + lane;
                const int krow = lin / CH;
                const int c = (lin % CH) ^ swz_b<CH, 16>(krow);
                voff[q] = c * 8 < count ? (uint32_t)(krow * ld2 + c * 16) : kParked;
            }
#pragma unroll
            for (int j = 0; j < TB; j++) {
                const int n = w * (R / 2) + j * 16 + 4 * (li & 3);
                const int krow = 8 * lg + (li >> 2);
                rd[j] = lds + krow * (R * 2) + (((n >> 3) ^ swz_b<CH, 16>(krow)) * 16) + (n & 7) * 2;
            }
        } else {
            base = ptr + (int64_t)r0 * ld;
            row_bytes = (int64_t)min(count, R) * ld * 2;
            // half h of a chunk holds rows w (R/2) + h (R/4) .. + R/4 - 1 of each
            // wave's share w; its local row is w (R/4) + x, and DMA q covers
            // local rows 32 q + 8 wave .. + 7.  The swizzle (bits 1-3 of the
            // local row) is the same for every q and h.
            const int lr0 = 8 * wave + (lane >> 3);
            const int c = (lane & 7) ^ swz_a<8>(lr0);
            kcol = c * 8;
            voff[0] = (uint32_t)(lr0 * ld2 + c * 16);
            const int lr = w * (R / 4) + li;
#pragma unroll
            for (int kk = 0; kk < 2; kk++) rd[kk] = lds + lr * 128 + (((kk * 4 + lg) ^ swz_a<8>(lr)) * 16);
        }
    }

    // The buffer descriptor of the fill that step t makes (t < 0: the
    // prologue); zero records past the segment's end.  Rows past the tile's
    // last one, and k-rows past k_rows, lie past the record count.
    __device__ __forceinline__ i32x4 rsrc(int t) const
    {
        if constexpr (KM) {
            const int s = t + LEAD, k0 = kb + s * 32;
            const int n = s < nk ? min(32, k_rows - k0) : 0;
            // a k-row's columns end ld - r0 elements past the base at most: the
            // record count may reach into the following columns of the last
            // row, which the parked lanes never touch
            return make_rsrc(base + (int64_t)k0 * ld, n > 0 ? (uint32_t)((int64_t)n * ld * 2) : 0u);
        } else {
            const int c = (t + LEAD) >> 1, k0 = kb + c * 64;
            return make_rsrc(base + k0, k0 < k_end ? (uint32_t)(row_bytes - (int64_t)k0 * 2) : 0u);
        }
    }
    // byte offset of DMA q of the fill that step t makes, half h.  A parked
    // lane's offset plus the row steps stays between 2^31 - 16 and 2^32, past
    // every record count.
    __device__ __forceinline__ int off(int t, int h, int q) const
    {
        if constexpr (KM) {
            return (int)(voff[q % NV] + (uint32_t)(q / NV * 16 * ld2));
        } else {
            const int row = (32 * q) / (R / 4) * (R / 2) + h * (R / 4) + (32 * q) % (R / 4);
            const uint32_t v = kb + ((t + LEAD) >> 1) * 64 + kcol < k_end ? voff[0] : kParked;
            return (int)(v + (uint32_t)(row * ld2));
        }
    }
};

template <int BM, int BN, bool AKM, bool BKM>
struct LinCfg {
    // (128 x 256 and 256 x 128 have room for six halves beside each other too,
    // and gain nothing from them: 2400 x 3232 x 4096 58.5 us with either)
    static constexpr bool BOTH_KC = !AKM && !BKM;
    static constexpr int NH = BOTH_KC ? 5 : 6;
    static constexpr int PERIOD = BOTH_KC ? 10 : (AKM && BKM ? 4 : 12);
    using OA = LinOperand<BM, AKM, NH>;
    using OB = LinOperand<BN, BKM, NH>;
    static constexpr int MAIN = OA::BYTES + OB::BYTES;
    // the epilogues' slabs: 64 rows a wave in fp32, or all its BM / 2 in 16
    // bits; then the rows' data
    static constexpr int SLAB32 = 64 * (BN / 2) * 4, SLAB16 = (BM / 2) * (BN / 2) * 2;
    static constexpr int SLABS = 4 * (SLAB32 > SLAB16 ? SLAB32 : SLAB16);
    static constexpr int EPI = SLABS + BM * 16;
    static constexpr int LDS = MAIN > EPI ? MAIN : EPI;
    static_assert(LDS <= 160 * 1024, "LDS budget");
};

template <int BM, int BN, bool AKM, bool BKM, bool BF>
__device__ __forceinline__ void mainloop_lin(f32x4 (&acc)[BM / 32][BN / 32], const LinParams &p, int m0, int n0,
                                             int kb, int k_end, char *smem)
{
    using C = LinCfg<BM, BN, AKM, BKM>;
    using OA = typename C::OA;
    using OB = typename C::OB;
    constexpr int TM = BM / 32, TN = BN / 32;
    constexpr int NMF = TM * TN, NDA = OA::ND, ND = OA::ND + OB::ND, NRA = OA::NR, NR = OA::NR + OB::NR;
    constexpr bool BOTH_KC = C::BOTH_KC;
    constexpr int PERIOD = C::PERIOD;
    // steps newer than the ones whose fills must have landed (see step below)
    constexpr int NEWER = BOTH_KC ? C::NH - 4 : 2;
    static_assert(NMF >= 3 * ND && NMF >= NR, "the gap schedule needs room");
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int nk = (k_end - kb + 31) >> 5;
    const uint32_t lds_w = (uint32_t)__builtin_amdgcn_readfirstlane((int)(lds_addr_of(smem) + wave * 1024));

    OA oa;
    OB ob;
    oa.init(p.A, p.lda, m0, (AKM ? p.m_read : p.M) - m0, p.k_rows, kb, k_end, nk, smem, lane, wave, wave >> 1);
    ob.init(p.B, p.ldb, n0, (BKM ? p.n_read : p.N) - n0, p.k_rows, kb, k_end, nk, smem + OA::BYTES, lane, wave,
            wave & 1);

    half8 fa[2][TM], fb[2][TN];
    fp16x4_t lo_a, lo_b;  // first half of a transposed read pair
    auto join = [](fp16x4_t lo, fp16x4_t hi) {
        const half4 l = __builtin_bit_cast(half4, lo), h = __builtin_bit_cast(half4, hi);
        return half8{l[0], l[1], l[2], l[3], h[0], h[1], h[2], h[3]};
    };
    // read r of operand o for the step d (its index modulo the period)
    auto read_op = [&](auto &o, auto R_, auto D_, half8 *dst, fp16x4_t &lo) {
        using O = typename std::remove_reference<decltype(o)>::type;
        constexpr int r = decltype(R_)::value, d = decltype(D_)::value;
        if constexpr (O::NSLOT == 4 && O::LEAD == 4) {  // k-major
            constexpr int rowb = O::CH * 16;
            const fp16x4_t v = __builtin_amdgcn_ds_read_tr16_b64_v4f16(
                (GE_LDS(fp16x4_t) *)(o.rd[r / 2] + (d % 4) * O::SLOT + (r & 1) * 4 * rowb));
            if constexpr ((r & 1) == 0)
                lo = v;
            else
                dst[r / 2] = join(lo, v);
        } else {
            constexpr int half = (d >> 1) * 2 + (r >= O::TB / 2 ? 1 : 0);
            constexpr int x = r % (O::TB / 2);
            dst[r] = *(const half8 *)(o.rd[d & 1] + (half % O::NSLOT) * O::SLOT + x * 2048);
        }
    };
    // read r of a step: A block 0 (both halves of it when k-major), every B block, the other A blocks
    constexpr int A0 = AKM ? 2 : 1;
    auto do_read = [&](auto R_, auto D_, auto P_) {
        constexpr int r = decltype(R_)::value, P = decltype(P_)::value;
        if constexpr (r < A0)
            read_op(oa, R_, D_, fa[P], lo_a);
        else if constexpr (r < A0 + OB::NR)
            read_op(ob, std::integral_constant<int, r - A0>{}, D_, fb[P], lo_b);
        else
            read_op(oa, std::integral_constant<int, r - OB::NR>{}, D_, fa[P], lo_a);
    };

    // prologue: the fills of the virtual steps before 0, in their order
    constexpr int FIRST = OA::LEAD > OB::LEAD ? OA::LEAD : OB::LEAD;
    static_for<FIRST>([&](auto V_) {
        constexpr int v = decltype(V_)::value - FIRST;
        if constexpr (v + OA::LEAD >= 0) {
            constexpr int f = v + OA::LEAD;
            const i32x4 r = oa.rsrc(v);
#pragma unroll
            for (int q = 0; q < OA::ND; q++)
                dma16(r, lds_w + (f % OA::NSLOT) * OA::SLOT + q * 4096, oa.off(v, f & 1, q));
        }
        if constexpr (v + OB::LEAD >= 0) {
            constexpr int f = v + OB::LEAD;
            const i32x4 r = ob.rsrc(v);
#pragma unroll
            for (int q = 0; q < OB::ND; q++)
                dma16(r, lds_w + OA::BYTES + (f % OB::NSLOT) * OB::SLOT + q * 4096, ob.off(v, f & 1, q));
        }
    });
    // step 0 reads the first k-major stage and chunk 0 (two halves)
    wait_vmcnt<(NEWER + 1) * ND>();
    barrier_lds();
    static_for<NR>([&](auto R_) {
        do_read(R_, std::integral_constant<int, 0>{}, std::integral_constant<int, 0>{});
    });
    agpr_fence(acc);  // the accumulators' zeroing (VALU) before the first MFMA reads them

    auto kstep = [&](auto D_, int t) {
        constexpr int D = decltype(D_)::value;
        constexpr int P = D & 1;
        constexpr int FA = D + OA::LEAD, FB = D + OB::LEAD;  // the fills this step makes
        using DN = std::integral_constant<int, (D + 1) % PERIOD>;
        i32x4 ra, rb;
        static_for<NMF>([&](auto M_) {
            constexpr int m = decltype(M_)::value;
            // B first: the block comes out transposed, a lane with 4 consecutive
            // columns of one row (what the epilogues store)
            mfma16_agpr<BF>(acc[m / TN][m % TN], fb[P][m % TN], fa[P][m / TN]);
            static_for<NR>([&](auto R_) {
                constexpr int r = decltype(R_)::value;
                if constexpr (r * NMF / NR == m) do_read(R_, DN{}, std::integral_constant<int, P ^ 1>{});
            });
            static_for<ND>([&](auto G_) {
                constexpr int g = decltype(G_)::value;
                constexpr int g0 = g * NMF / ND;
                if constexpr (m == g0) {
                    if constexpr (g == 0) ra = oa.rsrc(t);
                    if constexpr (g == NDA) rb = ob.rsrc(t);
                } else if constexpr (m == g0 + 1) {
                    constexpr uint32_t OFF =
                        g < NDA ? (uint32_t)((FA % OA::NSLOT) * OA::SLOT + g * 4096)
                                : (uint32_t)(OA::BYTES + (FB % OB::NSLOT) * OB::SLOT + (g - NDA) * 4096);
                    m0_set<OFF>(lds_w);
                } else if constexpr (m == g0 + 2) {
                    if constexpr (g < NDA)
                        dma16_issue(ra, oa.off(t, FA & 1, g));
                    else
                        dma16_issue(rb, ob.off(t, FB & 1, g - NDA));
                }
            });
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    // Step t publishes what it reads for step t+1: the k-major stage t+1
    // (filled in step t-3) and, for odd t, chunk (t+1)/2 (its last half filled
    // in step t-3 for NH = 6, t-2 for NH = 5).  The barrier also frees the
    // slots that this step's fills overwrite, the last step's included (its
    // fills write zeros).
    auto step = [&](auto D_, int t) {
        constexpr int D = decltype(D_)::value;
        if constexpr (!BOTH_KC) {
            wait_vmcnt<NEWER * ND>();
            barrier_lds();
        } else if constexpr (D & 1) {
            wait_vmcnt<NEWER * ND>();
            barrier_lds();
        }
        kstep(D_, t);
    };
#pragma unroll 1
    for (int t = 0; t < nk; t += PERIOD) {
        step(std::integral_constant<int, 0>{}, t);
        static_for<PERIOD - 1>([&](auto D_) {
            constexpr int d = decltype(D_)::value + 1;
            if (t + d < nk) step(std::integral_constant<int, d>{}, t + d);
        });
    }
    // the last fills (zero records) still write their slots, which the epilogue reuses
    wait_vmcnt<0>();
    agpr_fence(acc);
}

// 16-byte access at any element alignment (global memory takes it at the
// rate of the cache lines it touches)
typedef half8 half8u __attribute__((aligned(2)));
typedef f32x4 f32x4u __attribute__((aligned(4)));

// 8 consecutive elements, the first n of which exist (the rest read as zeros)
__device__ __forceinline__ half8 load8(const _Float16 *p, int n)
{
    if (n >= 8) return *(const half8u *)p;
    half8 v = {};
#pragma unroll
    for (int e = 0; e < 7; e++)
        if (e < n) v[e] = p[e];
    return v;
}
__device__ __forceinline__ void store8(_Float16 *p, half8 v, int n)
{
    if (n >= 8) {
        *(half8u *)p = v;
        return;
    }
#pragma unroll
    for (int e = 0; e < 7; e++)
        if (e < n) p[e] = v[e];
}

// Keeps one row of accumulator blocks in AGPRs up to here: without it the
// compiler copies many rows to VGPRs at the start of the epilogue and runs out.
template <int TN>
__device__ __forceinline__ void pin_row(f32x4 (&row)[TN])
{
#pragma unroll
    for (int j = 0; j < TN; j++) asm volatile("" : "+a"(row[j]));
}

// ---------------------------------------------------------------------------
// Epilogues.  Lane (li, lg) of wave (wm, wn) holds, of block (i, j), row
// wm BM/2 + 16 i + li, columns wn BN/2 + 16 j + 4 lg .. + 3.
//   fp32 outputs (partial sums, the accumulator) go out as they are, 16 bytes a
//     lane, 64 contiguous bytes a row.
//   16-bit outputs are rounded there and turned around in LDS (8-byte writes,
//     16-byte reads) so that a lane stores 16 bytes and 16 lanes a whole row of
//     the wave's block.
//   The forward needs its residual next to the fp32 value, so there 64 rows at
//     a time go through LDS in fp32.
//   The softmax statistics stay in the accumulator layout.
// The LDS rows are not padded: the 16-byte chunks of a row are XOR-swizzled
// with the row so that the writes (16 rows, 2 chunks) and the reads (2 or 4 whole
// rows) both cover all banks.  Against accumulators the other way around,
// which took four times the LDS writes and a reduction over 16 lanes for every
// row's statistics, 8192 x 8192 x 2048 with gelu, bias, residual and Z went from
// 259 to 251 us.
//
// With p.vec the outputs and the residual go through range-checked buffer
// accesses (rows past M and, parked, columns past N are dropped; an absent
// tensor is a descriptor of zero records, which reads as zeros); otherwise
// through guarded 16-byte accesses at any element alignment, element by element
// where a row ends inside one.
// ---------------------------------------------------------------------------
template <int BM, int BN, int EPI, int ACT, bool BF>
__device__ __forceinline__ void lin_epilogue(f32x4 (&acc)[BM / 32][BN / 32], const LinParams &p, int m0, int n0,
                                             int tile_n, int split, char *smem)
{
    using C = LinCfg<BM, BN, false, false>;
    constexpr int TM = BM / 32, TN = BN / 32, WM = BM / 2, WN = BN / 2;
    constexpr uint32_t kOut = 0x7FFFFFE0u;  // parked: past every record count, with 16 bytes to spare
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave >> 1, wn = wave & 1;
    const int li = lane & 15, lg = lane >> 4;
    const int rows_here = min(p.M - m0, BM);
    const int64_t m0l = m0;
    barrier_lds();  // every wave is done with the main loop's LDS

    if constexpr (EPI == LE_XFWD) {
        // a lane's maximum and sum over its 4 TN columns of a row; the 8 lanes
        // that share a row meet in LDS
        int *tcol = (int *)smem;                // the target's column in this tile, or -1
        float *red = (float *)(smem + BM * 4);  // [8][BM][2]
        if (tid < BM) {
            int64_t c = -1;
            if (tid < rows_here) {
                c = p.target[m0 + tid] - n0;
                if (c < 0 || c >= min(p.N - n0, BN)) c = -1;
            }
            tcol[tid] = (int)c;
        }
        barrier_lds();
        const bool edge = n0 + BN > p.N;
        const int col0 = wn * WN + 4 * lg;
#pragma unroll
        for (int i = 0; i < TM; i++) {
            pin_row<TN>(acc[i]);
            const int row = wm * WM + i * 16 + li;
            f32x4 x[TN];
#pragma unroll
            for (int j = 0; j < TN; j++) x[j] = acc[i][j];
            if (edge) {
#pragma unroll
                for (int j = 0; j < TN; j++)
#pragma unroll
                    for (int r = 0; r < 4; r++)
                        if (n0 + col0 + j * 16 + r >= p.N) x[j][r] = -__builtin_inff();
            }
            float m = x[0][0];
#pragma unroll
            for (int j = 0; j < TN; j++)
#pragma unroll
                for (int r = 0; r < 4; r++) m = __builtin_fmaxf(m, x[j][r]);
            // e^(x - m) as 2^(x log2 e - ref), one fma an element; what the
            // rounding of ref = m log2 e left out is put back once a row
            const float mf = m == -__builtin_inff() ? 0.0f : m;
            const float ref = mf * kLog2e;
            float s[4] = {};
#pragma unroll
            for (int j = 0; j < TN; j++)
#pragma unroll
                for (int r = 0; r < 4; r++) s[r] += exp2_hw(__builtin_fmaf(x[j][r], kLog2e, -ref));
            float2 ms;
            ms.x = m;
            ms.y = ((s[0] + s[1]) + (s[2] + s[3])) * exp2_hw(-__builtin_fmaf(mf, kLog2e, -ref));
            *(float2 *)(red + ((wn * 4 + lg) * BM + row) * 2) = ms;
            const int t = tcol[row] - col0;
            if (t >= 0 && t < WN && (t & 12) == 0) {  // this lane's columns: 16 j + r
                float v = x[0][0];
#pragma unroll
                for (int j = 0; j < TN; j++)
#pragma unroll
                    for (int r = 0; r < 4; r++)
                        if (t == 16 * j + r) v = x[j][r];
                p.tlogit[m0 + row] = v;
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        barrier_lds();
        if (tid < rows_here) {
            float m = red[tid * 2], s = red[tid * 2 + 1];
#pragma unroll
            for (int u = 1; u < 8; u++) softmax_join(m, s, red[(u * BM + tid) * 2], red[(u * BM + tid) * 2 + 1]);
            const int64_t o = (int64_t)(m0 + tid) * p.nparts + tile_n;
            p.part_max[o] = m;
            p.part_sum[o] = s;
        }
        return;
    }

    // descriptor of the tile's rows of a tensor of es-byte elements
    auto res_of = [&](const void *ptr, int64_t ld, int es) {
        return epi_rsrc((const char *)ptr + m0l * ld * es, ptr ? (uint32_t)((int64_t)rows_here * ld * es) : 0u);
    };
    // a lane's place in the row-wise passes: 8 columns from scol on, one of LPR lanes on a row
    constexpr int LPR = WN / 8, RPP = 64 / LPR;
    const int ncols = EPI == LE_XP ? p.n_store : p.N;
    const int scol = 8 * (lane % LPR), srow0 = lane / LPR;
    const int gcol = n0 + wn * WN + scol, ncol = ncols - gcol;
    auto off_of = [&](int row, int64_t ld) {
        return gcol < ncols ? (row * (int)ld + gcol) * 2 : (int)kOut;
    };
    const __amdgpu_buffer_rsrc_t rD = res_of(p.D, p.ldd, 2);

    if constexpr (EPI == LE_LINEAR) {
        const __amdgpu_buffer_rsrc_t rR = res_of(p.R, p.ldr, 2), rZ = res_of(p.Z, p.ldz, 2);
        float bias[8] = {};
        if (p.bias) {
            const half8 b8 = load8(p.bias + gcol, ncol);
#pragma unroll
            for (int e = 0; e < 8; e++) bias[e] = ld16<BF>(b8[e]);
        }
        char *slab = smem + wave * C::SLAB32;
        // 16-byte chunk c of a slab row: WN / 4 chunks, 128 words span one row
        // of 128 columns or two of 64
        auto chunk = [](int row, int c) {
            const int f = WN == 128 ? 2 * (row & 15) | (row & 1) : 2 * ((row >> 1) & 7) | ((row >> 1) & 1);
            return row * (WN * 4) + (c ^ f) * 16;
        };
        constexpr int PASSES = 16 / RPP;
#pragma unroll
        for (int ph = 0; ph < TM / 4; ph++) {
#pragma unroll
            for (int i = 0; i < 4; i++) {
                pin_row<TN>(acc[ph * 4 + i]);
#pragma unroll
                for (int j = 0; j < TN; j++)
                    *(f32x4 *)(slab + chunk(i * 16 + li, 4 * j + lg)) = acc[ph * 4 + i][j];
                __builtin_amdgcn_sched_barrier(0);
            }
            wave_lds_sync();
            const int row0 = wm * WM + ph * 64;
            auto slabs = [&](auto VEC_) {
                constexpr bool VEC = decltype(VEC_)::value;
                auto put8 = [&](half8 v, __amdgpu_buffer_rsrc_t r, _Float16 *t, int64_t ld, int row) {
                    if constexpr (VEC)
                        buf_store<half8, 2>(v, r, off_of(row, ld));
                    else if (t && row < rows_here)
                        store8(t + (m0l + row) * ld + gcol, v, ncol);
                };
                half8 rbuf[PASSES] = {};
                // At any alignment the loads are made without a branch too (rows past
                // the last repeat it, columns past N - 8 start there): inside one the
                // compiler would wait for them at once.  Lanes whose columns end
                // short read theirs again, in the tiles at the edge only.
                const bool edge = n0 + wn * WN + WN > p.N;
                auto fetch = [&](int s) {
#pragma unroll
                    for (int q = 0; q < PASSES; q++) {
                        const int row = row0 + s * 16 + q * RPP + srow0;
                        if constexpr (VEC)
                            rbuf[q] = buf_load<half8, 0>(rR, off_of(row, p.ldr));
                        else if (p.R && p.N >= 8)
                            rbuf[q] = *(const half8u *)(p.R + (m0l + min(row, rows_here - 1)) * p.ldr +
                                                        min(gcol, p.N - 8));
                    }
                };
                fetch(0);
#pragma unroll 1
                for (int s = 0; s < 4; s++) {
                    half8 rcur[PASSES];
#pragma unroll
                    for (int q = 0; q < PASSES; q++) rcur[q] = rbuf[q];
                    if (s < 3) fetch(s + 1);  // the next slab's residual flies beside this one's arithmetic
                    if (!VEC && edge && p.R && ncol < 8) {
#pragma unroll
                        for (int q = 0; q < PASSES; q++) {
                            const int row = row0 + s * 16 + q * RPP + srow0;
                            rcur[q] = load8(p.R + (m0l + min(row, rows_here - 1)) * p.ldr + gcol, ncol);
                        }
                    }
#pragma unroll
                    for (int q = 0; q < PASSES; q++) {
                        const int srow = s * 16 + q * RPP + srow0;
                        const f32x4 v0 = *(const f32x4 *)(slab + chunk(srow, scol / 4));
                        const f32x4 v1 = *(const f32x4 *)(slab + chunk(srow, scol / 4 + 1));
                        half8 d, z;
#pragma unroll
                        for (int e = 0; e < 8; e++) {
                            const float t = (e < 4 ? v0[e & 3] : v1[e & 3]) + bias[e];
                            z[e] = st16<BF>(t);
                            d[e] = st16<BF>(lin_act<ACT>(t) + ld16<BF>(rcur[q][e]));
                        }
                        put8(d, rD, p.D, p.ldd, row0 + srow);
                        put8(z, rZ, p.Z, p.ldz, row0 + srow);
                    }
                }
            };
            if (p.vec)
                slabs(std::true_type{});
            else
                slabs(std::false_type{});
            wave_lds_sync();  // this wave's reads are done before the next 64 rows overwrite its slab
        }
        return;
    }

    char *slab = smem + wave * C::SLAB16;
    // byte address of the 8 bytes (4 columns from col on) of a 16-bit slab row
    auto at16 = [](int row, int col) {
        const int f = WN == 128 ? row & 15 : (row >> 1) & 7;
        return row * (WN * 2) + ((col >> 3) ^ f) * 16 + (col & 4) * 2;
    };
    auto put4 = [&](int i, int j, f32x4 v, uint32_t keep) {
        half4 h;
#pragma unroll
        for (int r = 0; r < 4; r++) h[r] = st16<BF>(v[r]);
        i32x2 w = __builtin_bit_cast(i32x2, h);
        w[0] &= (int)keep;
        w[1] &= (int)keep;
        *(i32x2 *)(slab + at16(i * 16 + li, j * 16 + 4 * lg)) = w;
    };

    if constexpr (EPI == LE_OUT) {
        const __amdgpu_buffer_rsrc_t rC =
            res_of(p.C32 ? p.C32 + (int64_t)split * p.c_split : nullptr, p.ldc, 4);
        const float alpha = p.alpha ? *p.alpha : 1.0f;
        const int ccol = n0 + wn * WN + 4 * lg;  // (ldc is a multiple of 8: whole chunks exist)
        auto coff = [&](int i, int j) {
            return ccol + 16 * j < p.N ? ((wm * WM + i * 16 + li) * (int)p.ldc + ccol + 16 * j) * 4 : (int)kOut;
        };
        if (p.acc_out) {
#pragma unroll
            for (int i = 0; i < TM; i++) {
                pin_row<TN>(acc[i]);
                f32x4 c[TN] = {};
                if (p.acc_in)
#pragma unroll
                    for (int j = 0; j < TN; j++) c[j] = buf_load<f32x4, 0>(rC, coff(i, j));
#pragma unroll
                for (int j = 0; j < TN; j++) buf_store<f32x4, 0>(acc[i][j] + c[j], rC, coff(i, j));
                __builtin_amdgcn_sched_barrier(0);
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < TM; i++) {
            pin_row<TN>(acc[i]);
            f32x4 c[TN] = {};
            if (p.acc_in)
#pragma unroll
                for (int j = 0; j < TN; j++) c[j] = buf_load<f32x4, 0>(rC, coff(i, j));
#pragma unroll
            for (int j = 0; j < TN; j++) put4(i, j, (acc[i][j] + c[j]) * alpha, ~0u);
            __builtin_amdgcn_sched_barrier(0);
        }
    } else {  // LE_XP
        i32x4 *xrow = (i32x4 *)(smem + C::SLABS);  // the tile's XentRow entries
        if (tid < BM) xrow[tid] = tid < rows_here ? *(const i32x4 *)(p.rows + m0 + tid) : i32x4{0, 0, -1, 1};
        barrier_lds();
        const bool edge = n0 + BN > p.N;
        const int col0 = n0 + wn * WN + 4 * lg;
#pragma unroll
        for (int i = 0; i < TM; i++) {
            pin_row<TN>(acc[i]);
            // p = 2^(logit log2 e - lse log2 e); the target's 1 is taken off in
            // the few lanes that hold one.  An ignored row, and columns past
            // the vocabulary, are zeros whatever was computed there.
            const i32x4 xi = xrow[wm * WM + i * 16 + li];
            const f32x4 xf = __builtin_bit_cast(f32x4, xi);
            const float c = xf[0] * kLog2e, scale = xf[1];
            const int t = xi[2] - p.v0 - col0;
            const uint32_t keep = xi[3] ? 0u : ~0u;
            f32x4 x[TN];
#pragma unroll
            for (int j = 0; j < TN; j++)
#pragma unroll
                for (int r = 0; r < 4; r++) x[j][r] = exp2_hw(__builtin_fmaf(acc[i][j][r], kLog2e, -c));
            if (t >= 0 && t < WN && (t & 12) == 0) {
#pragma unroll
                for (int j = 0; j < TN; j++)
#pragma unroll
                    for (int r = 0; r < 4; r++)
                        if (t == 16 * j + r) x[j][r] -= 1.0f;
            }
#pragma unroll
            for (int j = 0; j < TN; j++) x[j] *= scale;
            if (edge) {
#pragma unroll
                for (int j = 0; j < TN; j++)
#pragma unroll
                    for (int r = 0; r < 4; r++)
                        if (col0 + j * 16 + r >= p.N) x[j][r] = 0.0f;
            }
#pragma unroll
            for (int j = 0; j < TN; j++) put4(i, j, x[j], keep);
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // the 16-bit slab, row by row
    wave_lds_sync();
    const bool vec = EPI == LE_XP || p.vec;
#pragma unroll 4
    for (int q = 0; q < WM / RPP; q++) {
        const int srow = q * RPP + srow0, row = wm * WM + srow;
        const half8 v = *(const half8 *)(slab + at16(srow, scol));
        // P is read again soon, so it is stored plainly
        if (vec)
            buf_store<half8, EPI == LE_XP ? 0 : 2>(v, rD, off_of(row, p.ldd));
        else if (row < rows_here)
            store8(p.D + (m0l + row) * p.ldd + gcol, v, ncol);
    }
}

// One tile: workgroup `block` of `blocks` of a product.
template <int BM, int BN, bool AKM, bool BKM, int EPI, int ACT, bool BF>
__device__ __forceinline__ void lin_tile(const LinParams &p, int block, int blocks, char *smem)
{
    const int lid = xcd_logical_id(blocks, block);
    const int split = lid / p.num_tiles, t = lid - split * p.num_tiles;
    // tiles in groups of group_m tile rows, column-major inside a group
    const int full = p.group_m * p.tiles_n, g = t / full, first = g * p.group_m;
    const int gm = min(p.tiles_m - first, p.group_m), rr = t - g * full;
    const int tm = first + rr % gm, tn = rr / gm;
    const int m0 = tm * BM, n0 = tn * BN;
    // (the split's length before the end: kb + k_split may pass 2^31)
    const int kb = split * p.k_split, k_end = kb + min(p.K - kb, p.k_split);

    f32x4 acc[BM / 32][BN / 32];
#pragma unroll
    for (int i = 0; i < BM / 32; i++)
#pragma unroll
        for (int j = 0; j < BN / 32; j++) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    mainloop_lin<BM, BN, AKM, BKM, BF>(acc, p, m0, n0, kb, k_end, smem);
    lin_epilogue<BM, BN, EPI, ACT, BF>(acc, p, m0, n0, tn, split, smem);
}

template <int BM, int BN, bool AKM, bool BKM, int EPI, int ACT, bool BF>
__global__ __launch_bounds__(256) void lin_gemm_kernel(LinParams p)
{
    __shared__ __attribute__((aligned(1024))) char smem[LinCfg<BM, BN, AKM, BKM>::LDS];
    lin_tile<BM, BN, AKM, BKM, EPI, ACT, BF>(p, (int)blockIdx.x, (int)gridDim.x, smem);
}

// A gradient's two products in one launch, on 128 x 128 tiles: where neither
// fills the chip they run beside each other instead of one after the other
// (1001 x 1003 x 1000 with dZ and dbias: 34 us apart, 24 in one launch).
struct LinPair {
    LinParams nn, tn;
    int nn_groups;
};
template <bool BF>
__global__ __launch_bounds__(256) void lin_grad_pair_kernel(LinPair p)
{
    constexpr int LN = LinCfg<128, 128, false, true>::LDS, LT = LinCfg<128, 128, true, true>::LDS;
    __shared__ __attribute__((aligned(1024))) char smem[LN > LT ? LN : LT];
    const int b = (int)blockIdx.x;
    if (b < p.nn_groups)
        lin_tile<128, 128, false, true, LE_OUT, 0, BF>(p.nn, b, p.nn_groups, smem);
    else
        lin_tile<128, 128, true, true, LE_OUT, 0, BF>(p.tn, b - p.nn_groups, (int)gridDim.x - p.nn_groups, smem);
}

}  // namespace gemm_epi
