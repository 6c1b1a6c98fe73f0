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
#include <stddef.h>
#include <stdint.h>

#include "linear_gemm.hpp"

namespace gemm_epi {

typedef int i32x8 __attribute__((ext_vector_type(8)));

struct Fp8Params {
    LinParams e;  // the epilogue's part, M, N, the tiles and the split
    const uint8_t *A, *B, *SA, *SB;
    int64_t lda, ldb, ldsa, ldsb;  // bytes: operand rows multiples of 16, scale rows multiples of 4
    int K, shift_b;
};

// 4-byte global -> LDS DMA: lane i's dword to LDS address M0 + 4 i (see dma16).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma4(const i32x4 &rsrc, uint32_t lds_addr, int voffset)
{
    const int m0v = __builtin_amdgcn_readfirstlane((int)lds_addr);
    asm volatile(
        "s_mov_b32 m0, %0\n\t"
        "s_nop 0\n\t"
        "buffer_load_dword %1, %2, 0 offen lds"
        :
        : "s"(m0v), "v"(voffset), "s"(rsrc)
        : "memory", "m0");
}
#pragma clang diagnostic pop

// acc += sb sa (b a^T), with byte D of the two scale registers.  b is e4m3, a
// e4m3 (FA = 0) or e5m2.
template <int D, int FA>
__device__ __forceinline__ void mfma8_agpr(f32x4 &acc, const i32x8 &b, const i32x8 &a, int sb, int sa)
{
#define GE_MFMA8(lo, hi, f)                                                                            \
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[" #lo "," #lo ",0] " \
                 "op_sel_hi:[" #hi "," #hi ",0] blgp:" #f                                               \
                 : "+a"(acc)                                                                           \
                 : "v"(b), "v"(a), "v"(sb), "v"(sa))
    if constexpr (FA == 0) {
        if constexpr (D == 0) GE_MFMA8(0, 0, 0);
        if constexpr (D == 1) GE_MFMA8(1, 0, 0);
        if constexpr (D == 2) GE_MFMA8(0, 1, 0);
        if constexpr (D == 3) GE_MFMA8(1, 1, 0);
    } else {
        if constexpr (D == 0) GE_MFMA8(0, 0, 1);
        if constexpr (D == 1) GE_MFMA8(1, 0, 1);
        if constexpr (D == 2) GE_MFMA8(0, 1, 1);
        if constexpr (D == 3) GE_MFMA8(1, 1, 1);
    }
#undef GE_MFMA8
}

// ---------------------------------------------------------------------------
// The main loop.  K is walked in chunks of 128 bytes, one MFMA deep.  Each wave
// owns (BM/2) x (BN/2): TM x TN accumulator blocks in AGPRs.  In step c the wave
// multiplies chunk c, column of blocks by column: A's fragments of the chunk lie
// in registers (read one step before), B's are read two columns ahead.  The
// order of all instructions is fixed by hand: operand reads and DMAs sit in the
// gaps between the MFMAs, as in the 16-bit loops.
//
// LDS holds half chunks (half of each wave's rows): a ring of 5 for A, 4 for B
// (5 and 5 would leave no room for the scales), and the scales of two groups of 4
// chunks, a dword a row, whose byte the MFMA selects.  There is one barrier a step, P_c,
// two columns before its end.  Between P_{c-1} and P_c (the window W_c) the waves
// read A's chunk c+1 and B's chunk c, so the slots of A's chunk c and B's chunk c-1
// are free, and W_c fills, in this order: B chunk c+1; A chunk c+2, second half;
// (every 4th step) the next group's scales; A chunk c+3, first half.  P_c waits
// for all but the last of these, which have until P_{c+1}.  DMAs are spread
// evenly over the window: bunched, they wait for each other in the memory pipe and
// the MFMAs behind them.
//
// A window of the 256 x 256 tile lasts 2048 cycles, longer than a load takes.  Of
// the 128 x 128 tile it lasts 512: there a second workgroup on the compute unit
// fills the wait.  Where the grid has none to spare, and in the 128 x 256 tile,
// both rings hold DEPTH = 4 or 3 whole chunks instead: W_c fills B's chunk
// c + DEPTH - 1 and A's chunk c + DEPTH, and P_c leaves the fills of the last DEPTH - 2
// windows in flight.
//
// In the 256 x 256 tile P_c waits for B's first half alone.  The second halves (B's
// chunk c, A's chunk c+1) are first read in column 2 of step c, and the waves meet a
// second time there (Q_c): that gives their loads 2300 cycles instead of 1300.
// ---------------------------------------------------------------------------
template <int R, int NH>
struct Fp8Operand {
    static constexpr int TB = R / 32;  // 16-row blocks per wave
    static constexpr int ND = R / 64;  // DMA instructions per wave and half chunk
    static constexpr int SLOT = 64 * R;
    static constexpr int BYTES = SLOT * NH;
    i32x4 rs;       // the descriptor of the chunk being filled: from its first column on
    int left;       // columns that exist from there on
    int ld;
    int kcol;       // this lane's column inside a chunk
    uint32_t voff;  // this lane's offset in DMA 0
    uint32_t vnow;  // the same for the chunk being filled: past every record count behind the row's end
    const char *rd[2];

    __device__ __forceinline__ void init(const uint8_t *ptr, int64_t ld_, int r0, int count, int kb, int k_end,
                                         const char *lds, int lane, int wave, int w)
    {
        ld = (int)ld_;
        left = k_end - kb;
        rs = make_rsrc(ptr + (int64_t)r0 * ld_ + kb, (uint32_t)((min(count, R) - 1) * ld + (left + 15) / 16 * 16));
        // local row w (R/4) + x of half h is row w (R/2) + h (R/4) + x of the tile;
        // DMA q covers local rows 32 q + 8 wave .. + 7
        const int lr0 = 8 * wave + (lane >> 3);
        kcol = ((lane & 7) ^ swz_a<8>(lr0)) * 16;
        voff = (uint32_t)(lr0 * ld + kcol);
        vnow = kcol < left ? voff : 0x7FFFFFF0u;
        const int lr = w * (R / 4) + (lane & 15);
#pragma unroll
        for (int kk = 0; kk < 2; kk++) rd[kk] = lds + lr * 128 + (((kk * 4 + (lane >> 4)) ^ swz_a<8>(lr)) * 16);
    }
    // Goes on to the next chunk.  (Addresses have 48 bits: the upper word's other half is the stride, 0.)
    __device__ __forceinline__ void advance()
    {
        const uint64_t at = ((uint64_t)(uint32_t)rs[1] << 32 | (uint32_t)rs[0]) + 128;
        rs[0] = (int)(uint32_t)at;
        rs[1] = (int)(uint32_t)(at >> 32);
        // (in scalar instructions: a vector one would need wait states before the DMA reads its result)
        int records = rs[2];
        asm volatile("s_add_i32 %0, %0, 0xffffff80\n\ts_max_i32 %0, %0, 0" : "+s"(records) : : "scc");
        rs[2] = records;
        left -= 128;
        vnow = kcol < left ? voff : 0x7FFFFFF0u;
    }
    __device__ __forceinline__ int off(int h, int q) const
    {
        // (the row steps' offsets are made anew each time: kept, they fill the scalar registers)
        int step = ld;
        asm volatile("" : "+s"(step));
        const int row = (32 * q) / (R / 4) * (R / 2) + h * (R / 4) + (32 * q) % (R / 4);
        return (int)(vnow + (uint32_t)(row * step));
    }
    // one of the two 16-byte pieces of block i, whose half lies in the slot at `at`
    __device__ __forceinline__ i32x4 piece(int at, int i, int kk) const
    {
        return *(const i32x4 *)(rd[kk] + at + (i % (TB / 2)) * 2048);
    }
    // Zeroes the bytes of the half chunk at `at` from byte `keep` on, in the 16 that
    // hold the row's end (what lies behind it may be anything).
    __device__ __forceinline__ static void mask(char *at, int keep)
    {
        asm volatile("" : "+s"(keep));  // (nothing of this is kept in registers through the loop)
        for (int r = threadIdx.x; r < R / 2; r += 256) {
            i32x4 *p = (i32x4 *)(at + r * 128 + (((keep >> 4) ^ swz_a<8>(r)) * 16));
            i32x4 v = *p;
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int left = (keep & 15) - 4 * e;
                v[e] = left >= 4 ? v[e] : left <= 0 ? 0 : v[e] & (int)((1u << (8 * left)) - 1);
            }
            *p = v;
        }
    }
};

// The scales of one operand: a dword (4 chunks) a row, in LDS in the order in
// which a lane needs them: rows li, 16 + li, 32 + li .. of its share side by side.
template <int R>
struct Fp8Scales {
    static constexpr int TB = R / 32;
    const uint8_t *base;
    int bytes;
    int voff;        // this lane's row
    uint32_t place;  // where this wave's 64 dwords go
    const char *rd;

    // shift: rows per scale, as a power of two
    __device__ __forceinline__ void init(const uint8_t *ptr, int64_t ld, int r0, int count, int kb, int K, int shift,
                                         const char *lds, int lane, int wave, int w)
    {
        const int last = (r0 + min(count, R) - 1) >> shift, first = r0 >> shift;
        base = ptr + (int64_t)first * ld + kb / 128;
        bytes = (last - first) * (int)ld + ((K + 127) / 128 + 3) / 4 * 4 - kb / 128;
        const int part = wave % (R / 64), pos = part * 64 + lane;  // (of 128 rows, two waves fetch the same)
        const int rem = pos % (R / 2);
        const int row = pos / (R / 2) * (R / 2) + rem % TB * 16 + rem / TB;
        voff = (((r0 + row) >> shift) - first) * (int)ld;
        place = (uint32_t)__builtin_amdgcn_readfirstlane((int)(lds_addr_of(lds) + part * 256));
        rd = lds + (w * (R / 2) + (lane & 15) * TB) * 4;
    }
    __device__ __forceinline__ void fill(int g) const
    {
        const int left = bytes - g * 4;
        dma4(make_rsrc(base + g * 4, left > 0 ? (uint32_t)left : 0u), place + (g & 1) * (R * 4), voff);
    }
    __device__ __forceinline__ void read(int g, int (&s)[TB]) const
    {
#pragma unroll
        for (int q = 0; q < TB / 4; q++) {
            const i32x4 v = *(const i32x4 *)(rd + (g & 1) * (R * 4) + q * 16);
#pragma unroll
            for (int e = 0; e < 4; e++) s[q * 4 + e] = v[e];
        }
    }
};

template <int BM, int BN, int DEPTH>
struct Fp8Cfg {
    using OA = Fp8Operand<BM, DEPTH ? 2 * DEPTH : 5>;
    using OB = Fp8Operand<BN, DEPTH ? 2 * DEPTH : 4>;
    static constexpr int B_BASE = OA::BYTES, S_BASE = B_BASE + OB::BYTES;
    static constexpr int MAIN = S_BASE + 8 * (BM + BN), EPI = LinCfg<BM, BN, false, false>::EPI;
    static constexpr int LDS = MAIN > EPI ? MAIN : EPI;
    static_assert(LDS <= 160 * 1024, "LDS budget");
};

// Covers VALU writes of the scale registers before an MFMA in inline asm reads them.
template <int N>
__device__ __forceinline__ void settle(int (&s)[N])
{
    static_assert(N == 4 || N == 8, "blocks");
    if constexpr (N == 8)
        asm volatile("s_nop 1" : "+v"(s[0]), "+v"(s[1]), "+v"(s[2]), "+v"(s[3]), "+v"(s[4]), "+v"(s[5]), "+v"(s[6]), "+v"(s[7]));
    else
        asm volatile("s_nop 1" : "+v"(s[0]), "+v"(s[1]), "+v"(s[2]), "+v"(s[3]));
}

template <int BM, int BN, int FA, int DEPTH>
__device__ __forceinline__ void mainloop_fp8(f32x4 (&acc)[BM / 32][BN / 32], const Fp8Params &p, int m0, int n0,
                                             int kb, int k_end, char *smem)
{
    using C = Fp8Cfg<BM, BN, DEPTH>;
    using OA = typename C::OA;
    using OB = typename C::OB;
    constexpr int TM = OA::TB, TN = OB::TB, NMF = TM * TN;
    constexpr int G0 = (TN - 2) * TM;               // the gap before which P_c stands
    constexpr int NDW = 2 * OB::ND + 2 * OA::ND;    // DMAs of a window, without the scales
    constexpr int MUST = 2 * OB::ND + OA::ND;       // of these, the ones P_c waits for
    constexpr bool DEEP = DEPTH > 0;
    constexpr int NC = DEEP ? DEPTH : 2;            // chunks of B's ring
    constexpr int PERIOD = DEPTH == 3 ? 12 : 4;     // steps after which slots and scale bytes repeat
    constexpr int GA = TN == 8 ? 5 * TM : 2 * TM - 1;  // gaps that hold A's reads
    constexpr bool TWICE = TN == 8 && !DEEP;        // a second meeting of the waves, Q_c
    constexpr int GQ = 2 * TM;                      // the gap before which it stands
    constexpr int SP = NMF / NDW;                   // gaps from one DMA to the next
    constexpr int BEFORE_Q = (GQ + NMF - G0) / SP;  // DMAs of W_c that are out at Q_c
    static_assert(SP >= 2 && SP * MUST >= NMF - G0, "the gap schedule needs room");
    static_assert(!TWICE || (BEFORE_Q <= MUST && (GQ + NMF - G0) % SP == 0), "the scales are out behind Q_c");
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int nk = (k_end - kb + 127) >> 7;
    const uint32_t lds_w = (uint32_t)__builtin_amdgcn_readfirstlane((int)(lds_addr_of(smem) + wave * 1024));
    OA oa;
    OB ob;
    Fp8Scales<BM> sca;
    Fp8Scales<BN> scb;
    oa.init(p.A, p.lda, m0, p.e.M - m0, kb, k_end, smem, lane, wave, wave >> 1);
    ob.init(p.B, p.ldb, n0, p.e.N - n0, kb, k_end, smem + C::B_BASE, lane, wave, wave & 1);
    sca.init(p.SA, p.ldsa, m0, p.e.M - m0, kb, p.K, 0, smem + C::S_BASE, lane, wave, wave >> 1);
    scb.init(p.SB, p.ldsb, n0, p.e.N - n0, kb, p.K, p.shift_b, smem + C::S_BASE + 8 * BM, lane, wave, wave & 1);
    const int tail = k_end & 15 ? k_end - kb - (nk - 1) * 128 : 0;  // bytes of the last chunk, where it needs a mask

    i32x8 fa[2][TM], fb[4];
    int sa[TM], sb[TN], sna[TM], snb[TN];
    // where A's half 2 c + k lies, by D = c mod PERIOD; the ring of 5 is kept turned so that its first slot is half 2 c's
    int ring[5] = {0, OA::SLOT, 2 * OA::SLOT, 3 * OA::SLOT, 4 * OA::SLOT};
    auto slot_a = [&](int D, int k) { return DEEP ? (2 * D + k) % (2 * NC) * OA::SLOT : ring[k]; };
    // slot of B's chunk x, half h, by x modulo PERIOD
    auto slot_b = [](int x, int h) { return (2 * (x % NC) + h) * OB::SLOT; };
    auto half_of = [](i32x8 &f, int kk, i32x4 v) {
#pragma unroll
        for (int e = 0; e < 4; e++) f[kk * 4 + e] = v[e];
    };
    // part `x` (0: descriptor and M0, 1: issue) of DMA d of the window W_c, D = c mod PERIOD
    auto fill = [&](auto D_, auto d_, auto x_) {
        constexpr int D = decltype(D_)::value, d = decltype(d_)::value, x = decltype(x_)::value;
        if constexpr (d < 2 * OB::ND) {
            constexpr int h = d / OB::ND, q = d % OB::ND;
            if constexpr (x == 0) {
                if constexpr (d == 0) ob.advance();
                constexpr int slot = 2 * ((D + NC - 1) % NC) + h;
                m0_set<(uint32_t)(C::B_BASE + slot * OB::SLOT + q * 4096)>(lds_w);
            } else {
                dma16_issue(ob.rs, ob.off(h, q));
            }
        } else {
            constexpr int e = d - 2 * OB::ND, n = e / OA::ND, q = e % OA::ND, h = DEEP ? n : 1 - n;
            if constexpr (x == 0) {
                if constexpr (q == 0 && h == 0) oa.advance();
                m0_set<(uint32_t)(q * 4096)>(lds_w + (uint32_t)slot_a(D, n));
            } else {
                dma16_issue(oa.rs, oa.off(h, q));
            }
        }
    };

    // prologue: what the windows before W_0 would have filled
    auto fill_whole = [&](auto &o, uint32_t at, int h) {
#pragma unroll
        for (int q = 0; q < std::remove_reference<decltype(o)>::type::ND; q++)
            dma16(o.rs, lds_w + at + q * 4096, o.off(h, q));
    };
    auto fill_a = [&](int c, int h) {
        if (c > 0 && h == 0) oa.advance();
        fill_whole(oa, (2 * c + h) * OA::SLOT, h);
    };
    auto fill_b = [&](int c, int h) {
        if (c > 0 && h == 0) ob.advance();
        fill_whole(ob, C::B_BASE + (2 * c + h) * OB::SLOT, h);
    };
    sca.fill(0);
    scb.fill(0);
    fill_a(0, 0);
    fill_a(0, 1);
    fill_b(0, 0);
    fill_b(0, 1);
    fill_a(1, 0);
    fill_a(1, 1);
    if constexpr (DEEP) {
#pragma unroll
        for (int c = 1; c < NC - 1; c++) {
            fill_b(c, 0);
            fill_b(c, 1);
            fill_a(c + 1, 0);
            fill_a(c + 1, 1);
        }
        wait_vmcnt<(NC - 2) * NDW>();
    } else {
        fill_a(2, 0);
        wait_vmcnt<OA::ND>();
    }
    barrier_lds();
    if (tail && nk <= 2) {
        if (nk == 1) {
            OA::mask(smem, tail);
            OA::mask(smem + OA::SLOT, tail);
            OB::mask(smem + C::B_BASE, tail);
            OB::mask(smem + C::B_BASE + OB::SLOT, tail);
        } else {
            OA::mask(smem + 2 * OA::SLOT, tail);
            OA::mask(smem + 3 * OA::SLOT, tail);
        }
        barrier_lds();
    }
#pragma unroll
    for (int i = 0; i < TM; i++)
#pragma unroll
        for (int kk = 0; kk < 2; kk++) half_of(fa[0][i], kk, oa.piece(i < TM / 2 ? 0 : OA::SLOT, i, kk));
#pragma unroll
    for (int j = 0; j < 2; j++)
#pragma unroll
        for (int kk = 0; kk < 2; kk++) half_of(fb[j], kk, ob.piece(0, j, kk));
    sca.read(0, sna);
    scb.read(0, snb);
    barrier_lds();
    static_for<2 * TM>([&](auto q_) {  // the window W_0 as far as the step before would have it
        constexpr int q = decltype(q_)::value;
        if constexpr (q / SP < NDW && q % SP < 2)
            fill(std::integral_constant<int, 0>{}, std::integral_constant<int, q / SP>{},
                 std::integral_constant<int, q % SP>{});
        if constexpr (q % SP == 0) asm volatile("s_nop 0");  // between the M0 write and the load
    });
    agpr_fence(acc);

    auto step = [&](auto D_, int c) {
        constexpr int D = decltype(D_)::value, P = D & 1, S = D & 3;
        if constexpr (S == 0) {
#pragma unroll
            for (int i = 0; i < TM; i++) sa[i] = sna[i];
#pragma unroll
            for (int j = 0; j < TN; j++) sb[j] = snb[j];
            settle(sa);
            settle(sb);
        }
        const int at0 = slot_a(D, 2), at1 = slot_a(D, 3);  // A's chunk c + 1
        static_for<NMF>([&](auto M_) {
            constexpr int m = decltype(M_)::value, j = m / TM, i = m % TM;
            if constexpr (TWICE && m == GQ) {
                // (nothing is overwritten behind Q_c, so the waves' own reads may still be in flight)
                asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" : : "i"(OA::ND + BEFORE_Q + (S == 1 ? 2 : 0))
                             : "memory");
                if (tail && (c == nk - 2 || c == nk - 1)) {
                    if (c == nk - 2) OA::mask(smem + at1, tail);
                    if (c == nk - 1) OB::mask(smem + C::B_BASE + slot_b(D, 1), tail);
                    barrier_lds();
                }
            }
            if constexpr (m == G0) {
                // (the next group's scales count in the window of S = 0)
                wait_vmcnt<TWICE  ? NDW - OB::ND + (S == 0 ? 2 : 0)
                           : DEEP ? (NC - 2) * NDW + (S < NC - 2 ? 2 : 0)
                                  : OA::ND>();
                barrier_lds();
                if (tail && (c == nk - 3 || c == nk - 2)) {  // the last chunk is in LDS: A's two steps ahead, B's one
                    if (c == nk - 3) {
                        OA::mask(smem + slot_a(D, 4), tail);
                        if constexpr (!TWICE) OA::mask(smem + slot_a(D, DEEP ? 5 : 0), tail);
                    } else {
                        OB::mask(smem + C::B_BASE + slot_b(D + 1, 0), tail);
                        if constexpr (!TWICE) OB::mask(smem + C::B_BASE + slot_b(D + 1, 1), tail);
                    }
                    barrier_lds();
                }
                // from here on the slots are the next step's
                if constexpr (!DEEP) {
                    const int r0 = ring[0], r1 = ring[1];
                    ring[0] = ring[2];
                    ring[1] = ring[3];
                    ring[2] = ring[4];
                    ring[3] = r0;
                    ring[4] = r1;
                }
            }
            mfma8_agpr<S, FA>(acc[i][j], fb[j & 3], fa[P][i], sb[j], sa[i]);
            // B's block j + 2, of this chunk or the next
            if constexpr (i < 2) {
                constexpr int b = j + 2, x = b < TN ? D : D + 1, jb = b < TN ? b : b - TN;
                half_of(fb[b & 3], i, ob.piece(slot_b(x, jb < TN / 2 ? 0 : 1), jb, i));
            }
            // A's chunk c + 1
            static_for<2 * TM>([&](auto R_) {
                constexpr int r = decltype(R_)::value;
                constexpr int g = TWICE ? (r < TM ? r * GQ / TM : GQ + (r - TM) * (GA - GQ) / TM) : r * GA / (2 * TM);
                if constexpr (g == m)
                    half_of(fa[P ^ 1][r / 2], r & 1, oa.piece(r / 2 < TM / 2 ? at0 : at1, r / 2, r & 1));
            });
            // the DMAs: of W_c up to P_c, of W_{c+1} behind it
            constexpr int q = m >= G0 ? m - G0 : m - G0 + NMF;
            if constexpr (S == 0 && q == SP * MUST && m < G0) {
                sca.fill((c >> 2) + 1);
                scb.fill((c >> 2) + 1);
            }
            if constexpr (q / SP < NDW && q % SP < 2)
                fill(std::integral_constant<int, m >= G0 ? (D + 1) % PERIOD : D>{}, std::integral_constant<int, q / SP>{},
                     std::integral_constant<int, q % SP>{});
            if constexpr (S == 3 && m == G0 + 1) {
                sca.read((c >> 2) + 1, sna);
                scb.read((c >> 2) + 1, snb);
            }
            __builtin_amdgcn_sched_barrier(0);
        });
    };
#pragma unroll 1
    for (int c = 0; c < nk; c += PERIOD) {
        step(std::integral_constant<int, 0>{}, c);
        static_for<PERIOD - 1>([&](auto D_) {
            constexpr int d = decltype(D_)::value + 1;
            if (c + d < nk) step(std::integral_constant<int, d>{}, c + d);
        });
    }
    wait_vmcnt<0>();  // the last fills still write their slots, which the epilogue reuses
    agpr_fence(acc);
}

typedef const __attribute__((address_space(4))) uint64_t *ArgWords;

// FA: the format of A, 0: e4m3, 1: e5m2.  Workgroup `block` of `blocks` of the
// product p; args: where p lies in the kernel's arguments.
template <int BM, int BN, int DEPTH, int EPI, int ACT, bool BF, int FA>
__device__ __forceinline__ void fp8_tile(const Fp8Params &p, ArgWords args, int block, int blocks, char *smem)
{
    const LinParams &e = p.e;
    const int lid = xcd_logical_id(blocks, block);
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
    mainloop_fp8<BM, BN, FA, DEPTH>(acc, p, m0, n0, kb, k_end, smem);
    // The epilogue's parameters are read again from the kernel's arguments: kept
    // in scalar registers from the start, they push the main loop's out of them.
    asm volatile("" : "+s"(args));
    static_assert(offsetof(Fp8Params, e) == 0 && sizeof(LinParams) % 8 == 0, "whole words from the start");
    union {
        LinParams e;
        uint64_t w[sizeof(LinParams) / 8];
    } again;
#pragma unroll
    for (int i = 0; i < (int)(sizeof(LinParams) / 8); i++) again.w[i] = args[i];
    lin_epilogue<BM, BN, EPI, ACT, BF>(acc, again.e, m0, n0, tn, split, smem);
}

template <int BM, int BN, int DEPTH, int EPI, int ACT, bool BF, int FA>
__global__ __launch_bounds__(256) void fp8_gemm_kernel(Fp8Params p)
{
    __shared__ __attribute__((aligned(1024))) char smem[Fp8Cfg<BM, BN, DEPTH>::LDS];
    fp8_tile<BM, BN, DEPTH, EPI, ACT, BF, FA>(p, (ArgWords)__builtin_amdgcn_kernarg_segment_ptr(), (int)blockIdx.x,
                                              (int)gridDim.x, smem);
}

// The sums of up to kBiasBands bands' column sums, one thread a column.
constexpr int kBiasBands = 64;
struct BiasSum {
    const float *partial;  // [bands][cols]
    float *out;
    int bands, cols;
};
__device__ __forceinline__ void bias_sum(const BiasSum &p, int group)
{
    const int c = group * 256 + (int)threadIdx.x;
    if (c >= p.cols) return;
    float v = 0.0f;
#pragma unroll 8
    for (int b = 0; b < p.bands; b++) v += p.partial[(int64_t)b * p.cols + c];
    p.out[c] = v;
}

// A gradient's two products in one launch, on the same tiles: where neither fills
// the chip they run beside each other (1001 x 1003 x 999 with dbias: 27.7 us
// apart, 12.1 in one launch).  The last workgroups sum the bias's gradient.
struct Fp8Pair {
    Fp8Params p[2];
    BiasSum bias;
    int groups[2];
};
template <int BM, int BN, int DEPTH, bool BF, int FA>
__global__ __launch_bounds__(256) void fp8_pair_kernel(Fp8Pair a)
{
    __shared__ __attribute__((aligned(1024))) char smem[Fp8Cfg<BM, BN, DEPTH>::LDS];
    int b = (int)blockIdx.x;
    if (b >= a.groups[0] + a.groups[1]) {
        bias_sum(a.bias, b - a.groups[0] - a.groups[1]);
        return;
    }
    const int second = b >= a.groups[0];
    static_assert(offsetof(Fp8Pair, p) == 0 && sizeof(Fp8Params) % 8 == 0, "whole words from the start");
    const ArgWords args = (ArgWords)__builtin_amdgcn_kernarg_segment_ptr() + second * (int)(sizeof(Fp8Params) / 8);
    union {
        Fp8Params p;
        uint64_t w[sizeof(Fp8Params) / 8];
    } mine;
#pragma unroll
    for (int i = 0; i < (int)(sizeof(Fp8Params) / 8); i++) mine.w[i] = args[i];
    fp8_tile<BM, BN, DEPTH, LE_OUT, 0, BF, FA>(mine.p, args, second ? b - a.groups[0] : b, a.groups[second], smem);
}

}  // namespace gemm_epi
