// moe.hpp -- a mixture-of-experts layer for a few tokens (include/fp8_ops.h).
//
// Three kernels for a chunk of up to 64 tokens: the router's logits; the
// chosen experts' up products with the activation; their down products with the
// weighted sum.  All are bound by reading the chosen experts' weights once.  They
// are one operand of 16x16x32 MFMAs, whose other operand are the tokens that
// chose the expert (16 rows), and the matrix units wait for memory.  No kernel waits for another's
// workgroups: each derives from the logits what it needs of the choice (one
// kernel for router and experts would need a wait across the whole grid).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "linear_gemm.hpp"
#include "ops_host.hpp"
#include "row_pieces.hpp"

namespace gemm_epi {

constexpr int kMoeChunk = 64;      // tokens that share one reading of the weights
constexpr int kMoeExperts = 1024;  // GE_MOE_MAX_EXPERTS
constexpr int kMoeTop = 32;        // GE_MOE_MAX_TOP_K

struct MoeParams {
    int T, H, E, I, k;  // T: of the chunk
    int gated, renormalize;
    const _Float16 *X, *Wr, *R;
    const void *Up, *Down;
    const uint8_t *US, *DS;
    int64_t ldx, ldwr, ldr, ldu, up_stride, ldus, us_stride, lddn, down_stride, ldds, ds_stride;
    _Float16 *D;
    int64_t ldd;
    float *logits;    // [T][E]
    int *chosen;      // [T][k]: expert
    float *weight;    // [T][k]: exp(logit - the token's largest)
    float *total;     // [T]: the sum of all experts' exp(logit - largest)
    _Float16 *hidden; // [T][k][I]
    uint8_t *low;     // [T][k][I]: what hidden's rounding left, see low_byte
};

// h is an operand of 16-bit MFMAs.  Rounded to 16 bits alone it makes the layer's error
// half as large again as the rounding of its result, so the remainder is kept
// as well, times 2^9 (bf16) or 2^12 (fp16), in e5m2: 3 bits more.  A remainder of |h|
// in [2^e, 2^(e+1)) is at most 2^(e+1) so, and e5m2 has steps of 2^-16 at least and ends
// at 57344, where larger ones are cut: the 3 bits hold for all of fp16 and for bf16 from
// 2^-15 to 2^16; outside bf16's h has between 0 and 3.  The down product takes 14.6 us instead of 14.0 for one token in 16 bits, 12.0
// for 10.4 in 8, 72 for 61 for 64 tokens.
template <bool BF>
constexpr float kLowScale = BF ? 0x1p9f : 0x1p12f;
template <bool BF>
__device__ __forceinline__ uint8_t low_byte(float h, _Float16 high)
{
    const float rest = (h - ld16<BF>(high)) * kLowScale<BF>;
    // (no NaN and no infinity: those are in the high part)
    const float r = __builtin_fabsf(rest) < __builtin_inff() ? __builtin_fminf(__builtin_fmaxf(rest, -57344.0f), 57344.0f) : 0.0f;
    return (uint8_t)__builtin_amdgcn_cvt_pk_bf8_f32(r, r, 0, false);
}

// Logits in an order that is total: a NaN below every number, -0 with +0.
__device__ __forceinline__ uint32_t logit_key(float v)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);
    if (v != v) return 0;
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// A lane's 16 consecutive columns of a row, as the operands of two MFMAs.
struct Pair8 {
    half8 v[2];
};
template <bool BF, bool E5M2 = false>
__device__ __forceinline__ Pair8 widen(i32x4 q)
{
    // both formats have fewer digits than either 16-bit type, and no larger range: exact
    i32x4 r[2];
#pragma unroll
    for (int u = 0; u < 4; u++) {
        int lo, hi;
        if constexpr (BF) {
            lo = __builtin_bit_cast(int, (E5M2 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(q[u], 1.0f, false)
                                                : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[u], 1.0f, false)));
            hi = __builtin_bit_cast(int, (E5M2 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(q[u], 1.0f, true)
                                                : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[u], 1.0f, true)));
        } else {
            lo = __builtin_bit_cast(int, (E5M2 ? __builtin_amdgcn_cvt_scalef32_pk_f16_bf8(q[u], 1.0f, false)
                                                : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(q[u], 1.0f, false)));
            hi = __builtin_bit_cast(int, (E5M2 ? __builtin_amdgcn_cvt_scalef32_pk_f16_bf8(q[u], 1.0f, true)
                                                : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(q[u], 1.0f, true)));
        }
        r[u >> 1][(u & 1) * 2] = lo;
        r[u >> 1][(u & 1) * 2 + 1] = hi;
    }
    return {{__builtin_bit_cast(half8, r[0]), __builtin_bit_cast(half8, r[1])}};
}
// Lane (li, lg) ends with 4 tokens (4 lg ..) of weight row li, so that a row's scale is the lane's own.
template <bool BF>
__device__ __forceinline__ f32x4 mfma_pair(const Pair8 &x, const Pair8 &w, f32x4 acc)
{
#pragma unroll
    for (int u = 0; u < 2; u++) {
        if constexpr (BF)
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x.v[u]),
                                                          __builtin_bit_cast(bf16x8, w.v[u]), acc, 0, 0, 0);
        else
            acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(x.v[u], w.v[u], acc, 0, 0, 0);
    }
    return acc;
}

// logits [T][E]: a wave takes one expert and up to 4 tokens, 8 columns a lane and turn.
// (In MFMAs, 16 experts a workgroup, the few workgroups' loads took 6.3 us for
// one token and 64 experts of 4096, and 10 us for 64 tokens; this 3.9 and 6.)
template <bool BF>
__global__ __launch_bounds__(256) void moe_router_kernel(MoeParams p)
{
    const int lane = threadIdx.x & 63, e = (int)blockIdx.x * 4 + ((int)threadIdx.x >> 6), t0 = (int)blockIdx.y * 4;
    if (e >= p.E) return;
    const _Float16 *w = p.Wr + (int64_t)e * p.ldwr;
    const _Float16 *x[4];
    float acc[4] = {};
#pragma unroll
    for (int t = 0; t < 4; t++) x[t] = p.X + (int64_t)min(t0 + t, p.T - 1) * p.ldx;
    auto add = [&](half8 wv, half8 xv, int t) {
#pragma unroll
        for (int i = 0; i < 8; i++) acc[t] = __builtin_fmaf(ld16<BF>(wv[i]), ld16<BF>(xv[i]), acc[t]);
    };
    int k = lane * 8;
    const int some = min(4, p.T - t0);
    for (; k + 1536 + 8 <= p.H; k += 2048) {
        half8 wv[4];
#pragma unroll
        for (int u = 0; u < 4; u++) wv[u] = *(const half8u *)(w + k + u * 512);
#pragma unroll
        for (int t = 0; t < 4; t++) {
            if (t >= some) break;
            half8 xv[4];
#pragma unroll
            for (int u = 0; u < 4; u++) xv[u] = *(const half8u *)(x[t] + k + u * 512);
#pragma unroll
            for (int u = 0; u < 4; u++) add(wv[u], xv[u], t);
        }
    }
    for (; k < p.H; k += 512) {
        const half8 wv = load8(w + k, p.H - k);
#pragma unroll
        for (int t = 0; t < 4; t++) add(wv, load8(x[t] + k, p.H - k), t);
    }
    float v = 0.0f;  // lane t: token t0 + t
#pragma unroll
    for (int t = 0; t < 4; t++) {
        float a = row16_sum(acc[t]);
        a += __shfl_xor(a, 16);
        a += __shfl_xor(a, 32);
        if (lane == t) v = a;
    }
    if (lane < some) p.logits[(int64_t)(t0 + lane) * p.E + e] = v;
}

// columns 64 u + 16 lg .. of row li of a block in LDS
template <int ES, bool BF>
__device__ __forceinline__ Pair8 get_pair(const char *lds, int u, int li, int lg)
{
    using R = RowBlocks<ES>;
    if constexpr (ES == 1)
        return widen<BF>(*(const i32x4 *)(lds + R::at(li, u * 4 + lg)));
    else
        return {{*(const half8 *)(lds + R::at(li, u * 8 + lg * 2)), *(const half8 *)(lds + R::at(li, u * 8 + lg * 2 + 1))}};
}

// The scales of 16 rows by tiles, for MFMA row li.
struct MoeScales {
    const uint8_t *s;  // of the first row's tile
    uint32_t off;      // from there to this lane's
    __device__ __forceinline__ void init(const uint8_t *scales, int64_t lds, int r0, int rows, int li)
    {
        s = scales + (int64_t)(r0 >> 7) * lds;
        off = (min(r0 + li, rows - 1) >> 7) > (r0 >> 7) ? (uint32_t)lds : 0u;
    }
    __device__ __forceinline__ uint32_t byte(int block) const { return s[off + (uint32_t)block]; }
    __device__ static __forceinline__ float value(uint32_t b)
    {
        return __builtin_bit_cast(float, b == 255 ? 0x7FC00000u : b ? b << 23 : 0x00400000u);
    }
};

template <bool W8, int G, int NB>
constexpr int moe_turn_bytes()
{
    return G * RowBlocks<W8 ? 1 : 2>::BYTES + NB * RowBlocks<2>::BYTES;
}

// One block of 128 columns: the weights of G times 16 rows and NB times 16 tokens, on their way.
template <bool BF, bool W8, int G, int NB>
struct MoeBlock {
    using W = RowBlocks<W8 ? 1 : 2>;
    using X = RowBlocks<2>;
    i32x4 w[G][W::NL];
    i32x4 x[NB][X::NL];
    uint32_t s[G];

    __device__ __forceinline__ void fetch(const W (&wr)[G], const MoeScales (&scales)[G], const X (&xr)[NB], int block)
    {
#pragma unroll
        for (int g = 0; g < G; g++) wr[g].load(w[g], block);
#pragma unroll
        for (int b = 0; b < NB; b++) xr[b].load(x[b], block);
        if constexpr (W8)
#pragma unroll
            for (int g = 0; g < G; g++) s[g] = scales[g].byte(block);
    }
    __device__ __forceinline__ void fetch_short(const W (&wr)[G], const MoeScales (&scales)[G], const X (&xr)[NB])
    {
#pragma unroll
        for (int g = 0; g < G; g++) wr[g].load_short(w[g]);
#pragma unroll
        for (int b = 0; b < NB; b++) xr[b].load_short(x[b]);
        if constexpr (W8)
#pragma unroll
            for (int g = 0; g < G; g++) s[g] = scales[g].byte(0);
    }
    // for the block in which the rows end, before use()
    __device__ __forceinline__ void finish(const W (&wr)[G], const X (&xr)[NB], int block)
    {
#pragma unroll
        for (int g = 0; g < G; g++) wr[g].finish(w[g], block);
#pragma unroll
        for (int b = 0; b < NB; b++) xr[b].finish(x[b], block);
    }
    // acc[g][b] += rows g times the tokens of block b; turned: moe_turn_bytes of LDS, the wave's own
    __device__ __forceinline__ void use(f32x4 (&acc)[G][NB], char *turned, int lane) const
    {
        const int li = lane & 15, lg = lane >> 4;
        char *xs = turned + G * W::BYTES;
#pragma unroll
        for (int g = 0; g < G; g++) W::put(turned + g * W::BYTES, w[g], lane);
#pragma unroll
        for (int b = 0; b < NB; b++) X::put(xs + b * X::BYTES, x[b], lane);
        wave_lds_sync();
        f32x4 part[G][NB];  // 8-bit: the sums of the block, before its scales
        if constexpr (W8)
#pragma unroll
            for (int g = 0; g < G; g++)
#pragma unroll
                for (int b = 0; b < NB; b++) part[g][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int u = 0; u < 2; u++) {
            Pair8 xv[NB];
#pragma unroll
            for (int b = 0; b < NB; b++) xv[b] = get_pair<2, BF>(xs + b * X::BYTES, u, li, lg);
#pragma unroll
            for (int g = 0; g < G; g++) {
                const Pair8 wv = get_pair<W8 ? 1 : 2, BF>(turned + g * W::BYTES, u, li, lg);
#pragma unroll
                for (int b = 0; b < NB; b++) {
                    if constexpr (W8)
                        part[g][b] = mfma_pair<BF>(xv[b], wv, part[g][b]);
                    else
                        acc[g][b] = mfma_pair<BF>(xv[b], wv, acc[g][b]);
                }
            }
        }
        if constexpr (W8)
#pragma unroll
            for (int g = 0; g < G; g++) {
                const float v = MoeScales::value(s[g]);
#pragma unroll
                for (int b = 0; b < NB; b++) acc[g][b] += v * part[g][b];
            }
        wave_lds_sync();
    }
};

// acc[g][b] += rows g times the 16 tokens of block b, over the blocks of
// stream_row_blocks.  turned: moe_turn_bytes of LDS, the wave's own.
template <bool BF, bool W8, int G, int NB, int DEPTH>
__device__ __forceinline__ void moe_product(f32x4 (&acc)[G][NB], const RowBlocks<W8 ? 1 : 2> (&w)[G],
                                            const MoeScales (&scales)[G], const RowBlocks<2> (&x)[NB], char *turned,
                                            int first, int step, int K, int turn, int lane)
{
    MoeBlock<BF, W8, G, NB> ring[DEPTH];
    if (K < kShortRow) {
        if (first == 0) {
            ring[0].fetch_short(w, scales, x);
            ring[0].use(acc, turned, lane);
        }
        return;
    }
    stream_row_blocks<DEPTH>(
        first, step, K, turn, [&](int d, int block) { ring[d].fetch(w, scales, x, block); },
        [&](int d, int finish) {
            if (finish >= 0) ring[d].finish(w, x, finish);
            ring[d].use(acc, turned, lane);
        });
}

// h = act(Up x) of one expert and some tiles of 16 of its inner rows, for the
// chunk's tokens that chose it.  A workgroup's expert is blockIdx.y, or, where the choices are
// fewer than the experts (by_choice), the one of rank blockIdx.y % k of token
// blockIdx.y / k, whose other choosers' workgroups then have nothing to do.
// Where there are few tiles (shared) the four waves share the contraction of one,
// otherwise each takes a tile of its own and streams its rows whole.  Experts of
// 2 x 1024 x 4096 in 8 bits: 64 of them 101 us with tiles of the waves' own, 122
// shared; the 8 of one token 21.8 and 17.2.
template <bool BF, bool W8, int ACT, bool GATED, int NB>
__global__ __launch_bounds__(256, 2) void moe_up_kernel(MoeParams p, int by_choice, int shared)
{
    constexpr int G = GATED ? 2 : 1;
    constexpr int DEPTH = NB == 1 ? (W8 ? 3 : 2) : (W8 ? 2 : 1);  // what the registers hold
    __shared__ uint32_t keys[kMoeExperts];
    __shared__ int ranks[kMoeChunk];  // the expert's rank in each token's choice; k and more: not chosen
    __shared__ int list[kMoeChunk];   // the tokens that chose it
    __shared__ int found;
    __shared__ float red[4][G][NB][64][4];
    __shared__ __attribute__((aligned(16))) char turned[4][moe_turn_bytes<W8, G, NB>()];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), li = lane & 15,
              lg = lane >> 4;
    int expert = (int)blockIdx.y, owner = 0;
    if (by_choice) {
        owner = expert / p.k;
        const int rank = expert - owner * p.k;
        for (int e = tid; e < p.E; e += 256) keys[e] = logit_key(p.logits[(int64_t)owner * p.E + e]);
        __syncthreads();
        for (int e = tid; e < p.E; e += 256) {
            const uint32_t mine = keys[e];
            int above = 0;
            for (int j = 0; j < p.E; j++) above += keys[j] > mine || (keys[j] == mine && j < e);
            if (above == rank) found = e;
        }
        __syncthreads();
        expert = __builtin_amdgcn_readfirstlane(found);
    }
    {  // four adjacent threads a token
        const int t = tid >> 2, part = tid & 3;
        int above = 0;
        if (t < p.T) {
            const float *row = p.logits + (int64_t)t * p.E;
            const uint32_t mine = logit_key(row[expert]);
#pragma unroll 8
            for (int j = part; j < p.E; j += 4) {
                const uint32_t key = logit_key(row[j]);
                above += key > mine || (key == mine && j < expert);
            }
        }
        above += __shfl_xor(above, 1);
        above += __shfl_xor(above, 2);
        if (part == 0) ranks[t] = t < p.T ? above : p.k;
    }
    __syncthreads();
    const unsigned long long who = __ballot(ranks[lane] < p.k);
    if (who == 0 || (by_choice && __ffsll(who) - 1 != owner)) return;  // (an earlier token's workgroup has the expert)
    const int n = __popcll(who);
    if (wave == 0 && (who >> lane & 1)) list[__popcll(who & ((1ull << lane) - 1))] = lane;
    if (blockIdx.x == 0) {  // this workgroup writes the choice down
        for (int t = wave; t < p.T; t += 4) {
            if (ranks[t] >= p.k) continue;
            const float *row = p.logits + (int64_t)t * p.E;
            float top = -__builtin_inff(), sum = 0.0f;
            for (int j = lane; j < p.E; j += 64) top = __builtin_fmaxf(top, row[j]);
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) top = __builtin_fmaxf(top, __shfl_xor(top, o));
            for (int j = lane; j < p.E; j += 64) sum += __expf(row[j] - top);
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) sum += __shfl_xor(sum, o);
            if (lane == 0) {
                p.chosen[t * p.k + ranks[t]] = expert;
                p.weight[t * p.k + ranks[t]] = __expf(row[expert] - top);
                p.total[t] = sum;  // (every expert of the token writes the same)
            }
        }
    }
    __syncthreads();

    const char *base = (const char *)p.Up + (int64_t)expert * p.up_stride * (W8 ? 1 : 2);
    const uint8_t *scales = W8 ? p.US + (int64_t)expert * p.us_stride : nullptr;
    const int i0 = (shared ? (int)blockIdx.x : (int)blockIdx.x * 4 + wave) * 16;
    if (i0 >= p.I) return;  // (of a shared tile all four waves stay)
    RowBlocks<W8 ? 1 : 2> w[G];
    MoeScales ws[G];
#pragma unroll
    for (int g = 0; g < G; g++) {
        const int r0 = g * p.I + i0, end = g ? 2 * p.I : p.I;
        w[g].init(base + (int64_t)r0 * p.ldu * (W8 ? 1 : 2), p.H, lane,
                  [&](int r) { return (uint32_t)(min(r, end - 1 - r0) * (int)p.ldu) * (W8 ? 1 : 2); });
        if constexpr (W8) ws[g].init(scales, p.ldus, r0, end, li);
    }
    const int turn = (i0 / 16 * 5 + expert * 3) % max(p.H >> 7, 1);
    // (an operand of the down product)
    auto store = [&](const float (&v)[G], int c, int r) {
        float h = lin_act<ACT>(v[0]);
        if constexpr (GATED) h *= v[1];
        const int t = list[c];
        const int64_t at = ((int64_t)t * p.k + ranks[t]) * p.I + i0 + r;
        const _Float16 high = st16<BF>(h);
        p.hidden[at] = high;
        p.low[at] = low_byte<BF>(h, high);
    };
    // 16 NB tokens at a time (more read the weights again, from the caches)
    for (int n0 = 0; n0 < n; n0 += 16 * NB) {
        RowBlocks<2> x[NB];
        f32x4 acc[G][NB];
#pragma unroll
        for (int b = 0; b < NB; b++) {
            // (rows past the last token repeat it)
            x[b].init((const char *)p.X, p.H, lane, [&](int r) {
                return (uint32_t)(list[min(n0 + b * 16 + r, n - 1)] * (int)p.ldx) * 2;
            });
#pragma unroll
            for (int g = 0; g < G; g++) acc[g][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        moe_product<BF, W8, G, NB, DEPTH>(acc, w, ws, x, turned[wave], shared ? wave : 0, shared ? 4 : 1, p.H, turn,
                                          lane);
        if (!shared) {
            // lane: row li, tokens 4 lg .. + 3 of a block
#pragma unroll
            for (int b = 0; b < NB; b++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const int c = n0 + b * 16 + lg * 4 + e;
                    float v[G];
#pragma unroll
                    for (int g = 0; g < G; g++) v[g] = acc[g][b][e];
                    if (c < n && i0 + li < p.I) store(v, c, li);
                }
            continue;
        }
#pragma unroll
        for (int g = 0; g < G; g++)
#pragma unroll
            for (int b = 0; b < NB; b++) *(f32x4 *)red[wave][g][b][lane] = acc[g][b];
        __syncthreads();
        // thread: column tid / 16 of a block, row tid % 16
        const int r = tid & 15, col = tid >> 4, at = (col >> 2) * 16 + r, el = col & 3;
#pragma unroll
        for (int b = 0; b < NB; b++) {
            const int c = n0 + b * 16 + col;
            float v[G];
#pragma unroll
            for (int g = 0; g < G; g++)
                v[g] = (red[0][g][b][at][el] + red[1][g][b][at][el]) + (red[2][g][b][at][el] + red[3][g][b][at][el]);
            if (c < n && i0 + r < p.I) store(v, c, r);
        }
        __syncthreads();
    }
}

// One block of 128 inner columns of 16 rows of Down and of h, high and low parts, on their way.
template <bool BF, bool W8>
struct DownBlock {
    using W = RowBlocks<W8 ? 1 : 2>;
    using High = RowBlocks<2>;
    using Low = RowBlocks<1>;
    static constexpr int BYTES = W::BYTES + High::BYTES + Low::BYTES;  // of LDS
    struct Rows {
        W w;
        MoeScales ws;
        High high;
        Low low;
    };
    i32x4 w[W::NL], high[High::NL], low[Low::NL];
    uint32_t s;

    __device__ __forceinline__ void fetch(const Rows &r, int block)
    {
        r.w.load(w, block);
        r.high.load(high, block);
        r.low.load(low, block);
        if constexpr (W8) s = r.ws.byte(block);
    }
    __device__ __forceinline__ void fetch_short(const Rows &r)
    {
        r.w.load_short(w);
        r.high.load_short(high);
        r.low.load_short(low);
        if constexpr (W8) s = r.ws.byte(0);
    }
    __device__ __forceinline__ void finish(const Rows &r, int block)
    {
        r.w.finish(w, block);
        r.high.finish(high, block);
        r.low.finish(low, block);
    }
    // acc, acc_low += the products with the high and the low parts
    __device__ __forceinline__ void use(f32x4 &acc, f32x4 &acc_low, char *turned, int lane) const
    {
        const int li = lane & 15, lg = lane >> 4;
        char *th = turned + W::BYTES, *tl = th + High::BYTES;
        W::put(turned, w, lane);
        High::put(th, high, lane);
        Low::put(tl, low, lane);
        wave_lds_sync();
        f32x4 part = {0.0f, 0.0f, 0.0f, 0.0f}, part_low = part;  // 8-bit: the sums of the block, before its scales
#pragma unroll
        for (int u = 0; u < 2; u++) {
            const Pair8 wv = get_pair<W8 ? 1 : 2, BF>(turned, u, li, lg), hv = get_pair<2, BF>(th, u, li, lg),
                        lv = widen<BF, true>(*(const i32x4 *)(tl + Low::at(li, u * 4 + lg)));
            f32x4 &to = W8 ? part : acc, &to_low = W8 ? part_low : acc_low;
            to = mfma_pair<BF>(hv, wv, to);
            to_low = mfma_pair<BF>(lv, wv, to_low);
        }
        if constexpr (W8) {
            const float v = MoeScales::value(s);
            acc += v * part;
            acc_low += v * part_low;
        }
        wave_lds_sync();
    }
};

// D = residual + sum of weight Down h for 16 of the layer's columns and all
// tokens of the chunk.  The work is a list of units: a chosen expert, up to 16 of
// its tokens and a part of its inner columns.  They are dealt out over the 8 waves,
// each of which adds up its own sums of all tokens in LDS, in a fixed order.  What
// bounds it is the bytes in flight: a wave streams over the ends of its units (64
// experts of 4096 x 1024 in 8 bits 61 us, 4.4 TB/s, before h had its low part, 72 with
// it and two blocks a ring instead of three; with units of 4 blocks that each
// drained before the next began 75 us).  Workgroups begin at different units.
// Where all began at the first one and the same rows of h, that was 101 us.
constexpr int kDownWaves = 8;
constexpr int kDownUnits = kMoeExperts + kMoeChunk * kMoeTop / 16;  // sum of ceil(tokens / 16) over the experts
template <bool BF, bool W8>
__global__ __launch_bounds__(64 * kDownWaves) void moe_down_kernel(MoeParams p)
{
    constexpr int THREADS = 64 * kDownWaves, PAIRS = kMoeChunk * kMoeTop / THREADS, DEPTH = 2;
    __shared__ unsigned long long users[kMoeExperts];  // tokens of each expert
    __shared__ uint16_t start[kMoeExperts];            // where its choices start in the list
    __shared__ uint16_t list[kMoeChunk * kMoeTop];     // the choices (t k + r), expert by expert, by token
    __shared__ uint16_t unit_expert[kDownUnits], unit_start[kDownUnits];
    __shared__ uint8_t unit_tokens[kDownUnits];
    __shared__ int count;
    __shared__ float share[kMoeChunk * kMoeTop];
    __shared__ float sums[kDownWaves][kMoeChunk][16];
    __shared__ __attribute__((aligned(16))) char turned[kDownWaves][DownBlock<BF, W8>::BYTES];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), li = lane & 15,
              lg = lane >> 4;
    const int h0 = (int)blockIdx.x * 16, rows = (p.T + 15) / 16 * 16;
    for (int e = tid; e < p.E; e += THREADS) users[e] = 0;
    int expert[PAIRS];
#pragma unroll
    for (int j = 0; j < PAIRS; j++) {
        const int i = tid + j * THREADS;
        expert[j] = -1;
        if (i >= p.T * p.k) continue;
        expert[j] = p.chosen[i];
        const int t = i / p.k;
        const float all = p.total[t];
        float sum = 0.0f;
        if (p.renormalize) {
#pragma unroll 8
            for (int r = 0; r < p.k; r++) sum += p.weight[t * p.k + r];
        }
        // (a NaN logit, chosen or not, is in `all` alone: the largest logit and the chosen ones' sum pass it by)
        share[i] = p.weight[i] / (p.renormalize && all == all ? sum : all);
    }
    for (int i = lane; i < rows * 16; i += 64) sums[wave][i >> 4][i & 15] = 0.0f;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < PAIRS; j++)
        if (expert[j] >= 0) atomicOr(&users[expert[j]], 1ull << ((tid + j * THREADS) / p.k));
    __syncthreads();
    if (wave == 0) {
        int n = 0, at = 0;  // units, choices
        for (int e0 = 0; e0 < p.E; e0 += 64) {
            const int tokens = e0 + lane < p.E ? __popcll(users[e0 + lane]) : 0, groups = (tokens + 15) / 16;
            int sum = tokens << 16 | groups;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int v = __shfl_up(sum, o);
                if (lane >= o) sum += v;
            }
            const int first = at + (sum >> 16) - tokens, unit = n + (sum & 0xFFFF) - groups;
            if (e0 + lane < p.E) start[e0 + lane] = (uint16_t)first;
            for (int g = 0; g < groups; g++) {
                unit_expert[unit + g] = (uint16_t)(e0 + lane);
                unit_start[unit + g] = (uint16_t)(first + g * 16);
                unit_tokens[unit + g] = (uint8_t)min(16, tokens - g * 16);
            }
            const int all = __shfl(sum, 63);
            n += all & 0xFFFF;
            at += all >> 16;
        }
        if (lane == 0) count = n;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < PAIRS; j++) {
        const int i = tid + j * THREADS, t = i / p.k;
        if (expert[j] >= 0) list[start[expert[j]] + __popcll(users[expert[j]] & ((1ull << t) - 1))] = (uint16_t)i;
    }
    __syncthreads();
    // parts of whole blocks of 128, so that every wave has a unit where that is possible
    const int entries = __builtin_amdgcn_readfirstlane(count), blocks = (p.I + 127) >> 7;
    const int len = blocks / min(blocks, (kDownWaves + entries - 1) / entries);
    const int parts = (blocks + len - 1) / len, units = entries * parts, tail = p.I & 127 ? blocks - 1 : -1;
    using Block = DownBlock<BF, W8>;
    struct Unit {
        typename Block::Rows rows;
        int first, n;    // blocks
        int at, tokens;  // in the list
    };
    const int shift = blockIdx.x * kDownWaves % units;
    auto place = [&](int u) { return u + shift < units ? u + shift : u + shift - units; };
    auto open = [&](int u) {
        Unit q;
        const int i = place(u) / parts, part = place(u) - i * parts, e = __builtin_amdgcn_readfirstlane(unit_expert[i]);
        q.at = __builtin_amdgcn_readfirstlane(unit_start[i]);
        q.tokens = __builtin_amdgcn_readfirstlane(unit_tokens[i]);
        q.first = part * len;
        q.n = min(blocks - q.first, len);
        q.rows.w.init((const char *)p.Down + ((int64_t)e * p.down_stride + h0 * p.lddn) * (W8 ? 1 : 2), p.I, lane,
                      [&](int r) { return (uint32_t)(min(r, p.H - 1 - h0) * (int)p.lddn) * (W8 ? 1 : 2); });
        if constexpr (W8) q.rows.ws.init(p.DS + (int64_t)e * p.ds_stride, p.ldds, h0, p.H, li);
        // (rows past the last token repeat it; below 2^32 bytes: 2048 rows of 2^20 elements)
        auto row = [&](int r) { return (uint32_t)list[q.at + min(r, q.tokens - 1)] * p.I; };
        q.rows.high.init((const char *)p.hidden, p.I, lane, [&](int r) { return row(r) * 2; });
        q.rows.low.init((const char *)p.low, p.I, lane, row);
        return q;
    };
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f}, acc_low = acc;
    auto close = [&](const Unit &q) {
        // the lane has tokens 4 lg .. of the 16, of column li
        float *at[4], old[4], by[4];
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const int c = list[q.at + min(lg * 4 + j, q.tokens - 1)];
            by[j] = share[c];
            at[j] = &sums[wave][c / p.k][li];
            old[j] = *at[j];
        }
#pragma unroll
        for (int j = 0; j < 4; j++) {
            // (what is not finite in Down is in the high part's sum; met by a remainder of 0 or of
            // the other sign, the low part's is a NaN or the other infinity)
            const float low = __builtin_fabsf(acc_low[j]) < __builtin_inff() ? (1.0f / kLowScale<BF>) * acc_low[j] : 0.0f;
            if (lg * 4 + j < q.tokens) *at[j] = old[j] + by[j] * (acc[j] + low);
        }
        acc = acc_low = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    };
    if (p.I < kShortRow) {
        for (int u = wave; u < units; u += kDownWaves) {
            const Unit q = open(u);
            Block f;
            f.fetch_short(q.rows);
            f.use(acc, acc_low, turned[wave], lane);
            close(q);
        }
    } else if (wave < units) {
        // A wave streams the blocks of its units: the first loads of the next unit
        // follow the last ones of this.  A unit's first group of DEPTH blocks is filled
        // up with blocks that are fetched and not used, so that its last one ends a group.
        Block ring[DEPTH];
        Unit q = open(wave);
        int g = 0;  // the number in the unit of ring[0]'s block
        auto fetch = [&](int d, const Unit &of, int block) {
            ring[d].fetch(of.rows, of.first + max(block, 0));
            __builtin_amdgcn_sched_barrier(0);
        };
        auto use = [&](int d) {
            if (g + d >= 0) ring[d].use(acc, acc_low, turned[wave], lane);
            __builtin_amdgcn_sched_barrier(0);
        };
        auto end = [&]() {
            if (q.first + q.n - 1 == tail) ring[DEPTH - 1].finish(q.rows, tail);
        };
        auto begin = [&](int n) { return n - (n + DEPTH - 1) / DEPTH * DEPTH; };
        g = begin(q.n);
#pragma unroll
        for (int d = 0; d < DEPTH; d++) fetch(d, q, g + d);
        for (int u = wave;;) {
#pragma unroll 1
            for (; g + DEPTH < q.n; g += DEPTH) {
#pragma unroll
                for (int d = 0; d < DEPTH; d++) {
                    use(d);
                    fetch(d, q, g + DEPTH + d);
                }
            }
            u += kDownWaves;
            if (u >= units) break;
            const Unit next = open(u);
            const int from = begin(next.n);
#pragma unroll
            for (int d = 0; d < DEPTH; d++) {
                if (d == DEPTH - 1) end();
                use(d);
                fetch(d, next, from + d);
            }
            close(q);
            q = next;
            g = from;
        }
        end();
#pragma unroll
        for (int d = 0; d < DEPTH; d++) use(d);
        close(q);
    }
    __syncthreads();
    for (int i = tid; i < rows * 16; i += THREADS) {
        const int t = i >> 4, r = i & 15;
        if (t >= p.T || h0 + r >= p.H) continue;
        float v = 0.0f;
#pragma unroll
        for (int u = 0; u < kDownWaves; u++) v += sums[u][t][r];
        if (p.R) v += ld16<BF>(p.R[t * p.ldr + h0 + r]);
        p.D[t * p.ldd + h0 + r] = st16<BF>(v);
    }
}

}  // namespace gemm_epi
