// moe.hpp -- a mixture-of-experts layer for a few tokens (include/fp8_ops.h).
//
// Three kernels for a chunk of up to 64 tokens: the router's logits; the
// chosen experts' up products with the activation; their down products with the
// weighted sum.  All are bound by reading the chosen experts' weights once, so
// the weights go from memory straight into the operand layout of 16x16x32
// MFMAs, against all the chunk's tokens (the columns of up to 4 blocks), and the
// matrix units wait for memory.  No kernel waits for another's workgroups: each
// derives from the logits what it needs of the choice.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "linear_gemm.hpp"
#include "ops_host.hpp"

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
};

// Logits in an order that is total: a NaN below every number, -0 with +0.
__device__ __forceinline__ uint32_t logit_key(float v)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);
    if (v != v) return 0;
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

typedef int i32x4b __attribute__((ext_vector_type(4), aligned(1)));

// A lane's 16 consecutive k of a row from column k on (n exist) as the operands of two MFMAs.
struct Pair8 {
    half8 v[2];
};
__device__ __forceinline__ Pair8 load16(const _Float16 *p, int n) { return {{load8(p, n), load8(p + 8, n - 8)}}; }
template <bool BF>
__device__ __forceinline__ Pair8 widen(i32x4 q)
{
    // e4m3 has fewer digits and a smaller range than either 16-bit type: exact
    Pair8 r;
#pragma unroll
    for (int u = 0; u < 4; u++) {
#pragma unroll
        for (int h = 0; h < 2; h++) {
            uint32_t w;
            if constexpr (BF)
                w = __builtin_bit_cast(uint32_t, h ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[u], 1.0f, true)
                                                   : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[u], 1.0f, false));
            else
                w = __builtin_bit_cast(uint32_t, h ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(q[u], 1.0f, true)
                                                   : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(q[u], 1.0f, false));
            const int at = (u & 1) * 4 + h * 2;
            r.v[u >> 1][at] = __builtin_bit_cast(_Float16, (uint16_t)w);
            r.v[u >> 1][at + 1] = __builtin_bit_cast(_Float16, (uint16_t)(w >> 16));
        }
    }
    return r;
}
// 16 bytes at any address, the first n of which exist (the rest read as zeros)
__device__ __forceinline__ i32x4 load_bytes16(const uint8_t *p, int n)
{
    if (n >= 16) return *(const i32x4b *)p;
    i32x4 v = {};
#pragma unroll
    for (int e = 0; e < 15; e++)
        if (e < n) v[e >> 2] |= (int)p[e] << (8 * (e & 3));
    return v;
}

template <bool BF>
__device__ __forceinline__ f32x4 mfma_pair(const Pair8 &w, const Pair8 &x, f32x4 acc)
{
#pragma unroll
    for (int u = 0; u < 2; u++) {
        if constexpr (BF)
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w.v[u]),
                                                          __builtin_bit_cast(bf16x8, x.v[u]), acc, 0, 0, 0);
        else
            acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(w.v[u], x.v[u], acc, 0, 0, 0);
    }
    return acc;
}

// logits [T][E]: a workgroup takes 16 experts and 16 tokens, its 16 waves parts of the contraction.
template <bool BF>
__global__ __launch_bounds__(1024) void moe_router_kernel(MoeParams p)
{
    __shared__ float red[16][64][4];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, li = lane & 15, lg = lane >> 4;
    const int e0 = (int)blockIdx.x * 16, t0 = (int)blockIdx.y * 16;
    const _Float16 *w = p.Wr + (int64_t)min(e0 + li, p.E - 1) * p.ldwr;
    const _Float16 *x = p.X + (int64_t)min(t0 + li, p.T - 1) * p.ldx;
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int k = wave * 64 + lg * 16; k - lg * 16 < p.H; k += 1024)
        acc = mfma_pair<BF>(load16(w + k, p.H - k), load16(x + k, p.H - k), acc);
    *(f32x4 *)red[wave][lane] = acc;
    __syncthreads();
    if (tid < 256) {
        const int t = tid >> 4, e = tid & 15;  // token t is lane t of a row of lanes, expert 4 lg + r
        float s = 0.0f;
#pragma unroll
        for (int u = 0; u < 16; u++) s += red[u][(e >> 2) * 16 + t][e & 3];
        if (t0 + t < p.T && e0 + e < p.E) p.logits[(int64_t)(t0 + t) * p.E + e0 + e] = s;
    }
}

// The weights of one operand row block: 16-bit, or 8-bit with block scales.
template <bool BF, bool W8>
struct MoeRows {
    const void *row;      // this lane's row
    const uint8_t *s[2];  // 8-bit: scales of the tile of the block's first and last row
    int edge;             // rows from this one on are of the second tile
    __device__ __forceinline__ void init(const void *base, int64_t ld, const uint8_t *scales, int64_t lds, int r0,
                                         int rows, int li)
    {
        const int64_t at = (int64_t)min(r0 + li, rows - 1) * ld;
        if constexpr (W8) {
            row = (const uint8_t *)base + at;
            const int last = min(r0 + 15, rows - 1);
            s[0] = scales + (int64_t)(r0 >> 7) * lds;
            s[1] = scales + (int64_t)(last >> 7) * lds;
            edge = (last >> 7 << 7) - r0;
        } else {
            row = (const _Float16 *)base + at;
        }
    }
    __device__ __forceinline__ Pair8 load(int k, int K) const
    {
        if constexpr (W8)
            return widen<BF>(load_bytes16((const uint8_t *)row + k, K - k));
        else
            return load16((const _Float16 *)row + k, K - k);
    }
    // the scales of a lane's four rows (4 lg + r) in block b
    __device__ __forceinline__ f32x4 scale(int b, int lg) const
    {
        const uint32_t a = s[0][b], c = s[1][b];
        f32x4 v;
#pragma unroll
        for (int r = 0; r < 4; r++) v[r] = e8m0(4 * lg + r < edge ? a : c);
        return v;
    }
    __device__ static __forceinline__ float e8m0(uint32_t b)
    {
        return __builtin_bit_cast(float, b == 255 ? 0x7FC00000u : b ? b << 23 : 0x00400000u);
    }
};

// h = act(Up x) of one expert and 16 of its inner rows, for the chunk's tokens
// that chose it.  A workgroup is (token, rank) of the choice, so that only chosen
// experts have workgroups; the first token of an expert serves all of its tokens.
// Four waves share the contraction.  TB: blocks of 16 tokens.
template <bool BF, bool W8, int ACT, bool GATED, int TB>
__global__ __launch_bounds__(256) void moe_up_kernel(MoeParams p)
{
    __shared__ uint32_t keys[kMoeExperts];
    __shared__ int ranks[kMoeChunk];  // the expert's rank in each token's choice; k and more: not chosen
    __shared__ int found;
    __shared__ float red[4][GATED ? 2 : 1][TB][64][4];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, li = lane & 15, lg = lane >> 4;
    const int owner = (int)blockIdx.y / p.k, rank = (int)blockIdx.y - owner * p.k;
    const int i0 = (int)blockIdx.x * 16;

    for (int e = tid; e < p.E; e += 256) keys[e] = logit_key(p.logits[(int64_t)owner * p.E + e]);
    __syncthreads();
    for (int e = tid; e < p.E; e += 256) {
        const uint32_t mine = keys[e];
        int above = 0;
        for (int j = 0; j < p.E; j++) above += keys[j] > mine || (keys[j] == mine && j < e);
        if (above == rank) found = e;
    }
    __syncthreads();
    const int expert = found;
    for (int t = wave; t < p.T; t += 4) {
        const float *row = p.logits + (int64_t)t * p.E;
        const uint32_t mine = logit_key(row[expert]);
        int above = 0;
        for (int j = lane; j < p.E; j += 64) {
            const uint32_t key = logit_key(row[j]);
            above += key > mine || (key == mine && j < expert);
        }
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) above += __shfl_xor(above, o);
        if (lane == 0) ranks[t] = above;
    }
    __syncthreads();
    for (int t = 0; t < owner; t++)
        if (ranks[t] < p.k) return;  // an earlier token's workgroup has this expert
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

    constexpr int G = GATED ? 2 : 1;
    const int rows = G * p.I;
    MoeRows<BF, W8> w[G];
    const char *base = (const char *)p.Up + (int64_t)expert * p.up_stride * (W8 ? 1 : 2);
    const uint8_t *scales = W8 ? p.US + (int64_t)expert * p.us_stride : nullptr;
#pragma unroll
    for (int g = 0; g < G; g++) w[g].init(base, p.ldu, scales, p.ldus, g * p.I + i0, g ? rows : p.I, li);
    // (the columns of tokens that did not choose the expert repeat the owner's; they are not stored)
    const _Float16 *x[TB];
#pragma unroll
    for (int b = 0; b < TB; b++) {
        const int t = b * 16 + li;
        x[b] = p.X + (int64_t)(t < p.T && ranks[min(t, p.T - 1)] < p.k ? t : owner) * p.ldx;
    }
    f32x4 acc[G][TB];
#pragma unroll
    for (int g = 0; g < G; g++)
#pragma unroll
        for (int b = 0; b < TB; b++) acc[g][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // 128 columns a turn: one block of the scales
    for (int k0 = wave * 128; k0 < p.H; k0 += 512) {
        f32x4 part[G][TB];
#pragma unroll
        for (int g = 0; g < G; g++)
#pragma unroll
            for (int b = 0; b < TB; b++) part[g][b] = W8 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : acc[g][b];
#pragma unroll
        for (int u = 0; u < 2; u++) {
            const int k = k0 + u * 64 + lg * 16;
            Pair8 xv[TB];
#pragma unroll
            for (int b = 0; b < TB; b++) xv[b] = load16(x[b] + k, p.H - k);
#pragma unroll
            for (int g = 0; g < G; g++) {
                const Pair8 wv = w[g].load(k, p.H);
#pragma unroll
                for (int b = 0; b < TB; b++) part[g][b] = mfma_pair<BF>(wv, xv[b], part[g][b]);
            }
        }
#pragma unroll
        for (int g = 0; g < G; g++) {
            if constexpr (W8) {
                const f32x4 s = w[g].scale(k0 >> 7, lg);
#pragma unroll
                for (int b = 0; b < TB; b++) acc[g][b] += s * part[g][b];
            } else {
#pragma unroll
                for (int b = 0; b < TB; b++) acc[g][b] = part[g][b];
            }
        }
    }
#pragma unroll
    for (int g = 0; g < G; g++)
#pragma unroll
        for (int b = 0; b < TB; b++) *(f32x4 *)red[wave][g][b][lane] = acc[g][b];
    __syncthreads();
    // thread: token tid / 16 of a block, inner row i0 + tid % 16
    const int r = tid & 15, at = (r >> 2) * 16 + (tid >> 4);
#pragma unroll
    for (int b = 0; b < TB; b++) {
        const int t = b * 16 + (tid >> 4);
        if (t >= p.T || i0 + r >= p.I || ranks[t] >= p.k) continue;
        float v[G];
#pragma unroll
        for (int g = 0; g < G; g++)
            v[g] = (red[0][g][b][at][r & 3] + red[1][g][b][at][r & 3]) +
                   (red[2][g][b][at][r & 3] + red[3][g][b][at][r & 3]);
        float h = lin_act<ACT>(v[0]);
        if constexpr (GATED) h *= v[1];
        // 16 bits: an operand of the down product
        p.hidden[((int64_t)t * p.k + ranks[t]) * p.I + i0 + r] = st16<BF>(h);
    }
}

// D = residual + sum of weight Down h for 16 of the layer's columns and all
// tokens of the chunk.  The experts that were chosen, and parts of 512 of their
// contraction, are dealt out over the 8 waves.
template <bool BF, bool W8, int TB>
__global__ __launch_bounds__(512) void moe_down_kernel(MoeParams p)
{
    __shared__ unsigned long long users[kMoeExperts];  // tokens of each expert
    __shared__ uint16_t list[kMoeExperts];
    __shared__ int count;
    __shared__ float share[kMoeChunk * kMoeTop];
    __shared__ uint16_t expert_of[kMoeChunk * kMoeTop];
    __shared__ float red[8][TB][64][4];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, li = lane & 15, lg = lane >> 4;
    const int h0 = (int)blockIdx.x * 16;
    for (int e = tid; e < p.E; e += 512) users[e] = 0;
    __syncthreads();
    for (int i = tid; i < p.T * p.k; i += 512) {
        const int t = i / p.k, e = p.chosen[i];
        float sum = 0.0f;
        if (p.renormalize)
            for (int j = 0; j < p.k; j++) sum += p.weight[t * p.k + j];
        else
            sum = p.total[t];
        share[i] = p.weight[i] / sum;
        expert_of[i] = (uint16_t)e;
        atomicOr(&users[e], 1ull << t);
    }
    __syncthreads();
    if (wave == 0) {
        int n = 0;
        for (int e0 = 0; e0 < p.E; e0 += 64) {
            const bool on = e0 + lane < p.E && users[e0 + lane];
            const unsigned long long m = __ballot(on);
            if (on) list[n + __popcll(m & ((1ull << lane) - 1))] = (uint16_t)(e0 + lane);
            n += __popcll(m);
        }
        if (lane == 0) count = n;
    }
    __syncthreads();
    const int parts = (p.I + 511) / 512, units = count * parts;
    f32x4 acc[TB];
#pragma unroll
    for (int b = 0; b < TB; b++) acc[b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int u = wave; u < units; u += 8) {
        const int e = list[u / parts], part = u % parts;
        const unsigned long long who = users[e];
        MoeRows<BF, W8> w;
        w.init((const char *)p.Down + (int64_t)e * p.down_stride * (W8 ? 1 : 2), p.lddn,
               W8 ? p.DS + (int64_t)e * p.ds_stride : nullptr, p.ldds, h0, p.H, li);
        // (the columns of tokens that did not choose the expert repeat those of one that did)
        const int some = __ffsll(who) - 1;
        const _Float16 *h[TB];
        float by[TB];
        uint32_t in = 0;
#pragma unroll
        for (int b = 0; b < TB; b++) {
            const bool here = who >> (b * 16 + li) & 1;
            const int t = here ? b * 16 + li : some;
            int r = 0;
            while (r < p.k - 1 && expert_of[t * p.k + r] != e) r++;
            in |= here ? 1u << b : 0u;
            by[b] = share[t * p.k + r];
            h[b] = p.hidden + ((int64_t)t * p.k + r) * p.I;
        }
        f32x4 sum[TB];
#pragma unroll
        for (int b = 0; b < TB; b++) sum[b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        const int end = min(p.I, part * 512 + 512);
        for (int k0 = part * 512; k0 < end; k0 += 128) {
            f32x4 s8[TB];
#pragma unroll
            for (int b = 0; b < TB; b++) s8[b] = W8 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : sum[b];
#pragma unroll
            for (int v = 0; v < 2; v++) {
                const int k = k0 + v * 64 + lg * 16;
                const Pair8 wv = w.load(k, p.I);
#pragma unroll
                for (int b = 0; b < TB; b++) {
                    s8[b] = mfma_pair<BF>(wv, load16(h[b] + k, p.I - k), s8[b]);
                }
            }
            if constexpr (W8) {
                const f32x4 s = w.scale(k0 >> 7, lg);
#pragma unroll
                for (int b = 0; b < TB; b++) sum[b] += s * s8[b];
            } else {
#pragma unroll
                for (int b = 0; b < TB; b++) sum[b] = s8[b];
            }
        }
        // (a token that did not choose the expert takes nothing of it, not a NaN either)
#pragma unroll
        for (int b = 0; b < TB; b++)
            if (in >> b & 1) acc[b] += by[b] * sum[b];
    }
#pragma unroll
    for (int b = 0; b < TB; b++) *(f32x4 *)red[wave][b][lane] = acc[b];
    __syncthreads();
    for (int i = tid; i < TB * 256; i += 512) {
        const int t = i >> 4, r = i & 15, at = (r >> 2) * 16 + (t & 15);
        if (t >= p.T || h0 + r >= p.H) continue;
        float v = 0.0f;
#pragma unroll
        for (int u = 0; u < 8; u++) v += red[u][t >> 4][at][r & 3];
        if (p.R) v += ld16<BF>(p.R[t * p.ldr + h0 + r]);
        p.D[t * p.ldd + h0 + r] = st16<BF>(v);
    }
}

}  // namespace gemm_epi
