// norm_residual.hpp -- the residual step between two blocks and its gradient:
//   H' = H + scale gate norm_post(Y) w_post,   X = norm_pre(H') w_pre.
//
// Bound by HBM bytes: each row is read once into registers, every statistic
// is taken from there, and each output is written once.  One workgroup of TPR
// threads holds a row, NV vectors of 8 elements per thread (16-byte accesses at
// any alignment); TPR follows the row length, so that a thread has one vector
// up to 4096 columns and a single row spreads over as many lanes as it has
// vectors.  Sums and norms are fp32; means are subtracted before squaring
// (two reductions), so that a large mean costs no digits.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "linear_small.hpp"

namespace gemm_epi {

enum NormKind : int { NORM_NONE = 0, NORM_RMS = 1, NORM_LAYER = 2 };

// 8 values of the residual stream: 16-bit, or fp32
template <bool BF, bool S32>
struct StreamVec {
    half8 h;
    __device__ __forceinline__ void load(const void *p, int64_t at, int n) { h = load8((const _Float16 *)p + at, n); }
    __device__ __forceinline__ float get(int e) const { return ld16<BF>(h[e]); }
    __device__ __forceinline__ void set(int e, float v) { h[e] = st16<BF>(v); }
    __device__ __forceinline__ void store(void *p, int64_t at, int n) { store8((_Float16 *)p + at, h, n); }
};
template <bool BF>
struct StreamVec<BF, true> {
    f32x4 v[2];
    __device__ __forceinline__ void load(const void *p, int64_t at, int n)
    {
        const float *q = (const float *)p + at;
        v[0] = v[1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (n >= 8) {
            v[0] = *(const f32x4u *)q;
            v[1] = *(const f32x4u *)(q + 4);
        } else {
#pragma unroll
            for (int e = 0; e < 7; e++)
                if (e < n) v[e >> 2][e & 3] = q[e];
        }
    }
    __device__ __forceinline__ float get(int e) const { return v[e >> 2][e & 3]; }
    __device__ __forceinline__ void set(int e, float x) { v[e >> 2][e & 3] = x; }
    __device__ __forceinline__ void store(void *p, int64_t at, int n)
    {
        float *q = (float *)p + at;
        if (n >= 8) {
            *(f32x4u *)q = v[0];
            *(f32x4u *)(q + 4) = v[1];
        } else {
#pragma unroll
            for (int e = 0; e < 7; e++)
                if (e < n) q[e] = v[e >> 2][e & 3];
        }
    }
};

// the last lane of a lower row (0x142: the row below; 0x143: row 1) in the rows
// of ROWS, zero in the others
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_rows(float x)
{
    return __builtin_bit_cast(float,
                              __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, ROWS, 0xF, false));
}

// Sums of N values over the workgroup of up to 16 waves, in a fixed order; every
// thread gets them.  The two LDS buffers alternate from call to call: a thread
// writes a buffer again only past the other one's barrier, which every thread
// reaches after its reads of the first.
template <int MAXN>
struct BlockSum {
    float (*lds)[16][MAXN];
    int waves;
    int phase = 0;
    template <int N>
    __device__ __forceinline__ void operator()(float (&v)[N])
    {
        static_assert(N <= MAXN, "LDS space");
#pragma unroll
        for (int i = 0; i < N; i++) {
            // rows of 16 lanes, then row 0 onto 1 and 2 onto 3, then the lower
            // half onto the upper: lane 63 has the wave's sum
            v[i] = row16_sum(v[i]);
            v[i] += dpp_rows<0x142, 0xA>(v[i]);
            v[i] += dpp_rows<0x143, 0xC>(v[i]);
        }
        if (waves == 1) {
#pragma unroll
            for (int i = 0; i < N; i++)
                v[i] = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v[i]), 63));
            return;
        }
        const int li = threadIdx.x & 15;
        if ((threadIdx.x & 63) == 63)
#pragma unroll
            for (int i = 0; i < N; i++) lds[phase][threadIdx.x >> 6][i] = v[i];
        barrier_lds();
        // lane li of each 16 takes wave li's sum
#pragma unroll
        for (int i = 0; i < N; i++) v[i] = row16_sum(li < waves ? lds[phase][li][i] : 0.0f);
        phase ^= 1;
    }
};

struct NormParams {
    const void *H;
    const _Float16 *Y, *w_post, *w_pre, *gate;
    void *H_out;
    _Float16 *X;
    int64_t ldh, ldy, ldho, ldx;
    int rows, hidden, rows_per_gate, post, pre;
    float scale, eps;
};

template <bool BF, bool S32, int TPR, int NV>
__global__ __launch_bounds__(TPR) void norm_residual_kernel(NormParams p)
{
    __shared__ float lds[2][16][1];
    BlockSum<1> sum{lds, TPR / 64};
    const int64_t row = block_row();
    if (row >= p.rows) return;
    const int H = p.hidden;
    const float inv_h = 1.0f / (float)H;
    const _Float16 *gate =
        p.gate ? p.gate + (int64_t)__builtin_amdgcn_readfirstlane((int)row / p.rows_per_gate) * H : nullptr;

    half8 y[NV], wpo[NV], wpr[NV], g[NV];
    StreamVec<BF, S32> h[NV];
#pragma unroll
    for (int u = 0; u < NV; u++) {
        const int c = (u * TPR + (int)threadIdx.x) * 8, n = H - c;
        y[u] = load8(p.Y + row * p.ldy + c, n);
        h[u].load(p.H, row * p.ldh + c, n);
        if (p.w_post) wpo[u] = load8(p.w_post + c, n);
        if (gate) g[u] = load8(gate + c, n);
        if (p.w_pre) wpr[u] = load8(p.w_pre + c, n);
    }
    // calls f(u, e) for the elements that exist
    auto each = [&](auto f) {
#pragma unroll
        for (int u = 0; u < NV; u++) {
            const int n = H - (u * TPR + (int)threadIdx.x) * 8;
#pragma unroll
            for (int e = 0; e < 8; e++)
                if (e < n) f(u, e);
        }
    };
    // 1 / sqrt(mean (v - mu)^2 + eps), mu = mean v (LAYER) or 0
    auto stats = [&](int kind, auto get, float &mu, float &r) {
        float s[1];
        mu = 0.0f;
        if (kind == NORM_LAYER) {
            s[0] = 0.0f;
            each([&](int u, int e) { s[0] += get(u, e); });
            sum(s);
            mu = s[0] * inv_h;
        }
        s[0] = 0.0f;
        each([&](int u, int e) {
            const float d = get(u, e) - mu;
            s[0] = __builtin_fmaf(d, d, s[0]);
        });
        sum(s);
        r = 1.0f / sqrtf(s[0] * inv_h + p.eps);
    };

    float mu = 0.0f, r = 1.0f;
    if (p.post != NORM_NONE) stats(p.post, [&](int u, int e) { return ld16<BF>(y[u][e]); }, mu, r);
    float hn[NV][8];
#pragma unroll
    for (int u = 0; u < NV; u++) {
#pragma unroll
        for (int e = 0; e < 8; e++) {
            float v = (ld16<BF>(y[u][e]) - mu) * r;
            if (p.w_post && p.post != NORM_NONE) v *= ld16<BF>(wpo[u][e]);
            v *= p.scale;
            if (gate) v *= ld16<BF>(g[u][e]);
            hn[u][e] = h[u].get(e) + v;
            h[u].set(e, hn[u][e]);
        }
        const int c = (u * TPR + (int)threadIdx.x) * 8;
        h[u].store(p.H_out, row * p.ldho + c, H - c);
    }
    stats(p.pre, [&](int u, int e) { return hn[u][e]; }, mu, r);
#pragma unroll
    for (int u = 0; u < NV; u++) {
        half8 x;
#pragma unroll
        for (int e = 0; e < 8; e++) {
            float v = (hn[u][e] - mu) * r;
            if (p.w_pre) v *= ld16<BF>(wpr[u][e]);
            x[e] = st16<BF>(v);
        }
        const int c = (u * TPR + (int)threadIdx.x) * 8;
        store8(p.X + row * p.ldx + c, x, H - c);
    }
}

// ---------------------------------------------------------------------------
// The gradient.  With n = (h' - mu) r the normalised row, dn = dX w_pre:
//   dH' total = dH' + r (dn - [mean dn] - n mean(dn n))      ([..]: LAYER only)
//   dH = dH' total
//   dyw = scale gate dH, dn' = dyw w_post, yn the normalised Y:
//   dY = r' (dn' - [mean dn'] - yn mean(dn' yn)),  dY = dyw for post = NONE
//   dw_pre += dX n,  dw_post += dyw yn,  dgate += scale yn w_post dH.
// One workgroup walks a run of rows that share a gate row and keeps the
// column sums of its rows in registers, so they cost one write of a partial
// row per workgroup; colsum_kernel adds those.  A run never crosses gate
// rows; where a gate row has a single run, its dgate needs no second pass,
// and a workgroup may take several such gate rows.
// ---------------------------------------------------------------------------
struct NormGradParams {
    const _Float16 *dX, *Y, *w_post, *w_pre, *gate;
    const void *dH_out, *H_out;
    void *dH;
    _Float16 *dY;
    int lddx, lddho, ldho, ldy, lddh, lddy;
    int hidden, post, pre;
    float scale, eps;
    int rows_per_gate, rows_per_run;
    int runs_per_gate;       // runs (of rows_per_run rows, the last one shorter) of one gate row
    int runs, runs_per_block;
    int gate_direct;         // runs_per_gate == 1: dgate is the output itself, else partial rows
    float *p_post, *p_pre;   // [blocks][hidden] partial sums, or NULL
    float *dgate;            // [G][hidden], or [runs][hidden] partial sums, or NULL
};

// The elements of one row that a thread of the gradient holds, as NU units
// of 4 consecutive ones: unit u starts at column (u threads + tid) 4.  Without
// TAIL the row length is a multiple of 4, so a unit exists whole or not at all;
// with it the row's last unit may be short.  Absent elements read as zeros.
// (Units of 8 took 25 more registers: past the 128 that let two workgroups
// share a compute unit.)
template <bool BF, typename T, bool TAIL, int NU>
struct RowPart {
    typedef T V __attribute__((ext_vector_type(4), aligned(sizeof(T))));
    V v[NU];
    // (a scalar row address plus a 32-bit offset: one register per unit)
    __device__ __forceinline__ void load(const T *row, int cols, int tid)
    {
        asm volatile("" : "+v"(tid));  // the masks are made again every time: kept, they take too many scalar registers
#pragma unroll
        for (int u = 0; u < NU; u++) {
            const int c = (u * (int)blockDim.x + tid) * 4;
            const char *at = (const char *)row + (uint32_t)c * (uint32_t)sizeof(T);
            v[u] = V{};
            if (TAIL ? c + 4 <= cols : c < cols) {
                v[u] = *(const V *)at;
            } else if (TAIL && c < cols) {
#pragma unroll
                for (int e = 0; e < 3; e++)
                    if (c + e < cols) v[u][e] = ((const T *)at)[e];
            }
        }
    }
    __device__ __forceinline__ void store(T *row, int cols, int tid) const
    {
        asm volatile("" : "+v"(tid));
#pragma unroll
        for (int u = 0; u < NU; u++) {
            const int c = (u * (int)blockDim.x + tid) * 4;
            char *at = (char *)row + (uint32_t)c * (uint32_t)sizeof(T);
            if (TAIL ? c + 4 <= cols : c < cols) {
                *(V *)at = v[u];
            } else if (TAIL && c < cols) {
#pragma unroll
                for (int e = 0; e < 3; e++)
                    if (c + e < cols) ((T *)at)[e] = v[u][e];
            }
        }
    }
    __device__ __forceinline__ void fill(T x)
    {
#pragma unroll
        for (int u = 0; u < NU; u++) v[u] = V{x, x, x, x};
    }
    __device__ __forceinline__ float get(int i) const
    {
        const T x = v[i / 4][i % 4];
        if constexpr (sizeof(T) == 2)
            return ld16<BF>(x);
        else
            return x;
    }
    __device__ __forceinline__ void set(int i, float f)
    {
        if constexpr (sizeof(T) == 2)
            v[i / 4][i % 4] = st16<BF>(f);
        else
            v[i / 4][i % 4] = f;
    }
};

template <bool BF, bool S32, int MAXT, int NU, bool TAIL>
__global__ __launch_bounds__(MAXT, 4) void norm_residual_grad_kernel(NormGradParams p)
{
    constexpr int NE = 4 * NU;
    // Past 4096 columns the registers (128 a lane: 16 waves on a compute unit)
    // hold a row's operands and little else: the sums of the two weights'
    // gradients and the weights themselves live in LDS, where each thread only
    // touches its own elements (with 12 elements the gate stays in registers:
    // 74 KB, so that two workgroups fit).
    constexpr bool LDS_ACC = MAXT > 512 || NU > 2;
    constexpr int LDS_W = !LDS_ACC ? 0 : NU > 2 ? 2 : 3;
    // Alone on its compute unit a workgroup loads the next row while it reduces
    // this one (short last units leave no scalar registers for it).
    constexpr bool PREFETCH = MAXT > 512 && !TAIL;
    using T = typename std::conditional<S32, float, _Float16>::type;
    using Half = RowPart<BF, _Float16, TAIL, NU>;
    using Stream = RowPart<BF, T, TAIL, NU>;
    __shared__ float lds[2][16][6];
    using HV = typename Half::V;
    __shared__ HV w_lds[LDS_ACC ? LDS_W : 1][LDS_ACC ? NU : 1][LDS_ACC ? MAXT : 1];
    __shared__ f32x4 acc_lds[LDS_ACC ? 2 : 1][LDS_ACC ? NE / 4 : 1][LDS_ACC ? MAXT : 1];
    BlockSum<6> sum{lds, (int)blockDim.x >> 6};
    const int H = p.hidden, tid = threadIdx.x;
    // (in vector registers: the scalar ones are short by a few)
    float inv_h = 1.0f / (float)H, scale = p.scale, eps = p.eps;
    asm volatile("" : "+v"(inv_h), "+v"(scale), "+v"(eps));
    const bool pre_mean = p.pre == NORM_LAYER, post_mean = p.post == NORM_LAYER, post_norm = p.post != NORM_NONE;

    // absent weights and gates are ones
    auto row_of = [&](const _Float16 *w) {
        Half r;
        if (w)
            r.load(w, H, tid);
        else
            r.fill(st16<BF>(1.0f));
        return r;
    };
    // does element i of this thread exist?
    auto in_row = [&](int i) {
        int t = tid;
        asm volatile("" : "+v"(t));
        return (i / 4 * (int)blockDim.x + t) * 4 + (TAIL ? i % 4 : 0) < H;
    };
    Half kept[3];  // w_post, w_pre, gate
    auto keep = [&](auto k, const Half &r) {
        if constexpr (k.value < LDS_W) {
#pragma unroll
            for (int u = 0; u < NU; u++) w_lds[k][u][tid] = r.v[u];
        } else {
            kept[k] = r;
        }
    };
    auto weight = [&](auto k) {
        if constexpr (k.value < LDS_W) {
            Half r;
#pragma unroll
            for (int u = 0; u < NU; u++) r.v[u] = w_lds[k][u][tid];
            return r;
        } else {
            return kept[k];
        }
    };
    float a_post[LDS_ACC ? 1 : NE], a_pre[LDS_ACC ? 1 : NE], a_gate[NE];
    keep(std::integral_constant<int, 0>{}, row_of(p.w_post));
    keep(std::integral_constant<int, 1>{}, row_of(p.w_pre));
    if constexpr (LDS_ACC) {
#pragma unroll
        for (int k = 0; k < NE / 4; k++) acc_lds[0][k][tid] = acc_lds[1][k][tid] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    } else {
#pragma unroll
        for (int i = 0; i < NE; i++) a_post[i] = a_pre[i] = 0.0f;
    }
    // (the block's share before the end: u0 + runs_per_block may pass 2^31)
    const int u0 = (int)blockIdx.x * p.runs_per_block, u1 = u0 + min(p.runs - u0, p.runs_per_block);
    for (int run = u0; run < u1; run++) {
        // (the quotient of two scalars is computed in vector registers: without
        // the readfirstlane every row address would live there too)
        const int gr = __builtin_amdgcn_readfirstlane(run / p.runs_per_gate);
        const int in_gate = (run - gr * p.runs_per_gate) * p.rows_per_run;
        const int64_t r0 = (int64_t)gr * p.rows_per_gate + in_gate;
        const int64_t r1 = r0 + min(p.rows_per_run, p.rows_per_gate - in_gate);
        keep(std::integral_constant<int, 2>{}, row_of(p.gate ? p.gate + (int64_t)gr * H : nullptr));
#pragma unroll
        for (int i = 0; i < NE; i++) a_gate[i] = 0.0f;
        Half dx, y;
        Stream dho, h;
        auto fetch = [&](int64_t row, Half &dx_, Stream &h_, Half &y_, Stream &dho_) {
            dx_.load(p.dX + row * p.lddx, H, tid);
            h_.load((const T *)p.H_out + row * p.ldho, H, tid);
            y_.load(p.Y + row * p.ldy, H, tid);
            dho_.load((const T *)p.dH_out + row * p.lddho, H, tid);
        };
        Half dx_next, y_next;
        Stream dho_next, h_next;
        if constexpr (PREFETCH) fetch(r0, dx_next, h_next, y_next, dho_next);
        for (int64_t row = r0; row < r1; row++) {
            if constexpr (PREFETCH) {
                dx = dx_next;
                h = h_next;
                y = y_next;
                dho = dho_next;
                if (row + 1 < r1) fetch(row + 1, dx_next, h_next, y_next, dho_next);
            } else {
                fetch(row, dx, h, y, dho);
            }
            float dn[NE];  // dX w_pre, then scale gate dH
            {
                const Half w = weight(std::integral_constant<int, 1>{});
#pragma unroll
                for (int i = 0; i < NE; i++) dn[i] = dx.get(i) * w.get(i);
            }
            // One pass gives the sums and the sums of squares.  Where a mean is
            // subtracted and is not small beside the deviation (mean^2 > 16
            // variance: the difference of the sums would lose more than 4 bits),
            // a second one takes them about the mean.  (Absent elements are
            // zeros: they only have to be kept out of that second pass.)
            float q[6] = {};
#pragma unroll
            for (int i = 0; i < NE; i++) {
                const float hv = h.get(i), yv = y.get(i);
                q[0] = __builtin_fmaf(hv, hv, q[0]);
                q[1] = __builtin_fmaf(yv, yv, q[1]);
                q[2] = __builtin_fmaf(dn[i], hv, q[2]);
                q[3] += hv;
                q[4] += yv;
                q[5] += dn[i];
            }
            sum(q);
            const float mu_h = pre_mean ? q[3] * inv_h : 0.0f, mu_y = post_mean ? q[4] * inv_h : 0.0f;
            const float m_dn = pre_mean ? q[5] * inv_h : 0.0f;
            float s[3] = {__builtin_fmaf(-mu_h, q[3], q[0]), __builtin_fmaf(-mu_y, q[4], q[1]),
                          __builtin_fmaf(-mu_h, q[5], q[2])};
            // (written so that a NaN, and a variance rounded below zero, take the second pass)
            if (!(mu_h * mu_h <= 16.0f * s[0] * inv_h && mu_y * mu_y <= 16.0f * s[1] * inv_h)) {
                s[0] = s[1] = s[2] = 0.0f;
#pragma unroll
                for (int i = 0; i < NE; i++) {
                    const float hc = in_row(i) ? h.get(i) - mu_h : 0.0f, yc = in_row(i) ? y.get(i) - mu_y : 0.0f;
                    s[0] = __builtin_fmaf(hc, hc, s[0]);
                    s[1] = __builtin_fmaf(yc, yc, s[1]);
                    s[2] = __builtin_fmaf(dn[i], hc, s[2]);
                }
                sum(s);
            }
            const float r_h = 1.0f / sqrtf(s[0] * inv_h + eps);
            const float r_y = post_norm ? 1.0f / sqrtf(s[1] * inv_h + eps) : 1.0f;
            const float c_h = s[2] * inv_h * r_h;  // mean(dn n)
            s[0] = s[1] = s[2] = 0.0f;
            {
                const Half wo = weight(std::integral_constant<int, 0>{}), ga = weight(std::integral_constant<int, 2>{});
#pragma unroll
                for (int k = 0; k < NE / 4; k++) {
                    f32x4 d_post, d_pre;
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const int i = 4 * k + e;
                        const float hn = (h.get(i) - mu_h) * r_h;
                        const float dh = dho.get(i) + (dn[i] - m_dn - hn * c_h) * r_h;
                        dho.set(i, dh);
                        d_pre[e] = dx.get(i) * hn;
                        const float yn = (y.get(i) - mu_y) * r_y, w = wo.get(i);
                        a_gate[i] = __builtin_fmaf(scale * dh, yn * w, a_gate[i]);
                        dn[i] = scale * dh * ga.get(i);
                        d_post[e] = dn[i] * yn;
                        if (in_row(i)) {
                            s[0] = __builtin_fmaf(dn[i], w, s[0]);
                            s[1] = __builtin_fmaf(d_post[e], w, s[1]);
                        }
                    }
                    if constexpr (LDS_ACC) {
                        acc_lds[0][k][tid] += d_post;
                        acc_lds[1][k][tid] += d_pre;
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            a_post[4 * k + e] += d_post[e];
                            a_pre[4 * k + e] += d_pre[e];
                        }
                    }
                }
            }
            dho.store((T *)p.dH + row * p.lddh, H, tid);
            float m_d = 0.0f, c_y = 0.0f;
            if (post_norm) {
                sum(s);
                m_d = post_mean ? s[0] * inv_h : 0.0f;
                c_y = s[1] * inv_h;
            }
            {
                const Half wo = weight(std::integral_constant<int, 0>{});
#pragma unroll
                for (int i = 0; i < NE; i++) {
                    const float yn = (y.get(i) - mu_y) * r_y;
                    y.set(i, (dn[i] * wo.get(i) - m_d - yn * c_y) * r_y);
                }
            }
            y.store(p.dY + row * p.lddy, H, tid);
        }
        if (p.dgate) {
            float *dst = p.dgate + (int64_t)(p.gate_direct ? gr : run) * H;
#pragma unroll
            for (int i = 0; i < NE; i++)
                if (in_row(i)) dst[(i / 4 * (int)blockDim.x + tid) * 4 + i % 4] = a_gate[i];
        }
    }
#pragma unroll
    for (int i = 0; i < NE; i++) {
        if (!in_row(i)) continue;
        const int64_t at = (int64_t)blockIdx.x * H + (i / 4 * (int)blockDim.x + tid) * 4 + i % 4;
        if (p.p_post) p.p_post[at] = LDS_ACC ? acc_lds[0][LDS_ACC ? i / 4 : 0][LDS_ACC ? tid : 0][i % 4] : a_post[LDS_ACC ? 0 : i];
        if (p.p_pre) p.p_pre[at] = LDS_ACC ? acc_lds[LDS_ACC ? 1 : 0][LDS_ACC ? i / 4 : 0][LDS_ACC ? tid : 0][i % 4] : a_pre[LDS_ACC ? 0 : i];
    }
}

}  // namespace gemm_epi
