// moe.hip -- the C ABI of the mixture-of-experts layer (include/fp8_ops.h):
// argument checks, workspace layout and launches.
#include <hip/hip_runtime.h>
#include <algorithm>
#include <stdint.h>

#include "fp8_ops.h"
#include "moe.hpp"
#include "ops_host.hpp"

using namespace gemm_epi;

namespace {

static_assert(kMoeExperts == GE_MOE_MAX_EXPERTS && kMoeTop == GE_MOE_MAX_TOP_K, "the header's limits");

// a weight matrix of every expert, in 16 bits or in 8 with scales
int check_experts(const void *w, int64_t ld, int64_t stride, const void *s, int64_t lds, int64_t s_stride, int64_t rows,
                  int64_t cols, int64_t experts)
{
    if (!w) return GEMM_EPI_ERR_NULL_INPUT;
    if (!s && !aligned(w, 2)) return GEMM_EPI_ERR_ALIGN;
    if (ld < cols || ld > GE_MAX_COLS) return GEMM_EPI_ERR_SHAPE;
    if (experts > 1 && stride < (rows - 1) * ld + cols) return GEMM_EPI_ERR_SHAPE;
    if (!s) return GEMM_EPI_OK;
    const int64_t rb = ceil_div(rows, 128), cb = ceil_div(cols, 128);
    if (lds < cb || lds > GE_MAX_COLS || (experts > 1 && s_stride < (rb - 1) * lds + cb)) return GEMM_EPI_ERR_SHAPE;
    return GEMM_EPI_OK;
}

int check_moe(const ge_moe_args *a)
{
    if (!a) return GEMM_EPI_ERR_NULL_INPUT;
    if (a->T < 0 || a->T > INT32_MAX - 256 || a->hidden < 1 || a->hidden > GE_MAX_COLS || a->inner < 1 ||
        a->inner > GE_MAX_COLS / 2 || a->experts < 1 || a->experts > GE_MOE_MAX_EXPERTS || a->top_k < 1 ||
        a->top_k > GE_MOE_MAX_TOP_K || a->top_k > a->experts)
        return GEMM_EPI_ERR_SHAPE;
    if (a->act < GE_ACT_IDENTITY || a->act > GE_ACT_SILU || a->gated < 0 || a->gated > 1 || a->renormalize < 0 ||
        a->renormalize > 1)
        return GEMM_EPI_ERR_KIND;
    GE_CHECK(check_dtype(a->dtype));
    if (!a->US != !a->DS) return GEMM_EPI_ERR_NULL_INPUT;
    GE_CHECK(check_matrix(a->Wr, a->ldwr, a->hidden, 2, GEMM_EPI_ERR_NULL_INPUT));
    GE_CHECK(check_experts(a->Up, a->ldu, a->up_stride, a->US, a->ldus, a->us_stride, (1 + a->gated) * a->inner,
                           a->hidden, a->experts));
    GE_CHECK(check_experts(a->Down, a->lddn, a->down_stride, a->DS, a->ldds, a->ds_stride, a->hidden, a->inner,
                           a->experts));
    if (a->T == 0) return GEMM_EPI_OK;
    GE_CHECK(check_matrix(a->X, a->ldx, a->hidden, 2, GEMM_EPI_ERR_NULL_INPUT));
    if (a->residual) GE_CHECK(check_matrix(a->residual, a->ldr, a->hidden, 2, GEMM_EPI_ERR_NULL_INPUT));
    return check_matrix(a->D, a->ldd, a->hidden, 2, GEMM_EPI_ERR_NULL_OUTPUT);
}

struct MoePlan {
    int64_t logits = 0, chosen = 0, weight = 0, total = 0, hidden = 0, low = 0, bytes = 0;
};

int plan_moe(const ge_moe_args *a, MoePlan &pl)
{
    GE_CHECK(check_moe(a));
    const int64_t t = std::min<int64_t>(a->T, kMoeChunk);
    if (t == 0) return GEMM_EPI_OK;
    Layout lay;
    pl.logits = lay.take(t * a->experts * 4);
    pl.chosen = lay.take(t * a->top_k * 4);
    pl.weight = lay.take(t * a->top_k * 4);
    pl.total = lay.take(t * 4);
    pl.hidden = lay.take(t * a->top_k * a->inner * 2);
    pl.low = lay.take(t * a->top_k * a->inner);
    pl.bytes = lay.bytes;
    return GEMM_EPI_OK;
}

// One block of 16 tokens at a time, or two where the experts have 12 and more on
// average: 64 tokens, 16 experts of 4096 x 1024, 4 each, in 8 bits 76.6 us with two and 80.2
// with one (16 bits 116 and 115), 8 experts of 4096 x 2048, 4 each, 16 bits 146 and 155.
template <bool BF, bool W8, int ACT, bool GATED>
hipError_t launch_up(const MoeParams &q, int by_choice, int shared, dim3 g, hipStream_t s)
{
    if (q.T > 16 && q.T * q.k >= 12 * q.E)
        return launch(moe_up_kernel<BF, W8, ACT, GATED, 2>, g, dim3(256), s, q, by_choice, shared);
    return launch(moe_up_kernel<BF, W8, ACT, GATED, 1>, g, dim3(256), s, q, by_choice, shared);
}
template <bool BF, bool W8, int ACT>
hipError_t launch_moe2(const MoeParams &q, hipStream_t s)
{
    hipError_t e = launch(moe_router_kernel<BF>, dim3((unsigned)ceil_div(q.E, 4), (unsigned)ceil_div(q.T, 4)), dim3(256),
                          s, q);
    if (e != hipSuccess) return e;
    // workgroups by expert, or by choice where those are fewer (one token, 8 of 64
    // experts in 8 bits: 32.8 us for the layer, 44.1 by expert; 4 tokens 82 and 79)
    const int by_choice = q.T * q.k < q.E;
    const int64_t rows = by_choice ? q.T * q.k : q.E;
    // a wave to a tile of 16 inner rows where that fills the chip's 8 waves a compute unit
    const int64_t row_tiles = ceil_div(q.I, 16);
    const int shared = rows * row_tiles < 8 * kCUs;
    const dim3 g((unsigned)(shared ? row_tiles : ceil_div(row_tiles, 4)), (unsigned)rows);
    e = q.gated ? launch_up<BF, W8, ACT, true>(q, by_choice, shared, g, s)
                : launch_up<BF, W8, ACT, false>(q, by_choice, shared, g, s);
    if (e != hipSuccess) return e;
    return launch(moe_down_kernel<BF, W8>, dim3((unsigned)ceil_div(q.H, 16)), dim3(64 * kDownWaves), s, q);
}
template <bool BF, bool W8>
hipError_t launch_moe(int act, const MoeParams &q, hipStream_t s)
{
    switch (act) {
    case ACT_RELU: return launch_moe2<BF, W8, ACT_RELU>(q, s);
    case ACT_GELU: return launch_moe2<BF, W8, ACT_GELU>(q, s);
    case ACT_SILU: return launch_moe2<BF, W8, ACT_SILU>(q, s);
    default: return launch_moe2<BF, W8, ACT_IDENTITY>(q, s);
    }
}

}  // namespace

extern "C" {

int ge_moe_workspace(const ge_moe_args *a, int64_t *bytes)
{
    MoePlan pl;
    GE_CHECK(plan_moe(a, pl));
    if (!bytes) return GEMM_EPI_ERR_NULL_OUTPUT;
    *bytes = pl.bytes;
    return GEMM_EPI_OK;
}

int ge_moe(const ge_moe_args *a)
{
    MoePlan pl;
    GE_CHECK(plan_moe(a, pl));
    GE_CHECK(check_workspace(a->workspace, a->workspace_bytes, pl.bytes));
    char *ws = (char *)a->workspace;
    MoeParams q = {};
    q.H = (int)a->hidden;
    q.E = (int)a->experts;
    q.I = (int)a->inner;
    q.k = (int)a->top_k;
    q.gated = (int)a->gated;
    q.renormalize = (int)a->renormalize;
    q.Wr = (const _Float16 *)a->Wr;
    q.Up = a->Up;
    q.Down = a->Down;
    q.US = (const uint8_t *)a->US;
    q.DS = (const uint8_t *)a->DS;
    q.ldx = a->ldx;
    q.ldwr = a->ldwr;
    q.ldr = a->ldr;
    q.ldu = a->ldu;
    q.up_stride = a->up_stride;
    q.ldus = a->ldus;
    q.us_stride = a->us_stride;
    q.lddn = a->lddn;
    q.down_stride = a->down_stride;
    q.ldds = a->ldds;
    q.ds_stride = a->ds_stride;
    q.ldd = a->ldd;
    q.logits = (float *)(ws + pl.logits);
    q.chosen = (int *)(ws + pl.chosen);
    q.weight = (float *)(ws + pl.weight);
    q.total = (float *)(ws + pl.total);
    q.hidden = (_Float16 *)(ws + pl.hidden);
    q.low = (uint8_t *)ws + pl.low;
    const bool bf = a->dtype == GEMM_EPI_BF16;
    hipStream_t s = (hipStream_t)a->stream;
    for (int64_t t = 0; t < a->T; t += kMoeChunk) {
        q.T = (int)std::min<int64_t>(a->T - t, kMoeChunk);
        q.X = (const _Float16 *)a->X + t * a->ldx;
        q.R = a->residual ? (const _Float16 *)a->residual + t * a->ldr : nullptr;
        q.D = (_Float16 *)a->D + t * a->ldd;
        const int act = (int)a->act;
        hipError_t e;
        if (a->US)
            e = bf ? launch_moe<true, true>(act, q, s) : launch_moe<false, true>(act, q, s);
        else
            e = bf ? launch_moe<true, false>(act, q, s) : launch_moe<false, false>(act, q, s);
        GE_TRY(e);
    }
    return GEMM_EPI_OK;
}

}  // extern "C"
