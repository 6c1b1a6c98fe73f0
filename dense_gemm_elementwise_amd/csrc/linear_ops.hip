// linear_ops.hip -- the C ABI of include/linear_ops.h: argument checks, plans
// (tiles, splits, pieces of the vocabulary, workspace layout) and launches.
//
// Every check runs on the host before any HIP call.  A plan depends on the
// arguments alone, so the workspace query and the call lay the workspace out
// alike.
#include <hip/hip_runtime.h>
#include <algorithm>
#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include "linear_launch.hpp"
#include "linear_ops.h"
#include "linear_small.hpp"
#include "norm_residual.hpp"

namespace gemm_epi {
void set_last_hip_error(int e);  // gemm_epi.hip
}

using namespace gemm_epi;

namespace {

constexpr int kCUs = 256;

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
int64_t ceil_div(int64_t v, int64_t m) { return (v + m - 1) / m; }

int hip_status(hipError_t e)
{
    if (e == hipSuccess) return GEMM_EPI_OK;
    set_last_hip_error((int)e);
    return GEMM_EPI_ERR_HIP;
}

#define GE_TRY(call)                                  \
    do {                                              \
        const int ge_rc = hip_status(call);           \
        if (ge_rc != GEMM_EPI_OK) return ge_rc;       \
    } while (0)

// (arguments convert to the kernel's own parameter types)
template <typename T>
struct Same {
    using type = T;
};
template <typename... P>
hipError_t launch(void (*kernel)(P...), dim3 grid, dim3 block, hipStream_t s, typename Same<P>::type... a)
{
    void *args[] = {(void *)&a...};
    return hipLaunchKernel((const void *)kernel, grid, block, args, 0, s);
}

// a matrix operand: NULL, alignment and row stride
int check_matrix(const void *p, int64_t ld, int64_t cols, uintptr_t es, int null_status)
{
    if (!p) return null_status;
    if (!aligned(p, es)) return GEMM_EPI_ERR_ALIGN;
    if (ld < cols || ld > GE_MAX_COLS) return GEMM_EPI_ERR_SHAPE;
    return GEMM_EPI_OK;
}
#define GE_CHECK(call)                          \
    do {                                        \
        const int ge_rc = (call);               \
        if (ge_rc != GEMM_EPI_OK) return ge_rc; \
    } while (0)

int check_dims(int64_t rows, int64_t rows2, int64_t cols)
{
    if (rows < 0 || rows > INT32_MAX - 256 || rows2 < 1 || rows2 > INT32_MAX - 256 || cols < 1 || cols > GE_MAX_COLS)
        return GEMM_EPI_ERR_SHAPE;
    return GEMM_EPI_OK;
}
int check_dtype(int64_t dtype) { return dtype == GEMM_EPI_F16 || dtype == GEMM_EPI_BF16 ? GEMM_EPI_OK : GEMM_EPI_ERR_DTYPE; }

// A region of the workspace.
struct Layout {
    int64_t bytes = 0;
    int64_t take(int64_t n)
    {
        const int64_t at = bytes;
        bytes = round_up(bytes + n, 256);
        return at;
    }
};

int check_workspace(const void *ws, int64_t have, int64_t need)
{
    if (need == 0) return GEMM_EPI_OK;
    if (!ws || have < need) return GEMM_EPI_ERR_WORKSPACE;
    return aligned(ws, 16) ? GEMM_EPI_OK : GEMM_EPI_ERR_ALIGN;
}

constexpr unsigned kAllTiles = 0xF;  // bits: indices into kLinTiles

// ---- tiles and splits ---------------------------------------------------------
// One product M x N x K on `tile`, its contraction cut into `splits` pieces of
// k_split (a multiple of 64).
struct ProductPlan {
    int tile = kLinSmall, splits = 1;
    int tiles_m = 0, tiles_n = 0;
    int64_t k_split = 0;
    int64_t part_bytes = 0;  // fp32 partial sums of the splits
    double cost = 0;         // estimated microseconds
};

// Estimated microseconds of a plan, from timings of every tile and split on 54
// shapes (64^3 to 8192^2 x 2048, and 1 to 40 rows against 8192 x 4096): each
// round of workgroups costs a fixed time (first loads, epilogue) and a time
// per unit of K, which grows with the share of the chip at work (its clock
// falls under full load).  Measured (fixed us; ns per unit of K, from few
// workgroups to a full chip):
//   256 x 256           13;   15.6 .. 22
//   128 x 256, 256 x 128  9;    8   .. 11.8
//   128 x 128            5;    7.2 .. 8.6, and 5.5; 13.2 for two on a CU
// Past two rounds the workgroups drift apart and the last round costs half of
// one.  A split adds a launch, its workgroups and the partial sums'
// round trip.  The pick was
// within 8% of the fastest form on all but 3 of the 54.
double product_cost(int64_t M, int64_t N, int64_t K, int tile, int splits)
{
    const LinTile t = kLinTiles[tile];
    const double groups = (double)(ceil_div(M, t.bm) * ceil_div(N, t.bn) * splits);
    const double k = (double)round_up(ceil_div(K, splits), 32) * 1e-3;
    const double share = std::min(1.0, groups / kCUs);
    double slots = kCUs, round;
    if (tile == kLinBig) {
        round = 13.0 + k * (15.6 + 6.4 * share);
    } else if (tile != kLinSmall) {
        round = 9.0 + k * (8.0 + 3.8 * share);
    } else if (groups <= kCUs) {
        round = 5.0 + k * (7.2 + 1.4 * share);
    } else {
        slots = 2 * kCUs;
        round = 5.5 + k * 13.2;
    }
    const double rounds = groups / slots;
    double us = round * (rounds <= 2.0 ? ceil(rounds) : rounds + 0.5);
    if (splits > 1) us += 2.0 + 0.25 * splits + (double)splits * M * N * 8 / 4.0e6;
    return us;
}

// a launch holds fewer than 2^32 threads: 2^24 workgroups of 256
constexpr int64_t kMaxGroups = (1 << 24) - 1;
int64_t product_groups(const ProductPlan &pl) { return (int64_t)pl.tiles_m * pl.tiles_n * pl.splits; }
bool product_fits(const ProductPlan &pl) { return product_groups(pl) <= kMaxGroups; }

// tiles: bit mask of the tiles that exist for this product, split_tiles: of
// those whose split form exists; small: the best plan on the 128 x 128 tile, if
// it is wanted too.  Of the tiles whose grid one launch holds the cheapest (a
// larger tile where a smaller one would be too many); where none is, the plan does
// not pass product_fits.
ProductPlan plan_product(int64_t M, int64_t N, int64_t K, unsigned tiles, unsigned split_tiles,
                         ProductPlan *small = nullptr)
{
    ProductPlan best;
    for (int i = 0; i < 4; i++) {
        if (!(tiles >> i & 1)) continue;
        const LinTile t = kLinTiles[i];
        ProductPlan of_tile;
        of_tile.tile = i;
        of_tile.cost = 1e300;
        of_tile.tiles_m = (int)ceil_div(M, t.bm);
        of_tile.tiles_n = (int)ceil_div(N, t.bn);
        const int64_t grid = (int64_t)of_tile.tiles_m * of_tile.tiles_n;
        for (int want = 1; want <= 64; want *= 2) {
            if (want > 1 && (!(split_tiles >> i & 1) || K < want * 256 || grid * want > 4 * kCUs)) break;
            const int64_t k_split = round_up(ceil_div(K, want), 64);
            const int splits = (int)ceil_div(K, k_split);
            const double c = product_cost(M, N, K, i, splits);
            if (c < of_tile.cost) {
                of_tile.cost = c;
                of_tile.splits = splits;
                of_tile.k_split = k_split;
            }
        }
        of_tile.part_bytes = of_tile.splits > 1 ? of_tile.splits * M * round_up(N, 8) * 4 : 0;
        if (small && i == kLinSmall) *small = of_tile;
        const bool fits = product_fits(of_tile), best_fits = best.tiles_m > 0 && product_fits(best);
        if (best.tiles_m == 0 || (fits == best_fits ? of_tile.cost < best.cost : fits)) best = of_tile;
    }
    return best;
}

// The grid of a kernel that takes its row, or its block of columns, from block_row.
dim3 row_grid(int64_t rows)
{
    return dim3((unsigned)std::min(rows, kRowGrid), (unsigned)ceil_div(rows, kRowGrid));
}

void set_product(LinParams &p, const ProductPlan &pl, int64_t M, int64_t N, int64_t K)
{
    p.M = (int)M;
    p.N = (int)N;
    p.K = (int)K;
    p.tiles_m = pl.tiles_m;
    p.tiles_n = pl.tiles_n;
    p.num_tiles = pl.tiles_m * pl.tiles_n;
    p.group_m = 8;
    p.k_split = (int)pl.k_split;
}

// rows that the 16-byte DMA of the products can read
bool dma_rows(const void *p, int64_t ld, int64_t cols) { return cols % 8 == 0 && ld % 8 == 0 && aligned(p, 16); }

// An operand as the products read it: in place, or a padded copy.
struct Operand16 {
    const _Float16 *p;
    int64_t ld;
};
struct StagePlan2 {
    bool on[2] = {false, false};
    int64_t off[2] = {0, 0};
    int64_t ldo = 0;
};
// The copies of a staging plan (`cols` columns); the operands then are the copies.
struct StageSet {
    PadParams q = {};
    int n = 0;
    unsigned blocks = 0;
};
StageSet stage_set(const StagePlan2 &st, char *ws, int64_t cols, Operand16 &a, int64_t a_rows, Operand16 &b,
                   int64_t b_rows)
{
    StageSet r;
    Operand16 *op[2] = {&a, &b};
    const int64_t rows[2] = {a_rows, b_rows};
    for (int i = 0; i < 2; i++) {
        if (!st.on[i]) continue;
        r.q.src[r.n] = op[i]->p;
        r.q.lds[r.n] = op[i]->ld;
        r.q.rows[r.n] = rows[i];
        r.q.dst[r.n] = (_Float16 *)(ws + st.off[i]);
        op[i]->p = r.q.dst[r.n];
        op[i]->ld = st.ldo;
        r.n++;
    }
    r.q.cols = (int)cols;
    r.q.ldo = (int)st.ldo;
    r.blocks = (unsigned)std::min<int64_t>(ceil_div(std::max(r.q.rows[0], r.q.rows[1]) * (st.ldo / 8), 256), 4096);
    return r;
}
hipError_t run_staging(const StageSet &st, hipStream_t s)
{
    return st.n ? launch(pad_rows_kernel, dim3(st.blocks, st.n), dim3(256), s, st.q) : hipSuccess;
}
StagePlan2 plan_staging2(const void *a, int64_t lda, int64_t a_rows, const void *b, int64_t ldb, int64_t b_rows,
                         int64_t cols, Layout &lay)
{
    StagePlan2 st;
    st.ldo = round_up(cols, 8);
    st.on[0] = !dma_rows(a, lda, cols);
    st.on[1] = !dma_rows(b, ldb, cols);
    if (st.on[0]) st.off[0] = lay.take(a_rows * st.ldo * 2);
    if (st.on[1]) st.off[1] = lay.take(b_rows * st.ldo * 2);
    return st;
}

template <bool BF, int EPI>
hipError_t launch_split_sum(int act, SplitSumParams q, hipStream_t s)
{
    // several lanes for an output while that does not fill the chip
    const int64_t outputs = (int64_t)q.M * ((q.N + 7) / 8);
    q.lanes = outputs * 8 <= 512 * kCUs ? (q.splits >= 16 ? 8 : q.splits >= 8 ? 4 : 1) : 1;
    const int64_t blocks = std::min<int64_t>(ceil_div(outputs * q.lanes, 256), 4096);
    const dim3 g((unsigned)blocks), b(256);
    if constexpr (EPI == LE_LINEAR) {
        switch (act) {
        case ACT_RELU: return launch(split_sum_kernel<BF, EPI, ACT_RELU>, g, b, s, q);
        case ACT_GELU: return launch(split_sum_kernel<BF, EPI, ACT_GELU>, g, b, s, q);
        case ACT_SILU: return launch(split_sum_kernel<BF, EPI, ACT_SILU>, g, b, s, q);
        default: break;
        }
    }
    return launch(split_sum_kernel<BF, EPI, ACT_IDENTITY>, g, b, s, q);
}

// A gradient product (NN or TN) into D (16-bit), or into / onto the fp32
// accumulator acc, through partial sums where the plan splits it.
struct GradProduct {
    LinParams p;
    SplitSumParams sum;
    int tile, groups;
    bool split;
};
// p holds the operands
GradProduct grad_product(LinParams p, const ProductPlan &pl, int64_t M, int64_t N, int64_t K, void *D, int64_t ldd,
                         float *acc, bool acc_in, bool acc_out, const float *alpha, float *part)
{
    GradProduct g = {};
    set_product(p, pl, M, N, K);
    const int64_t ldc = round_up(N, 8);
    p.ldc = ldc;
    p.ldd = ldd;
    g.tile = pl.tile;
    g.groups = p.num_tiles * pl.splits;
    g.split = pl.splits > 1;
    if (g.split) {
        p.C32 = part;
        p.c_split = M * ldc;
        p.acc_out = 1;
        SplitSumParams &q = g.sum;
        q.part = part;
        q.splits = pl.splits;
        q.M = (int)M;
        q.N = (int)N;
        q.ldc = ldc;
        q.c_split = M * ldc;
        q.D = (_Float16 *)D;
        q.ldd = ldd;
        q.C32 = acc;
        q.acc_in = acc_in;
        q.acc_out = acc_out;
        q.alpha = alpha;
    } else {
        p.C32 = acc;
        p.acc_in = acc_in;
        p.acc_out = acc_out;
        p.alpha = alpha;
        p.D = (_Float16 *)D;
        p.vec = dma_rows(D, ldd, N);
    }
    g.p = p;
    return g;
}
template <bool BF>
hipError_t run_grad_sum(const GradProduct &g, hipStream_t s)
{
    return g.split ? launch_split_sum<BF, LE_OUT>(0, g.sum, s) : hipSuccess;
}
template <bool BF>
hipError_t run_grad_product(bool tn, const GradProduct &g, hipStream_t s)
{
    hipError_t e;
    if (tn)
        e = BF ? lin_launch_tn_bf16(g.tile, g.p, g.groups, s) : lin_launch_tn_f16(g.tile, g.p, g.groups, s);
    else
        e = BF ? lin_launch_nn_bf16(g.tile, g.p, g.groups, s) : lin_launch_nn_f16(g.tile, g.p, g.groups, s);
    return e == hipSuccess ? run_grad_sum<BF>(g, s) : e;
}

// The two products of a gradient, dX (M x K over N) and dW (N x K over M):
// each by its own plan, or both in one launch.
struct GradPlan {
    ProductPlan dx, dw;
    bool pair = false;
    int64_t off_dx = 0, off_dw = 0;  // partial sums, relative to the plan's own region
    int64_t part_bytes = 0;
    bool fits = true;
};
GradPlan plan_grad(int64_t M, int64_t N, int64_t K, bool want_dx, bool want_dw)
{
    GradPlan g;
    ProductPlan x, w;  // on the small tile
    g.dx = plan_product(M, K, round_up(N, 8), kAllTiles, kAllTiles, &x);
    g.dw = plan_product(N, K, M, kAllTiles, kAllTiles, &w);
    g.fits = (!want_dx || product_fits(g.dx)) && (!want_dw || product_fits(g.dw));
    if (want_dx && want_dw) {
        // Beside each other two products cost the longer one, and the shorter one
        // as far as their workgroups are more than the compute units: all of it
        // from twice 256 more on, less a launch and an idle tail, 5 us.  On 32
        // shapes: 64^3 14.7 us apart, 10.9 in one launch; 333 x 9999 x 1000 (P in
        // between) 55 and 45; 512 x 4096 x 4096 59 and 53; 4096^3, where the
        // large tile wins, 222 and 255.
        // The contraction stays cut where the product alone would cut it: a gradient
        // has the same bits whether or not the other one is wanted (the tile does
        // not change them, the order of the sum along K does).
        const bool same = x.k_split == g.dx.k_split && w.k_split == g.dw.k_split;
        const int64_t groups = product_groups(x) + product_groups(w);
        const double beside = std::min(1.0, std::max(0.0, (double)(groups - kCUs) / (2.0 * kCUs)));
        const double pair =
            std::max(x.cost, w.cost) + beside * std::min(x.cost, w.cost) - (beside == 1.0 ? 5.0 : 0.0);
        if (same && groups <= kMaxGroups && pair < g.dx.cost + g.dw.cost) {
            g.pair = true;
            g.dx = x;
            g.dw = w;
        }
    }
    g.off_dw = want_dx ? round_up(g.dx.part_bytes, 256) : 0;
    g.part_bytes = g.off_dw + (want_dw ? g.dw.part_bytes : 0);
    return g;
}
template <bool BF>
hipError_t run_grad(const GradPlan &pl, const GradProduct *dx, const GradProduct *dw, hipStream_t s)
{
    if (pl.pair && dx && dw) {
        const LinPair p = {dx->p, dw->p, dx->groups};
        const int groups = dx->groups + dw->groups;
        hipError_t e = BF ? lin_launch_pair_bf16(p, groups, s) : lin_launch_pair_f16(p, groups, s);
        if (e == hipSuccess) e = run_grad_sum<BF>(*dx, s);
        return e == hipSuccess ? run_grad_sum<BF>(*dw, s) : e;
    }
    hipError_t e = dx ? run_grad_product<BF>(false, *dx, s) : hipSuccess;
    return e == hipSuccess && dw ? run_grad_product<BF>(true, *dw, s) : e;
}

hipError_t run_zero(void *p, int64_t ld_bytes, int64_t rows, int64_t bytes, hipStream_t s)
{
    const int64_t blocks = std::min<int64_t>(ceil_div(rows * (bytes / 2), 256), 4096);
    return launch(zero_rows_kernel, dim3((unsigned)blocks), dim3(256), s, (char *)p, ld_bytes, rows, bytes / 2);
}

// ---- linear -------------------------------------------------------------------
// Rows of X up to which a product reads W through row_dot_kernel, and through
// skinny_kernel (one MFMA block); past them it takes the tiles.  linear_small.hpp
// has the times on both sides of the first.
constexpr int64_t dot_rows(bool bf) { return bf ? 1 : 2; }
constexpr int64_t kSkinnyRows = 16;
// workgroups of row_dot_kernel: eight of four waves on every CU, fewer where
// there are fewer rows of W
int row_dot_groups(int64_t N) { return (int)std::min<int64_t>(ceil_div(N, 4), 8 * kCUs); }

// columns of the vocabulary per workgroup of skinny_kernel
constexpr int64_t kSkinnyWide = 32768;
int64_t skinny_cols(int64_t V) { return V < kSkinnyWide ? 16 : 64; }

template <bool BF, int MODE, int ACT>
hipError_t launch_skinny(const SkinnyParams &q, hipStream_t s)
{
    const dim3 b(256);
    if constexpr (MODE != SK_LINEAR)
        if (skinny_cols(q.N) == 64)
            return launch(skinny_kernel<BF, MODE, ACT, false>, row_grid(ceil_div(q.N, 64)), b, s, q);
    return launch(skinny_kernel<BF, MODE, ACT, true>, row_grid(ceil_div(q.N, 16)), b, s, q);
}

template <bool BF, bool XENT, int ACT>
hipError_t launch_few_rows(const SkinnyParams &q, hipStream_t s)
{
    const dim3 b(256);
    const dim3 g((unsigned)row_dot_groups(q.N));
    if (q.M == 1) return launch(row_dot_kernel<BF, XENT, ACT, 1>, g, b, s, q);
    if constexpr (dot_rows(BF) == 2)
        if (q.M == 2) return launch(row_dot_kernel<BF, XENT, ACT, 2>, g, b, s, q);
    return launch_skinny<BF, XENT ? SK_STATS : SK_LINEAR, ACT>(q, s);
}

struct LinearPlan {
    bool skinny = false;
    StagePlan2 st;  // X, W
    ProductPlan pl;
    int64_t off_part = 0, bytes = 0;
};

int check_linear(const ge_linear_args *a)
{
    if (!a) return GEMM_EPI_ERR_NULL_INPUT;
    GE_CHECK(check_dims(a->M, a->N, a->K));
    if (a->N > GE_MAX_COLS) return GEMM_EPI_ERR_SHAPE;
    if (!a->W || (a->M > 0 && !a->X)) return GEMM_EPI_ERR_NULL_INPUT;
    if (a->M > 0 && !a->D) return GEMM_EPI_ERR_NULL_OUTPUT;
    if (a->act < GE_ACT_IDENTITY || a->act > GE_ACT_SILU) return GEMM_EPI_ERR_KIND;
    GE_CHECK(check_dtype(a->dtype));
    GE_CHECK(check_matrix(a->W, a->ldw, a->K, 2, GEMM_EPI_ERR_NULL_INPUT));
    if (a->X) GE_CHECK(check_matrix(a->X, a->ldx, a->K, 2, GEMM_EPI_ERR_NULL_INPUT));
    if (a->D) GE_CHECK(check_matrix(a->D, a->ldd, a->N, 2, GEMM_EPI_ERR_NULL_OUTPUT));
    if (a->residual) GE_CHECK(check_matrix(a->residual, a->ldr, a->N, 2, GEMM_EPI_ERR_NULL_INPUT));
    if (a->Z) GE_CHECK(check_matrix(a->Z, a->ldz, a->N, 2, GEMM_EPI_ERR_NULL_OUTPUT));
    if (a->bias && !aligned(a->bias, 2)) return GEMM_EPI_ERR_ALIGN;
    return GEMM_EPI_OK;
}

int plan_linear(const ge_linear_args *a, LinearPlan &pl)
{
    GE_CHECK(check_linear(a));
    if (a->M == 0) return GEMM_EPI_OK;
    pl.skinny = a->M <= kSkinnyRows;
    if (pl.skinny) return GEMM_EPI_OK;
    Layout lay;
    pl.st = plan_staging2(a->X, a->ldx, a->M, a->W, a->ldw, a->N, a->K, lay);
    pl.pl = plan_product(a->M, a->N, a->K, 0xF, 1u << kLinSmall);
    if (!product_fits(pl.pl)) return GEMM_EPI_ERR_SHAPE;
    pl.off_part = lay.take(pl.pl.part_bytes);
    pl.bytes = lay.bytes;
    return GEMM_EPI_OK;
}

template <bool BF>
int run_linear(const ge_linear_args *a, const LinearPlan &pl)
{
    hipStream_t s = (hipStream_t)a->stream;
    char *ws = (char *)a->workspace;
    const int act = (int)a->act;
    if (pl.skinny) {
        SkinnyParams q = {};
        q.X = (const _Float16 *)a->X;
        q.W = (const _Float16 *)a->W;
        q.ldx = a->ldx;
        q.ldw = a->ldw;
        q.M = (int)a->M;
        q.N = (int)a->N;
        q.K = (int)a->K;
        q.bias = (const _Float16 *)a->bias;
        q.R = (const _Float16 *)a->residual;
        q.D = (_Float16 *)a->D;
        q.Z = (_Float16 *)a->Z;
        q.ldr = a->ldr;
        q.ldd = a->ldd;
        q.ldz = a->ldz;
        switch (act) {
        case ACT_RELU: return hip_status(launch_few_rows<BF, false, ACT_RELU>(q, s));
        case ACT_GELU: return hip_status(launch_few_rows<BF, false, ACT_GELU>(q, s));
        case ACT_SILU: return hip_status(launch_few_rows<BF, false, ACT_SILU>(q, s));
        default: return hip_status(launch_few_rows<BF, false, ACT_IDENTITY>(q, s));
        }
    }
    Operand16 x = {(const _Float16 *)a->X, a->ldx}, w = {(const _Float16 *)a->W, a->ldw};
    GE_TRY(run_staging(stage_set(pl.st, ws, a->K, x, a->M, w, a->N), s));
    LinParams p = {};
    set_product(p, pl.pl, a->M, a->N, round_up(a->K, 8));
    p.A = x.p;
    p.lda = x.ld;
    p.B = w.p;
    p.ldb = w.ld;
    const int groups = p.num_tiles * pl.pl.splits;
    if (pl.pl.splits > 1) {
        const int64_t ldc = round_up(a->N, 8);
        p.C32 = (float *)(ws + pl.off_part);
        p.ldc = ldc;
        p.c_split = a->M * ldc;
        p.acc_out = 1;
        GE_TRY(BF ? lin_launch_fwd_split_bf16(p, groups, s) : lin_launch_fwd_split_f16(p, groups, s));
        SplitSumParams q = {};
        q.part = p.C32;
        q.splits = pl.pl.splits;
        q.M = (int)a->M;
        q.N = (int)a->N;
        q.ldc = ldc;
        q.c_split = p.c_split;
        q.bias = (const _Float16 *)a->bias;
        q.R = (const _Float16 *)a->residual;
        q.D = (_Float16 *)a->D;
        q.Z = (_Float16 *)a->Z;
        q.ldr = a->ldr;
        q.ldd = a->ldd;
        q.ldz = a->ldz;
        return hip_status(launch_split_sum<BF, LE_LINEAR>(act, q, s));
    }
    p.bias = (const _Float16 *)a->bias;
    p.R = (const _Float16 *)a->residual;
    p.D = (_Float16 *)a->D;
    p.Z = (_Float16 *)a->Z;
    p.ldr = a->ldr;
    p.ldd = a->ldd;
    p.ldz = a->ldz;
    p.vec = dma_rows(a->D, a->ldd, a->N) && (!a->Z || dma_rows(a->Z, a->ldz, a->N)) &&
            (!a->residual || dma_rows(a->residual, a->ldr, a->N));
    if (pl.pl.tile == kLinBig)
        return hip_status(BF ? lin_launch_fwd_big_bf16(act, p, groups, s) : lin_launch_fwd_big_f16(act, p, groups, s));
    return hip_status(BF ? lin_launch_fwd_bf16(act, pl.pl.tile, p, groups, s)
                         : lin_launch_fwd_f16(act, pl.pl.tile, p, groups, s));
}

// ---- linear, backward -----------------------------------------------------------
struct LinearGradPlan {
    bool direct = false;  // dD itself is dZ
    int64_t N8 = 0;
    int strips = 0, rows_per_strip = 0;
    StagePlan2 st;  // X, W
    GradPlan grad;
    int64_t off_dz = 0, off_bias = 0, off_part = 0, bytes = 0;
};

int check_linear_grad(const ge_linear_backward_args *a)
{
    if (!a) return GEMM_EPI_ERR_NULL_INPUT;
    GE_CHECK(check_dims(a->M, a->N, a->K));
    if (a->N > GE_MAX_COLS) return GEMM_EPI_ERR_SHAPE;
    // (with no rows dX is empty: an allocator gives it no address)
    if (a->M > 0 && !a->dX && !a->dW && !a->dbias) return GEMM_EPI_ERR_NULL_OUTPUT;
    if (a->act < GE_ACT_IDENTITY || a->act > GE_ACT_SILU) return GEMM_EPI_ERR_KIND;
    GE_CHECK(check_dtype(a->dtype));
    if (a->M > 0) {
        GE_CHECK(check_matrix(a->dD, a->lddd, a->N, 2, GEMM_EPI_ERR_NULL_INPUT));
        if (a->act != GE_ACT_IDENTITY) GE_CHECK(check_matrix(a->Z, a->ldz, a->N, 2, GEMM_EPI_ERR_NULL_INPUT));
        if (a->dW) GE_CHECK(check_matrix(a->X, a->ldx, a->K, 2, GEMM_EPI_ERR_NULL_INPUT));
        if (a->dX) GE_CHECK(check_matrix(a->W, a->ldw, a->K, 2, GEMM_EPI_ERR_NULL_INPUT));
    }
    if (a->dX) GE_CHECK(check_matrix(a->dX, a->lddx, a->K, 2, GEMM_EPI_ERR_NULL_OUTPUT));
    if (a->dW) GE_CHECK(check_matrix(a->dW, a->lddw, a->K, 2, GEMM_EPI_ERR_NULL_OUTPUT));
    if (a->dbias && !aligned(a->dbias, 4)) return GEMM_EPI_ERR_ALIGN;
    return GEMM_EPI_OK;
}

int plan_linear_grad(const ge_linear_backward_args *a, LinearGradPlan &pl)
{
    GE_CHECK(check_linear_grad(a));
    if (a->M == 0) return GEMM_EPI_OK;
    pl.N8 = round_up(a->N, 8);
    Layout lay;
    pl.direct = a->act == GE_ACT_IDENTITY && dma_rows(a->dD, a->lddd, a->N);
    if (!pl.direct) pl.off_dz = lay.take(a->M * pl.N8 * 2);
    // strips of rows: about 2048 blocks of 256 columns, at least 32 rows each (a
    // thread's four loads in flight), 16 (two rows a thread, one after the other)
    // where 32 leave most compute units fewer than three blocks: 1001 x 1003 of K = 1000, gelu, fp16, 24.0 us the call
    // with 32 and 22.0 with 16, 200 x 4099 x 1023 35.3 and 29.5, 1500 x 3000 x
    // 1000 47.6 and 45.9; but 2000 x 3001 x 2001 (756 blocks) 76.4 and 77.8, and
    // 8 rows are no faster than 16 anywhere.  One strip, whose sums are dbias
    // itself, up to 128 rows.
    const int64_t cols = ceil_div(a->N, 256), least = cols * ceil_div(a->M, 32) < 5 * kCUs / 2 ? 16 : 32;
    pl.rows_per_strip = (int)round_up(std::max(least, ceil_div(a->M, std::max<int64_t>(1, 2048 / cols))), 8);
    if (a->M <= 128) pl.rows_per_strip = 128;
    pl.strips = (int)ceil_div(a->M, pl.rows_per_strip);
    if (a->dbias && pl.strips > 1) pl.off_bias = lay.take((int64_t)pl.strips * a->N * 4);
    // an unwanted product's operand is not staged (the other operand stands in)
    const void *x = a->dW ? a->X : a->W, *w = a->dX ? a->W : a->X;
    const int64_t ldx = a->dW ? a->ldx : a->ldw, ldw = a->dX ? a->ldw : a->ldx;
    if (a->dX || a->dW) {
        pl.st = plan_staging2(x, ldx, a->dW ? a->M : 0, w, ldw, a->dX ? a->N : 0, a->K, lay);
        pl.st.on[0] &= a->dW != nullptr;
        pl.st.on[1] &= a->dX != nullptr;
    }
    if (a->dX || a->dW) {
        pl.grad = plan_grad(a->M, a->N, a->K, a->dX, a->dW);
        if (!pl.grad.fits) return GEMM_EPI_ERR_SHAPE;
        pl.off_part = lay.take(pl.grad.part_bytes);
    }
    pl.bytes = lay.bytes;
    return GEMM_EPI_OK;
}

template <bool BF>
hipError_t launch_dz(int act, const DzParams &q, dim3 g, hipStream_t s)
{
    switch (act) {
    case ACT_RELU: return launch(dz_kernel<BF, ACT_RELU>, g, dim3(256), s, q);
    case ACT_GELU: return launch(dz_kernel<BF, ACT_GELU>, g, dim3(256), s, q);
    case ACT_SILU: return launch(dz_kernel<BF, ACT_SILU>, g, dim3(256), s, q);
    default: return launch(dz_kernel<BF, ACT_IDENTITY>, g, dim3(256), s, q);
    }
}

template <bool BF>
int run_linear_grad(const ge_linear_backward_args *a, const LinearGradPlan &pl)
{
    hipStream_t s = (hipStream_t)a->stream;
    char *ws = (char *)a->workspace;
    if (a->M == 0) {
        if (a->dW) GE_TRY(run_zero(a->dW, a->lddw * 2, a->N, a->K * 2, s));
        if (a->dbias) GE_TRY(run_zero(a->dbias, a->N * 4, 1, a->N * 4, s));
        return GEMM_EPI_OK;
    }
    Operand16 dz = {(const _Float16 *)a->dD, a->lddd};
    Operand16 x = {(const _Float16 *)a->X, a->ldx}, w = {(const _Float16 *)a->W, a->ldw};
    const StageSet stage = stage_set(pl.st, ws, a->K, x, a->M, w, a->N);
    if (pl.direct && !a->dbias) {
        GE_TRY(run_staging(stage, s));
    } else {
        DzParams q = {};
        q.dD = (const _Float16 *)a->dD;
        q.Z = (const _Float16 *)a->Z;
        q.ldd = a->lddd;
        q.ldz = a->ldz;
        q.ldo = pl.N8;
        q.out = pl.direct ? nullptr : (_Float16 *)(ws + pl.off_dz);
        q.partial = pl.strips == 1 ? a->dbias : a->dbias ? (float *)(ws + pl.off_bias) : nullptr;
        q.M = (int)a->M;
        q.N = (int)a->N;
        q.N8 = (int)pl.N8;
        q.rows_per_strip = pl.rows_per_strip;
        q.cols_blocks = (int)ceil_div(a->N, 256);
        q.dz_blocks = q.cols_blocks * pl.strips;
        q.pad = stage.q;
        q.pads = stage.n;
        GE_TRY(launch_dz<BF>((int)a->act, q, dim3((unsigned)q.dz_blocks + (stage.n ? stage.blocks : 0u)), s));
        if (!pl.direct) dz = {q.out, pl.N8};
        if (a->dbias && pl.strips > 1) {
            ColSumParams c = {};
            c.partial[0] = q.partial;
            c.out[0] = a->dbias;
            c.parts[0] = pl.strips;
            c.ld = c.cols = (int)a->N;
            GE_TRY(launch(colsum_kernel, dim3((unsigned)ceil_div(a->N, 64)), dim3(1024), s, c));
        }
    }
    GradProduct dx, dw;
    if (a->dX) {
        LinParams p = {};
        p.A = dz.p;
        p.lda = dz.ld;
        p.B = w.p;
        p.ldb = w.ld;
        p.n_read = (int)round_up(a->K, 8);
        p.k_rows = (int)a->N;
        dx = grad_product(p, pl.grad.dx, a->M, a->K, pl.N8, a->dX, a->lddx, nullptr, false, false, nullptr,
                          (float *)(ws + pl.off_part));
    }
    if (a->dW) {
        LinParams p = {};
        p.A = dz.p;
        p.lda = dz.ld;
        p.m_read = (int)pl.N8;
        p.B = x.p;
        p.ldb = x.ld;
        p.n_read = (int)round_up(a->K, 8);
        p.k_rows = (int)a->M;
        dw = grad_product(p, pl.grad.dw, a->N, a->K, a->M, a->dW, a->lddw, nullptr, false, false, nullptr,
                          (float *)(ws + pl.off_part + pl.grad.off_dw));
    }
    return hip_status(run_grad<BF>(pl.grad, a->dX ? &dx : nullptr, a->dW ? &dw : nullptr, s));
}

// ---- cross entropy ---------------------------------------------------------------
constexpr unsigned kSquareTiles = 1u << kLinBig | 1u << kLinSmall;

struct XentPlan {
    bool skinny = false;
    StagePlan2 st;
    ProductPlan pl;
    int nparts = 0;
    int64_t off_max = 0, off_sum = 0, off_tlogit = 0, bytes = 0;
};

int check_xent(const ge_linear_xent_args *a)
{
    if (!a) return GEMM_EPI_ERR_NULL_INPUT;
    GE_CHECK(check_dims(a->T, a->V, a->K));
    if (!a->W || (a->T > 0 && (!a->X || !a->target))) return GEMM_EPI_ERR_NULL_INPUT;
    if (a->T > 0 && (!a->loss || !a->lse)) return GEMM_EPI_ERR_NULL_OUTPUT;
    GE_CHECK(check_dtype(a->dtype));
    GE_CHECK(check_matrix(a->W, a->ldw, a->K, 2, GEMM_EPI_ERR_NULL_INPUT));
    if (a->X) GE_CHECK(check_matrix(a->X, a->ldx, a->K, 2, GEMM_EPI_ERR_NULL_INPUT));
    if (!aligned(a->target, 8) || !aligned(a->loss, 4) || !aligned(a->lse, 4)) return GEMM_EPI_ERR_ALIGN;
    return GEMM_EPI_OK;
}

int plan_xent(const ge_linear_xent_args *a, XentPlan &pl)
{
    GE_CHECK(check_xent(a));
    if (a->T == 0) return GEMM_EPI_OK;
    Layout lay;
    pl.skinny = a->T <= kSkinnyRows;
    if (pl.skinny) {
        pl.nparts = a->T <= dot_rows(a->dtype == GEMM_EPI_BF16) ? row_dot_groups(a->V) : (int)ceil_div(a->V, skinny_cols(a->V));
    } else {
        pl.st = plan_staging2(a->X, a->ldx, a->T, a->W, a->ldw, a->V, a->K, lay);
        pl.pl = plan_product(a->T, a->V, a->K, kSquareTiles, 0);
        if (!product_fits(pl.pl)) return GEMM_EPI_ERR_SHAPE;
        pl.nparts = pl.pl.tiles_n;
    }
    pl.off_max = lay.take(a->T * pl.nparts * 4);
    pl.off_sum = lay.take(a->T * pl.nparts * 4);
    pl.off_tlogit = lay.take(a->T * 4);
    pl.bytes = lay.bytes;
    return GEMM_EPI_OK;
}

template <bool BF>
int run_xent(const ge_linear_xent_args *a, const XentPlan &pl)
{
    hipStream_t s = (hipStream_t)a->stream;
    char *ws = (char *)a->workspace;
    float *pmax = (float *)(ws + pl.off_max), *psum = (float *)(ws + pl.off_sum),
          *tlogit = (float *)(ws + pl.off_tlogit);
    if (pl.skinny) {
        SkinnyParams q = {};
        q.X = (const _Float16 *)a->X;
        q.W = (const _Float16 *)a->W;
        q.ldx = a->ldx;
        q.ldw = a->ldw;
        q.M = (int)a->T;
        q.N = (int)a->V;
        q.K = (int)a->K;
        q.target = a->target;
        q.part_max = pmax;
        q.part_sum = psum;
        q.tlogit = tlogit;
        q.nparts = pl.nparts;
        GE_TRY((launch_few_rows<BF, true, ACT_IDENTITY>(q, s)));
    } else {
        Operand16 x = {(const _Float16 *)a->X, a->ldx}, w = {(const _Float16 *)a->W, a->ldw};
        GE_TRY(run_staging(stage_set(pl.st, ws, a->K, x, a->T, w, a->V), s));
        LinParams p = {};
        set_product(p, pl.pl, a->T, a->V, round_up(a->K, 8));
        p.A = x.p;
        p.lda = x.ld;
        p.B = w.p;
        p.ldb = w.ld;
        p.target = a->target;
        p.part_max = pmax;
        p.part_sum = psum;
        p.nparts = pl.nparts;
        p.tlogit = tlogit;
        GE_TRY(BF ? lin_launch_xent_bf16(LE_XFWD, pl.pl.tile, p, p.num_tiles, s)
                  : lin_launch_xent_f16(LE_XFWD, pl.pl.tile, p, p.num_tiles, s));
    }
    return hip_status(launch(xent_loss_kernel, row_grid(a->T), dim3(pl.nparts > 128 ? 256 : 64), s, a->T,
                             (const float *)pmax, (const float *)psum, pl.nparts, (const float *)tlogit, a->target,
                             a->V, a->ignore_index, a->loss, a->lse));
}

// The vocabulary goes in pieces of `piece` columns: P of one piece is written
// by one product and read by two.  A piece as large as 128 MiB of P (half the
// last-level cache) keeps those reads off HBM; more pieces cost a round trip of
// dX's fp32 accumulator each, T K 8 bytes against 2 T K piece operations, so a
// piece is not made shorter than 8192 columns (P then takes 16 KiB a row of X
// past 8192 rows, whatever the vocabulary).  Within that it is a length that
// fills whole rounds of tiles, with the rest in a shorter last piece: 4096 x
// 100003 in 6 pieces of 16384 and one of 1699 takes 25 rounds for each of its
// products, in 7 even ones (3.5 rounds each) 28.
constexpr int64_t kPieceBytes = 128 << 20, kPieceMin = 8192;

struct XentGradPlan {
    StagePlan2 st;
    int64_t piece = 0, pld = 0;
    int pieces = 0;
    ProductPlan p, p_last;  // of a full piece, of the last one
    GradPlan grad, grad_last;
    int64_t off_rows = 0, off_alpha = 0, off_p = 0, off_acc = 0, off_part = 0, bytes = 0;
};

int check_xent_grad(const ge_linear_xent_backward_args *a)
{
    if (!a) return GEMM_EPI_ERR_NULL_INPUT;
    GE_CHECK(check_dims(a->T, a->V, a->K));
    if (a->T > 0 && !a->dX && !a->dW) return GEMM_EPI_ERR_NULL_OUTPUT;
    if (!a->W || (a->T > 0 && (!a->X || !a->target || !a->lse || !a->dloss))) return GEMM_EPI_ERR_NULL_INPUT;
    GE_CHECK(check_dtype(a->dtype));
    GE_CHECK(check_matrix(a->W, a->ldw, a->K, 2, GEMM_EPI_ERR_NULL_INPUT));
    if (a->X) GE_CHECK(check_matrix(a->X, a->ldx, a->K, 2, GEMM_EPI_ERR_NULL_INPUT));
    if (a->dX) GE_CHECK(check_matrix(a->dX, a->lddx, a->K, 2, GEMM_EPI_ERR_NULL_OUTPUT));
    if (a->dW) GE_CHECK(check_matrix(a->dW, a->lddw, a->K, 2, GEMM_EPI_ERR_NULL_OUTPUT));
    if (!aligned(a->target, 8) || !aligned(a->dloss, 4) || !aligned(a->lse, 4)) return GEMM_EPI_ERR_ALIGN;
    return GEMM_EPI_OK;
}

int plan_xent_grad(const ge_linear_xent_backward_args *a, XentGradPlan &pl)
{
    GE_CHECK(check_xent_grad(a));
    if (a->T == 0) return GEMM_EPI_OK;
    Layout lay;
    pl.st = plan_staging2(a->X, a->ldx, a->T, a->W, a->ldw, a->V, a->K, lay);
    // a piece is a row of P, at most GE_MAX_COLS long (few rows of X would take longer ones)
    const int64_t limit =
        std::min<int64_t>(std::max(kPieceMin, kPieceBytes / (a->T * 2) / 256 * 256), GE_MAX_COLS);
    pl.pieces = (int)ceil_div(a->V, limit);
    pl.piece = a->V;
    if (pl.pieces > 1) {
        pl.piece = std::min<int64_t>(round_up(ceil_div(a->V, pl.pieces), 256), limit / 256 * 256);  // even pieces
        // columns that make whole rounds of 256 x 256 tiles over the chip
        int64_t tiles_m = ceil_div(a->T, 256), step = 256 * kCUs;
        for (; tiles_m % 2 == 0 && step > 256; tiles_m /= 2) step /= 2;
        if (step <= limit) pl.piece = limit / step * step;
        pl.pieces = (int)ceil_div(a->V, pl.piece);
    }
    pl.pld = round_up(pl.piece, 8);
    const int64_t last = a->V - (pl.pieces - 1) * pl.piece;
    pl.p = plan_product(a->T, pl.piece, a->K, kSquareTiles, 0);
    pl.grad = plan_grad(a->T, pl.piece, a->K, a->dX, a->dW);
    pl.p_last = last == pl.piece ? pl.p : plan_product(a->T, last, a->K, kSquareTiles, 0);
    pl.grad_last = last == pl.piece ? pl.grad : plan_grad(a->T, last, a->K, a->dX, a->dW);
    if (!product_fits(pl.p) || !product_fits(pl.p_last) || !pl.grad.fits || !pl.grad_last.fits)
        return GEMM_EPI_ERR_SHAPE;
    const int64_t part = std::max(pl.grad.part_bytes, pl.grad_last.part_bytes);
    pl.off_rows = lay.take(a->T * (int64_t)sizeof(XentRow));
    pl.off_alpha = lay.take(4);
    pl.off_p = lay.take(a->T * pl.pld * 2);
    if (a->dX && pl.pieces > 1) pl.off_acc = lay.take(a->T * round_up(a->K, 8) * 4);
    pl.off_part = lay.take(part);
    pl.bytes = lay.bytes;
    return GEMM_EPI_OK;
}

template <bool BF>
int run_xent_grad(const ge_linear_xent_backward_args *a, const XentGradPlan &pl)
{
    hipStream_t s = (hipStream_t)a->stream;
    char *ws = (char *)a->workspace;
    if (a->T == 0) return a->dW ? hip_status(run_zero(a->dW, a->lddw * 2, a->V, a->K * 2, s)) : GEMM_EPI_OK;
    XentRow *rows = (XentRow *)(ws + pl.off_rows);
    float *alpha = (float *)(ws + pl.off_alpha);
    GE_TRY(launch(xent_rows_kernel, dim3(1), dim3(1024), s, (int)a->T, a->V, a->ignore_index, a->dloss, a->lse,
                  a->target, rows, alpha));
    Operand16 x = {(const _Float16 *)a->X, a->ldx}, w = {(const _Float16 *)a->W, a->ldw};
    GE_TRY(run_staging(stage_set(pl.st, ws, a->K, x, a->T, w, a->V), s));
    _Float16 *P = (_Float16 *)(ws + pl.off_p);
    float *acc = pl.pieces > 1 ? (float *)(ws + pl.off_acc) : nullptr;
    float *part = (float *)(ws + pl.off_part);
    for (int c = 0; c < pl.pieces; c++) {
        const bool last = c == pl.pieces - 1;
        const int64_t v0 = c * pl.piece, n = last ? a->V - v0 : pl.piece;
        LinParams p = {};
        set_product(p, last ? pl.p_last : pl.p, a->T, n, round_up(a->K, 8));
        p.A = x.p;
        p.lda = x.ld;
        p.B = w.p + v0 * w.ld;
        p.ldb = w.ld;
        p.rows = rows;
        p.v0 = (int)v0;
        p.D = P;
        p.ldd = pl.pld;
        p.n_store = (int)round_up(n, 8);
        const int tile = last ? pl.p_last.tile : pl.p.tile;
        if (a->T <= kSkinnyRows) {
            SkinnyParams q = {};
            q.X = x.p;
            q.W = p.B;
            q.ldx = x.ld;
            q.ldw = w.ld;
            q.M = (int)a->T;
            q.N = (int)n;
            q.K = (int)a->K;
            q.D = P;
            q.ldd = pl.pld;
            q.rows = rows;
            q.v0 = (int)v0;
            GE_TRY((launch_skinny<BF, SK_P, ACT_IDENTITY>(q, s)));
        } else {
            GE_TRY(BF ? lin_launch_xent_bf16(LE_XP, tile, p, p.num_tiles, s)
                      : lin_launch_xent_f16(LE_XP, tile, p, p.num_tiles, s));
        }
        const GradPlan &g = last ? pl.grad_last : pl.grad;
        GradProduct dx, dw;
        if (a->dX) {
            LinParams q = {};
            q.A = P;
            q.lda = pl.pld;
            q.B = p.B;
            q.ldb = w.ld;
            q.n_read = (int)round_up(a->K, 8);
            q.k_rows = (int)n;
            dx = grad_product(q, g.dx, a->T, a->K, round_up(n, 8), a->dX, a->lddx, acc, c > 0, !last, alpha, part);
        }
        if (a->dW) {
            LinParams q = {};
            q.A = P;
            q.lda = pl.pld;
            q.m_read = (int)round_up(n, 8);
            q.B = x.p;
            q.ldb = x.ld;
            q.n_read = (int)round_up(a->K, 8);
            q.k_rows = (int)a->T;
            dw = grad_product(q, g.dw, n, a->K, a->T, (char *)a->dW + v0 * a->lddw * 2, a->lddw, nullptr, false, false,
                              alpha, (float *)((char *)part + g.off_dw));
        }
        GE_TRY(run_grad<BF>(g, a->dX ? &dx : nullptr, a->dW ? &dw : nullptr, s));
    }
    return GEMM_EPI_OK;
}

// ---- norms and the residual step ----------------------------------------------
int check_norm(int64_t T, int64_t H, int64_t G, int64_t post, int64_t pre, const void *gate, double scale, double eps,
               int64_t dtype, int64_t sdtype)
{
    if (T < 0 || T > INT32_MAX || H < 1 || H > GE_MAX_HIDDEN || G < 1 || T % G != 0) return GEMM_EPI_ERR_SHAPE;
    if (!gate && G != 1) return GEMM_EPI_ERR_SHAPE;
    if (post < GE_NORM_NONE || post > GE_NORM_LAYER || (pre != GE_NORM_RMS && pre != GE_NORM_LAYER))
        return GEMM_EPI_ERR_KIND;
    GE_CHECK(check_dtype(dtype));
    if (sdtype != dtype && sdtype != GEMM_EPI_F32) return GEMM_EPI_ERR_DTYPE;
    if (!(eps >= 0.0) || scale != scale) return GEMM_EPI_ERR_SHAPE;
    return GEMM_EPI_OK;
}

int check_norm_args(const ge_norm_residual_args *a)
{
    if (!a) return GEMM_EPI_ERR_NULL_INPUT;
    GE_CHECK(check_norm(a->T, a->hidden, a->G, a->post, a->pre, a->gate, a->scale, a->eps, a->dtype, a->stream_dtype));
    const uintptr_t es = a->stream_dtype == GEMM_EPI_F32 ? 4 : 2;
    for (const void *v : {a->w_post, a->w_pre, a->gate})
        if (!aligned(v, 2)) return GEMM_EPI_ERR_ALIGN;
    if (a->T == 0) return GEMM_EPI_OK;
    GE_CHECK(check_matrix(a->H, a->ldh, a->hidden, es, GEMM_EPI_ERR_NULL_INPUT));
    GE_CHECK(check_matrix(a->Y, a->ldy, a->hidden, 2, GEMM_EPI_ERR_NULL_INPUT));
    GE_CHECK(check_matrix(a->H_out, a->ldho, a->hidden, es, GEMM_EPI_ERR_NULL_OUTPUT));
    return check_matrix(a->X, a->ldx, a->hidden, 2, GEMM_EPI_ERR_NULL_OUTPUT);
}

// Calls f(threads per row, vectors per thread) for a row length.
template <typename F>
hipError_t dispatch_row(int64_t H, F &&f)
{
    if (H <= 512) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
    if (H <= 1024) return f(std::integral_constant<int, 128>{}, std::integral_constant<int, 1>{});
    if (H <= 2048) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 1>{});
    if (H <= 4096) return f(std::integral_constant<int, 512>{}, std::integral_constant<int, 1>{});
    if (H <= 8192) return f(std::integral_constant<int, 512>{}, std::integral_constant<int, 2>{});
    return f(std::integral_constant<int, 1024>{}, std::integral_constant<int, 2>{});
}

template <bool BF, bool S32>
hipError_t run_norm(const ge_norm_residual_args *a)
{
    NormParams p = {};
    p.H = a->H;
    p.Y = (const _Float16 *)a->Y;
    p.w_post = (const _Float16 *)a->w_post;
    p.w_pre = (const _Float16 *)a->w_pre;
    p.gate = (const _Float16 *)a->gate;
    p.H_out = a->H_out;
    p.X = (_Float16 *)a->X;
    p.ldh = a->ldh;
    p.ldy = a->ldy;
    p.ldho = a->ldho;
    p.ldx = a->ldx;
    p.rows = (int)a->T;
    p.hidden = (int)a->hidden;
    p.rows_per_gate = (int)(a->T / a->G);
    p.post = (int)a->post;
    p.pre = (int)a->pre;
    p.scale = (float)a->scale;
    p.eps = (float)a->eps;
    return dispatch_row(a->hidden, [&](auto tpr, auto nv) {
        constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
        return launch(norm_residual_kernel<BF, S32, TPR, NV>, row_grid(a->T), dim3(TPR),
                      (hipStream_t)a->stream, p);
    });
}

// Elements a thread of the gradient holds.  A row of 8 a thread past 4096
// columns is a workgroup that has its compute unit alone; with 12 a thread two
// workgroups of up to 512 threads share it up to 6144 columns, one's reductions
// beside the other's loads.  8190 rows, us with 8 and with 12, 16-bit stream:
// 4100 columns 152 and 115, 5120 157 and 123, 6144 168 and 143; rows of an odd
// length (no loads in flight behind the reductions with 8): 4101 215 and 153.
// An fp32 stream of whole units stays with 8, whose next row's loads are in
// flight: 4100 columns 133 and 142, 6144 196 and 202; odd 4101: 225 and 163.
int norm_grad_elements(int64_t H, bool s32)
{
    return H > 4096 && H <= 6144 && !(s32 && H % 4 == 0) ? 12 : 8;
}
// its threads, in whole waves
int64_t norm_grad_threads(int64_t H, bool s32) { return round_up(ceil_div(H, norm_grad_elements(H, s32)), 64); }

// Runs of rows that share a gate row, and workgroups: as many as the compute
// units hold at once (one of more than 512 threads, two of 512, more of the
// small ones), so that the partial column sums, a row per workgroup, stay small
// beside the rows themselves.  8192 rows: 4100 columns at 8 a thread 149 us
// with 256, 167 with 1024; 4096 columns 127 with 256, 102 with 512; 1024
// columns 40 with 512, 36 with 1024.  At least 2 rows each, from 256 rows on.
struct NormGradPlan {
    int64_t rows_per_gate = 0, rows_per_run = 0, runs = 0, runs_per_block = 1, blocks = 0;
    int runs_per_gate = 1;
    int64_t off_post = 0, off_pre = 0, off_gate = 0, bytes = 0;
};
int plan_norm_grad(const ge_norm_residual_backward_args *a, NormGradPlan &pl)
{
    if (!a) return GEMM_EPI_ERR_NULL_INPUT;
    GE_CHECK(check_norm(a->T, a->hidden, a->G, a->post, a->pre, a->gate, a->scale, a->eps, a->dtype, a->stream_dtype));
    if (a->hidden > GE_MAX_HIDDEN_GRAD) return GEMM_EPI_ERR_SHAPE;
    const uintptr_t es = a->stream_dtype == GEMM_EPI_F32 ? 4 : 2;
    for (const void *v : {a->w_post, a->w_pre, a->gate})
        if (!aligned(v, 2)) return GEMM_EPI_ERR_ALIGN;
    for (const void *v : {a->dw_post, a->dw_pre, a->dgate})
        if (!aligned(v, 4)) return GEMM_EPI_ERR_ALIGN;
    if (a->T == 0) return GEMM_EPI_OK;
    GE_CHECK(check_matrix(a->dX, a->lddx, a->hidden, 2, GEMM_EPI_ERR_NULL_INPUT));
    GE_CHECK(check_matrix(a->dH_out, a->lddho, a->hidden, es, GEMM_EPI_ERR_NULL_INPUT));
    GE_CHECK(check_matrix(a->H_out, a->ldho, a->hidden, es, GEMM_EPI_ERR_NULL_INPUT));
    GE_CHECK(check_matrix(a->Y, a->ldy, a->hidden, 2, GEMM_EPI_ERR_NULL_INPUT));
    GE_CHECK(check_matrix(a->dH, a->lddh, a->hidden, es, GEMM_EPI_ERR_NULL_OUTPUT));
    GE_CHECK(check_matrix(a->dY, a->lddy, a->hidden, 2, GEMM_EPI_ERR_NULL_OUTPUT));
    pl.rows_per_gate = a->T / a->G;
    const int64_t threads = norm_grad_threads(a->hidden, a->stream_dtype == GEMM_EPI_F32);
    const int64_t most = kCUs * (threads > 512 ? 1 : threads > 256 ? 2 : 4);
    const int64_t blocks = a->T <= kCUs ? a->T : std::min(most, ceil_div(a->T, 2));
    pl.rows_per_run = std::min(pl.rows_per_gate, ceil_div(a->T, blocks));
    pl.runs_per_gate = (int)ceil_div(pl.rows_per_gate, pl.rows_per_run);
    pl.runs = a->G * pl.runs_per_gate;
    pl.runs_per_block = pl.runs_per_gate > 1 ? 1 : ceil_div(pl.runs, blocks);
    pl.blocks = ceil_div(pl.runs, pl.runs_per_block);
    Layout lay;
    if (a->dw_post && a->post != GE_NORM_NONE) pl.off_post = lay.take(pl.blocks * a->hidden * 4);
    if (a->dw_pre) pl.off_pre = lay.take(pl.blocks * a->hidden * 4);
    if (a->dgate && pl.runs_per_gate > 1) pl.off_gate = lay.take(pl.runs * a->hidden * 4);
    pl.bytes = lay.bytes;
    return GEMM_EPI_OK;
}

template <bool BF, bool S32>
int run_norm_grad(const ge_norm_residual_backward_args *a, const NormGradPlan &pl)
{
    hipStream_t s = (hipStream_t)a->stream;
    char *ws = (char *)a->workspace;
    const int64_t H = a->hidden;
    const bool post = a->dw_post && a->post != GE_NORM_NONE;
    if (a->dw_post && !post) GE_TRY(run_zero(a->dw_post, H * 4, 1, H * 4, s));
    if (a->T == 0) {
        if (post) GE_TRY(run_zero(a->dw_post, H * 4, 1, H * 4, s));
        if (a->dw_pre) GE_TRY(run_zero(a->dw_pre, H * 4, 1, H * 4, s));
        if (a->dgate) GE_TRY(run_zero(a->dgate, H * 4, a->G, H * 4, s));
        return GEMM_EPI_OK;
    }
    NormGradParams p = {};
    p.dX = (const _Float16 *)a->dX;
    p.Y = (const _Float16 *)a->Y;
    p.w_post = a->post != GE_NORM_NONE ? (const _Float16 *)a->w_post : nullptr;
    p.w_pre = (const _Float16 *)a->w_pre;
    p.gate = (const _Float16 *)a->gate;
    p.dH_out = a->dH_out;
    p.H_out = a->H_out;
    p.dH = a->dH;
    p.dY = (_Float16 *)a->dY;
    p.lddx = (int)a->lddx;
    p.lddho = (int)a->lddho;
    p.ldho = (int)a->ldho;
    p.ldy = (int)a->ldy;
    p.lddh = (int)a->lddh;
    p.lddy = (int)a->lddy;
    p.hidden = (int)H;
    p.post = (int)a->post;
    p.pre = (int)a->pre;
    p.scale = (float)a->scale;
    p.eps = (float)a->eps;
    p.rows_per_gate = (int)pl.rows_per_gate;
    p.rows_per_run = (int)pl.rows_per_run;
    p.runs_per_gate = pl.runs_per_gate;
    p.runs = (int)pl.runs;
    p.runs_per_block = (int)pl.runs_per_block;
    p.gate_direct = pl.runs_per_gate == 1;
    p.p_post = post ? (float *)(ws + pl.off_post) : nullptr;
    p.p_pre = a->dw_pre ? (float *)(ws + pl.off_pre) : nullptr;
    p.dgate = !a->dgate || p.gate_direct ? a->dgate : (float *)(ws + pl.off_gate);
    const dim3 g((unsigned)pl.blocks), b((unsigned)norm_grad_threads(H, S32));
    auto run = [&](auto most, auto units) {
        constexpr int MAXT = decltype(most)::value, NU = decltype(units)::value;
        if (H % 4 != 0) return launch(norm_residual_grad_kernel<BF, S32, MAXT, NU, true>, g, b, s, p);
        if constexpr (!(S32 && NU == 3))
            return launch(norm_residual_grad_kernel<BF, S32, MAXT, NU, false>, g, b, s, p);
        return hipErrorInvalidValue;  // norm_grad_elements
    };
    using std::integral_constant;
    if (norm_grad_elements(H, S32) == 12)
        GE_TRY(run(integral_constant<int, 512>{}, integral_constant<int, 3>{}));
    else if (H <= 4096)
        GE_TRY(run(integral_constant<int, 512>{}, integral_constant<int, 2>{}));
    else
        GE_TRY(run(integral_constant<int, 1024>{}, integral_constant<int, 2>{}));
    ColSumParams c = {};
    c.partial[0] = p.p_post;
    c.out[0] = post ? a->dw_post : nullptr;
    c.partial[1] = p.p_pre;
    c.out[1] = a->dw_pre;
    c.parts[0] = c.parts[1] = (int)pl.blocks;
    c.partial[2] = p.dgate;
    const bool gates = a->dgate && !p.gate_direct;
    c.out[2] = gates ? a->dgate : nullptr;
    c.parts[2] = pl.runs_per_gate;
    c.ld = c.cols = (int)H;
    if (!c.out[0] && !c.out[1] && !gates) return GEMM_EPI_OK;
    return hip_status(launch(colsum_kernel, dim3((unsigned)ceil_div(H, 64), 2 + (gates ? (unsigned)a->G : 0u)),
                             dim3(1024), s, c));
}

}  // namespace

extern "C" {

int ge_linear_workspace(const ge_linear_args *a, int64_t *bytes)
{
    LinearPlan pl;
    GE_CHECK(plan_linear(a, pl));
    if (!bytes) return GEMM_EPI_ERR_NULL_OUTPUT;
    *bytes = pl.bytes;
    return GEMM_EPI_OK;
}

int ge_linear(const ge_linear_args *a)
{
    LinearPlan pl;
    GE_CHECK(plan_linear(a, pl));
    GE_CHECK(check_workspace(a->workspace, a->workspace_bytes, pl.bytes));
    if (a->M == 0) return GEMM_EPI_OK;
    return a->dtype == GEMM_EPI_BF16 ? run_linear<true>(a, pl) : run_linear<false>(a, pl);
}

int ge_linear_backward_workspace(const ge_linear_backward_args *a, int64_t *bytes)
{
    LinearGradPlan pl;
    GE_CHECK(plan_linear_grad(a, pl));
    if (!bytes) return GEMM_EPI_ERR_NULL_OUTPUT;
    *bytes = pl.bytes;
    return GEMM_EPI_OK;
}

int ge_linear_backward(const ge_linear_backward_args *a)
{
    LinearGradPlan pl;
    GE_CHECK(plan_linear_grad(a, pl));
    GE_CHECK(check_workspace(a->workspace, a->workspace_bytes, pl.bytes));
    return a->dtype == GEMM_EPI_BF16 ? run_linear_grad<true>(a, pl) : run_linear_grad<false>(a, pl);
}

int ge_linear_xent_workspace(const ge_linear_xent_args *a, int64_t *bytes)
{
    XentPlan pl;
    GE_CHECK(plan_xent(a, pl));
    if (!bytes) return GEMM_EPI_ERR_NULL_OUTPUT;
    *bytes = pl.bytes;
    return GEMM_EPI_OK;
}

int ge_linear_xent(const ge_linear_xent_args *a)
{
    XentPlan pl;
    GE_CHECK(plan_xent(a, pl));
    GE_CHECK(check_workspace(a->workspace, a->workspace_bytes, pl.bytes));
    if (a->T == 0) return GEMM_EPI_OK;
    return a->dtype == GEMM_EPI_BF16 ? run_xent<true>(a, pl) : run_xent<false>(a, pl);
}

int ge_linear_xent_backward_workspace(const ge_linear_xent_backward_args *a, int64_t *bytes)
{
    XentGradPlan pl;
    GE_CHECK(plan_xent_grad(a, pl));
    if (!bytes) return GEMM_EPI_ERR_NULL_OUTPUT;
    *bytes = pl.bytes;
    return GEMM_EPI_OK;
}

int ge_linear_xent_backward(const ge_linear_xent_backward_args *a)
{
    XentGradPlan pl;
    GE_CHECK(plan_xent_grad(a, pl));
    GE_CHECK(check_workspace(a->workspace, a->workspace_bytes, pl.bytes));
    return a->dtype == GEMM_EPI_BF16 ? run_xent_grad<true>(a, pl) : run_xent_grad<false>(a, pl);
}

int ge_norm_residual(const ge_norm_residual_args *a)
{
    GE_CHECK(check_norm_args(a));
    if (a->T == 0) return GEMM_EPI_OK;
    if (a->stream_dtype == GEMM_EPI_F32)
        return hip_status(a->dtype == GEMM_EPI_BF16 ? run_norm<true, true>(a) : run_norm<false, true>(a));
    return hip_status(a->dtype == GEMM_EPI_BF16 ? run_norm<true, false>(a) : run_norm<false, false>(a));
}

int ge_norm_residual_backward_workspace(const ge_norm_residual_backward_args *a, int64_t *bytes)
{
    NormGradPlan pl;
    GE_CHECK(plan_norm_grad(a, pl));
    if (!bytes) return GEMM_EPI_ERR_NULL_OUTPUT;
    *bytes = pl.bytes;
    return GEMM_EPI_OK;
}

int ge_norm_residual_backward(const ge_norm_residual_backward_args *a)
{
    NormGradPlan pl;
    GE_CHECK(plan_norm_grad(a, pl));
    GE_CHECK(check_workspace(a->workspace, a->workspace_bytes, pl.bytes));
    if (a->stream_dtype == GEMM_EPI_F32)
        return a->dtype == GEMM_EPI_BF16 ? run_norm_grad<true, true>(a, pl) : run_norm_grad<false, true>(a, pl);
    return a->dtype == GEMM_EPI_BF16 ? run_norm_grad<true, false>(a, pl) : run_norm_grad<false, false>(a, pl);
}

}  // extern "C"
