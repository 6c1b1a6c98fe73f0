// fp8_ops.hip -- the C ABI of include/fp8_ops.h for the 8-bit products:
// argument checks, plans (tiles, splits, workspace layout) and launches.
#include <hip/hip_runtime.h>
#include <algorithm>
#include <math.h>
#include <stdint.h>

#include "fp8_launch.hpp"
#include "fp8_ops.h"
#include "fp8_quant.hpp"
#include "fp8_rows.hpp"
#include "ops_host.hpp"

using namespace gemm_epi;

namespace {

int64_t blocks_of(int64_t n) { return ceil_div(n, kBlock); }

int check_bytes(const void *p, int64_t ld, int64_t cols, int64_t limit, int null_status)
{
    if (!p) return null_status;
    return ld < cols || ld > limit ? GEMM_EPI_ERR_SHAPE : GEMM_EPI_OK;
}
int check_format(int64_t f) { return f == GE_FP8_E4M3 || f == GE_FP8_E5M2 ? GEMM_EPI_OK : GEMM_EPI_ERR_DTYPE; }

// ---- quantisation ---------------------------------------------------------------
int64_t quant_groups(int64_t R, int64_t C) { return blocks_of(R) * blocks_of(C); }
// 512 threads each, below 2^32 in all, with room for the staging of operands
bool quant_fits(int64_t R, int64_t C) { return quant_groups(R, C) <= (1 << 23) - 16 * kCUs; }
template <int SRC, bool TILE, bool BOTH>
hipError_t launch_quant3(int format, const QuantParams &q, hipStream_t s)
{
    const dim3 g((unsigned)quant_groups(q.R, q.C)), b(512);
    return format == GE_FP8_E4M3 ? launch(quant_kernel<SRC, TILE, BOTH, 0, kNoGrad>, g, b, s, q)
                                 : launch(quant_kernel<SRC, TILE, BOTH, 1, kNoGrad>, g, b, s, q);
}
template <int SRC>
hipError_t launch_quant2(bool tile, int format, const QuantParams &q, hipStream_t s)
{
    if (tile) return q.QT ? launch_quant3<SRC, true, true>(format, q, s) : launch_quant3<SRC, true, false>(format, q, s);
    return q.QT ? launch_quant3<SRC, false, true>(format, q, s) : launch_quant3<SRC, false, false>(format, q, s);
}
hipError_t launch_quant(int64_t dtype, bool tile, int format, const QuantParams &q, hipStream_t s)
{
    switch (dtype) {
    case GEMM_EPI_F32: return launch_quant2<QS_F32>(tile, format, q, s);
    case GEMM_EPI_BF16: return launch_quant2<QS_BF16>(tile, format, q, s);
    default: return launch_quant2<QS_F16>(tile, format, q, s);
    }
}

int check_quantize(const ge_quantize_fp8_args *a)
{
    if (!a) return GEMM_EPI_ERR_NULL_INPUT;
    if (a->R < 0 || a->R > GE_MAX_COLS || a->C < 1 || a->C > GE_MAX_COLS) return GEMM_EPI_ERR_SHAPE;
    if (a->block != GE_BLOCK_ROW && a->block != GE_BLOCK_TILE) return GEMM_EPI_ERR_KIND;
    GE_CHECK(check_format(a->format));
    if (a->dtype < GEMM_EPI_F16 || a->dtype > GEMM_EPI_F32) return GEMM_EPI_ERR_DTYPE;
    if (a->R == 0) return GEMM_EPI_OK;
    if (!quant_fits(a->R, a->C)) return GEMM_EPI_ERR_SHAPE;
    const int64_t rb = blocks_of(a->R), cb = blocks_of(a->C);
    GE_CHECK(check_matrix(a->X, a->ldx, a->C, a->dtype == GEMM_EPI_F32 ? 4 : 2, GEMM_EPI_ERR_NULL_INPUT));
    GE_CHECK(check_bytes(a->Q, a->ldq, a->C, GE_MAX_COLS + 128, GEMM_EPI_ERR_NULL_OUTPUT));
    GE_CHECK(check_bytes(a->S, a->lds, cb, GE_MAX_COLS + 128, GEMM_EPI_ERR_NULL_OUTPUT));
    if (!a->QT != !a->ST) return GEMM_EPI_ERR_NULL_OUTPUT;
    if (a->QT) {
        GE_CHECK(check_bytes(a->QT, a->ldqt, a->R, GE_MAX_COLS + 128, GEMM_EPI_ERR_NULL_OUTPUT));
        GE_CHECK(check_bytes(a->ST, a->ldst, rb, GE_MAX_COLS + 128, GEMM_EPI_ERR_NULL_OUTPUT));
    }
    return GEMM_EPI_OK;
}

// ---- operands -------------------------------------------------------------------
// An 8-bit matrix with its scales as the products read them: in place, or a copy.
struct Operand8 {
    const uint8_t *q, *s;
    int64_t ldq, lds;
};
struct Staging {
    PadBytes p = {};
    int64_t pieces = 0;
    void add(const uint8_t *&src, int64_t &ld, int64_t rows, int64_t cols, uint8_t *dst)
    {
        const int n = p.n++;
        p.src[n] = src;
        p.lds[n] = ld;
        p.rows[n] = (int)rows;
        p.cols[n] = (int)cols;
        p.ldo[n] = round_up(cols, 16);
        p.dst[n] = dst;
        pieces += rows * p.ldo[n] / 16;
        src = dst;
        ld = p.ldo[n];
    }
    int64_t groups(int threads) const { return std::min<int64_t>(ceil_div(pieces, threads), 8 * kCUs); }
    hipError_t run(hipStream_t s) const
    {
        return p.n ? launch(pad_bytes_kernel, dim3((unsigned)groups(256)), dim3(256), s, p) : hipSuccess;
    }
};
// rows that all begin at multiples of `unit` bytes (a single one has no pitch)
bool rows_at(int64_t unit, const void *p, int64_t ld, int64_t rows) { return aligned(p, unit) && (rows == 1 || ld % unit == 0); }

// Where an operand's copies lie; negative: read in place.
struct StageAt {
    int64_t q = -1, s = -1;
};
StageAt plan_operand(const void *q, int64_t ldq, const void *s, int64_t lds, int64_t rows, int64_t srows, int64_t cols,
                     Layout &lay)
{
    StageAt at;
    if (!rows_at(16, q, ldq, rows)) at.q = lay.take(rows * round_up(cols, 16));
    if (!rows_at(4, s, lds, srows)) at.s = lay.take(srows * round_up(blocks_of(cols), 16));
    return at;
}
void stage_operand(const StageAt &at, Operand8 &o, int64_t rows, int64_t srows, int64_t cols, char *ws, Staging &st)
{
    if (at.q >= 0) st.add(o.q, o.ldq, rows, cols, (uint8_t *)ws + at.q);
    if (at.s >= 0) st.add(o.s, o.lds, srows, blocks_of(cols), (uint8_t *)ws + at.s);
    // (a single row's pitch is raised to the rule: rows that do not exist then lie behind the descriptors' ends)
    o.ldq = round_up(o.ldq, 16);
    o.lds = round_up(o.lds, 4);
}

// ---- products -------------------------------------------------------------------
struct Plan8 {
    int tile = kFp8Small, splits = 1;
    int64_t tiles_m = 0, tiles_n = 0, k_split = 0, part_bytes = 0;
};
int64_t plan_groups(const Plan8 &p) { return p.tiles_m * p.tiles_n * p.splits; }
bool plan_fits(const Plan8 &p) { return plan_groups(p) <= kMaxGroups; }

// Estimated microseconds of a tile and split, fitted to timings of all of them on
// 34 shapes (128^3 to 8192^3, 32 rows against 4096 x 4096, 300 x 300 x 8192): a
// round of workgroups costs a fixed time and a time per unit of K, which grows
// with the share of the chip at work.  Fixed us, and ns per unit of K from few
// workgroups to a full chip:
//   256 x 256               10.7;  7.7 .. 8.6
//   128 x 256                7.7;  4.0 .. 5.2
//   128 x 128, deep rings    5.5;  2.5 .. 3.1   (4.7; 3.1 .. 5.6 with the others)
//   128 x 128, two on a CU   6.5;  5.9
// Past two rounds the last one costs a third of one.  A split adds a launch and its
// partial sums' round trip.  The pick was within 5% of the fastest on all 34 (for
// instance 2400 x 3232 x 4096: 128 x 256 29.7, 128 x 128 32.5, 256 x 256 43.2;
// 1536 x 1536 x 4096: deep 16.6, 24.1 without; 1024 x 1024 x 8192: 27.3, in
// 4 splits 21.0).
double cost8(int64_t M, int64_t N, int64_t K, int tile, int splits)
{
    const Fp8Tile t = kFp8Tiles[tile];
    const double groups = (double)(ceil_div(M, t.bm) * ceil_div(N, t.bn) * splits);
    const double k = (double)round_up(ceil_div(K, splits), splits > 1 ? 512 : 128) * 1e-3;
    const double share = std::min(1.0, groups / kCUs);
    double slots = kCUs, round;
    switch (tile) {
    case kFp8Big: round = 10.7 + k * (7.7 + 0.9 * share); break;
    case kFp8Wide: round = 7.7 + k * (4.0 + 1.1 * share); break;
    case kFp8Deep: round = 5.5 + k * (2.5 + 0.6 * share); break;
    default:
        if (groups > kCUs) slots = 2 * kCUs;
        round = groups > kCUs ? 6.5 + k * 5.9 : 4.7 + k * (3.1 + 2.5 * share);
    }
    const double rounds = groups / slots;
    double us = round * (rounds <= 2.0 ? ceil(rounds) : rounds + 0.34);
    if (splits > 1) us += 3.5 + 0.04 * splits + (double)splits * M * N * 8 / 8.8e6;
    return us;
}

// The cheapest plan of those whose grid one launch holds.  k_split is a multiple of
// 512: four blocks, a dword of scales.
Plan8 plan_fp8(int64_t M, int64_t N, int64_t K)
{
    Plan8 best;
    double least = 0;
    for (int i = 0; i < (int)(sizeof(kFp8Tiles) / sizeof(kFp8Tiles[0])); i++) {
        const Fp8Tile t = kFp8Tiles[i];
        for (int want = 1; want <= 16; want *= 2) {
            Plan8 p;
            p.tile = i;
            p.tiles_m = ceil_div(M, t.bm);
            p.tiles_n = ceil_div(N, t.bn);
            if (want > 1 && (K < want * 512 || p.tiles_m * p.tiles_n * want > 4 * kCUs)) break;
            p.k_split = round_up(ceil_div(K, want), 512);
            p.splits = (int)ceil_div(K, p.k_split);
            p.part_bytes = p.splits > 1 ? p.splits * M * round_up(N, 8) * 4 : 0;
            const double c = cost8(M, N, K, i, p.splits);
            const bool fits = plan_fits(p), best_fits = best.tiles_m > 0 && plan_fits(best);
            if (best.tiles_m == 0 || (fits == best_fits ? c < least : fits)) {
                best = p;
                least = c;
            }
        }
    }
    return best;
}

// The plan of another tile for the split of `like`: the sums along K keep their order.
Plan8 plan_tile8(const Plan8 &like, int tile, int64_t M, int64_t N)
{
    Plan8 p = like;
    p.tile = tile;
    p.tiles_m = ceil_div(M, kFp8Tiles[tile].bm);
    p.tiles_n = ceil_div(N, kFp8Tiles[tile].bn);
    return p;
}

void set_product8(Fp8Params &p, const Plan8 &pl, int64_t M, int64_t N, int64_t K, const Operand8 &a, const Operand8 &b,
                  int shift_b)
{
    p.A = a.q;
    p.SA = a.s;
    p.lda = a.ldq;
    p.ldsa = a.lds;
    p.B = b.q;
    p.SB = b.s;
    p.ldb = b.ldq;
    p.ldsb = b.lds;
    p.K = (int)K;
    p.shift_b = shift_b;
    p.e.M = (int)M;
    p.e.N = (int)N;
    p.e.tiles_m = (int)pl.tiles_m;
    p.e.tiles_n = (int)pl.tiles_n;
    p.e.num_tiles = (int)(pl.tiles_m * pl.tiles_n);
    p.e.group_m = 8;
    p.e.k_split = (int)pl.k_split;
}

hipError_t launch_fwd8(bool bf, bool e5m2, int act, int tile, const Fp8Params &p, int groups, hipStream_t s)
{
    if (e5m2)
        return bf ? fp8_launch_fwd_e5m2_bf16(act, tile, p, groups, s) : fp8_launch_fwd_e5m2_f16(act, tile, p, groups, s);
    return bf ? fp8_launch_fwd_e4m3_bf16(act, tile, p, groups, s) : fp8_launch_fwd_e4m3_f16(act, tile, p, groups, s);
}
hipError_t launch_out8(bool bf, bool e5m2, int tile, const Fp8Params &p, int groups, hipStream_t s)
{
    if (e5m2) return bf ? fp8_launch_out_e5m2_bf16(tile, p, groups, s) : fp8_launch_out_e5m2_f16(tile, p, groups, s);
    return bf ? fp8_launch_out_e4m3_bf16(tile, p, groups, s) : fp8_launch_out_e4m3_f16(tile, p, groups, s);
}

// Turns a product into one that leaves fp32 partial sums at `part`; returns their sum's operands.
SplitSumParams set_split8(Fp8Params &p, const Plan8 &pl, float *part)
{
    const int64_t ldc = round_up(p.e.N, 8);
    p.e.C32 = part;
    p.e.ldc = ldc;
    p.e.c_split = p.e.M * ldc;
    p.e.acc_out = 1;
    SplitSumParams q = {};
    q.part = part;
    q.splits = pl.splits;
    q.M = p.e.M;
    q.N = p.e.N;
    q.ldc = ldc;
    q.c_split = p.e.c_split;
    return q;
}

// C = A B^T into D (16-bit), in parts where it is split: p is set up for the
// launch, sum for the one behind it that adds up the parts.
struct Product8 {
    Fp8Params p = {};
    SplitSumParams sum = {};
    int groups = 0;
    bool split = false;
};
void set_out8(Product8 &o, const Plan8 &pl, void *D, int64_t ldd, float *part)
{
    o.groups = (int)plan_groups(pl);
    o.split = pl.splits > 1;
    if (o.split) {
        o.sum = set_split8(o.p, pl, part);
        o.sum.D = (_Float16 *)D;
        o.sum.ldd = ldd;
    } else {
        o.p.e.D = (_Float16 *)D;
        o.p.e.ldd = ldd;
        o.p.e.vec = dma_rows(D, ldd, o.p.e.N);
    }
}
hipError_t run_sum8(bool bf, const Product8 &o, hipStream_t s)
{
    return o.split ? run_split_sum_out(bf, o.sum, s) : hipSuccess;
}
hipError_t run_product8(bool bf, bool e5m2, const Plan8 &pl, const Product8 &o, hipStream_t s)
{
    const hipError_t e = launch_out8(bf, e5m2, pl.tile, o.p, o.groups, s);
    return e == hipSuccess ? run_sum8(bf, o, s) : e;
}
hipError_t launch_pair8(bool bf, bool e5m2, int tile, const Fp8Pair &p, hipStream_t s)
{
    if (e5m2) return bf ? fp8_launch_pair_e5m2_bf16(tile, p, s) : fp8_launch_pair_e5m2_f16(tile, p, s);
    return bf ? fp8_launch_pair_e4m3_bf16(tile, p, s) : fp8_launch_pair_e4m3_f16(tile, p, s);
}

// ---- linear ---------------------------------------------------------------------
struct LinearPlan8 {
    bool few = false;  // rows: fp8_rows.hpp
    StageAt x, w;
    Plan8 pl;
    int64_t off_q = 0, off_s = 0, off_part = 0, bytes = 0;
};

int check_linear8(const ge_linear_fp8_args *a)
{
    if (!a) return GEMM_EPI_ERR_NULL_INPUT;
    GE_CHECK(check_dims(a->M, a->N, a->K));
    if (a->N > GE_MAX_COLS) return GEMM_EPI_ERR_SHAPE;
    if (a->act < GE_ACT_IDENTITY || a->act > GE_ACT_SILU) return GEMM_EPI_ERR_KIND;
    GE_CHECK(check_dtype(a->dtype));
    GE_CHECK(check_format(a->format));
    GE_CHECK(check_bytes(a->W, a->ldw, a->K, GE_MAX_COLS + 128, GEMM_EPI_ERR_NULL_INPUT));
    GE_CHECK(check_bytes(a->WS, a->ldws, blocks_of(a->K), GE_MAX_COLS + 128, GEMM_EPI_ERR_NULL_INPUT));
    if (a->M == 0) return GEMM_EPI_OK;
    if (a->XS) {
        GE_CHECK(check_bytes(a->X, a->ldx, a->K, GE_MAX_COLS + 128, GEMM_EPI_ERR_NULL_INPUT));
        GE_CHECK(check_bytes(a->XS, a->ldxs, blocks_of(a->K), GE_MAX_COLS + 128, GEMM_EPI_ERR_NULL_INPUT));
    } else {
        GE_CHECK(check_matrix(a->X, a->ldx, a->K, 2, GEMM_EPI_ERR_NULL_INPUT));
    }
    GE_CHECK(check_matrix(a->D, a->ldd, a->N, 2, GEMM_EPI_ERR_NULL_OUTPUT));
    if (a->residual) GE_CHECK(check_matrix(a->residual, a->ldr, a->N, 2, GEMM_EPI_ERR_NULL_INPUT));
    if (a->Z) GE_CHECK(check_matrix(a->Z, a->ldz, a->N, 2, GEMM_EPI_ERR_NULL_OUTPUT));
    if (a->bias && !aligned(a->bias, 2)) return GEMM_EPI_ERR_ALIGN;
    return GEMM_EPI_OK;
}

int plan_linear8(const ge_linear_fp8_args *a, LinearPlan8 &pl)
{
    GE_CHECK(check_linear8(a));
    if (a->M == 0) return GEMM_EPI_OK;
    if (!a->XS && !quant_fits(a->M, a->K)) return GEMM_EPI_ERR_SHAPE;
    Layout lay;
    pl.few = a->M <= kFewRows;
    if (pl.few) {
        if (!a->XS && a->M > kFewRows16Bit) {
            pl.off_q = lay.take(a->M * round_up(a->K, 16));
            pl.off_s = lay.take(a->M * round_up(blocks_of(a->K), 4));
        }
        pl.bytes = lay.bytes;
        return GEMM_EPI_OK;
    }
    if (a->XS) {
        pl.x = plan_operand(a->X, a->ldx, a->XS, a->ldxs, a->M, a->M, a->K, lay);
    } else {
        pl.off_q = lay.take(a->M * round_up(a->K, 16));
        pl.off_s = lay.take(a->M * round_up(blocks_of(a->K), 4));
    }
    pl.w = plan_operand(a->W, a->ldw, a->WS, a->ldws, a->N, blocks_of(a->N), a->K, lay);
    pl.pl = plan_fp8(a->M, a->N, a->K);
    if (!plan_fits(pl.pl)) return GEMM_EPI_ERR_SHAPE;
    pl.off_part = lay.take(pl.pl.part_bytes);
    pl.bytes = lay.bytes;
    return GEMM_EPI_OK;
}

int run_linear8(const ge_linear_fp8_args *a, const LinearPlan8 &pl)
{
    hipStream_t s = (hipStream_t)a->stream;
    char *ws = (char *)a->workspace;
    const bool bf = a->dtype == GEMM_EPI_BF16;
    Operand8 x = {(const uint8_t *)a->X, (const uint8_t *)a->XS, a->ldx, a->ldxs};
    Operand8 w = {(const uint8_t *)a->W, (const uint8_t *)a->WS, a->ldw, a->ldws};
    const bool e5m2 = a->format == GE_FP8_E5M2;
    Staging st;
    if (pl.few && (a->XS || a->M <= kFewRows16Bit)) {
        // X is read as it is
    } else if (a->XS) {
        stage_operand(pl.x, x, a->M, a->M, a->K, ws, st);
    } else {
        QuantParams q = {};
        q.X = a->X;
        q.ldx = a->ldx;
        q.R = (int)a->M;
        q.C = (int)a->K;
        q.Q = (uint8_t *)ws + pl.off_q;
        q.ldq = round_up(a->K, 16);
        q.S = (uint8_t *)ws + pl.off_s;
        q.lds = round_up(blocks_of(a->K), 4);
        GE_TRY(launch_quant(a->dtype, false, (int)a->format, q, s));
        x = {q.Q, q.S, q.ldq, q.lds};
    }
    if (pl.few) {
        FewRows8 f = {};
        f.X = x.q;
        f.XS = x.s;
        f.ldx = x.ldq;
        f.ldxs = x.lds;
        f.W = w.q;
        f.WS = w.s;
        f.ldw = w.ldq;
        f.ldws = w.lds;
        f.M = (int)a->M;
        f.N = (int)a->N;
        f.K = (int)a->K;
        f.act = (int)a->act;
        f.bias = (const _Float16 *)a->bias;
        f.R = (const _Float16 *)a->residual;
        f.D = (_Float16 *)a->D;
        f.Z = (_Float16 *)a->Z;
        f.ldr = a->ldr;
        f.ldd = a->ldd;
        f.ldz = a->ldz;
        return hip_status(fp8_launch_rows(bf, e5m2, f, s));
    }
    stage_operand(pl.w, w, a->N, blocks_of(a->N), a->K, ws, st);
    GE_TRY(st.run(s));
    Fp8Params p = {};
    set_product8(p, pl.pl, a->M, a->N, a->K, x, w, 7);
    const int groups = (int)plan_groups(pl.pl);
    if (pl.pl.splits > 1) {
        SplitSumParams q = set_split8(p, pl.pl, (float *)(ws + pl.off_part));
        q.bias = (const _Float16 *)a->bias;
        q.R = (const _Float16 *)a->residual;
        q.D = (_Float16 *)a->D;
        q.Z = (_Float16 *)a->Z;
        q.ldr = a->ldr;
        q.ldd = a->ldd;
        q.ldz = a->ldz;
        GE_TRY(launch_out8(bf, e5m2, pl.pl.tile, p, groups, s));
        return hip_status(run_split_sum_linear(bf, (int)a->act, q, s));
    }
    p.e.bias = (const _Float16 *)a->bias;
    p.e.R = (const _Float16 *)a->residual;
    p.e.D = (_Float16 *)a->D;
    p.e.Z = (_Float16 *)a->Z;
    p.e.ldr = a->ldr;
    p.e.ldd = a->ldd;
    p.e.ldz = a->ldz;
    p.e.vec = dma_rows(a->D, a->ldd, a->N) && (!a->Z || dma_rows(a->Z, a->ldz, a->N)) &&
              (!a->residual || dma_rows(a->residual, a->ldr, a->N));
    return hip_status(launch_fwd8(bf, e5m2, (int)a->act, pl.pl.tile, p, groups, s));
}

__global__ __launch_bounds__(256) void bias_sum_kernel(BiasSum p) { bias_sum(p, (int)blockIdx.x); }

// ---- linear, backward -------------------------------------------------------------
struct LinearGradPlan8 {
    StageAt x, w;
    Plan8 dx, dw;
    bool pair = false;  // both in one launch, on dx's tile
    int64_t off_dw = 0;
    int64_t off_q = 0, off_s = 0, off_qt = 0, off_st = 0, off_bias = 0, off_part = 0, bytes = 0;
};

int check_linear_grad8(const ge_linear_fp8_backward_args *a)
{
    if (!a) return GEMM_EPI_ERR_NULL_INPUT;
    GE_CHECK(check_dims(a->M, a->N, a->K));
    if (a->N > GE_MAX_COLS || a->M > GE_MAX_COLS) return GEMM_EPI_ERR_SHAPE;
    if (a->M > 0 && !a->dX && !a->dW && !a->dbias) return GEMM_EPI_ERR_NULL_OUTPUT;
    if (a->act < GE_ACT_IDENTITY || a->act > GE_ACT_SILU) return GEMM_EPI_ERR_KIND;
    GE_CHECK(check_dtype(a->dtype));
    GE_CHECK(check_format(a->format));
    if (a->M > 0) {
        GE_CHECK(check_matrix(a->dD, a->lddd, a->N, 2, GEMM_EPI_ERR_NULL_INPUT));
        if (a->act != GE_ACT_IDENTITY) GE_CHECK(check_matrix(a->Z, a->ldz, a->N, 2, GEMM_EPI_ERR_NULL_INPUT));
        if (a->dW) {
            GE_CHECK(check_bytes(a->XT, a->ldxt, a->M, GE_MAX_COLS + 128, GEMM_EPI_ERR_NULL_INPUT));
            GE_CHECK(check_bytes(a->XTS, a->ldxts, blocks_of(a->M), GE_MAX_COLS + 128, GEMM_EPI_ERR_NULL_INPUT));
        }
        if (a->dX) {
            GE_CHECK(check_bytes(a->WT, a->ldwt, a->N, GE_MAX_COLS + 128, GEMM_EPI_ERR_NULL_INPUT));
            GE_CHECK(check_bytes(a->WTS, a->ldwts, blocks_of(a->N), GE_MAX_COLS + 128, GEMM_EPI_ERR_NULL_INPUT));
        }
    }
    if (a->dX) GE_CHECK(check_matrix(a->dX, a->lddx, a->K, 2, GEMM_EPI_ERR_NULL_OUTPUT));
    if (a->dW) GE_CHECK(check_matrix(a->dW, a->lddw, a->K, 2, GEMM_EPI_ERR_NULL_OUTPUT));
    if (a->dbias && !aligned(a->dbias, 4)) return GEMM_EPI_ERR_ALIGN;
    return GEMM_EPI_OK;
}

int plan_linear_grad8(const ge_linear_fp8_backward_args *a, LinearGradPlan8 &pl)
{
    GE_CHECK(check_linear_grad8(a));
    if (a->M == 0) return GEMM_EPI_OK;
    if (!quant_fits(a->M, a->N)) return GEMM_EPI_ERR_SHAPE;
    Layout lay;
    pl.off_q = lay.take(a->M * round_up(a->N, 16));
    pl.off_s = lay.take(a->M * round_up(blocks_of(a->N), 4));
    pl.off_qt = lay.take(a->N * round_up(a->M, 16));
    pl.off_st = lay.take(a->N * round_up(blocks_of(a->M), 4));
    if (a->dbias && a->M > kBlock) pl.off_bias = lay.take(blocks_of(a->M) * a->N * 4);
    if (a->dX) {
        pl.w = plan_operand(a->WT, a->ldwt, a->WTS, a->ldwts, a->K, blocks_of(a->K), a->N, lay);
        pl.dx = plan_fp8(a->M, a->K, a->N);
        if (!plan_fits(pl.dx)) return GEMM_EPI_ERR_SHAPE;
    }
    if (a->dW) {
        pl.x = plan_operand(a->XT, a->ldxt, a->XTS, a->ldxts, a->K, a->K, a->M, lay);
        pl.dw = plan_fp8(a->N, a->K, a->M);
        if (!plan_fits(pl.dw)) return GEMM_EPI_ERR_SHAPE;
    }
    // Where both fit on the chip together, one launch on a tile that both share, if
    // the longer one then takes less than both one after the other by a tenth (the
    // estimates' error).  Apart and together, with dbias, us: 1001 x 1003 x 999 27.7 and 12.1,
    // 1024^3 18.6 and 9.0, 2048 x 2048 x 1024 25.9 and 14.7, 1400^3 26.0 and 12.8,
    // 700 x 300 x 5001 19.9 and 12.7, 2816^3 (256 x 256) 51.9 and 42.3.
    if (a->dX && a->dW) {
        double least = 0.9 * (cost8(a->M, a->K, a->N, pl.dx.tile, pl.dx.splits) +
                              cost8(a->N, a->K, a->M, pl.dw.tile, pl.dw.splits));
        const Plan8 x0 = pl.dx, w0 = pl.dw;
        for (const int tile : {kFp8Deep, kFp8Wide, kFp8Big}) {
            const Plan8 x = plan_tile8(x0, tile, a->M, a->K), w = plan_tile8(w0, tile, a->N, a->K);
            const double c = std::max(cost8(a->M, a->K, a->N, tile, x.splits), cost8(a->N, a->K, a->M, tile, w.splits));
            if (plan_groups(x) + plan_groups(w) > kCUs || c >= least) continue;
            least = c;
            pl.pair = true;
            pl.dx = x;
            pl.dw = w;
        }
    }
    pl.off_dw = pl.pair ? round_up(pl.dx.part_bytes, 256) : 0;
    pl.off_part = lay.take(std::max(a->dX ? pl.dx.part_bytes : 0, pl.off_dw + (a->dW ? pl.dw.part_bytes : 0)));
    pl.bytes = lay.bytes;
    return GEMM_EPI_OK;
}

template <int SRC, int ACT>
hipError_t launch_dz3(int format, const QuantParams &q, int64_t pad_groups, hipStream_t s)
{
    const dim3 g((unsigned)(quant_groups(q.R, q.C) + pad_groups)), b(512);
    return format == GE_FP8_E4M3 ? launch(quant_kernel<SRC, false, true, 0, ACT>, g, b, s, q)
                                 : launch(quant_kernel<SRC, false, true, 1, ACT>, g, b, s, q);
}
template <int SRC>
hipError_t launch_dz2(int act, int format, const QuantParams &q, int64_t pad_groups, hipStream_t s)
{
    switch (act) {
    case ACT_RELU: return launch_dz3<SRC, ACT_RELU>(format, q, pad_groups, s);
    case ACT_GELU: return launch_dz3<SRC, ACT_GELU>(format, q, pad_groups, s);
    case ACT_SILU: return launch_dz3<SRC, ACT_SILU>(format, q, pad_groups, s);
    default: return launch_dz3<SRC, ACT_IDENTITY>(format, q, pad_groups, s);
    }
}

int run_linear_grad8(const ge_linear_fp8_backward_args *a, const LinearGradPlan8 &pl)
{
    hipStream_t s = (hipStream_t)a->stream;
    char *ws = (char *)a->workspace;
    const bool bf = a->dtype == GEMM_EPI_BF16, e5m2 = a->format == GE_FP8_E5M2;
    if (a->M == 0) {
        if (a->dW) GE_TRY(run_zero(a->dW, a->lddw * 2, a->N, a->K * 2, s));
        if (a->dbias) GE_TRY(run_zero(a->dbias, a->N * 4, 1, a->N * 4, s));
        return GEMM_EPI_OK;
    }
    QuantParams q = {};
    q.X = a->dD;
    q.ldx = a->lddd;
    q.Z = a->Z;
    q.ldz = a->ldz;
    q.R = (int)a->M;
    q.C = (int)a->N;
    q.Q = (uint8_t *)ws + pl.off_q;
    q.ldq = round_up(a->N, 16);
    q.S = (uint8_t *)ws + pl.off_s;
    q.lds = round_up(blocks_of(a->N), 4);
    q.QT = (uint8_t *)ws + pl.off_qt;
    q.ldqt = round_up(a->M, 16);
    q.ST = (uint8_t *)ws + pl.off_st;
    q.ldst = round_up(blocks_of(a->M), 4);
    q.bands = (int)blocks_of(a->M);
    q.partial = !a->dbias ? nullptr : q.bands == 1 ? a->dbias : (float *)(ws + pl.off_bias);
    Staging st;
    Operand8 w = {(const uint8_t *)a->WT, (const uint8_t *)a->WTS, a->ldwt, a->ldwts};
    Operand8 x = {(const uint8_t *)a->XT, (const uint8_t *)a->XTS, a->ldxt, a->ldxts};
    if (a->dX) stage_operand(pl.w, w, a->K, blocks_of(a->K), a->N, ws, st);
    if (a->dW) stage_operand(pl.x, x, a->K, a->K, a->M, ws, st);
    q.pad = st.p;
    GE_TRY(bf ? launch_dz2<QS_BF16>((int)a->act, (int)a->format, q, st.groups(512), s)
              : launch_dz2<QS_F16>((int)a->act, (int)a->format, q, st.groups(512), s));
    float *part = (float *)(ws + pl.off_part);
    Product8 dx, dw;
    if (a->dX) {
        set_product8(dx.p, pl.dx, a->M, a->K, a->N, {q.Q, q.S, q.ldq, q.lds}, w, 7);
        set_out8(dx, pl.dx, a->dX, a->lddx, part);
    }
    if (a->dW) {
        set_product8(dw.p, pl.dw, a->N, a->K, a->M, {q.QT, q.ST, q.ldqt, q.ldst}, x, 0);
        set_out8(dw, pl.dw, a->dW, a->lddw, part + pl.off_dw / 4);
    }
    const bool sum_bias = a->dbias && q.bands > 1;
    if (pl.pair) {
        Fp8Pair pair = {{dx.p, dw.p}, {}, {dx.groups, dw.groups}};
        const bool here = sum_bias && q.bands <= kBiasBands;
        if (here) pair.bias = {q.partial, a->dbias, q.bands, (int)a->N};
        GE_TRY(launch_pair8(bf, e5m2, pl.dx.tile, pair, s));
        GE_TRY(run_sum8(bf, dx, s));
        GE_TRY(run_sum8(bf, dw, s));
        return sum_bias && !here ? hip_status(run_colsum(q.partial, a->dbias, q.bands, (int)a->N, s)) : GEMM_EPI_OK;
    }
    if (sum_bias) {
        // (the same order of the sum as in a pair's launch: dbias has the same bits
        // whichever other gradients are wanted)
        GE_TRY(q.bands <= kBiasBands ? launch(bias_sum_kernel, dim3((unsigned)ceil_div(a->N, 256)), dim3(256), s,
                                              BiasSum{q.partial, a->dbias, q.bands, (int)a->N})
                                     : run_colsum(q.partial, a->dbias, q.bands, (int)a->N, s));
    }
    if (a->dX) GE_TRY(run_product8(bf, e5m2, pl.dx, dx, s));
    if (a->dW) GE_TRY(run_product8(bf, e5m2, pl.dw, dw, s));
    return GEMM_EPI_OK;
}

}  // namespace

extern "C" {

int ge_quantize_fp8(const ge_quantize_fp8_args *a)
{
    GE_CHECK(check_quantize(a));
    if (a->R == 0) return GEMM_EPI_OK;
    QuantParams q = {};
    q.X = a->X;
    q.ldx = a->ldx;
    q.R = (int)a->R;
    q.C = (int)a->C;
    q.Q = (uint8_t *)a->Q;
    q.ldq = a->ldq;
    q.S = (uint8_t *)a->S;
    q.lds = a->lds;
    q.QT = (uint8_t *)a->QT;
    q.ldqt = a->ldqt;
    q.ST = (uint8_t *)a->ST;
    q.ldst = a->ldst;
    return hip_status(
        launch_quant(a->dtype, a->block == GE_BLOCK_TILE, (int)a->format, q, (hipStream_t)a->stream));
}

int ge_linear_fp8_workspace(const ge_linear_fp8_args *a, int64_t *bytes)
{
    LinearPlan8 pl;
    GE_CHECK(plan_linear8(a, pl));
    if (!bytes) return GEMM_EPI_ERR_NULL_OUTPUT;
    *bytes = pl.bytes;
    return GEMM_EPI_OK;
}

int ge_linear_fp8(const ge_linear_fp8_args *a)
{
    LinearPlan8 pl;
    GE_CHECK(plan_linear8(a, pl));
    GE_CHECK(check_workspace(a->workspace, a->workspace_bytes, pl.bytes));
    return a->M == 0 ? GEMM_EPI_OK : run_linear8(a, pl);
}

int ge_linear_fp8_backward_workspace(const ge_linear_fp8_backward_args *a, int64_t *bytes)
{
    LinearGradPlan8 pl;
    GE_CHECK(plan_linear_grad8(a, pl));
    if (!bytes) return GEMM_EPI_ERR_NULL_OUTPUT;
    *bytes = pl.bytes;
    return GEMM_EPI_OK;
}

int ge_linear_fp8_backward(const ge_linear_fp8_backward_args *a)
{
    LinearGradPlan8 pl;
    GE_CHECK(plan_linear_grad8(a, pl));
    GE_CHECK(check_workspace(a->workspace, a->workspace_bytes, pl.bytes));
    return run_linear_grad8(a, pl);
}

}  // extern "C"
