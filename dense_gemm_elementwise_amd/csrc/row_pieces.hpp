// row_pieces.hpp -- rows of any length and alignment, read 16 bytes a lane.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "linear_gemm.hpp"

namespace gemm_epi {

typedef int i32x4b __attribute__((ext_vector_type(4), aligned(1)));

// v moved down by n bytes (0 .. 16), zeros behind
__device__ __forceinline__ i32x4 move_down(i32x4 v, int n)
{
    const uint64_t lo = (uint64_t)(uint32_t)v[1] << 32 | (uint32_t)v[0], hi = (uint64_t)(uint32_t)v[3] << 32 | (uint32_t)v[2];
    const int s = n * 8 & 63;
    const uint64_t high = hi >> s, low = lo >> s | (s ? hi << (64 - s) : 0);
    const uint64_t a = n >= 16 ? 0 : n >= 8 ? high : low, b = n >= 8 ? 0 : high;
    return i32x4{(int)(uint32_t)a, (int)(uint32_t)(a >> 32), (int)(uint32_t)b, (int)(uint32_t)(b >> 32)};
}
// 16 bytes at any element-aligned address
template <int ES>
__device__ __forceinline__ i32x4 load_piece(const char *p) { return *(const i32x4b *)p; }
// The same of a row that has fewer than 16 bytes, element by element: the first n
// exist (the last of them at p + n - 1 where n is not positive), the rest are zeros.
template <int ES>
__device__ __forceinline__ i32x4 load_piece_short(const char *p, int n)
{
    constexpr int P = 16 / ES;
    uint32_t v[4] = {};
#pragma unroll 1
    for (int e = 0; e < P; e++) {  // (the elements move down, one after the other)
        const char *at = p + (int64_t)min(e, n - 1) * ES;
        const uint32_t x = ES == 1 ? *(const uint8_t *)at : ES == 2 ? *(const uint16_t *)at : *(const uint32_t *)at;
#pragma unroll
        for (int d = 0; d < 3; d++) v[d] = (uint64_t)v[d] >> (8 * ES) | v[d + 1] << (32 - 8 * ES);
        v[3] = (uint64_t)v[3] >> (8 * ES) | (e < n ? x << (32 - 8 * ES) : 0);
    }
    return i32x4{(int)v[0], (int)v[1], (int)v[2], (int)v[3]};
}
// 16 rows of a matrix, blocks of 128 columns at a time (ES: bytes of an element).
// A load takes 16 bytes a lane, adjacent lanes along a row: 8 rows of 128 bytes or 4 of 256.  That is not
// the layout of an MFMA operand (lane l has row l % 16), so a block is turned
// around in the wave's own LDS.  Loads in the operand layout, 64 bytes of 16 rows
// each, ask the L1 for four times as many lines and made it the bound: 64
// experts of 2 x 1024 x 4096 in 8 bits 122 us, 101 us (5.3 TB/s) this way.
template <int ES>
struct RowBlocks {
    static constexpr int LPR = 8 * ES, NL = 2 * ES, RPL = 8 / ES;  // lanes a row, loads a block, rows a load
    static constexpr int BYTES = 16 * 128 * ES;                   // of a block
    const char *base;   // shared by all lanes
    uint32_t off[NL];   // this lane's rows
    int col, last;      // its bytes of a block's rows; where the last 16 bytes of a row begin
    // row(i): the byte offset of row i, of K elements
    template <typename F>
    __device__ __forceinline__ void init(const char *ptr, int K, int lane, F &&row)
    {
        base = ptr;
        col = lane % LPR * 16;
        last = K * ES - 16;
#pragma unroll
        for (int v = 0; v < NL; v++) off[v] = row(v * RPL + lane / LPR);
    }
    // (of rows of 16 bytes and more; where they end in the block, finish() follows)
    // L: the loads that are made, of the first L RPL rows
    template <int L>
    __device__ __forceinline__ void load(i32x4 (&f)[L], int block) const
    {
        const uint32_t at = (uint32_t)min(col + block * (128 * ES), last);
#pragma unroll
        for (int v = 0; v < L; v++) f[v] = load_piece<ES>(base + (off[v] + at));
    }
    template <int L>
    __device__ __forceinline__ void finish(i32x4 (&f)[L], int block) const
    {
        const int miss = min(max(col + block * (128 * ES) - last, 0), 16);
#pragma unroll
        for (int v = 0; v < L; v++) f[v] = move_down(f[v], miss);
    }
    // the only block of shorter rows
    template <int L>
    __device__ __forceinline__ void load_short(i32x4 (&f)[L]) const
    {
        const int K = (last + 16) / ES;
#pragma unroll
        for (int v = 0; v < L; v++) f[v] = load_piece_short<ES>(base + (off[v] + (uint32_t)col), K - col / ES);
    }
    __device__ static __forceinline__ int at(int row, int piece) { return row * (128 * ES) + (piece ^ swz_a<LPR>(row)) * 16; }
    template <int L>
    __device__ static __forceinline__ void put(char *lds, const i32x4 (&f)[L], int lane)
    {
#pragma unroll
        for (int v = 0; v < L; v++) *(i32x4 *)(lds + at(v * RPL + lane / LPR, lane % LPR)) = f[v];
    }
};

constexpr int kShortRow = 16;  // elements; of shorter rows there is no piece of 16 bytes in 8 bits

// A wave takes every step-th block of 128 of K columns (kShortRow and more) from
// block `first` on: fetch(d, block) issues the loads of slot d, use(d, finish) uses
// them, with the block's number in finish where the rows end in it, otherwise -1.
// DEPTH blocks' loads are in flight together.  The blocks are taken from block `turn` on,
// around the end, so that workgroups do not all walk their rows from the start.
template <int DEPTH, typename Fetch, typename Use>
__device__ __forceinline__ void stream_row_blocks(int first, int step, int K, int turn, Fetch &&fetch, Use &&use)
{
    // The steady loop has no branch around its loads, and the order of loads and uses
    // is fixed, before it too: where paths join, the compiler waits for as many loads
    // as either path would need.
    const int whole = K >> 7;
    const bool tail = (K & 127) && first <= whole && (whole - first) % step == 0;  // the last block this wave takes
    int left = (whole > first ? (whole - first + step - 1) / step : 0) + tail;
    int j = first + turn;  // the block, before it is wrapped around
    j -= j >= whole ? whole : 0;
    auto number = [&](int d) {  // of the d-th block from j on
        const int i = j + d * step;
        return tail && d == left - 1 ? whole : i >= whole ? i - whole : i;
    };
    if (left >= DEPTH) {
#pragma unroll
        for (int d = 0; d < DEPTH; d++) {
            fetch(d, number(d));
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll 1
        while (left >= 2 * DEPTH) {
#pragma unroll
            for (int d = 0; d < DEPTH; d++) {
                use(d, -1);
                __builtin_amdgcn_sched_barrier(0);
                fetch(d, number(d + DEPTH));
                __builtin_amdgcn_sched_barrier(0);
            }
            left -= DEPTH;
            j += DEPTH * step;
            j -= j >= whole ? whole : 0;
        }
#pragma unroll
        for (int d = 0; d < DEPTH; d++) {
            use(d, d == DEPTH - 1 && tail && left == DEPTH ? whole : -1);
        }
        left -= DEPTH;
        j += DEPTH * step;
        j -= j >= whole ? whole : 0;
    }
    if (left > 0) {  // fewer than DEPTH: together, the last one again where there is none
#pragma unroll
        for (int d = 0; d < DEPTH; d++) fetch(d, number(min(d, left - 1)));
#pragma unroll
        for (int d = 0; d < DEPTH; d++) {
            if (d >= left) continue;
            use(d, tail && d == left - 1 ? whole : -1);
        }
    }
}

}  // namespace gemm_epi
