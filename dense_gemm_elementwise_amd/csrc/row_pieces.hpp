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
    __device__ __forceinline__ void load(i32x4 (&f)[NL], int block) const
    {
        const uint32_t at = (uint32_t)min(col + block * (128 * ES), last);
#pragma unroll
        for (int v = 0; v < NL; v++) f[v] = load_piece<ES>(base + (off[v] + at));
    }
    __device__ __forceinline__ void finish(i32x4 (&f)[NL], int block) const
    {
        const int miss = min(max(col + block * (128 * ES) - last, 0), 16);
#pragma unroll
        for (int v = 0; v < NL; v++) f[v] = move_down(f[v], miss);
    }
    // the only block of shorter rows
    __device__ __forceinline__ void load_short(i32x4 (&f)[NL]) const
    {
        const int K = (last + 16) / ES;
#pragma unroll
        for (int v = 0; v < NL; v++) f[v] = load_piece_short<ES>(base + (off[v] + (uint32_t)col), K - col / ES);
    }
    __device__ static __forceinline__ int at(int row, int piece) { return row * (128 * ES) + (piece ^ swz_a<LPR>(row)) * 16; }
    __device__ static __forceinline__ void put(char *lds, const i32x4 (&f)[NL], int lane)
    {
#pragma unroll
        for (int v = 0; v < NL; v++) *(i32x4 *)(lds + at(v * RPL + lane / LPR, lane % LPR)) = f[v];
    }
};

}  // namespace gemm_epi
