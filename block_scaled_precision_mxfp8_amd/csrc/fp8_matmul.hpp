// fp8_matmul.hpp -- what the kernels of products with 8-bit operands share (gfx950).
#pragma once

#include "mxq_device.hpp"

namespace mxq {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// What a product is ragged along: nothing, its rows (tokens sorted by expert),
// or its contraction (a weight gradient's tokens sorted by expert).
enum Ragged { kDense, kRows, kContraction };

// y[r, c] = sum_k x[r, k] w[c, k]; x and w are E4M3 codes.  Scales: fp32, x one
// for 128 k and w one for 128 rows and 128 k; or E8M0 bytes, one for 32 k of a
// row, for both.  Strides in elements of what they stride over (bytes of codes,
// scales, elements of y).
struct Fp8Matmul {
    const uint8_t *x, *w;
    const void *sx, *sw;
    void *y;
    const int32_t *offsets;  // groups + 1 of them; null if dense
    int64_t ldx, ldw, ld_sx, ld_sw, ldy;
    int64_t w_stride, sw_stride;  // between groups (kRows)
    int64_t y_stride;             // between groups (kContraction)
    int32_t m, n, k, groups;
    int32_t out_f32;
};

// offsets[i] as a row of 0..most.
__device__ __forceinline__ int32_t offset_at(const Fp8Matmul &a, int i, int32_t most)
{
    return min(max(a.offsets[i], 0), most);
}

// offsets[i] as a place of the contraction: a multiple of 32, or its end.
__device__ __forceinline__ int32_t k_offset_at(const Fp8Matmul &a, int i)
{
    const int32_t v = offset_at(a, i, a.k);
    return v == a.k ? v : v & ~31;
}

// The first n < 16 bytes at p, zeros behind them; reads no others.
__device__ __forceinline__ uint4 first_bytes(const uint8_t *p, int n)
{
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 15; ++i)
        if (i < n) w[i / 4] |= (uint32_t)p[i] << (i % 4 * 8);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Which group the t-th tile of `rows` rows belongs to when every group is cut
// into tiles by itself, and the rows of that tile: [first, end).  False past the
// last tile.  Every wave counts for itself, 64 groups at a time.
__device__ __forceinline__ bool find_row_tile(const Fp8Matmul &a, int rows, int32_t t, int &group,
                                              int32_t &first, int32_t &end)
{
    const int lane = threadIdx.x & (kWave - 1);
    int32_t before = 0;
    for (int g0 = 0; g0 < a.groups; g0 += kWave) {
        const int g = g0 + lane;
        int32_t b = 0, e = 0;
        if (g < a.groups) {
            b = offset_at(a, g, a.m);
            e = max(b, offset_at(a, g + 1, a.m));
        }
        const int32_t tiles = (e - b + rows - 1) / rows;
        int32_t upto = tiles;
#pragma unroll
        for (int off = 1; off < kWave; off <<= 1) {
            const int32_t v = __shfl_up(upto, off, kWave);
            if (lane >= off) upto += v;
        }
        const uint64_t past = __builtin_amdgcn_ballot_w64(before + upto > t);
        if (past) {
            const int l = __builtin_ctzll(past);
            const int32_t at = t - before - (__builtin_amdgcn_readlane(upto, l) -
                                             __builtin_amdgcn_readlane(tiles, l));
            group = g0 + l;
            end = __builtin_amdgcn_readlane(e, l);
            first = __builtin_amdgcn_readlane(b, l) + at * rows;
            end = min(end, first + rows);
            return true;
        }
        before += __builtin_amdgcn_readlane(upto, kWave - 1);
    }
    return false;
}

// 16 bytes at any address
struct __attribute__((packed, aligned(1))) Bytes16 { uint32_t w[4]; };
struct __attribute__((packed, aligned(4))) Words4 { uint32_t w[4]; };

__device__ __forceinline__ void store_product(void *y, int64_t at, float v, bool f32)
{
    if (f32)
        static_cast<float *>(y)[at] = v;
    else
        static_cast<__bf16 *>(y)[at] = (__bf16)v;
}

}  // namespace mxq
