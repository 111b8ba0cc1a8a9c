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

constexpr int kStep = 128;  // k of one step: one line of every row

// 64 lanes' 16 bytes at base + voff + soff into LDS at `lds` + 16 * lane, with no
// register in between.  In assembly because the compiler would have every later read
// of LDS wait for it; the loops wait where they have to.  (m0 is set right before
// its use, and the compiler has none of its own for it here.)
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t rsrc, uint32_t lds,
                                            uint32_t voff, uint32_t soff)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"(lds), "v"(voff), "s"(rsrc), "s"(soff)
                 : "memory");
}

__device__ __forceinline__ i32x8 join(uint4 a, uint4 b)
{
    return i32x8{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}

// 16 codes times a power of two (1 or a lifted MXFP8 scale) as bf16: exact wherever bf16 holds
// the value.  An infinite scale makes NaN of every code, 0 too.
__device__ __forceinline__ void decode16(bf16x8 (&d)[2], uint4 q, float scale)
{
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint2 a = mx_dequant4_hw(w[2 * j], scale), b = mx_dequant4_hw(w[2 * j + 1], scale);
        d[j] = __builtin_bit_cast(bf16x8, make_uint4(a.x, a.y, b.x, b.y));
    }
}

// 16 bytes at any address
struct __attribute__((packed, aligned(1))) Bytes16 { uint32_t w[4]; };

// Bytes at .. at + 15 of a run of `total`, zeros behind its end; reads nothing
// outside the run.  Near the end the run's last 16 bytes are read and moved down: one
// load, where a load for each byte would take the load path many times as long.
__device__ __forceinline__ uint4 bytes16_of(const uint8_t *run, int32_t at, int32_t total)
{
    if (total < 16) return first_bytes(run + at, max(min(total - at, 15), 0));
    const int over = max(at + 16 - total, 0);
    const Bytes16 v = *reinterpret_cast<const Bytes16 *>(run + (at - over));
    uint64_t lo = v.w[0] | (uint64_t)v.w[1] << 32, hi = v.w[2] | (uint64_t)v.w[3] << 32;
    if (over >= 8) lo = hi, hi = 0;
    const int bits = 8 * (over & 7);
    if (bits) {
        lo = lo >> bits | hi << (64 - bits);
        hi >>= bits;
    }
    if (over >= 16) lo = 0;
    return make_uint4((uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32));
}

// A buffer of 2^31 - 1 bytes from p on: an offset of kNowhere is outside it, and what
// is loaded from there is zero.
constexpr uint32_t kNowhere = 0x80000000u;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_at(const uint8_t *p)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(p), 0, 0x7FFFFFFF, 0x00020000);
}

// Block-FP8: the product of two scales may leave fp32 where the sum does not (2^100 and
// 2^100 over codes of 0; 2^-100 and 2^-41 under a sum of 2^24).  Such a sum is seen when it
// is done: one past fp32 has made it infinite or NaN, and what a subnormal one has lost,
// at most 2^-125 for each 128 k, counts only in sums below 2^-90.  Those are worked out
// again, one at a time in 64 bits, if a pair of their scales is the reason: 0.1 ms for a
// few tokens, 0.7 for one among 8192 (x 7168 x 7168).  So the loops have nothing of it; with
// the powers of two of both scales in the matrix cores' scales 8192 x 7168 x 7168 took 5 %
// longer.
constexpr uint32_t kUnsure = 0xDA000000u;
__device__ __forceinline__ uint32_t unsure(float v)  // kUnsure or more: not finite, or below 2^-90
{
    return (__float_as_uint(v) << 1) - 0x25000000u;
}

// Whether the product of two scales is no normal number, though neither is 0 or not finite.
__device__ __forceinline__ bool odd_pair(uint32_t sx, uint32_t sw)
{
    const float x = __uint_as_float(sx), w = __uint_as_float(sw);
    return x != 0.f && w != 0.f && __builtin_isfinite(x) && __builtin_isfinite(w) && !__builtin_isnormal(x * w);
}

__device__ __forceinline__ float block_product_again(const uint8_t *x, const float *sx, const uint8_t *w,
                                                     const float *sw, int32_t k)
{
    double sum = 0;
    for (int32_t i = 0; i * 128 < k; ++i) {
        double part = 0;
#pragma unroll 1  // little code: unrolled, though not run, it cost 33 x 4097 x 7168 in fp32 1.6 us of 16.9
        for (int32_t at = i * 128; at < min(k, i * 128 + 128); at += 16) {
            bf16x8 p[2], q[2];
            decode16(p, *reinterpret_cast<const uint4 *>(x + at), 1.0f);
            decode16(q, *reinterpret_cast<const uint4 *>(w + at), 1.0f);
#pragma unroll
            for (int j = 0; j < 16; ++j) part += (float)p[j / 8][j % 8] * (float)q[j / 8][j % 8];  // exact: four bits each
        }
        sum += part * ((double)sx[i] * (double)sw[i]);
    }
    return (float)sum;
}

// MXFP8 results in fp32: with both operands lifted by 2^10, codes are normal numbers of bf16
// under every byte up to 236, so nothing is lost at that end, and sums come out 2^20 times
// themselves.  At the other end codes become infinite (bytes above 236, where they are not 0
// or the lifted scale is infinite) or sums do (of 2^108 and more): all of it ends in a
// result that is not finite, which is then worked out again unless a scale of NaN is why.
constexpr uint32_t kLift = 10;
constexpr float kLowered = 0x1p-20f;
__device__ __forceinline__ float lifted(uint32_t byte)
{
    return __uint_as_float(min(byte + kLift, 255u) << 23);
}

// Whether one of n scale bytes is NaN's.
__device__ __forceinline__ bool nan_scale(const uint8_t *s, int32_t n)
{
    for (int32_t at = 0; at < n; at += 16) {
        const uint4 v = bytes16_of(s, at, n);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        bool found = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) found |= (((w[i] & 0x7F7F7F7Fu) + 0x01010101u) & w[i] & 0x80808080u) != 0;
        if (found) return true;
    }
    return false;
}

// A result v that is not finite, of k values whose first scales are at sx and sw.
__device__ __forceinline__ float mx_product_again(float v, const uint8_t *x, const uint8_t *sx, const uint8_t *w,
                                                  const uint8_t *sw, int32_t k)
{
    const int32_t groups = (k + 31) / 32;
    if (nan_scale(sx, groups) || nan_scale(sw, groups)) return __builtin_nanf("");
    bool large = false;  // else a code is NaN
#pragma unroll 1
    for (int32_t i = 0; i < groups; ++i)
        large |= max(sx[i], sw[i]) > 236 || sx[i] + sw[i] > 254 + 60;  // 2^22 products below 2^18 each
    if (!large) return v;
    double sum = 0;
#pragma unroll 1  // little code, as above
    for (int32_t at = 0; at < k; at += 16) {
        auto load = [&](const uint8_t *row) {
            return at + 16 <= k ? *reinterpret_cast<const uint4 *>(row + at) : first_bytes(row + at, k - at);
        };
        bf16x8 p[2], q[2];
        decode16(p, load(x), 1.0f);
        decode16(q, load(w), 1.0f);
        double part = 0;
#pragma unroll
        for (int j = 0; j < 16; ++j) part += (float)p[j / 8][j % 8] * (float)q[j / 8][j % 8];
        sum += __builtin_ldexp(part, sx[at / 32] + sw[at / 32] - 254);
    }
    return (float)sum;
}

__device__ __forceinline__ void store_product(void *y, int64_t at, float v, bool f32)
{
    if (f32)
        static_cast<float *>(y)[at] = v;
    else
        static_cast<__bf16 *>(y)[at] = (__bf16)v;
}

}  // namespace mxq
