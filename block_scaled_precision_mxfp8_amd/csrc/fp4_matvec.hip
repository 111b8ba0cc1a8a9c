// fp4_matvec.hip -- products of a few tokens with 4-bit weights for gfx950.
//
//   y[t, n] = sum_k x[t, k] * w[n, k],  w = E2M1(q) * 2^(s - 127)       (MXFP4)
//                                       w = E2M1(q) * E4M3(s) * g       (NVFP4)
//
// x bf16, q and s as the quantizers write them, sums in fp32, y bf16 or fp32.
//
// Both kernels multiply on the matrix cores (v_mfma_f32_16x16x32_bf16, weights
// as the A operand, tokens as B); lane (m, kg) = (lane % 16, lane / 16) holds
// 8 elements of row or column m.  The contraction may take k in any order as
// long as both operands agree.
//
// MXFP4 weights are exact in bf16 and decoded with their scale by one
// conversion for two.  NVFP4's E2M1 x E4M3 has at most 6 significant bits, also
// exact in bf16; g multiplies the fp32 sum.
//
// What limits these kernels is how a wave's loads fall on cache lines: a
// 16-byte-per-lane load costs about a clock for every line that a group of 16
// neighbouring lanes touches.  Lane m holding row m, as the matrix cores want
// it, touches 64 (measured: 72 clocks a load, 37 us for 64 tokens x [16384,
// 7168]); four neighbouring lanes on 64 bytes of one row touch 16 (27 us).  One
// token is bound by bytes: x [8192, 8192] reads 36 MB in 8 us.  With 64, the
// loads' address work, the exchanges through LDS (every workgroup exchanges all
// tokens anew), the matrix cores and the decoding take 6 to 9 us each and hardly
// overlap.  More than 64 are tiles that read and decode the weights again: 1024 x
// [16384, 7168] take 357 us, NVFP4 405 (240 GFLOP).

#include "fp4_mfma.hpp"
#include "launch.hpp"

namespace mxq {

namespace {

template <int N>
__device__ __forceinline__ void load_words(uint32_t (&d)[N], const uint8_t *p)
{
    const Bytes<4 * N> v = *reinterpret_cast<const Bytes<4 * N> *>(p);
    __builtin_memcpy(d, &v, sizeof v);
}

template <int kByte>
__device__ __forceinline__ uint32_t nv_pair(uint32_t codes, float scale)
{
    const f32x2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, kByte);
    return bf16x2_exact(v.x * scale, v.y * scale);
}

// 8 weights.  Scale word: the E8M0 byte in bits 23..30, or the E4M3 byte kByte.
template <bool kNV, int kByte>
__device__ __forceinline__ bf16x8 weights8(uint32_t codes, uint32_t scale)
{
    if constexpr (kNV) {
        const float f = __builtin_amdgcn_cvt_f32_fp8((int)scale, kByte);
        return as_bf16x8(nv_pair<0>(codes, f), nv_pair<1>(codes, f), nv_pair<2>(codes, f),
                         nv_pair<3>(codes, f));
    } else {
        return fp4_frag(codes, scale);
    }
}

__device__ __forceinline__ void store_y(void *y, int64_t at, float v, int out_f32)
{
    if (out_f32)
        static_cast<float *>(y)[at] = v;
    else
        static_cast<__bf16 *>(y)[at] = (__bf16)v;
}

struct MatvecArgs {
    const uint16_t *x;
    int64_t tokens, ldx;
    const uint8_t *q, *s;
    const float *g;
    int64_t n, k;
    void *y;
    int64_t ldy;
    int out_f32;
};

// ---------------------------------------------------------------------------
// One token: the 16 rows of A are 4 weight rows x 4 slices of k, column p of B
// the same slice p of the token (all columns alike modulo 4); of the product
// only the elements of equal slices are used, their sum over the slices is the
// result.  A quad of lanes then reads 64 contiguous bytes of one row and lane
// (kg, row, p) = (lane / 16, lane / 4 % 4, lane % 4) holds 16 of them, k = 128
// kg + 32 p .. of a step of 512: one MXFP4 group, and exactly what four products
// want, with no exchange between lanes.  The matrix cores do sixteen times the
// work needed, still under the time of the loads.  The token is loaded with the
// weights (16 lanes touch two lines); staging it in LDS cost 1.3 us of 8.7
// (x [8192, 8192]).
//
// The waves of a workgroup take the steps of k in turn, kDepth of them
// in flight; sums are added through LDS in a fixed order.
// ---------------------------------------------------------------------------
template <bool kNV, int RS, int kWaves, int kDepth>
__device__ __forceinline__ void one_body(const MatvecArgs &a)
{
    constexpr int kGroup = kNV ? 16 : 32, kSb = 32 / kGroup;  // scale bytes per lane and step
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int kg = lane >> 4, row = (lane >> 2) & 3, p = lane & 3, piece = kg * 4 + p;
    const int64_t row0 = (int64_t)blockIdx.x * (RS * 4);
    const int k = (int)a.k;
    const int full = k / 512, steps = (k + 511) / 512;

    const uint8_t *qr[RS], *sr[RS];
#pragma unroll
    for (int i = 0; i < RS; ++i) {  // rows past the end repeat the last: their sums are dropped
        const int64_t r = min(row0 + 4 * i + row, a.n - 1);
        qr[i] = a.q + r * (a.k >> 1) + piece * 16;
        sr[i] = a.s + r * (a.k / kGroup) + piece * kSb;
    }
    const float gs = kNV && a.k > 0 ? *a.g : 1.0f;  // an empty sum is 0 whatever g is
    struct Step { uint32_t w[RS][4], s[RS]; uint4 x[4]; } ring[kDepth];
    auto load = [&](Step &t, int st) {
#pragma unroll
        for (int j = 0; j < 4; ++j) t.x[j] = ld16<false>(a.x + st * 512 + piece * 32 + 8 * j);
#pragma unroll
        for (int i = 0; i < RS; ++i) {
            const Words<4> v = *reinterpret_cast<const Words<4> *>(qr[i] + (int64_t)st * 256);
#pragma unroll
            for (int j = 0; j < 4; ++j) t.w[i][j] = v.w[j];
            const uint8_t *sp = sr[i] + (int64_t)st * (16 * kSb);
            if constexpr (kNV) {
                const Bytes<2> b = *reinterpret_cast<const Bytes<2> *>(sp);
                t.s[i] = (uint32_t)b.b[0] | (uint32_t)b.b[1] << 8;
            } else {
                t.s[i] = *sp;
            }
        }
    };
    if (full > 0) {  // steps past the last repeat it, unused: no branch between the loads
#pragma unroll
        for (int u = 0; u < kDepth; ++u) load(ring[u], min(wave + u * kWaves, full - 1));
    }

    f32x4 acc[RS];
#pragma unroll
    for (int i = 0; i < RS; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto multiply = [&](const Step &t) {
        static_for<0, 4, 1>([&](auto J) {
            constexpr int j = J;
            const bf16x8 b = __builtin_bit_cast(bf16x8, t.x[j]);
#pragma unroll
            for (int i = 0; i < RS; ++i)
                acc[i] = mfma(weights8<kNV, j / 2>(t.w[i][j], kNV ? t.s[i] : t.s[i] << 23), b, acc[i]);
        });
    };
    for (int base = wave; base < full; base += kDepth * kWaves) {
        static_for<0, kDepth, 1>([&](auto U) {
            const int st = base + U * kWaves;
            if (st < full) {
                multiply(ring[U]);
                if (st + kDepth * kWaves < full) load(ring[U], st + kDepth * kWaves);
            }
        });
    }
    if (full < steps && wave == full % kWaves) {  // a partial step: what lies past k counts as zero
        const int valid = k - full * 512 - piece * 32;
        Step &t = ring[0];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            t.x[j] = make_uint4(0, 0, 0, 0);
            if (8 * j < valid) t.x[j] = ld16<false>(a.x + full * 512 + piece * 32 + 8 * j);
        }
#pragma unroll
        for (int i = 0; i < RS; ++i) {
            t.s[i] = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                t.w[i][j] = 8 * j < valid ? reinterpret_cast<const Words<4> *>(qr[i] + (int64_t)full * 256)->w[j] : 0u;
#pragma unroll
            for (int j = 0; j < kSb; ++j)
                if (kGroup * j < valid) t.s[i] |= (uint32_t)sr[i][(int64_t)full * (16 * kSb) + j] << (8 * j);
        }
        multiply(t);
    }

    // lane (kg, any, p) holds rows 4 kg + 0..3 of the product, slices 0..3 of
    // weight row kg, in a column of slice p
    __shared__ float red[kWaves][RS][4];
#pragma unroll
    for (int i = 0; i < RS; ++i) {
        float v = p == 0 ? acc[i][0] : p == 1 ? acc[i][1] : p == 2 ? acc[i][2] : acc[i][3];
        v += __uint_as_float(dpp_swap1(__float_as_uint(v)));
        v += __uint_as_float(dpp_swap2(__float_as_uint(v)));
        if ((lane & 15) == 0) red[wave][i][kg] = v;
    }
    __syncthreads();
    if (threadIdx.x < RS * 4) {
        const int i = threadIdx.x >> 2, row_of = threadIdx.x & 3;
        float v = red[0][i][row_of];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) v += red[w][i][row_of];
        if (row0 + threadIdx.x < a.n) store_y(a.y, row0 + threadIdx.x, v * gs, a.out_f32);
    }
}

template <bool kNV, int RS, int kWaves, int kDepth>
__global__ __launch_bounds__(kWaves * 64) void matvec_one_kernel(MatvecArgs a)
{
    one_body<kNV, RS, kWaves, kDepth>(a);
}

// ---------------------------------------------------------------------------
// More tokens: RT strips of 16 rows by NT tiles of 16 tokens per workgroup,
// whose waves split k in contiguous runs of chunks of 128.
//
// Loads have four neighbouring lanes on the four 16-byte pieces of a row (or
// token) r, lane 4 r + (p ^ 2 (r / 8)) on piece p; ds_bpermute then gives lane
// (m, kg) piece kg of row m.  (The exclusive or lets the 32 lanes that pass
// together read from 32 different lanes modulo 32; without it a third of the
// LDS cycles were conflicts.)  For tokens that is the operand (k = 32 j + 8 kg ..
// from the j-th load).  For weights a 4 x 4 transposition over kg (four permlane
// swaps) makes it dword kg of piece j, the same k.  One scale load covers four
// chunks.  kDepth chunks of weights, one of tokens are in flight.
// ---------------------------------------------------------------------------

// w[j] of lane group kg <- w[kg] of lane group j
__device__ __forceinline__ void transpose_kg(uint32_t (&w)[4])
{
    auto r = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    w[0] = r[0];
    w[2] = r[1];
    r = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    w[1] = r[0];
    w[3] = r[1];
    r = __builtin_amdgcn_permlane16_swap(w[0], w[1], false, false);
    w[0] = r[0];
    w[1] = r[1];
    r = __builtin_amdgcn_permlane16_swap(w[2], w[3], false, false);
    w[2] = r[0];
    w[3] = r[1];
}

__device__ __forceinline__ uint32_t from_lane(int lane4, uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_ds_bpermute(lane4, (int)v);
}

template <bool kNV, int RT, int NT, int kWaves, int kDepth>
__device__ __forceinline__ void many_body(const MatvecArgs &a)
{
    constexpr int kGroup = kNV ? 16 : 32, SW = kNV ? 2 : 1;  // scale words per row and chunk
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int m = lane & 15, kg = lane >> 4, r4 = lane >> 2, p4 = (lane & 3) ^ ((r4 >> 3) << 1);
    const int64_t row0 = (int64_t)blockIdx.x * (RT * 16), tok0 = (int64_t)blockIdx.y * (NT * 16);
    const int64_t n = a.n, k = a.k;

    // rows and tokens past the end repeat the last: their sums are dropped
    const uint8_t *qr[RT], *sr[RT];
    const uint16_t *xr[NT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const int64_t r = min(row0 + i * 16 + r4, n - 1);
        qr[i] = a.q + r * (k >> 1) + p4 * 16;
        sr[i] = a.s + r * (k / kGroup) + p4 * (4 * SW);
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) xr[i] = a.x + min(tok0 + i * 16 + r4, a.tokens - 1) * a.ldx + p4 * 8;

    const float gs = kNV && a.k > 0 ? *a.g : 1.0f;  // an empty sum is 0 whatever g is
    const int chunks = (int)(k / 128), per = (chunks + kWaves - 1) / kWaves;
    const int c0 = wave * per, c1 = min(chunks, c0 + per), last = chunks - 1;
    const int flip = (m >> 3) << 1, from_mk = 4 * (4 * m + (kg ^ flip));

    f32x4 acc[RT][NT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[i][t] = f32x4{0.f, 0.f, 0.f, 0.f};

    uint32_t wb[kDepth][RT][4], sb[2][RT][SW];
    uint4 xc[4][NT];
    auto load_w = [&](uint32_t(&d)[RT][4], int c) {
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const Words<4> v = *reinterpret_cast<const Words<4> *>(qr[i] + (int64_t)min(c, last) * 64);
#pragma unroll
            for (int j = 0; j < 4; ++j) d[i][j] = v.w[j];
        }
    };
    auto load_s = [&](uint32_t(&d)[RT][SW], int c) {  // chunk c + p4
        const int64_t at = (int64_t)(min(c + p4, last) - p4) * (4 * SW);
#pragma unroll
        for (int i = 0; i < RT; ++i) load_words<SW>(d[i], sr[i] + at);
    };
    auto load_x = [&](int j, int c) {
        const int64_t at = (int64_t)min(c, last) * 128 + 32 * j;
#pragma unroll
        for (int t = 0; t < NT; ++t) xc[j][t] = ld16<false>(xr[t] + at);
    };
    if (c0 < c1) {
#pragma unroll
        for (int j = 0; j < 4; ++j) load_x(j, c0);
        load_s(sb[0], c0);
#pragma unroll
        for (int d = 0; d < kDepth; ++d) load_w(wb[d], c0 + d);
    }
    static_assert(8 % kDepth == 0, "ring positions are constants in the unrolled loop");
    for (int base = c0; base < c1; base += 8) {
        static_for<0, 8, 1>([&](auto U) {
            constexpr int u = U;
            const int c = base + u;
            if (c < c1) {
                if constexpr (u % 4 == 0) load_s(sb[(u / 4 + 1) & 1], c + 4);
                uint32_t w[RT][4], s[RT][SW];
#pragma unroll
                for (int i = 0; i < RT; ++i) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[i][j] = from_lane(from_mk, wb[u % kDepth][i][j]);
#pragma unroll
                    for (int j = 0; j < SW; ++j) s[i][j] = from_lane(16 * m + 4 * ((u & 3) ^ flip), sb[(u / 4) & 1][i][j]);
                    if constexpr (kNV) {  // bytes 2 j + kg / 2 to bytes 0 and 2
#pragma unroll
                        for (int j = 0; j < SW; ++j) s[i][j] = kg & 2 ? s[i][j] >> 8 : s[i][j];
                    }
                    transpose_kg(w[i]);
                }
                load_w(wb[u % kDepth], c + kDepth);
                static_for<0, 4, 1>([&](auto J) {
                    constexpr int j = J;
                    bf16x8 b[NT];
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const uint4 v = xc[j][t];
                        b[t] = as_bf16x8(from_lane(from_mk, v.x), from_lane(from_mk, v.y),
                                         from_lane(from_mk, v.z), from_lane(from_mk, v.w));
                    }
                    load_x(j, c + 1);
#pragma unroll
                    for (int i = 0; i < RT; ++i) {
                        uint32_t sw;
                        if constexpr (kNV) sw = s[i][j / 2];
                        else sw = scale_at<j>(s[i][0]);
                        const bf16x8 wf = weights8<kNV, 2 * (j & 1)>(w[i][j], sw);
#pragma unroll
                        for (int t = 0; t < NT; ++t) acc[i][t] = mfma(wf, b[t], acc[i][t]);
                    }
                });
            }
        });
    }
    if (chunks * 128 < k && wave == kWaves - 1) {
        // the last, partial chunk: lane (m, kg) takes k = 32 kg + 8 j .. of it,
        // as far as it goes, straight from its row
        const int64_t at = (int64_t)chunks * 128 + kg * 32;
        const int valid = (int)(k - at);  // 16 (NVFP4) or 32 divides it
        uint32_t w[RT][4], s[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int64_t r = min(row0 + i * 16 + m, n - 1);
            s[i] = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[i][j] = 8 * j < valid ? reinterpret_cast<const Words<4> *>(a.q + r * (k >> 1) + (at >> 1))->w[j] : 0u;
#pragma unroll
            for (int j = 0; j < 32 / kGroup; ++j)
                if (kGroup * j < valid)
                    s[i] |= (uint32_t)a.s[r * (k / kGroup) + at / kGroup + j] << (kNV ? 8 * j : 23);
        }
        static_for<0, 4, 1>([&](auto J) {
            constexpr int j = J;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const uint16_t *xp = a.x + min(tok0 + t * 16 + m, a.tokens - 1) * a.ldx + at;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (8 * j < valid) v = ld16<false>(xp + 8 * j);
#pragma unroll
                for (int i = 0; i < RT; ++i)
                    acc[i][t] = mfma(weights8<kNV, j / 2>(w[i][j], s[i]), __builtin_bit_cast(bf16x8, v), acc[i][t]);
            }
        });
    }

    // Add the waves' tiles in order.  A tile's 64 lanes are stored with a gap
    // after every 16, so that neighbouring threads, which take neighbouring
    // rows of one token, read different banks and write contiguous bytes.
    constexpr int kTile = 68;
    __shared__ f32x4 red[kWaves][RT * NT][kTile];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t) red[wave][t * RT + i][lane + kg] = acc[i][t];
    __syncthreads();
    for (int e = threadIdx.x; e < RT * NT * 256; e += kWaves * kWave) {
        const int row = e % (RT * 16), tok = e / (RT * 16);
        const int tile = (tok >> 4) * RT + (row >> 4), l = (tok & 15) + 17 * ((row >> 2) & 3);
        float v = red[0][tile][l][row & 3];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) v += red[w][tile][l][row & 3];
        if (tok0 + tok < a.tokens && row0 + row < n)
            store_y(a.y, (tok0 + tok) * a.ldy + row0 + row, v * gs, a.out_f32);
    }
}

template <bool kNV, int RT, int NT, int kWaves, int kDepth>
__global__ __launch_bounds__(kWaves * 64) void matvec_many_kernel(MatvecArgs a)
{
    many_body<kNV, RT, NT, kWaves, kDepth>(a);
}

template <bool kNV, int RS, int kWaves, int kDepth>
hipError_t go_one(const MatvecArgs &a, hipStream_t stream)
{
    const int64_t gx = (a.n + RS * 4 - 1) / (RS * 4);
    if (gx > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((matvec_one_kernel<kNV, RS, kWaves, kDepth>), dim3((unsigned)gx),
                       dim3(kWaves * kWave), 0, stream, a);
    return hipGetLastError();
}

template <bool kNV, int RT, int NT, int kWaves, int kDepth>
hipError_t go_many(const MatvecArgs &a, hipStream_t stream)
{
    const int64_t gx = (a.n + RT * 16 - 1) / (RT * 16);
    if (gx > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
    constexpr int64_t kMost = 65535 * NT * 16;  // tokens of one launch
    for (int64_t t = 0; t < a.tokens; t += kMost) {
        MatvecArgs part = a;
        part.x += t * a.ldx;
        part.y = static_cast<uint8_t *>(a.y) + t * a.ldy * (a.out_f32 ? 4 : 2);
        part.tokens = a.tokens - t < kMost ? a.tokens - t : kMost;
        hipLaunchKernelGGL((matvec_many_kernel<kNV, RT, NT, kWaves, kDepth>),
                           dim3((unsigned)gx, (unsigned)((part.tokens + NT * 16 - 1) / (NT * 16))),
                           dim3(kWaves * kWave), 0, stream, part);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// Measured on MI355X (us, weights from the memory-side cache).  One token x
// [8192, 8192] MXFP4: 8.1 with 8 rows and 4 waves a workgroup, 8.5 with 8 and 8,
// 9.5 with 16 and 8, 9.0 through matvec_many; x [16384, 7168]: 12.2, 13.7, 15.4.
// A plain read of the codes takes 5.8 and 9.1.  (With several tokens, staged in
// LDS, such products took 12.7 for 4 x [8192, 8960] and 4.5 for 2 x [512, 7168],
// matvec_many 10.3 and 5.5.)
//
// More tokens: small tiles read weights and tokens more often, large ones leave
// CUs without work.  The smallest that needs no more than one workgroup per CU
// measured best or next to it, though the step to twice the tile leaves half of
// the CUs idle (5 tokens x [4096, 7168] take 7.2 us, NVFP4 8.2, x [4097, 7168] 8.3
// and 10.1).  64 tokens x [512, 7168] take 5.6, 6.7, 9.3,
// 12.4, 19.7 with (1, 1), (2, 1), (2, 2), (4, 2), (4, 4) strips and tiles of
// tokens; x [2048, 7168] 11.0, 7.9, 10.4, 14.0, 22.1; x [8192, 7168] 37.5, 26.9,
// 20.8, 16.2, 23.3; x [16384, 7168] 77, 57, 40, 34, 27.  16 tokens x [4096, 7168]
// 7.3, 7.9, 11.2 with 1, 2, 4 strips; x [16384, 7168] 21.3, 17.3, 15.7.
template <bool kNV>
hipError_t pick(const MatvecArgs &a, hipStream_t stream)
{
    if (a.tokens == 1 && a.k <= 1 << 30) return go_one<kNV, 2, 4, 4>(a, stream);
    constexpr int64_t kCus = 256;
    const auto fits = [&](int64_t rt, int64_t nt) {
        const int64_t y = (a.tokens + nt * 16 - 1) / (nt * 16);
        return y <= kCus && (a.n + rt * 16 - 1) / (rt * 16) * y <= kCus;
    };
    if (fits(1, 1)) return go_many<kNV, 1, 1, 8, 2>(a, stream);
    if (fits(2, 1)) return go_many<kNV, 2, 1, 8, 2>(a, stream);
    if (a.tokens <= 16) return go_many<kNV, 4, 1, 8, 2>(a, stream);
    if (fits(2, 2)) return go_many<kNV, 2, 2, 8, 2>(a, stream);
    if (a.tokens <= 32 || fits(4, 2)) return go_many<kNV, 4, 2, 8, 2>(a, stream);
    return go_many<kNV, 4, 4, 8, 2>(a, stream);
}

}  // namespace

hipError_t launch_fp4_matvec(bool nv, const uint16_t *x, int64_t tokens, int64_t ldx,
                             const uint8_t *q, const uint8_t *s, const float *g, int64_t n,
                             int64_t k, void *y, int64_t ldy, bool out_f32, hipStream_t stream)
{
    const MatvecArgs a{x, tokens, ldx, q, s, g, n, k, y, ldy, (int)out_f32};
    return nv ? pick<true>(a, stream) : pick<false>(a, stream);
}

}  // namespace mxq
