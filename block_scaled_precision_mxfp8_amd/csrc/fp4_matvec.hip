// fp4_matvec.hip -- products of a few tokens with 4-bit weights for gfx950.
//
//   y[t, n] = sum_k x[t, k] * w[n, k],  w = E2M1(q) * 2^(s - 127)       (MXFP4)
//                                       w = E2M1(q) * E4M3(s) * g       (NVFP4)
//
// x bf16, q and s as the quantizers write them, sums in fp32, y bf16 or fp32.
//
// Each wave multiplies 16-row strips of weights with up to 64 tokens on the
// matrix cores (v_mfma_f32_16x16x32_bf16, weights as the A operand).  The
// contraction runs over k, so any order of k serves as long as both operands
// agree: lane (m, kg) = (lane % 16, lane / 16) loads the 16 contiguous code
// bytes of row m, k = 32 kg .. 32 kg + 31 of a 128-wide chunk -- for MXFP4
// exactly one scale group -- and the j-th of four matrix instructions takes
// its j-th dword (8 elements).  A row's 64 bytes of a chunk are contiguous
// over the kg lanes, so codes come straight from row-major storage.
//
// MXFP4 weights are exact in bf16, and v_cvt_scalef32_pk_bf16_fp4 applies the
// scale while it decodes: it reads only the exponent field of its scale
// operand, so a rotated scale word serves without masking (checked for every
// code and scale byte, junk in sign and fraction included).  NVFP4's E2M1 x
// E4M3 has at most 6 significant bits, also exact in bf16; g multiplies the
// fp32 sum.

#include "launch.hpp"
#include "mxq_device.hpp"

namespace mxq {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// 16 and 8 bytes from addresses aligned to 4 and 1
struct __attribute__((packed, aligned(4))) Codes16 { uint32_t w[4]; };
struct __attribute__((packed, aligned(1))) Bytes8 { uint32_t w[2]; };
struct __attribute__((packed, aligned(1))) Bytes2 { uint16_t w; };

__device__ __forceinline__ bf16x8 as_bf16x8(uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    return __builtin_bit_cast(bf16x8, make_uint4(a, b, c, d));
}

template <int kByte>
__device__ __forceinline__ uint32_t mx_pair(uint32_t codes, float scale)
{
    return __builtin_bit_cast(uint32_t,
                              __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, kByte));
}

__device__ __forceinline__ bf16x8 mx_frag(uint32_t codes, float scale)
{
    return as_bf16x8(mx_pair<0>(codes, scale), mx_pair<1>(codes, scale), mx_pair<2>(codes, scale),
                     mx_pair<3>(codes, scale));
}

template <int kByte>
__device__ __forceinline__ uint32_t nv_pair(uint32_t codes, float scale)
{
    const f32x2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, kByte);
    return bf16x2_exact(v.x * scale, v.y * scale);
}

__device__ __forceinline__ bf16x8 nv_frag(uint32_t codes, float scale)
{
    return as_bf16x8(nv_pair<0>(codes, scale), nv_pair<1>(codes, scale), nv_pair<2>(codes, scale),
                     nv_pair<3>(codes, scale));
}

// One wave's share of RT strips of 16 rows and NT tiles of 16 tokens; the
// workgroup's kWaves waves take the 256-wide steps of k in turn and add their
// sums through LDS in a fixed order.
template <bool kNV, int RT, int NT, int kWaves>
__global__ __launch_bounds__(kWaves * 64) void fp4_matvec_kernel(
    const uint16_t *__restrict__ x, int64_t tokens, int64_t ldx, const uint8_t *__restrict__ q,
    const uint8_t *__restrict__ s, const float *__restrict__ g, int64_t n, int64_t k,
    void *__restrict__ y, int64_t ldy, int out_f32)
{
    constexpr int kGroup = kNV ? 16 : 32;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int m = lane & 15, kg = lane >> 4;
    const int64_t row0 = (int64_t)blockIdx.x * (RT * 16);
    const int64_t tok0 = (int64_t)blockIdx.y * (NT * 16);

    const uint8_t *qrow[RT], *srow[RT];
    const uint16_t *xrow[NT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {  // rows past the end repeat the last: their sums are dropped
        const int64_t r = min(row0 + i * 16 + m, n - 1);
        qrow[i] = q + r * (k >> 1) + kg * 16;
        srow[i] = s + r * (k / kGroup);
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) xrow[i] = x + min(tok0 + i * 16 + m, tokens - 1) * ldx + kg * 32;

    f32x4 acc[RT][NT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    // one chunk of 128 from its codes, scale bits and the tokens
    auto chunk = [&](const Codes16(&w)[RT], const uint32_t(&sc)[RT], int64_t k0, int valid) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            bf16x8 b[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (8 * j < valid) v = *reinterpret_cast<const uint4 *>(xrow[t] + k0 + 8 * j);
                b[t] = __builtin_bit_cast(bf16x8, v);
            }
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                bf16x8 a;
                if constexpr (kNV)
                    a = nv_frag(w[i].w[j],
                                j < 2 ? __builtin_amdgcn_cvt_f32_fp8((int)sc[i], 0)
                                      : __builtin_amdgcn_cvt_f32_fp8((int)sc[i], 1));
                else
                    a = mx_frag(w[i].w[j], __uint_as_float(sc[i]));
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    acc[i][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b[t], acc[i][t], 0, 0, 0);
            }
        }
    };

    const int64_t full = k / 256;
    const int rot = (8 * kg + 9) & 31;  // scale byte kg of a word -> bits 23..30
    for (int64_t step = wave; step < full; step += kWaves) {
        const int64_t k0 = step * 256;
        Codes16 w[2][RT];
        uint32_t sc[2][RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            w[0][i] = *reinterpret_cast<const Codes16 *>(qrow[i] + (k0 >> 1));
            w[1][i] = *reinterpret_cast<const Codes16 *>(qrow[i] + (k0 >> 1) + 64);
            if constexpr (kNV) {
                const uint8_t *p = srow[i] + (k0 >> 4) + 2 * kg;
                sc[0][i] = reinterpret_cast<const Bytes2 *>(p)->w;
                sc[1][i] = reinterpret_cast<const Bytes2 *>(p + 8)->w;
            } else {
                const Bytes8 b = *reinterpret_cast<const Bytes8 *>(srow[i] + (k0 >> 5));
                sc[0][i] = __builtin_amdgcn_alignbit(b.w[0], b.w[0], rot);
                sc[1][i] = __builtin_amdgcn_alignbit(b.w[1], b.w[1], rot);
            }
        }
        chunk(w[0], sc[0], k0, 32);
        chunk(w[1], sc[1], k0 + 128, 32);
    }
    if (full * 256 < k && wave == (int)(full % kWaves)) {  // the last, partial step
        for (int64_t k0 = full * 256; k0 < k; k0 += 128) {
            // what of this lane's 32 elements exists: 0, 16 (NVFP4) or 32
            const int valid = (int)min((int64_t)32, max((int64_t)0, k - k0 - kg * 32));
            Codes16 w[RT];
            uint32_t sc[RT];
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                sc[i] = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w[i].w[j] = 8 * j < valid ? reinterpret_cast<const uint32_t *>(
                                                    qrow[i] + (k0 >> 1))[j]
                                              : 0u;
#pragma unroll
                for (int j = 0; j < 32 / kGroup; ++j)
                    if (kGroup * j < valid)
                        sc[i] |= (uint32_t)srow[i][(k0 + kg * 32) / kGroup + j] << (kNV ? 8 * j : 23);
            }
            chunk(w, sc, k0, valid);
        }
    }

    __shared__ f32x4 red[kWaves][RT * NT][kWave];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t) red[wave][i * NT + t][lane] = acc[i][t];
    __syncthreads();
    const float gs = kNV ? *g : 1.0f;
    for (int e = threadIdx.x; e < RT * NT * kWave; e += kWaves * kWave) {
        const int tile = e / kWave, l = e % kWave;
        f32x4 v = red[0][tile][l];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) v += red[w][tile][l];
        const int64_t t = tok0 + (tile % NT) * 16 + (l & 15);
        const int64_t r = row0 + (tile / NT) * 16 + (l >> 4) * 4;
        if (t >= tokens) continue;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if (r + c >= n) break;
            const float o = kNV ? v[c] * gs : v[c];
            if (out_f32)
                static_cast<float *>(y)[t * ldy + r + c] = o;
            else
                static_cast<__bf16 *>(y)[t * ldy + r + c] = (__bf16)o;
        }
    }
}

template <bool kNV, int RT, int NT, int kWaves>
hipError_t go(const uint16_t *x, int64_t tokens, int64_t ldx, const uint8_t *q, const uint8_t *s,
              const float *g, int64_t n, int64_t k, void *y, int64_t ldy, bool f32,
              hipStream_t stream)
{
    const int64_t gx = (n + RT * 16 - 1) / (RT * 16), gy = (tokens + NT * 16 - 1) / (NT * 16);
    if (gx > 0x7FFFFFFF || gy > 65535) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((fp4_matvec_kernel<kNV, RT, NT, kWaves>), dim3((unsigned)gx, (unsigned)gy),
                       dim3(kWaves * kWave), 0, stream, x, tokens, ldx, q, s, g, n, k, y, ldy,
                       (int)f32);
    return hipGetLastError();
}

template <bool kNV>
hipError_t pick(const uint16_t *x, int64_t tokens, int64_t ldx, const uint8_t *q, const uint8_t *s,
                const float *g, int64_t n, int64_t k, void *y, int64_t ldy, bool f32,
                hipStream_t stream)
{
    if (tokens <= 16) return go<kNV, 1, 1, 8>(x, tokens, ldx, q, s, g, n, k, y, ldy, f32, stream);
    if (tokens <= 32) return go<kNV, 2, 2, 8>(x, tokens, ldx, q, s, g, n, k, y, ldy, f32, stream);
    return go<kNV, 2, 4, 8>(x, tokens, ldx, q, s, g, n, k, y, ldy, f32, stream);
}

}  // namespace

hipError_t launch_fp4_matvec(bool nv, const uint16_t *x, int64_t tokens, int64_t ldx,
                             const uint8_t *q, const uint8_t *s, const float *g, int64_t n,
                             int64_t k, void *y, int64_t ldy, bool out_f32, hipStream_t stream)
{
    return nv ? pick<true>(x, tokens, ldx, q, s, g, n, k, y, ldy, out_f32, stream)
              : pick<false>(x, tokens, ldx, q, s, g, n, k, y, ldy, out_f32, stream);
}

}  // namespace mxq
