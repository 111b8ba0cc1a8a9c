// fp4_mfma.hpp -- E2M1 codes as operands of the bf16 matrix cores (gfx950).
#pragma once

#include "mxq_device.hpp"

namespace mxq {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// N dwords at an address aligned to 4, N bytes at any address
template <int N>
struct __attribute__((packed, aligned(4))) Words { uint32_t w[N]; };
template <int N>
struct __attribute__((packed, aligned(1))) Bytes { uint8_t b[N]; };

__device__ __forceinline__ bf16x8 as_bf16x8(uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    return __builtin_bit_cast(bf16x8, make_uint4(a, b, c, d));
}

// 16 x 16 fp32 += A (16 x 32) B (32 x 16): lane (m, kg) = (lane % 16, lane /
// 16) holds 8 elements of A's row m and of B's column m, and of the result
// column m in rows 4 kg + 0..3.
__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// The two E2M1 codes of byte kByte times 2^(e - 127) as bf16 (exact), e the
// exponent field of scale_bits, 255 giving NaN; past bf16's range (253 and 254
// with large codes) Inf.  v_cvt_scalef32_pk_bf16_fp4 reads nothing else of its
// scale operand (checked for every code and exponent with junk in the sign and
// the fraction), so a scale word need only be shifted into place.
template <int kByte>
__device__ __forceinline__ uint32_t fp4_pair(uint32_t codes, uint32_t scale_bits)
{
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(
                                            codes, __uint_as_float(scale_bits), kByte));
}

__device__ __forceinline__ bf16x8 fp4_frag(uint32_t codes, uint32_t scale_bits)
{
    return as_bf16x8(fp4_pair<0>(codes, scale_bits), fp4_pair<1>(codes, scale_bits),
                     fp4_pair<2>(codes, scale_bits), fp4_pair<3>(codes, scale_bits));
}

// Byte i of a word to bits 23..30, the other bits junk.
template <int i>
__device__ __forceinline__ uint32_t scale_at(uint32_t w)
{
    if constexpr (i == 3) return w >> 1;
    else return w << (23 - 8 * i);
}

}  // namespace mxq
