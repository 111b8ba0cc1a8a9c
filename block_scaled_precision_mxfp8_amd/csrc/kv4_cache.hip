// kv4_cache.hip -- writing into and copying pages of the paged MXFP4 key/value
// cache for gfx950 (layout: kv4.hpp).

#include "kv4.hpp"
#include "launch.hpp"
#include "mxq_device.hpp"

namespace mxq {

namespace {

// One lane quantizes 8 consecutive dims of one (token, K or V, head); a lane
// quad holds one group of 32, as in the MXFP4 quantizer.
__global__ __launch_bounds__(256) void kv4_append_kernel(
    Kv4Geom geo, uint8_t *__restrict__ cache, const uint16_t *__restrict__ kx, int64_t k_tok,
    int64_t k_head, const uint16_t *__restrict__ vx, int64_t v_tok, int64_t v_head,
    const int64_t *__restrict__ slots, int64_t tokens, uint16_t *__restrict__ k_fq,
    uint16_t *__restrict__ v_fq)
{
    const int d8 = geo.dim >> 3;  // lanes per (token, K or V, head)
    const int64_t per_tok = (int64_t)2 * geo.heads * d8;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= tokens * per_tok) return;  // whole quads: dim % 32 == 0
    const int64_t t = i / per_tok;
    int r = (int)(i - t * per_tok);
    const bool is_v = r >= geo.heads * d8;
    if (is_v) r -= geo.heads * d8;
    const int h = r / d8, d = (r - h * d8) * 8;

    const uint16_t *src = is_v ? vx + t * v_tok + h * v_head : kx + t * k_tok + h * k_head;
    const uint4 v = ld16<false>(src + d);
    const uint32_t sb = mx4_scale_byte(quad_max(amax8(v)));
    const bool nan_group = sb == 0xFFu;
    const float sf = e8m0_to_f32(sb);
    const uint32_t codes = nan_group ? e2m1x8_nan(v) : e2m1x8_hw(v, sf);

    uint16_t *fq = is_v ? v_fq : k_fq;
    if (fq) {
        uint4 o = e2m1x8_dequant_hw(codes, sf);
        if (nan_group) o = e2m1x8_dequant_nan(codes);
        st16<false>(fq + (t * geo.heads + h) * geo.dim + d, o);
    }
    const int64_t slot = slots[t];
    const int64_t page = slot / geo.page;
    if (slot < 0 || page >= geo.pages) return;  // a token without a place is not stored
    const int in = (int)(slot - page * geo.page);
    uint8_t *base = cache + page * geo.page_stride;
    if (is_v) {
        uint8_t *p = base + geo.v_codes() + geo.v_code(h, in, d >> 1);
#pragma unroll
        for (int c = 0; c < 4; ++c) p[16 * c] = (uint8_t)(codes >> (8 * c));
    } else {
        st4<false>(base + geo.k_code(h, in) + (d >> 1), codes);
    }
    // the quad's four lanes hold the same byte
    base[(is_v ? geo.v_scales() : geo.k_scales()) + geo.scale(h, in, d >> 5)] = (uint8_t)sb;
}

// Each workgroup copies 4 KiB pieces of one page of one layer.
__global__ __launch_bounds__(256) void kv4_copy_kernel(uint8_t *__restrict__ cache,
                                                       int64_t layer_stride, int64_t pages,
                                                       int64_t page_stride, int64_t page_bytes,
                                                       const int32_t *__restrict__ src,
                                                       const int32_t *__restrict__ dst,
                                                       unsigned pieces)
{
    const unsigned i = blockIdx.x / pieces;
    const int64_t s = src[i], d = dst[i];
    if (s < 0 || d < 0 || s >= pages || d >= pages || s == d) return;
    uint8_t *base = cache + (int64_t)blockIdx.y * layer_stride;
    const int64_t at = ((int64_t)(blockIdx.x - i * pieces) * 256 + threadIdx.x) * 16;
    if (at < page_bytes) st16<true>(base + d * page_stride + at, ld16<true>(base + s * page_stride + at));
}

}  // namespace

hipError_t launch_kv4_append(const Kv4Geom &geo, uint8_t *cache, const uint16_t *k, int64_t k_tok,
                             int64_t k_head, const uint16_t *v, int64_t v_tok, int64_t v_head,
                             const int64_t *slots, int64_t tokens, uint16_t *k_fq, uint16_t *v_fq,
                             hipStream_t stream)
{
    const int64_t lanes = tokens * 2 * geo.heads * (geo.dim >> 3);
    const int64_t grid = (lanes + 255) / 256;
    if (grid > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(kv4_append_kernel, dim3((unsigned)grid), dim3(256), 0, stream, geo, cache, k,
                       k_tok, k_head, v, v_tok, v_head, slots, tokens, k_fq, v_fq);
    return hipGetLastError();
}

hipError_t launch_kv4_copy(uint8_t *cache, int64_t layers, int64_t layer_stride, int64_t pages,
                           int64_t page_stride, int64_t page_bytes, const int32_t *src,
                           const int32_t *dst, int64_t n, hipStream_t stream)
{
    const int64_t pieces = (page_bytes + 4095) / 4096;
    if (n > 0x7FFFFFFF || pieces > 0x7FFFFFFF / n || layers > 65535)
        return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(kv4_copy_kernel, dim3((unsigned)(pieces * n), (unsigned)layers), dim3(256), 0,
                       stream, cache, layer_stride, pages, page_stride, page_bytes, src, dst,
                       (unsigned)pieces);
    return hipGetLastError();
}

}  // namespace mxq
