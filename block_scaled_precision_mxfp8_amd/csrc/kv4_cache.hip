// kv4_cache.hip -- writing into and copying pages of the paged MXFP4 key/value
// cache for gfx950 (layout: kv4.hpp).

#include "kv4.hpp"
#include "launch.hpp"
#include "mxq_device.hpp"

namespace mxq {

namespace {

// A workgroup stores one head of kTok consecutive tokens of the call.  One lane
// quantizes 8 consecutive dims of one token; a lane quad holds one group of 32,
// as in the MXFP4 quantizer.  K codes go straight to their rows.  V codes and
// all scales lie 16 tokens together in the cache, so they pass through LDS:
// where a whole block of 16 tokens is appended, in order, by this workgroup,
// its bytes are transposed in registers and leave as 16-byte stores; tokens of
// other blocks (both ends of a run, single tokens) are stored byte by byte.
//
// Bound by bytes: 16384 tokens of 8 heads x 128 read 67 MB and write 18 MB, in
// 23.4 us (3.6 TB/s; the median of launches in a row).  With bytes stored one by
// one throughout they took 46 us, the 16 partial writes of each 16 bytes being
// what L2 was busy with.  A workgroup's tokens start at multiples of kTok of the
// call, blocks at multiples of 16 slots: of a run that does not begin at one, 16
// of every 64 tokens lie in blocks that two workgroups share and go byte by byte
// (a run from slot 0 takes 20.3 us, from slot 5 22.3).  Small calls are one
// launch and one trip to memory.
template <int D, int kTok>
__global__ __launch_bounds__(256) void kv4_append_kernel(
    Kv4Geom geo, uint8_t *__restrict__ cache, const uint16_t *__restrict__ kx, int64_t k_tok,
    int64_t k_head, const uint16_t *__restrict__ vx, int64_t v_tok, int64_t v_head,
    const int64_t *__restrict__ slots, int64_t tokens, uint16_t *__restrict__ k_fq,
    uint16_t *__restrict__ v_fq)
{
    constexpr int kLanes = D / 8, NG = D / 32;  // lanes and groups per token
    __shared__ int64_t slot_of[kTok], base_of[kTok];
    __shared__ int in_of[kTok], lead[kTok / 16];
    __shared__ bool whole[kTok];
    __shared__ uint32_t vcode[kTok][kLanes + 1];
    __shared__ uint8_t scales[2][kTok][NG];  // K, V
    const int h = blockIdx.y, tid = threadIdx.x;
    const int64_t t0 = (int64_t)blockIdx.x * kTok;
    const int n = (int)min((int64_t)kTok, tokens - t0);

    if (tid < kTok) {
        int64_t slot = tid < n ? slots[t0 + tid] : -1;
        const int64_t page = slot / geo.page;
        if (slot < 0 || page >= geo.pages) slot = -1;  // a token without a place is not stored
        slot_of[tid] = slot;
        base_of[tid] = slot < 0 ? 0 : page * geo.page_stride;
        in_of[tid] = slot < 0 ? 0 : (int)(slot - page * geo.page);
    }
    if (tid < kTok / 16) lead[tid] = -1;
    __syncthreads();
    if (tid < kTok) {  // is the token's block of 16 all here, in order?
        const int64_t slot = slot_of[tid];
        const int first = tid - (in_of[tid] & 15);
        bool all = slot >= 0 && first >= 0 && first + 16 <= n;
        for (int j = 0; j < 16 && all; ++j) all = slot_of[first + j] == slot - tid + first + j;
        whole[tid] = all;
        if (all && first == tid) lead[tid >> 4] = tid;  // starts are 16 apart at least
    }

    const uint16_t *const src[2] = {kx + h * k_head, vx + h * v_head};
    constexpr int kBatch = 4;  // loads in flight per lane
    for (int at = tid; at < n * 2 * kLanes; at += 256 * kBatch) {
        uint4 v[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int e = at + 256 * u, t = e / (2 * kLanes), r = e - t * (2 * kLanes), kv = r / kLanes;
            v[u] = make_uint4(0, 0, 0, 0);
            if (t < n) v[u] = ld16<true>(src[kv] + (t0 + t) * (kv ? v_tok : k_tok) + (r - kv * kLanes) * 8);
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int e = at + 256 * u, t = e / (2 * kLanes), r = e - t * (2 * kLanes), kv = r / kLanes;
            const int c = r - kv * kLanes;
            const uint32_t sb = mx4_scale_byte(quad_max(amax8(v[u])));
            const bool nan_group = sb == 0xFFu;
            const float sf = e8m0_to_f32(sb);
            const uint32_t codes = nan_group ? e2m1x8_nan(v[u]) : e2m1x8_hw(v[u], sf);
            if (t >= n) continue;
            if (uint16_t *fq = kv ? v_fq : k_fq) {
                uint4 o = e2m1x8_dequant_hw(codes, sf);
                if (nan_group) o = e2m1x8_dequant_nan(codes);
                st16<true>(fq + ((t0 + t) * geo.heads + h) * D + c * 8, o);
            }
            scales[kv][t][c >> 2] = (uint8_t)sb;  // the quad's four lanes hold the same byte
            if (kv)
                vcode[t][c] = codes;
            else if (slot_of[t] >= 0)
                st4<false>(cache + base_of[t] + geo.k_code(h, in_of[t]) + c * 4, codes);
        }
    }
    __syncthreads();

    for (int e = tid; e < kTok / 16 * kLanes; e += 256) {  // V codes of whole blocks, four dim pairs a thread
        const int t = lead[e / kLanes], c = e % kLanes;
        if (t < 0) continue;
        uint32_t out[4][4];  // [dim pair][token / 4]
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const uint32_t a = vcode[t + 4 * w][c], b = vcode[t + 4 * w + 1][c];
            const uint32_t d = vcode[t + 4 * w + 2][c], f = vcode[t + 4 * w + 3][c];
            const uint32_t ab0 = __builtin_amdgcn_perm(b, a, 0x05010400u), ab1 = __builtin_amdgcn_perm(b, a, 0x07030602u);
            const uint32_t df0 = __builtin_amdgcn_perm(f, d, 0x05010400u), df1 = __builtin_amdgcn_perm(f, d, 0x07030602u);
            out[0][w] = __builtin_amdgcn_perm(df0, ab0, 0x05040100u);
            out[1][w] = __builtin_amdgcn_perm(df0, ab0, 0x07060302u);
            out[2][w] = __builtin_amdgcn_perm(df1, ab1, 0x05040100u);
            out[3][w] = __builtin_amdgcn_perm(df1, ab1, 0x07060302u);
        }
        uint8_t *p = cache + base_of[t] + geo.v_codes() + geo.v_code(h, in_of[t], 4 * c);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            st16<false>(p + 16 * i, make_uint4(out[i][0], out[i][1], out[i][2], out[i][3]));
    }
    for (int e = tid; e < kTok / 16 * 2 * NG; e += 256) {  // scales of whole blocks
        const int t = lead[e / (2 * NG)], kv = e / NG & 1, g = e % NG;
        if (t < 0) continue;
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i / 4] |= (uint32_t)scales[kv][t + i][g] << (8 * (i & 3));
        st16<false>(cache + base_of[t] + (kv ? geo.v_scales() : geo.k_scales()) + geo.scale(h, in_of[t], g),
                    make_uint4(w[0], w[1], w[2], w[3]));
    }
    for (int e = tid; e < n * kLanes; e += 256) {  // the other tokens
        const int t = e / kLanes, c = e % kLanes;
        if (slot_of[t] < 0 || whole[t]) continue;
        uint8_t *base = cache + base_of[t];
        uint8_t *p = base + geo.v_codes() + geo.v_code(h, in_of[t], 4 * c);
#pragma unroll
        for (int i = 0; i < 4; ++i) p[16 * i] = (uint8_t)(vcode[t][c] >> (8 * i));
        if (c < 2 * NG) {
            const int kv = c / NG, g = c % NG;
            base[(kv ? geo.v_scales() : geo.k_scales()) + geo.scale(h, in_of[t], g)] = scales[kv][t][g];
        }
    }
}

// cache[l, dst[i]] = cache[l, src[i]].  A workgroup copies 4 KiB of one page of
// one layer: nothing is kept between the 16 bytes of its threads, so many small
// workgroups do as well as few that loop, and a call of few pages spreads over
// the CUs.  Bound by bytes: 512 pages of 8 layers, 285 MB each way, take 98 us
// (5.8 TB/s); 8 pages of 4 layers 2.4 us, a launch.
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

namespace {

struct AppendArgs {
    const Kv4Geom &geo;
    uint8_t *cache;
    const uint16_t *k, *v;
    int64_t k_tok, k_head, v_tok, v_head;
    const int64_t *slots;
    int64_t tokens;
    uint16_t *k_fq, *v_fq;
};

template <int D, int kTok>
hipError_t go_append(const AppendArgs &a, hipStream_t stream)
{
    const int64_t gx = (a.tokens + kTok - 1) / kTok;
    hipLaunchKernelGGL((kv4_append_kernel<D, kTok>), dim3((unsigned)gx, (unsigned)a.geo.heads), dim3(256), 0,
                       stream, a.geo, a.cache, a.k, a.k_tok, a.k_head, a.v, a.v_tok, a.v_head, a.slots,
                       a.tokens, a.k_fq, a.v_fq);
    return hipGetLastError();
}

// Tokens of a workgroup: short windows spread a small call over more CUs, long
// ones have fewer ends of runs.  With 16 and 64, runs over 8 heads of 128: 33
// tokens 4.8 and 7.5 us, 2048 tokens 7.5 and 8.1, 4096 tokens 12.6 and 9.6, 16384
// tokens 37.0 and 23.6; single tokens of 2048 pages 13.0 and 14.7.
template <int D>
hipError_t pick_append(const AppendArgs &a, hipStream_t stream)
{
    return a.tokens * a.geo.heads >= 64 * 512 ? go_append<D, 64>(a, stream) : go_append<D, 16>(a, stream);
}

}  // namespace

hipError_t launch_kv4_append(const Kv4Geom &geo, uint8_t *cache, const uint16_t *k, int64_t k_tok,
                             int64_t k_head, const uint16_t *v, int64_t v_tok, int64_t v_head,
                             const int64_t *slots, int64_t tokens, uint16_t *k_fq, uint16_t *v_fq,
                             hipStream_t stream)
{
    const AppendArgs a{geo, cache, k, v, k_tok, k_head, v_tok, v_head, slots, tokens, k_fq, v_fq};
    switch (geo.dim) {
    case 64: return pick_append<64>(a, stream);
    case 96: return pick_append<96>(a, stream);
    case 128: return pick_append<128>(a, stream);
    case 192: return pick_append<192>(a, stream);
    case 256: return pick_append<256>(a, stream);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_kv4_copy(uint8_t *cache, int64_t layers, int64_t layer_stride, int64_t pages,
                           int64_t page_stride, int64_t page_bytes, const int32_t *src,
                           const int32_t *dst, int64_t n, hipStream_t stream)
{
    const int64_t pieces = (page_bytes + 4095) / 4096;
    hipLaunchKernelGGL(kv4_copy_kernel, dim3((unsigned)(pieces * n), (unsigned)layers), dim3(256), 0,
                       stream, cache, layer_stride, pages, page_stride, page_bytes, src, dst,
                       (unsigned)pieces);
    return hipGetLastError();
}

}  // namespace mxq
