// kv4_attention.hip -- attention over the paged MXFP4 key/value cache for
// gfx950 (cache layout: kv4.hpp).
//
//   o[b, t, h] = sum_j p_j v_j,  p = softmax over the visible j of scale q.k_j
//
// Query t of sequence b stands at position lengths[b] - tokens + t; it sees
// the cached positions j < lengths[b] that are not after it (causal) and less
// than `window` before it (window > 0).  A query that sees nothing gets zeros
// and lse -inf.
//
// A tile of the computation is 16 rows (query tokens x query heads of one kv
// head) by 64 cached tokens, all in registers.  It computes S^T = K Q^T and
// O^T += V^T P^T with v_mfma_f32_16x16x32_bf16, lane (m, kg) = (lane % 16,
// lane / 16) holding column m = row of the query tile in S^T, P^T and O^T, so
// the running maximum and sum of a row live in the lanes that hold its scores
// and no transposition is needed between the two products:
//   - S^T tile u (of four) takes as its row 4 a + r the token 16 a + 4 u + r.
//     The result puts the 16 tokens 16 kg .. 16 kg + 15 in lane kg's registers,
//     in order.
//   - The second product contracts over tokens, in two steps of 32; lane kg's
//     eight operand elements of step s are its tokens 16 kg + 8 s ..: the P
//     values it already has, rounded to bf16 (relative error 2^-9 each, on
//     weights whose sum is taken from the fp32 values).
//   - V^T's rows are dims, two of which share a byte of 16 neighbouring tokens
//     (the cache's V layout): one 16-byte load gives a lane both dims for all
//     its tokens, v_cvt_scalef32_pk_bf16_fp4 decodes a byte with its token's
//     scale, and v_perm pairs tokens.  One product takes the even dims, one
//     the odd ones.
// The scaled conversion reads only the exponent field of its scale operand
// (checked for every code and scale byte), so scale bytes are rotated into
// place and not masked; a NaN scale (0xFF) decodes to NaN.
//
// Masked tokens count for nothing whatever they hold: their scores are
// replaced, codes are finite by themselves, and V scales are cleared where no
// row of the tile sees the token.  Where some rows see a token and others do
// not, a NaN scale is taken out of the product and put into the rows that see
// it.

#include "fp4_mfma.hpp"
#include "kv4.hpp"


namespace mxq {

namespace {

// Bytes [0, n) of a word.
__device__ __forceinline__ uint32_t low_bytes(int n)
{
    return n <= 0 ? 0u : n >= 4 ? ~0u : (1u << (8 * n)) - 1u;
}

// 0x80 in every byte of w that is 0xFF (exact as a test of the whole word;
// a byte above a hit may show as well, so callers look at bytes again).
__device__ __forceinline__ uint32_t has_ff(uint32_t w)
{
    return (~w - 0x01010101u) & w & 0x80808080u;
}

__device__ __forceinline__ float max_over_kg(float v)
{
    v = fmaxf(v, __shfl_xor(v, 16, kWave));
    return fmaxf(v, __shfl_xor(v, 32, kWave));
}

__device__ __forceinline__ float sum_over_kg(float v)
{
    v += __shfl_xor(v, 16, kWave);
    return v + __shfl_xor(v, 32, kWave);
}

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// What a lane loads of a tile: K codes of its four tokens, their scales, V
// codes of 16 tokens x NG dim pairs, their scales.
template <int D>
struct Tile {
    static constexpr int NG = D / 32;
    static constexpr int kScaleSets = D == 64 || D == 128 ? 1 : 2;  // K scale groups a lane's dims touch
    Words<NG> kc[4];
    uint4 ks[kScaleSets];
    uint4 vc[NG], vs[NG];
    bool ok;  // the page of the lane's 16 tokens (kg) is in the cache
};

template <int D>
__device__ __forceinline__ void load_tile(const Kv4Attn &a, const uint8_t *cache, const int32_t *table,
                                          int h, int tile, int m, int kg, Tile<D> &t)
{
    constexpr int NG = D / 32;
    const Kv4Geom &geo = a.geo;
    const int bpp = geo.page >> 4;  // blocks of 16 tokens in a page
    auto place = [&](int blk, int &in) {
        const int p = blk / bpp;
        in = (blk - p * bpp) * 16;
        int pg = p < a.width ? table[p] : -1;
        return pg;
    };
    int in;
    int pg = place(tile * 4 + (m >> 2), in);
    bool ok = pg >= 0 && pg < geo.pages;
    {
        const uint8_t *base = cache + (ok ? pg : 0) * geo.page_stride;
        const uint8_t *kc = base + geo.k_code(h, in + (m & 3)) + kg * (D / 8);
#pragma unroll
        for (int u = 0; u < 4; ++u) t.kc[u] = *reinterpret_cast<const Words<NG> *>(kc + u * 4 * (D / 2));
        const int g0 = kg * (D / 4) / 32;
        const uint8_t *ks = base + geo.k_scales() + geo.scale(h, in, g0);
        t.ks[0] = ld16<false>(ks);
        if constexpr (Tile<D>::kScaleSets == 2) t.ks[1] = ld16<false>(ks + (g0 + 1 < NG ? 16 : 0));
    }
    pg = place(tile * 4 + kg, in);
    t.ok = pg >= 0 && pg < geo.pages;
    {
        const uint8_t *base = cache + (t.ok ? pg : 0) * geo.page_stride;
        const uint8_t *vc = base + geo.v_codes() + geo.v_code(h, in, m);
        const uint8_t *vs = base + geo.v_scales() + geo.scale(h, in, 0);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            t.vc[g] = ld16<false>(vc + g * 256);
            t.vs[g] = ld16<false>(vs + g * 16);
        }
    }
}

// kWaves waves take the 64-token tiles of one split in turn, each with its own
// running maximum and sum, and are joined through LDS in a fixed order.
template <int D, int kWaves>
__global__ __launch_bounds__(kWaves * 64) void kv4_attention_kernel(Kv4Attn a)
{
    constexpr int NG = D / 32;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int m = lane & 15, kg = lane >> 4;
    const int heads = a.geo.heads, group = a.q_heads / heads, T = a.tokens;
    const int h = blockIdx.x % heads, b = blockIdx.x / heads, split = blockIdx.z;
    const int rows = T * group, row0 = blockIdx.y * 16;

    const int cap = a.width * a.geo.page;
    const int len = a.geo.pages > 0 ? min(max(a.lengths[b], 0), cap) : 0;
    const int row = min(row0 + m, rows - 1);
    const int t = row / group, hq = h * group + (row - t * group);
    // visible tokens of this lane's row: [jlo, jhi)
    const int pos = len - T + t;
    const int jhi = a.causal ? max(pos + 1, 0) : len;
    const int jlo = a.window > 0 ? max(pos - a.window + 1, 0) : 0;
    // of any and of every row of the tile
    const int tf = row0 / group, tl = min(row0 + 15, rows - 1) / group;
    const int any_lo = a.window > 0 ? max(len - T + tf - a.window + 1, 0) : 0;
    const int any_hi = a.causal ? max(len - T + tl + 1, 0) : len;
    const int all_lo = a.window > 0 ? max(len - T + tl - a.window + 1, 0) : 0;
    const int all_hi = a.causal ? max(len - T + tf + 1, 0) : len;
    const int tile0 = any_lo / 64, ntiles = any_hi > any_lo ? (any_hi + 63) / 64 - tile0 : 0;
    const int per = (ntiles + a.splits - 1) / a.splits;
    const int tile_end = tile0 + min(ntiles, (split + 1) * per);

    bf16x8 qf[NG];
    {
        const uint16_t *qp = a.q + b * a.q_seq + t * a.q_tok + hq * a.q_head + kg * (D / 4);
#pragma unroll
        for (int j = 0; j < NG; ++j) qf[j] = __builtin_bit_cast(bf16x8, ld16<false>(qp + 8 * j));
    }
    const int32_t *table = a.table + b * a.table_stride;
    const float c = a.scale * kLog2e;
    const int rot = (8 * (m & 3) + 9) & 31;  // scale byte m % 4 of a word -> bits 23..30

    f32x4 oe[NG], oo[NG];  // even and odd dims
#pragma unroll
    for (int g = 0; g < NG; ++g) oe[g] = oo[g] = f32x4{0.f, 0.f, 0.f, 0.f};
    float mx = -INFINITY, sum = 0.f;

    for (int tile = tile0 + split * per + wave; tile < tile_end; tile += kWaves) {
        Tile<D> tl_;
        load_tile<D>(a, a.cache, table, h, tile, m, kg, tl_);

        float x[16];  // tokens 16 kg + 0..15 of the tile
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const uint32_t w0 = u == 0 ? tl_.ks[0].x : u == 1 ? tl_.ks[0].y : u == 2 ? tl_.ks[0].z : tl_.ks[0].w;
            const uint32_t s0 = __builtin_amdgcn_alignbit(w0, w0, rot);
            uint32_t s1 = s0;
            if constexpr (Tile<D>::kScaleSets == 2) {
                const uint32_t w1 = u == 0 ? tl_.ks[1].x : u == 1 ? tl_.ks[1].y : u == 2 ? tl_.ks[1].z : tl_.ks[1].w;
                s1 = __builtin_amdgcn_alignbit(w1, w1, rot);
            }
            f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                // dims kg D/4 + 8 j ..: the lane's first or second scale group
                const uint32_t s = 8 * j + kg * (D / 4) % 32 < 32 ? s0 : s1;
                const uint32_t w = tl_.kc[u].w[j];
                acc = mfma(
                    fp4_frag(w, s),
                    qf[j], acc);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) x[4 * u + r] = acc[r] * c;
        }

        const int first = tile * 64 + 16 * kg;  // the lane's first token
        if (tile * 64 < all_lo || tile * 64 + 64 > all_hi || wave_any(!tl_.ok)) {
            const int lo = tl_.ok ? jlo - first : 16, hi = jhi - first;
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = i >= lo && i < hi ? x[i] : -INFINITY;
            // V scales of tokens no row sees
            const int alo = tl_.ok ? any_lo - first : 16, ahi = any_hi - first;
            uint32_t bad = 0;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const uint32_t keep = low_bytes(ahi - 4 * w) & ~low_bytes(alo - 4 * w);
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    uint32_t &v = w == 0 ? tl_.vs[g].x : w == 1 ? tl_.vs[g].y : w == 2 ? tl_.vs[g].z : tl_.vs[g].w;
                    v &= keep;
                    bad |= has_ff(v);
                }
            }
            if (wave_any(bad != 0)) {  // a NaN group that only some rows may see
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    bool hit = false;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        uint32_t &v = i / 4 == 0 ? tl_.vs[g].x : i / 4 == 1 ? tl_.vs[g].y : i / 4 == 2 ? tl_.vs[g].z : tl_.vs[g].w;
                        const uint32_t byte = 0xFFu << (8 * (i & 3));
                        if ((v & byte) == byte) {
                            v &= ~byte;
                            // the row of lane m; all its lanes look at their own tokens
                            hit |= i >= lo && i < hi;
                        }
                    }
                    int any = hit;
                    any |= __shfl_xor(any, 16, kWave);
                    any |= __shfl_xor(any, 32, kWave);
                    if (any) {
                        oe[g] += f32x4{NAN, NAN, NAN, NAN};
                        oo[g] += f32x4{NAN, NAN, NAN, NAN};
                    }
                }
            }
        }

        float top = x[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) top = fmaxf(top, x[i]);
        const float mx_new = fmaxf(mx, max_over_kg(top));
        const float base = mx_new == -INFINITY ? 0.f : mx_new;
        if (wave_any(mx_new > mx)) {
            const float f = __builtin_amdgcn_exp2f(mx - base);
            sum *= f;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                oe[g] *= f;
                oo[g] *= f;
            }
            mx = mx_new;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            x[i] = __builtin_amdgcn_exp2f(x[i] - base);
            sum += x[i];
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const bf16x8 p = as_bf16x8(bf16x2_rne(x[8 * s], x[8 * s + 1]), bf16x2_rne(x[8 * s + 2], x[8 * s + 3]),
                                       bf16x2_rne(x[8 * s + 4], x[8 * s + 5]), bf16x2_rne(x[8 * s + 6], x[8 * s + 7]));
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                uint32_t e[4], o[4];
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const uint32_t codes = s == 0 ? (w == 0 ? tl_.vc[g].x : tl_.vc[g].y) : (w == 0 ? tl_.vc[g].z : tl_.vc[g].w);
                    const uint32_t sc = s == 0 ? (w == 0 ? tl_.vs[g].x : tl_.vs[g].y) : (w == 0 ? tl_.vs[g].z : tl_.vs[g].w);
                    const uint32_t t0 = fp4_pair<0>(codes, scale_at<0>(sc)), t1 = fp4_pair<1>(codes, scale_at<1>(sc));
                    const uint32_t t2 = fp4_pair<2>(codes, scale_at<2>(sc)), t3 = fp4_pair<3>(codes, scale_at<3>(sc));
                    e[2 * w] = __builtin_amdgcn_perm(t1, t0, 0x05040100u);
                    e[2 * w + 1] = __builtin_amdgcn_perm(t3, t2, 0x05040100u);
                    o[2 * w] = __builtin_amdgcn_perm(t1, t0, 0x07060302u);
                    o[2 * w + 1] = __builtin_amdgcn_perm(t3, t2, 0x07060302u);
                }
                oe[g] = mfma(as_bf16x8(e[0], e[1], e[2], e[3]), p, oe[g]);
                oo[g] = mfma(as_bf16x8(o[0], o[1], o[2], o[3]), p, oo[g]);
            }
        }
    }

    // join the waves: lane (m, kg) holds dims 32 g + 8 kg + 0..7 of row m
    constexpr int kPitch = D + 4;  // rows 4 banks apart
    __shared__ float so[kWaves][16][kPitch];
    __shared__ float sm[kWaves][16], sl[kWaves][16];
    sum = sum_over_kg(sum);
    if (kg == 0) {
        sm[wave][m] = mx;
        sl[wave][m] = sum;
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        float *p = &so[wave][m][32 * g + 8 * kg];
        *reinterpret_cast<f32x4 *>(p) = f32x4{oe[g][0], oo[g][0], oe[g][1], oo[g][1]};
        *reinterpret_cast<f32x4 *>(p + 4) = f32x4{oe[g][2], oo[g][2], oe[g][3], oo[g][3]};
    }
    __syncthreads();
    constexpr int kPer = 16 * D / (kWaves * 64);  // dims of one row per thread
    static_assert(kPer >= 1 && D % kPer == 0, "a thread stays in one row");
    const int r = threadIdx.x / (D / kPer), d0 = threadIdx.x % (D / kPer) * kPer;
    if (row0 + r >= rows) return;
    float top = sm[0][r];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) top = fmaxf(top, sm[w][r]);
    const float base = top == -INFINITY ? 0.f : top;
    float total = 0.f, o[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) o[i] = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const float f = __builtin_amdgcn_exp2f(sm[w][r] - base);
        total += sl[w][r] * f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) o[i] += so[w][r][d0 + i] * f;
    }
    const int tr = (row0 + r) / group;
    const int64_t line = ((int64_t)b * T + tr) * a.q_heads + h * group + (row0 + r - tr * group);
    if (a.splits > 1) {
        const int64_t lines = (int64_t)a.seqs * T * a.q_heads;
        float *part = a.part + (split * lines + line) * D + d0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) part[i] = o[i];
        if (d0 == 0) {
            float *ml = a.part + a.splits * lines * D + (split * lines + line) * 2;
            ml[0] = top;
            ml[1] = total;
        }
        return;
    }
    const float inv = total == 0.f ? 0.f : 1.0f / total;
    __bf16 *out = reinterpret_cast<__bf16 *>(a.out) + line * D + d0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) out[i] = (__bf16)(o[i] * inv);
    if (a.lse && d0 == 0) a.lse[line] = (top + __builtin_log2f(total)) * kLn2;
}

// Joins the splits of one row per workgroup of D / 2 threads.
__global__ __launch_bounds__(128) void kv4_join_kernel(const float *__restrict__ part, int64_t lines,
                                                       int splits, int dim, uint16_t *__restrict__ out,
                                                       float *__restrict__ lse)
{
    const int64_t line = blockIdx.x;
    const float *ml = part + splits * lines * dim;
    float top = -INFINITY;
    for (int s = 0; s < splits; ++s) top = fmaxf(top, ml[(s * lines + line) * 2]);
    const float base = top == -INFINITY ? 0.f : top;
    float total = 0.f, o0 = 0.f, o1 = 0.f;
    for (int s = 0; s < splits; ++s) {
        const float f = __builtin_amdgcn_exp2f(ml[(s * lines + line) * 2] - base);
        total += ml[(s * lines + line) * 2 + 1] * f;
        const float2 v = reinterpret_cast<const float2 *>(part + (s * lines + line) * dim)[threadIdx.x];
        o0 += v.x * f;
        o1 += v.y * f;
    }
    const float inv = total == 0.f ? 0.f : 1.0f / total;
    reinterpret_cast<uint32_t *>(out + line * dim)[threadIdx.x] =
        (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)(o0 * inv)) |
        (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)(o1 * inv)) << 16;
    if (lse && threadIdx.x == 0) lse[line] = (top + __builtin_log2f(total)) * kLn2;
}

constexpr int kWavesPerGroup = 4;

template <int D>
hipError_t go(const Kv4Attn &a, hipStream_t stream)
{
    const int64_t mt = ((int64_t)a.tokens * (a.q_heads / a.geo.heads) + 15) / 16;
    const int64_t gx = (int64_t)a.seqs * a.geo.heads;
    if (gx > 0x7FFFFFFF || mt > 65535) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((kv4_attention_kernel<D, kWavesPerGroup>),
                       dim3((unsigned)gx, (unsigned)mt, (unsigned)a.splits), dim3(kWavesPerGroup * kWave),
                       0, stream, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.splits == 1) return e;
    const int64_t lines = (int64_t)a.seqs * a.tokens * a.q_heads;
    if (lines > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(kv4_join_kernel, dim3((unsigned)lines), dim3(D / 2), 0, stream, a.part, lines,
                       a.splits, D, a.out, a.lse);
    return hipGetLastError();
}

}  // namespace

int32_t kv4_attention_splits(int64_t seqs, int64_t tokens, int64_t q_heads, int64_t kv_heads,
                             int64_t dim, int64_t page, int64_t width)
{
    (void)dim;
    const int64_t groups = (tokens * (q_heads / kv_heads) + 15) / 16 * seqs * kv_heads;
    const int64_t tiles = (width * page + 63) / 64;
    const int64_t fill = (1024 + groups - 1) / groups;  // 4 workgroups per CU
    int64_t s = fill < tiles / kWavesPerGroup ? fill : tiles / kWavesPerGroup;
    return (int32_t)(s < 1 ? 1 : s > 128 ? 128 : s);
}

hipError_t launch_kv4_attention(const Kv4Attn &a, hipStream_t stream)
{
    switch (a.geo.dim) {
    case 64: return go<64>(a, stream);
    case 96: return go<96>(a, stream);
    case 128: return go<128>(a, stream);
    case 192: return go<192>(a, stream);
    case 256: return go<256>(a, stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace mxq
