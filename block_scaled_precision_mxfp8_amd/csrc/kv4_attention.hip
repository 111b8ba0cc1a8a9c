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
//     values it already has, as a sum of two bf16 numbers (off by 2^-16 at
//     most), so there are two products.  One bf16 number would be off by 2^-8,
//     more than the output's own rounding where values cancel.
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
// replaced, and V scales are cleared where no row of the tile sees the token.
// Where some rows see a token and others do not, a weight of 0 does not silence
// a V that is not finite.  There "wild" scales (255, NaN; 253 and 254, which
// pass bf16's range with large codes) are taken out of the product, and
// add_wild gives them to the rows that see them after the last tile.

#include <limits.h>

#include "fp4_mfma.hpp"
#include "kv4.hpp"

namespace mxq {

namespace {

// Bytes [0, n) of a word.
__device__ __forceinline__ uint32_t low_bytes(int n)
{
    return n <= 0 ? 0u : n >= 4 ? ~0u : (1u << (8 * n)) - 1u;
}

// 0xFF in every byte of w that is 253 or more: the low seven bits are then 125
// or more, and adding 3 carries into bit 7.
__device__ __forceinline__ uint32_t wild_bytes(uint32_t w)
{
    return ((((w & 0x7F7F7F7Fu) + 0x03030303u) & w & 0x80808080u) >> 7) * 0xFFu;
}

// 0xFF in every byte that is 255, of those that wild_bytes found (253..255).
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w, uint32_t wild)
{
    return (w & (w >> 1) & wild & 0x01010101u) * 0xFFu;
}

// Over the four lanes of a column, kg = 0..3 (lanes 16 apart), by swaps of half
// and quarter waves: no trip through LDS, which costs some 130 clocks each.
__device__ __forceinline__ float max_over_kg(float v)
{
    const uint32_t u = __float_as_uint(v);
    const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const uint32_t w = __float_as_uint(fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1])));
    const auto b = __builtin_amdgcn_permlane16_swap(w, w, false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

__device__ __forceinline__ float sum_over_kg(float v)
{
    const uint32_t u = __float_as_uint(v);
    const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const uint32_t w = __float_as_uint(__uint_as_float(a[0]) + __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane16_swap(w, w, false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// NG dwords that are read once: 16-byte pieces with the streaming hint where
// the address allows them (64 sequences of 4096..8192 tokens, 8 heads of 128:
// 89 us with the hint on K and V codes, 94 without).
template <int NG>
__device__ __forceinline__ Words<NG> load_once(const uint8_t *p)
{
    if constexpr (NG % 4 == 0) {
        uint4 v[NG / 4];
#pragma unroll
        for (int i = 0; i < NG / 4; ++i) v[i] = ld16<true>(p + 16 * i);
        return __builtin_bit_cast(Words<NG>, v);
    } else {
        return *reinterpret_cast<const Words<NG> *>(p);
    }
}

constexpr int scale_sets(int dim) { return dim == 64 || dim == 128 ? 1 : 2; }

// Where a tile lies.  In general each block of 16 tokens may be in a page of its
// own, and a lane follows the block it loads from.  With pages of a multiple of
// 64 tokens (kWide) a tile is in one page: place and address are then the same
// for the whole wave, kept in scalar registers, and a lane only adds an offset
// that never changes.
template <bool kWide>
struct Place {
    int entry, in;  // of the page table, block in the page
    int loaded;     // the table's entry, -1 for none: read ahead, looked at when used
    __device__ __forceinline__ void start(const Kv4Attn &a, const int32_t *table, int per_page, int tile, int block)
    {
        const int blk = tile * 4 + (kWide ? 0 : block);
        entry = blk / per_page;
        in = blk - entry * per_page;
        look(a, table);
    }
    __device__ __forceinline__ void advance(const Kv4Attn &a, const int32_t *table, int entries, int blocks, int per_page)
    {
        entry += entries;
        in += blocks;
        if (in >= per_page) {
            in -= per_page;
            ++entry;
        }
        look(a, table);
    }
    __device__ __forceinline__ void look(const Kv4Attn &a, const int32_t *table)
    {
        loaded = entry < a.width ? table[entry] : -1;
    }
    __device__ __forceinline__ int page() const
    {
        return kWide ? __builtin_amdgcn_readfirstlane(loaded) : loaded;
    }
    __device__ __forceinline__ bool ok(const Kv4Attn &a) const { return page() >= 0 && page() < a.geo.pages; }
    // Its page; page 0 stands in for one not in the cache, whose tokens are masked.
    __device__ __forceinline__ const uint8_t *base(const Kv4Attn &a) const
    {
        return a.cache + (int64_t)(ok(a) ? page() : 0) * a.geo.page_stride;
    }
};

// Bytes of a block of 16 tokens of one head, in codes and in scales; offsets in
// a page fit 32 bits.
constexpr int code_block(int dim) { return 8 * dim; }
constexpr int scale_block(int dim) { return dim / 2; }

// What a lane loads of K: codes of its four tokens, the scales of their block.
template <int D, bool kWide>
struct KTile {
    static constexpr int NG = D / 32;
    Words<NG> codes[4];
    uint4 scales[scale_sets(D)];  // the groups its D / 4 dims touch
    uint32_t code_at, scale_at;   // in the page, from the tile's (or its block's) first token

    __device__ __forceinline__ void init(const Kv4Geom &geo, int h, int m, int kg)
    {
        const int first = kWide ? 16 * (m >> 2) : 0;
        code_at = (uint32_t)(geo.k_code(h, first + (m & 3)) + kg * (D / 8));
        scale_at = (uint32_t)(geo.k_scales() + geo.scale(h, first, kg * (D / 4) / 32));
    }
    __device__ __forceinline__ void load(const Kv4Attn &a, const Place<kWide> &at, int kg)
    {
        const uint8_t *base = at.base(a);
        const uint8_t *kc = base + at.in * code_block(D) + code_at;
#pragma unroll
        for (int u = 0; u < 4; ++u) codes[u] = load_once<NG>(kc + u * 4 * (D / 2));
        const uint8_t *ks = base + at.in * scale_block(D) + scale_at;
        scales[0] = ld16<false>(ks);
        if constexpr (scale_sets(D) == 2) scales[1] = ld16<false>(ks + (kg * (D / 4) / 32 + 1 < NG ? 16 : 0));
    }
};

// Of V: codes of 16 tokens x NG dim pairs and their scales.
template <int D, bool kWide>
struct VTile {
    static constexpr int NG = D / 32;
    uint4 codes[NG], scales[NG];
    uint32_t code_at, scale_at;
    bool ok;  // the block's page is in the cache

    __device__ __forceinline__ void init(const Kv4Geom &geo, int h, int m, int kg)
    {
        const int first = kWide ? 16 * kg : 0;
        code_at = (uint32_t)(geo.v_codes() + geo.v_code(h, first, m));
        scale_at = (uint32_t)(geo.v_scales() + geo.scale(h, first, 0));
    }
    __device__ __forceinline__ void load(const Kv4Attn &a, const Place<kWide> &at)
    {
        ok = at.ok(a);
        const uint8_t *base = at.base(a);
        const uint8_t *vc = base + at.in * code_block(D) + code_at;
        const uint8_t *vs = base + at.in * scale_block(D) + scale_at;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            codes[g] = ld16<true>(vc + g * 256);
            scales[g] = ld16<false>(vs + g * 16);
        }
    }
};

__device__ __forceinline__ uint32_t word(const uint4 &v, int i)
{
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

__device__ __forceinline__ uint32_t &word(uint4 &v, int i)
{
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// Which tokens rows [row0, row0 + n) of one sequence see: [any_lo, any_hi) by
// any of them, [all_lo, all_hi) by every one.
struct Range {
    int any_lo, any_hi, all_lo, all_hi;
    __device__ __forceinline__ Range(const Kv4Attn &a, int len, int group, int row0, int n)
    {
        const int rows = a.tokens * group;
        const int first = len - a.tokens + row0 / group, last = len - a.tokens + min(row0 + n - 1, rows - 1) / group;
        any_lo = a.window > 0 ? max(first - a.window + 1, 0) : 0;
        any_hi = a.causal ? max(last + 1, 0) : len;
        all_lo = a.window > 0 ? max(last - a.window + 1, 0) : 0;
        all_hi = a.causal ? max(first + 1, 0) : len;
    }
};

__device__ __forceinline__ int context_length(const Kv4Attn &a, int b)
{
    return a.geo.pages > 0 ? min(max(a.lengths[b], 0), a.width * a.geo.page) : 0;
}

// Scores to base-2 exponents: exp(scale s) = 2^(c s).  A negative scale is
// carried by q's signs, so that c is positive and the largest score can be
// found before multiplying.  Scales of zero and NaN are carried by q as well
// (times 0, which makes q.k 0 or, where q is not finite, NaN; and NaN), with a c
// of 1, so that masked scores stay -inf.
__device__ __forceinline__ float exponent_factor(float scale)
{
    const float c = __builtin_fabsf(scale) * kLog2e;
    return c > 0.f ? c : 1.f;
}

// 0 times two bf16 numbers.
__device__ __forceinline__ uint32_t zero_times(uint32_t w)
{
    return ((w & 0x7F80u) == 0x7F80u ? 0x7FC0u : 0u) | ((w & 0x7F800000u) == 0x7F800000u ? 0x7FC00000u : 0u);
}

__device__ __forceinline__ bf16x8 load_q(const uint16_t *p, float scale)
{
    const uint32_t flip = scale < 0.f ? 0x80008000u : 0u;
    const uint4 v = ld16<false>(p);
    if (!(__builtin_fabsf(scale) * kLog2e > 0.f)) {
        const uint32_t nan = scale != scale ? 0x7FC07FC0u : 0u;
        return as_bf16x8(zero_times(v.x) | nan, zero_times(v.y) | nan, zero_times(v.z) | nan, zero_times(v.w) | nan);
    }
    return as_bf16x8(v.x ^ flip, v.y ^ flip, v.z ^ flip, v.w ^ flip);
}

// What a row's scores are taken from in the softmax: its running maximum (of q.k,
// unscaled), 0 while it has none.  The first product starts at minus that, and
// so gives the difference: exp(scale s - max) = 2^(c (s - max)) for scores of any
// size, where c s - (c max, rounded) is off by that rounding, whole powers of two
// for scores past 2^24, and overflows past 2^31.
__device__ __forceinline__ float softmax_from(float mx) { return mx == -INFINITY ? 0.f : mx; }

// One step of a row's running softmax over the 16 scores of each of its four
// lanes, less softmax_from(mx): x becomes the weights, the running maximum and
// this lane's sum move on, and the row's earlier sums want the returned factor
// when `moved`.
__device__ __forceinline__ float softmax_step(float (&x)[16], float c, float &mx, float &sum, bool &moved)
{
    float top = x[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) top = fmaxf(top, x[i]);
    top = max_over_kg(top);
    const bool up = top > (mx == -INFINITY ? -INFINITY : 0.f);
    float f = 1.f;
    moved = wave_any(up);
    if (moved) {
        const float by = up ? top : 0.f;
        f = mx == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(-by * c);
        sum *= f;
        if (up) mx = softmax_from(mx) + by;
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] -= by;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        x[i] = __builtin_amdgcn_exp2f(x[i] * c);
        sum += x[i];
    }
    return f;
}

// Weights of tokens 8 s .. as a sum of two bf16 numbers.  What the second costs,
// with its products: 64 sequences of 4096..8192 tokens 77 us (73 without), the
// chunk of 2 x 512 tokens 320 to 332 us (252 to 267).
struct Weights { bf16x8 hi, lo; };

__device__ __forceinline__ Weights weights_frag(const float (&x)[16], int s)
{
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = x[8 * s + 2 * i], b = x[8 * s + 2 * i + 1];
        hi[i] = bf16x2_rne(a, b);
        lo[i] = bf16x2_rne(a - bf16lo_to_f32(hi[i]), b - bf16hi_to_f32(hi[i]));
    }
    return {as_bf16x8(hi[0], hi[1], hi[2], hi[3]), as_bf16x8(lo[0], lo[1], lo[2], lo[3])};
}

__device__ __forceinline__ f32x4 weigh(bf16x8 v, const Weights &p, f32x4 acc) { return mfma(v, p.hi, mfma(v, p.lo, acc)); }

// V^T operands of 8 tokens (code and scale words of tokens 0..3 and 4..7) for
// a lane's even and odd dim.
__device__ __forceinline__ void v_frags(uint32_t c0, uint32_t c1, uint32_t s0, uint32_t s1, bf16x8 &even, bf16x8 &odd)
{
    uint32_t e[4], o[4];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const uint32_t c = w ? c1 : c0, s = w ? s1 : s0;
        const uint32_t t0 = fp4_pair<0>(c, scale_at<0>(s)), t1 = fp4_pair<1>(c, scale_at<1>(s));
        const uint32_t t2 = fp4_pair<2>(c, scale_at<2>(s)), t3 = fp4_pair<3>(c, scale_at<3>(s));
        e[2 * w] = __builtin_amdgcn_perm(t1, t0, 0x05040100u);
        e[2 * w + 1] = __builtin_amdgcn_perm(t3, t2, 0x05040100u);
        o[2 * w] = __builtin_amdgcn_perm(t1, t0, 0x07060302u);
        o[2 * w + 1] = __builtin_amdgcn_perm(t3, t2, 0x07060302u);
    }
    even = as_bf16x8(e[0], e[1], e[2], e[3]);
    odd = as_bf16x8(o[0], o[1], o[2], o[3]);
}

// Scale byte m % 4 of a word -> bits 23..30, by rotation.
__device__ __forceinline__ int scale_rotation(int m) { return (8 * (m & 3) + 9) & 31; }

// q.k - from of 64 tokens, 16 kg + 0..15 of them in this lane.
template <int D, bool kWide>
__device__ __forceinline__ void scores(const KTile<D, kWide> &kt, const bf16x8 (&qf)[D / 32], int m, int kg, float from,
                                       float (&x)[16])
{
    const int rot = scale_rotation(m);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const uint32_t w0 = word(kt.scales[0], u), s0 = __builtin_amdgcn_alignbit(w0, w0, rot);
        uint32_t s1 = s0;
        if constexpr (scale_sets(D) == 2) {
            const uint32_t w1 = word(kt.scales[1], u);
            s1 = __builtin_amdgcn_alignbit(w1, w1, rot);
        }
        f32x4 acc = {-from, -from, -from, -from};
#pragma unroll
        for (int j = 0; j < D / 32; ++j)  // dims kg D/4 + 8 j ..: the lane's first or second scale group
            acc = mfma(fp4_frag(kt.codes[u].w[j], 8 * j + kg * (D / 4) % 32 < 32 ? s0 : s1), qf[j], acc);
#pragma unroll
        for (int r = 0; r < 4; ++r) x[4 * u + r] = acc[r];
    }
}

// Adds to one strip of rows what a masked tile's product has left out: tokens of
// wild V scales, for the rows that see them ([jlo, jhi), c and mx as in the
// softmax, which is over).  2^8 of the weights times 2^-8 of the values is
// finite, so that rows that do not see them get 0; NaN goes to the rows that do.
template <int D>
__device__ __forceinline__ void add_wild(const Kv4Attn &a, const int32_t *table, int h, int tile, int m, int kg,
                                         const bf16x8 (&qf)[D / 32], int jlo, int jhi, float c, float mx,
                                         f32x4 (&oe)[D / 32], f32x4 (&oo)[D / 32])
{
    constexpr int NG = D / 32;
    Place<false> kp, vp;
    KTile<D, false> kt;
    VTile<D, false> vt;
    kt.init(a.geo, h, m, kg);
    vt.init(a.geo, h, m, kg);
    kp.start(a, table, a.geo.page >> 4, tile, m >> 2);
    vp.start(a, table, a.geo.page >> 4, tile, kg);
    kt.load(a, kp, kg);
    vt.load(a, vp);
    float x[16];
    scores<D, false>(kt, qf, m, kg, softmax_from(mx), x);
    const int first = tile * 64 + 16 * kg, lo = vt.ok ? jlo - first : 16, hi = jhi - first;
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = i >= lo && i < hi ? __builtin_amdgcn_exp2f(x[i] * c) * 256.f : 0.f;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        bool nan_seen = false;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            uint32_t &v = word(vt.scales[g], w);
            const uint32_t wild = wild_bytes(v), nan = nan_bytes(v, wild);
            nan_seen |= (nan & low_bytes(hi - 4 * w) & ~low_bytes(lo - 4 * w)) != 0;
            word(vt.codes[g], w) &= wild & ~nan;
            v = (v & wild & ~nan) - (0x08080808u & wild & ~nan);
        }
        int any = nan_seen;  // by the row of lane m: all its lanes look at their own tokens
        any |= __shfl_xor(any, 16, kWave);
        any |= __shfl_xor(any, 32, kWave);
        if (any) {
            oe[g] += f32x4{NAN, NAN, NAN, NAN};
            oo[g] += f32x4{NAN, NAN, NAN, NAN};
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            bf16x8 e, o;
            v_frags(word(vt.codes[g], 2 * s), word(vt.codes[g], 2 * s + 1), word(vt.scales[g], 2 * s),
                    word(vt.scales[g], 2 * s + 1), e, o);
            const Weights p = weights_frag(x, s);
            oe[g] = weigh(e, p, oe[g]);
            oo[g] = weigh(o, p, oo[g]);
        }
    }
}

// Sequences are started longest first when the workgroups do not all fit at
// once, so that the last to run are short: the sequence of rank `r` by length,
// ties in order.  For at most kRanked sequences; with more of them there are
// enough workgroups to even out.
constexpr int kRanked = 128;

template <int kThreads>
__device__ __forceinline__ int sequence_of_rank(const Kv4Attn &a, int r)
{
    __shared__ int length[kRanked], rank[kRanked], found;
    const int t = threadIdx.x % kRanked, part = threadIdx.x / kRanked, parts = kThreads / kRanked;
    if (part == 0 && t < a.seqs) {
        length[t] = context_length(a, t);
        rank[t] = 0;
    }
    __syncthreads();
    if (t < a.seqs) {
        const int mine = length[t];
        int before = 0;
#pragma unroll 4
        for (int j = part; j < a.seqs; j += parts) before += length[j] > mine || (length[j] == mine && j < t);
        atomicAdd(&rank[t], before);
    }
    __syncthreads();
    if (part == 0 && t < a.seqs && rank[t] == r) found = t;
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(found);
}

// Few rows: 16 of one kv head per workgroup, whose kWaves waves take the 64-token
// tiles of one split in turn, each with its own running maximum and sum, and are
// joined through LDS in a fixed order.  A wave loads the next tile's codes and
// scales before it multiplies this one's.
//
// Bound by bytes, and nearly as much by vector issue, where the cache is large:
// one query token of 64 sequences of 4096..8192 tokens, 64 query heads on 8 kv
// heads of 128, reads 418 MB of codes and scales in 86 us (4.9 TB/s; the median
// of launches in a row, 79 the least).  A short context is one wave's chain of
// loads and products: a sequence of 1000 tokens takes 9.5 us, two tiles a wave.
template <int D, int kWaves, bool kWide>
__global__ __launch_bounds__(kWaves * 64, kWaves == 4 ? 3 : 1) void kv4_attention_kernel(Kv4Attn a)
{
    constexpr int NG = D / 32;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int m = lane & 15, kg = lane >> 4;
    const int heads = a.geo.heads, group = a.q_heads / heads, T = a.tokens;
    const int h = blockIdx.x % heads, split = blockIdx.z;
    const int b = a.ranked ? sequence_of_rank<kWaves * kWave>(a, blockIdx.x / heads) : blockIdx.x / heads;
    const int rows = T * group, row0 = blockIdx.y * 16;

    const int len = context_length(a, b);
    const int row = min(row0 + m, rows - 1);
    const int t = row / group, hq = h * group + (row - t * group);
    // visible tokens of this lane's row: [jlo, jhi)
    const int pos = len - T + t;
    const int jhi = a.causal ? max(pos + 1, 0) : len;
    const int jlo = a.window > 0 ? max(pos - a.window + 1, 0) : 0;
    const Range see(a, len, group, row0, 16);
    const int tile0 = see.any_lo / 64, ntiles = see.any_hi > see.any_lo ? (see.any_hi + 63) / 64 - tile0 : 0;
    const int per = (ntiles + a.splits - 1) / a.splits;
    const int tile_end = tile0 + min(ntiles, (split + 1) * per);

    bf16x8 qf[NG];
    {
        const uint16_t *qp = a.q + b * a.q_seq + t * a.q_tok + hq * a.q_head + kg * (D / 4);
#pragma unroll
        for (int j = 0; j < NG; ++j) qf[j] = load_q(qp + 8 * j, a.scale);
    }
    const int32_t *table = a.table + b * a.table_stride;
    const float c = exponent_factor(a.scale);

    f32x4 oe[NG], oo[NG];  // even and odd dims
#pragma unroll
    for (int g = 0; g < NG; ++g) oe[g] = oo[g] = f32x4{0.f, 0.f, 0.f, 0.f};
    float mx = -INFINITY, sum = 0.f;

    const int bpp = a.geo.page >> 4;  // blocks in a page
    const int step_pages = 4 * kWaves / bpp, step_blocks = 4 * kWaves - step_pages * bpp;
    int tile = tile0 + split * per + wave;
    Place<kWide> kp, vp;  // of the next tile
    KTile<D, kWide> kt;
    VTile<D, kWide> vt;
    if (tile < tile_end) {
        kt.init(a.geo, h, m, kg);
        vt.init(a.geo, h, m, kg);
        kp.start(a, table, bpp, tile, m >> 2);
        vp.start(a, table, bpp, tile, kg);
        kt.load(a, kp, kg);
        vt.load(a, vp);
        kp.advance(a, table, step_pages, step_blocks, bpp);
        vp.advance(a, table, step_pages, step_blocks, bpp);
    }
    auto masked = [&](int t, bool ok) {
        return t * 64 < see.all_lo || t * 64 + 64 > see.all_hi || wave_any(!ok);
    };
    int wild_lo = INT_MAX, wild_hi = -1;  // masked tiles that wild scales were taken out of
    // Each operand's registers are loaded anew as soon as they are used: K of
    // the next tile is in flight during the softmax and the second product, V
    // during the first product, page numbers one tile longer.
    for (; tile < tile_end; tile += kWaves) {
        const bool more = tile + kWaves < tile_end;
        float x[16];  // tokens 16 kg + 0..15 of the tile
        scores<D, kWide>(kt, qf, m, kg, softmax_from(mx), x);
        if (more) {
            kt.load(a, kp, kg);
            kp.advance(a, table, step_pages, step_blocks, bpp);
        }

        const int first = tile * 64 + 16 * kg;  // the lane's first token
        if (masked(tile, vt.ok)) {
            const int lo = vt.ok ? jlo - first : 16, hi = jhi - first;
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = i >= lo && i < hi ? x[i] : -INFINITY;
            // V scales of tokens no row sees
            const int alo = vt.ok ? see.any_lo - first : 16, ahi = see.any_hi - first;
            uint32_t hits = 0;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const uint32_t keep = low_bytes(ahi - 4 * w) & ~low_bytes(alo - 4 * w);
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    uint32_t &v = word(vt.scales[g], w);
                    v &= keep;
                    const uint32_t wild = wild_bytes(v);
                    v &= ~wild;
                    word(vt.codes[g], w) &= ~wild;
                    hits |= wild;
                }
            }
            if (wave_any(hits != 0)) {
                wild_lo = min(wild_lo, tile);
                wild_hi = tile;
            }
        }

        bool moved;
        const float f = softmax_step(x, c, mx, sum, moved);
        if (moved) {
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                oe[g] *= f;
                oo[g] *= f;
            }
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const Weights p = weights_frag(x, s);
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                bf16x8 e, o;
                v_frags(word(vt.codes[g], 2 * s), word(vt.codes[g], 2 * s + 1), word(vt.scales[g], 2 * s),
                        word(vt.scales[g], 2 * s + 1), e, o);
                oe[g] = weigh(e, p, oe[g]);
                oo[g] = weigh(o, p, oo[g]);
            }
        }
        if (more) {
            vt.load(a, vp);
            vp.advance(a, table, step_pages, step_blocks, bpp);
        }
    }

    for (int t = wild_lo; t <= wild_hi; t += kWaves) {
        vp.start(a, table, bpp, t, kg);
        if (masked(t, vp.ok(a))) add_wild<D>(a, table, h, t, m, kg, qf, jlo, jhi, c, mx, oe, oo);
    }

    // join the waves: lane (m, kg) holds dims 32 g + 8 kg + 0..7 of row m
    constexpr int kPitch = D + 4;  // rows 4 banks apart
    __shared__ float so[kWaves][16][kPitch];
    __shared__ float sm[kWaves][16], sl[kWaves][16];
    sum = sum_over_kg(sum);
    if (kg == 0) {
        sm[wave][m] = mx * c;
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

// ---------------------------------------------------------------------------
// Many rows: eight waves of MT x 16 rows each share the tiles.  A tile's K and V
// are decoded once, an eighth by each wave, into LDS as whole matrix operands
// (1 KiB each, lane by lane, so that reads and writes are free of conflicts),
// two buffers deep: while a tile is multiplied the next is decoded, and the
// codes of the two after it are on their way from memory.  One barrier a tile.
//
// Bound by issue: 512 query tokens over 12..16 k cached tokens (2 sequences, 32
// query heads on 8 kv heads of 128; 234 GFLOP, 351 with the second product of
// the weights) take 327 us.  A tile costs a wave some 400 vector and 96 matrix
// instructions; most of the vector ones are the softmax's and the weights', of
// the same wave's chain of scores, softmax and second product, so that they add
// up to the products rather than run beside them (the matrix cores are busy 46 %
// of the time).  MT = 1: 376 us, where this takes 332.  Measured with one product
// for the weights, when this took 278: waves 4..7 half a tile behind the others
// (two barriers a tile) 342 us, one tile less in flight 291, no reads ahead of
// the products in LDS 308, addresses kept in scalar registers as the few-row
// kernel has them 284.
// ---------------------------------------------------------------------------
constexpr int kShareWaves = 8;

template <int D, int MT>
__global__ __launch_bounds__(kShareWaves * 64) void kv4_attention_rows_kernel(Kv4Attn a)
{
    constexpr int NG = D / 32, kHalf = (NG + 1) / 2;
    constexpr int kVRounds = (2 * NG + kShareWaves - 1) / kShareWaves;
    extern __shared__ __align__(16) uint4 shared_frags[];
    uint4 *const kf = shared_frags, *const vf = kf + 2 * 4 * NG * kWave;  // [buffer][frag][lane]
    __shared__ int wild_tiles[2][kShareWaves];  // masked tiles, first and last, that a wave took wild scales out of
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int m = lane & 15, kg = lane >> 4;
    const int heads = a.geo.heads, group = a.q_heads / heads, T = a.tokens;
    const int h = blockIdx.x % heads, b = blockIdx.x / heads, split = blockIdx.z;
    const int rows = T * group, block0 = blockIdx.y * (kShareWaves * MT * 16), row0 = block0 + wave * (MT * 16);

    const int len = context_length(a, b);
    const Range see(a, len, group, block0, kShareWaves * MT * 16);
    const int tile0 = see.any_lo / 64, ntiles = see.any_hi > see.any_lo ? (see.any_hi + 63) / 64 - tile0 : 0;
    const int per = (ntiles + a.splits - 1) / a.splits;
    const int begin = tile0 + split * per, end = tile0 + min(ntiles, (split + 1) * per);

    bf16x8 qf[MT][NG];
    int jlo[MT], jhi[MT];
    int64_t line[MT];
    const float c = exponent_factor(a.scale);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int row = min(row0 + 16 * i + m, rows - 1), t = row / group, hq = h * group + (row - t * group);
        const int pos = len - T + t;
        jhi[i] = a.causal ? max(pos + 1, 0) : len;
        jlo[i] = a.window > 0 ? max(pos - a.window + 1, 0) : 0;
        line[i] = ((int64_t)b * T + t) * a.q_heads + hq;
        const uint16_t *qp = a.q + b * a.q_seq + t * a.q_tok + hq * a.q_head + kg * (D / 4);
#pragma unroll
        for (int j = 0; j < NG; ++j) qf[i][j] = load_q(qp + 8 * j, a.scale);
    }
    f32x4 oe[MT][NG], oo[MT][NG];  // even and odd dims
    float mx[MT], sum[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        mx[i] = -INFINITY;
        sum[i] = 0.f;
#pragma unroll
        for (int g = 0; g < NG; ++g) oe[i][g] = oo[i][g] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    // This wave's share of a tile: K of tokens u = wave / 2, half the dwords;
    // V of (g, s) = (unit / 2, unit % 2), unit = wave + 8 r.
    const int32_t *table = a.table + b * a.table_stride;
    const int bpp = a.geo.page >> 4, step_pages = 4 / bpp, step_blocks = 4 - step_pages * bpp;
    const int ku = wave >> 1, kj = (wave & 1) * kHalf, kn = wave & 1 ? NG - kHalf : kHalf;
    const int rot = scale_rotation(m);
    Place<false> kp, vp;  // of the next tile
    struct Share {  // of one tile
        uint32_t kc[kHalf], ks[scale_sets(D)];
        uint2 vc[kVRounds], vs[kVRounds];
        bool v_ok;
    } share[2];
    // Past the last tile the loads find some page or none; what they bring is
    // not used.
    auto load = [&](Share &t) {
        {
            const uint8_t *base = kp.base(a);
            const uint8_t *p = base + a.geo.k_code(h, kp.in * 16 + 4 * ku + (m & 3)) + kg * (D / 8) + 4 * kj;
            if (NG % 2 == 0 || kn == kHalf) {
                const Words<kHalf> v = *reinterpret_cast<const Words<kHalf> *>(p);
#pragma unroll
                for (int j = 0; j < kHalf; ++j) t.kc[j] = v.w[j];
            } else {
#pragma unroll
                for (int j = 0; j < kHalf; ++j) t.kc[j] = j < kn ? reinterpret_cast<const uint32_t *>(p)[j] : 0u;
            }
            // the group of this wave's first dim of the lane, and the one after it
            const int g0 = D == 256 ? 2 * kg + (wave & 1) : kg * (D / 4) / 32;
            const uint8_t *sp = base + a.geo.k_scales() + a.geo.scale(h, kp.in * 16, g0) + 4 * ku;
            t.ks[0] = ld4<false>(sp);
            if constexpr (scale_sets(D) == 2) t.ks[1] = D == 256 ? t.ks[0] : ld4<false>(sp + (g0 + 1 < NG ? 16 : 0));
        }
        t.v_ok = vp.ok(a);
        const uint8_t *base = vp.base(a);
#pragma unroll
        for (int r = 0; r < kVRounds; ++r) {
            const int unit = wave + kShareWaves * r, g = unit >> 1, s = unit & 1;
            if (unit < 2 * NG) {
                t.vc[r] = ld8<false>(base + a.geo.v_codes() + a.geo.v_code(h, vp.in * 16, 16 * g + m) + 8 * s);
                t.vs[r] = ld8<false>(base + a.geo.v_scales() + a.geo.scale(h, vp.in * 16, g) + 8 * s);
            }
        }
        kp.advance(a, table, step_pages, step_blocks, bpp);
        vp.advance(a, table, step_pages, step_blocks, bpp);
    };
    auto masked = [&](int tile, bool ok) {
        return tile * 64 < see.all_lo || tile * 64 + 64 > see.all_hi || wave_any(!ok);
    };
    int wild_lo = INT_MAX, wild_hi = -1;
    auto decode = [&](Share &sh, int tile, int buf) {
#pragma unroll
        for (int j = 0; j < kHalf; ++j) {
            if (j < kn) {
                uint32_t w = sh.ks[0];
                if constexpr (scale_sets(D) == 2)
                    w = D == 256 || 8 * (kj + j) + kg * (D / 4) % 32 < 32 ? sh.ks[0] : sh.ks[1];
                const bf16x8 f = fp4_frag(sh.kc[j], __builtin_amdgcn_alignbit(w, w, rot));
                kf[((buf * 4 + ku) * NG + kj + j) * kWave + lane] = __builtin_bit_cast(uint4, f);
            }
        }
        const bool mask = masked(tile, sh.v_ok);
#pragma unroll
        for (int r = 0; r < kVRounds; ++r) {
            const int unit = wave + kShareWaves * r, s = unit & 1;
            if (unit < 2 * NG) {
                if (mask) {  // scales of tokens no row sees, and wild ones, leave the product
                    const int first = tile * 64 + 16 * kg + 8 * s;
                    const int lo = sh.v_ok ? see.any_lo - first : 8, hi = see.any_hi - first;
                    sh.vs[r].x &= low_bytes(hi) & ~low_bytes(lo);
                    sh.vs[r].y &= low_bytes(hi - 4) & ~low_bytes(lo - 4);
                    const uint32_t wild0 = wild_bytes(sh.vs[r].x), wild1 = wild_bytes(sh.vs[r].y);
                    sh.vs[r].x &= ~wild0;
                    sh.vs[r].y &= ~wild1;
                    sh.vc[r].x &= ~wild0;
                    sh.vc[r].y &= ~wild1;
                    if (wave_any((wild0 | wild1) != 0)) {
                        wild_lo = min(wild_lo, tile);
                        wild_hi = tile;
                    }
                }
                bf16x8 e, o;
                v_frags(sh.vc[r].x, sh.vc[r].y, sh.vs[r].x, sh.vs[r].y, e, o);
                uint4 *p = vf + ((buf * 2 * NG + unit) * 2) * kWave + lane;
                p[0] = __builtin_bit_cast(uint4, e);
                p[kWave] = __builtin_bit_cast(uint4, o);
            }
        }
    };

    bool ok = true, ok_next = true;  // of this lane's block of the tile multiplied, and of the next
    if (begin < end) {
        kp.start(a, table, bpp, begin, m >> 2);
        vp.start(a, table, bpp, begin, kg);
        load(share[0]);
        load(share[1]);
        ok_next = share[0].v_ok;
        decode(share[0], begin, 0);
        load(share[0]);
    }
    __syncthreads();
    const bool work = row0 < rows;  // a wave without rows only decodes
    auto step = [&](int tile, int buf) {
        ok = ok_next;
        if (tile + 1 < end) {
            ok_next = share[buf ^ 1].v_ok;
            decode(share[buf ^ 1], tile + 1, buf ^ 1);
            load(share[buf ^ 1]);
        }
        if (work) {
            float x[MT][16], from[MT];  // tokens 16 kg + 0..15 of the tile
#pragma unroll
            for (int i = 0; i < MT; ++i) from[i] = softmax_from(mx[i]);
            uint4 kk[2][NG], vv[2][4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (u == 0) {
#pragma unroll
                    for (int j = 0; j < NG; ++j) kk[0][j] = kf[((buf * 4) * NG + j) * kWave + lane];
                }
                if (u < 3) {
#pragma unroll
                    for (int j = 0; j < NG; ++j) kk[(u + 1) & 1][j] = kf[((buf * 4 + u + 1) * NG + j) * kWave + lane];
                }
                __builtin_amdgcn_sched_barrier(0);
                f32x4 acc[MT];
#pragma unroll
                for (int i = 0; i < MT; ++i) acc[i] = f32x4{-from[i], -from[i], -from[i], -from[i]};
#pragma unroll
                for (int j = 0; j < NG; ++j) {
                    const bf16x8 f = __builtin_bit_cast(bf16x8, kk[u & 1][j]);
#pragma unroll
                    for (int i = 0; i < MT; ++i) acc[i] = mfma(f, qf[i][j], acc[i]);
                }
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) x[i][4 * u + r] = acc[i][r];
            }
            if (masked(tile, ok)) {
                const int first = tile * 64 + 16 * kg;
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    const int lo = ok ? jlo[i] - first : 16, hi = jhi[i] - first;
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[i][e] = e >= lo && e < hi ? x[i][e] : -INFINITY;
                }
            }
            Weights p[MT][2];
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                bool moved;
                const float f = softmax_step(x[i], c, mx[i], sum[i], moved);
                if (moved) {
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        oe[i][g] *= f;
                        oo[i][g] *= f;
                    }
                }
                p[i][0] = weights_frag(x[i], 0);
                p[i][1] = weights_frag(x[i], 1);
            }
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                if (g == 0) {
#pragma unroll
                    for (int s = 0; s < 4; ++s) vv[0][s] = vf[(buf * 4 * NG + s) * kWave + lane];
                }
                if (g + 1 < NG) {
#pragma unroll
                    for (int s = 0; s < 4; ++s) vv[(g + 1) & 1][s] = vf[(buf * 4 * NG + 4 * g + 4 + s) * kWave + lane];
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const bf16x8 e = __builtin_bit_cast(bf16x8, vv[g & 1][2 * s]), o = __builtin_bit_cast(bf16x8, vv[g & 1][2 * s + 1]);
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        oe[i][g] = mfma(e, p[i][s].lo, oe[i][g]);
                        oo[i][g] = mfma(o, p[i][s].lo, oo[i][g]);
                    }
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        oe[i][g] = mfma(e, p[i][s].hi, oe[i][g]);
                        oo[i][g] = mfma(o, p[i][s].hi, oo[i][g]);
                    }
                }
            }
        }
        __syncthreads();
    };
    for (int tile = begin; tile < end; tile += 2) {
        step(tile, 0);
        if (tile + 1 < end) step(tile + 1, 1);
    }

    if (lane == 0) {
        wild_tiles[0][wave] = wild_lo;
        wild_tiles[1][wave] = wild_hi;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kShareWaves; ++w) {
        wild_lo = min(wild_lo, wild_tiles[0][w]);
        wild_hi = max(wild_hi, wild_tiles[1][w]);
    }
    for (int tile = wild_lo; tile <= wild_hi; ++tile) {
        vp.start(a, table, bpp, tile, kg);
        if (!masked(tile, vp.ok(a))) continue;
#pragma unroll
        for (int i = 0; i < MT; ++i) add_wild<D>(a, table, h, tile, m, kg, qf[i], jlo[i], jhi[i], c, mx[i], oe[i], oo[i]);
    }

    // lane (m, kg) holds dims 32 g + 8 kg + 0..7 of row m
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        if (row0 + 16 * i + m >= rows) continue;
        const float total = sum_over_kg(sum[i]), top = mx[i] * c;
        if (a.splits > 1) {
            const int64_t lines = (int64_t)a.seqs * T * a.q_heads;
            float *part = a.part + (split * lines + line[i]) * D + 8 * kg;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                *reinterpret_cast<f32x4 *>(part + 32 * g) = f32x4{oe[i][g][0], oo[i][g][0], oe[i][g][1], oo[i][g][1]};
                *reinterpret_cast<f32x4 *>(part + 32 * g + 4) = f32x4{oe[i][g][2], oo[i][g][2], oe[i][g][3], oo[i][g][3]};
            }
            if (kg == 0) {
                float *ml = a.part + a.splits * lines * D + (split * lines + line[i]) * 2;
                ml[0] = top;
                ml[1] = total;
            }
        } else {
            const float inv = total == 0.f ? 0.f : 1.0f / total;
            uint16_t *out = a.out + line[i] * D + 8 * kg;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const bf16x8 v = {(__bf16)(oe[i][g][0] * inv), (__bf16)(oo[i][g][0] * inv), (__bf16)(oe[i][g][1] * inv),
                                  (__bf16)(oo[i][g][1] * inv), (__bf16)(oe[i][g][2] * inv), (__bf16)(oo[i][g][2] * inv),
                                  (__bf16)(oe[i][g][3] * inv), (__bf16)(oo[i][g][3] * inv)};
                *reinterpret_cast<bf16x8 *>(out + 32 * g) = v;
            }
            if (a.lse && kg == 0) a.lse[line[i]] = (top + __builtin_log2f(total)) * kLn2;
        }
    }
}

constexpr int kMaxSplits = 128;

__device__ __forceinline__ uint2 bf16x4(f32x4 v)
{
    return make_uint2(bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]));
}

// Joins the splits of many rows: D / 4 lanes a row, four dims a lane.
template <int D>
__global__ __launch_bounds__(256) void kv4_join_rows_kernel(const float *__restrict__ part, int64_t lines,
                                                            int splits, uint16_t *__restrict__ out,
                                                            float *__restrict__ lse)
{
    constexpr int kLanes = D / 4, kRows = 256 / kLanes;
    const int d = threadIdx.x % kLanes, r = threadIdx.x / kLanes;
    const int64_t line = (int64_t)blockIdx.x * kRows + r;
    if (r >= kRows || line >= lines) return;
    const float2 *ml = reinterpret_cast<const float2 *>(part + splits * lines * D) + line;
    float top = -INFINITY;
    for (int s = 0; s < splits; ++s) top = fmaxf(top, ml[s * lines].x);
    const float base = top == -INFINITY ? 0.f : top;
    float total = 0.f;
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
    for (int s = 0; s < splits; ++s) {
        const float2 v = ml[s * lines];
        const float f = __builtin_amdgcn_exp2f(v.x - base);
        total += v.y * f;
        o += reinterpret_cast<const f32x4 *>(part + (s * lines + line) * D)[d] * f;
    }
    o *= total == 0.f ? 0.f : 1.0f / total;
    reinterpret_cast<uint2 *>(out + line * D)[d] = bf16x4(o);
    if (lse && d == 0) lse[line] = (top + __builtin_log2f(total)) * kLn2;
}

// Joins the splits of one row per workgroup: 256 / (D / 4) of them at a time,
// four dims a thread, then those groups through LDS.
template <int D>
__global__ __launch_bounds__(256) void kv4_join_kernel(const float *__restrict__ part, int64_t lines,
                                                       int splits, uint16_t *__restrict__ out,
                                                       float *__restrict__ lse)
{
    constexpr int kLanes = D / 4, kGroups = 256 / kLanes;
    const int64_t line = blockIdx.x;
    __shared__ float sm[kMaxSplits], sl[kMaxSplits];
    __shared__ f32x4 so[kGroups][kLanes];
    const int t = threadIdx.x, d = t % kLanes, group = t / kLanes;
    if (t < splits) {
        const float2 v = reinterpret_cast<const float2 *>(part + splits * lines * D)[t * lines + line];
        sm[t] = v.x;
        sl[t] = v.y;
    }
    __syncthreads();
    float top = -INFINITY;
    for (int s = 0; s < splits; ++s) top = fmaxf(top, sm[s]);
    const float base = top == -INFINITY ? 0.f : top;
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    if (group < kGroups) {
#pragma unroll 4
        for (int s = group; s < splits; s += kGroups) {
            const f32x4 v = reinterpret_cast<const f32x4 *>(part + (s * lines + line) * D)[d];
            o += v * __builtin_amdgcn_exp2f(sm[s] - base);
        }
        so[group][d] = o;
    }
    __syncthreads();
    if (t >= kLanes) return;
    float total = 0.f;
    for (int s = 0; s < splits; ++s) total += sl[s] * __builtin_amdgcn_exp2f(sm[s] - base);
    o = so[0][t];
#pragma unroll
    for (int i = 1; i < kGroups; ++i) o += so[i][t];
    o *= total == 0.f ? 0.f : 1.0f / total;
    reinterpret_cast<uint2 *>(out + line * D)[t] = bf16x4(o);
    if (lse && t == 0) lse[line] = (top + __builtin_log2f(total)) * kLn2;
}

// Waves of a workgroup of the few-row kernel.  Eight finish a sequence sooner
// and need fewer splits; four (three workgroups a CU up to 128 dims, whose
// beginnings and ends then overlap) do better once there are that many.  128
// sequences of 0..4096 tokens, 8 heads of 128: 75 us with eight, 62 with four; 96
// of 4096..8192: 125 and 115; 64 of them: 87 and 85; 48 of 0..8192: 48 and 61.
constexpr int kFewWaves = 8;
constexpr int64_t kManyGroups = 768;

// Row tiles of a wave of the many-row kernel.
constexpr int row_tiles(int dim, int64_t rows) { return dim <= 128 && rows > 128 ? 2 : 1; }

constexpr int64_t kCus = 256;

// Whether K and V are decoded once for all rows (query tokens x query heads of
// one kv head) and not for each 16 of them.  That takes 33 rows (49 up to 128
// dims) to pay, and more workgroups than half the CUs: with fewer, the context
// is split between them either way, and the few-row kernel's waves, which work
// alone, split it finer.  8 heads of 128, few rows' kernel and many rows', us:
// 32 sequences of 4096, 32 rows 58 and 86, 48 rows 75 and 86, 64 rows 98 and 86;
// one of 8192, 64 rows 14 and 21, 128 rows (64 workgroups) 19 and 29, 512 rows
// (256) 42 and 50; four of 16384, 128 rows (256) 81 and 71.  32 sequences of 4096
// with heads of 256: 32 rows 113 and 131, 36 rows 170 and 133; of 192: 32 rows 77
// and 113, 48 rows 114 and 115; of 64: 48 rows 43 and 73, 64 rows 54 and 74, where
// the rule is early, as it is with 96: 64 rows 77 and 84.  Five of 8192 with heads
// of 256, 48 rows (120 workgroups): 51 and 58.
constexpr bool many_rows(int dim, int64_t rows, int64_t heads)
{
    return rows > (dim <= 128 ? 48 : 32) && (rows + 15) / 16 * heads > kCus / 2;
}

template <int D, int MT>
hipError_t go_rows(const Kv4Attn &a, int64_t rows, hipStream_t stream)
{
    const int64_t gx = (int64_t)a.seqs * a.geo.heads, gy = (rows + kShareWaves * MT * 16 - 1) / (kShareWaves * MT * 16);
    const dim3 grid((unsigned)gx, (unsigned)gy, (unsigned)a.splits), block(kShareWaves * kWave);
    constexpr unsigned lds = 2 * 8 * (D / 32) * kWave * sizeof(uint4);
    hipLaunchKernelGGL((kv4_attention_rows_kernel<D, MT>), grid, block, lds, stream, a);
    return hipGetLastError();
}

template <int D, int kWaves>
hipError_t go_few(const Kv4Attn &a, int64_t gx, int64_t gy, hipStream_t stream)
{
    Kv4Attn ordered = a;
    ordered.ranked = a.seqs > 1 && a.seqs <= kRanked && gx * gy * a.splits > kCus;
    const dim3 grid((unsigned)gx, (unsigned)gy, (unsigned)a.splits), block(kWaves * kWave);
    if (a.geo.page % 64 == 0)
        hipLaunchKernelGGL((kv4_attention_kernel<D, kWaves, true>), grid, block, 0, stream, ordered);
    else
        hipLaunchKernelGGL((kv4_attention_kernel<D, kWaves, false>), grid, block, 0, stream, ordered);
    return hipGetLastError();
}

template <int D>
hipError_t go(const Kv4Attn &a, hipStream_t stream)
{
    const int64_t rows = (int64_t)a.tokens * (a.q_heads / a.geo.heads);
    const int64_t gx = (int64_t)a.seqs * a.geo.heads;
    const int64_t lines = gx * rows;
    hipError_t e;
    if (many_rows(D, rows, gx)) {
        e = row_tiles(D, rows) == 2 ? go_rows<D, D <= 128 ? 2 : 1>(a, rows, stream) : go_rows<D, 1>(a, rows, stream);
    } else {
        const int64_t gy = (rows + 15) / 16;
        e = D <= 128 && gx * gy * a.splits >= kManyGroups ? go_few<D, D <= 128 ? 4 : kFewWaves>(a, gx, gy, stream)
                                                          : go_few<D, kFewWaves>(a, gx, gy, stream);
    }
    if (e != hipSuccess || a.splits == 1) return e;
    // Few rows, or many splits, are joined in parallel; many rows fill the GPU
    // without that.  A workgroup a row and D / 4 lanes a row measured (D = 128)
    // 22.4 and 8.0 us for 32768 rows of 2 splits, 4.3 and 3.6 for 4096 of 8,
    // 13.3 and 18.0 for 4096 of 32, 3.6 and 3.6 for 2048 of 4.
    constexpr int64_t kRows = 256 / (D / 4);
    if (lines >= 16 * kCus && a.splits <= 8)
        hipLaunchKernelGGL((kv4_join_rows_kernel<D>), dim3((unsigned)((lines + kRows - 1) / kRows)), dim3(256), 0,
                           stream, a.part, lines, a.splits, a.out, a.lse);
    else
        hipLaunchKernelGGL((kv4_join_kernel<D>), dim3((unsigned)lines), dim3(256), 0, stream, a.part, lines,
                           a.splits, a.out, a.lse);
    return hipGetLastError();
}

}  // namespace

// Splitting the context fills the CUs when there are few rows, but costs a
// second launch and the partial sums, in all about the time of three or four
// tiles (2 us each, alone): up to four tiles a wave there is one split, else no
// less than one tile for a wave (with many rows, eight for the workgroup).
// Seven sequences that see 1088 tokens: 8.6 us, 9.5 with two splits.  All
// workgroups run at once: one more than a CU each costs a second round (seven
// sequences of 8192, 8 heads of 128: 19.3 us with 4 splits, 27.0 with 5).
int32_t kv4_attention_splits(int64_t seqs, int64_t tokens, int64_t q_heads, int64_t kv_heads,
                             int64_t dim, int64_t page, int64_t width, int64_t window)
{
    const int64_t rows = tokens * (q_heads / kv_heads);
    // enough workgroups as it is, whatever the tiles (and no product below overflows)
    if (seqs * kv_heads > kCus || rows > kCus * 256) return 1;
    const bool many = many_rows((int)dim, rows, seqs * kv_heads);
    const int64_t tile = many ? kShareWaves * row_tiles((int)dim, rows) * 16 : 16;
    const int64_t groups = (rows + tile - 1) / tile * seqs * kv_heads;
    int64_t seen = width * page;
    if (window > 0 && window + tokens + 64 < seen) seen = window + tokens + 64;
    const int64_t fill = kCus / groups;
    const int64_t tiles = (seen + 63) / 64;
    const int64_t most = many ? tiles / 8 : tiles > 4 * kFewWaves ? tiles / kFewWaves : 1;
    const int64_t s = fill < most ? fill : most;
    return (int32_t)(s < 1 ? 1 : s > kMaxSplits ? kMaxSplits : s);
}

int64_t kv4_attention_most_rows(int64_t dim)
{
    return 65535 * (int64_t)(kShareWaves * row_tiles((int)dim, INT_MAX) * 16);  // as many strips as a grid's y holds
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
