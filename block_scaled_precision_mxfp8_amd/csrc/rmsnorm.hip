// rmsnorm.hip -- RMS norm with the residual's addition and 8-bit output, and its
// gradient, for gfx950.
//
//   h = bf16(x + residual),  r = (mean(h^2) + eps)^-1/2,  y = h * r * weight
//
// y, in fp32, is quantized as it stands: block-FP8 (one fp32 scale for 128 values, as
// blockfp8_quantize_1x128) or MXFP8 (E8M0 for 32, as mxq_quantize_rowwise).  It is not
// rounded to bf16 first, so codes can differ from those of a separate norm and
// quantizer by that rounding.  Gradient, u = h * r, g = dy * weight:
//   dx = r * (g - u * mean(g * u)) + dh,  dweight = sum over the rows of dy * u
// (the quantizer counts as the identity).  Sums are of 8 values of a lane in fp32, then
// over lanes and waves in a fixed order, in fp64 for the norm and fp32 for the gradient;
// rows whose squares leave fp32 (below 2^-45 or from 2^62 on) are summed in fp64 throughout.
//
// Bound by bytes: the norm reads 4 and writes 3 for a value (h, q), the gradient reads 6
// and writes 2.  So a row is read once and stays in registers from the sum to the
// output, up to 32 values a lane, and as few waves share it as hold it: their sum costs a
// barrier.  Rows stream past the caches (non-temporal): 16384 x 7168 with residual 146 us
// (5.7 TB/s) where ordinary accesses took 157, the gradient 164 (5.7 TB/s) where 183; of what
// that does to the kernel that reads them next, and to small batches, nothing is measured.
// One row is a chain of latencies, 6.2 us of which a launch is 3.9: four pieces of x and the
// residual, each pair waited for before the next is asked for, the sum over lanes and a
// barrier, then four pieces of the weight, again one after the other.

#include "launch.hpp"
#include "mxq_device.hpp"

namespace mxq {

namespace {

constexpr int kVecs = 4;  // most 16-byte pieces a lane holds

struct Row8 { float f[8]; };

__device__ __forceinline__ Row8 floats(uint4 v)
{
    return Row8{{bf16lo_to_f32(v.x), bf16hi_to_f32(v.x), bf16lo_to_f32(v.y), bf16hi_to_f32(v.y),
                 bf16lo_to_f32(v.z), bf16hi_to_f32(v.z), bf16lo_to_f32(v.w), bf16hi_to_f32(v.w)}};
}

__device__ __forceinline__ uint4 bf16s(const Row8 &r)
{
    return make_uint4(bf16x2_rne(r.f[0], r.f[1]), bf16x2_rne(r.f[2], r.f[3]),
                      bf16x2_rne(r.f[4], r.f[5]), bf16x2_rne(r.f[6], r.f[7]));
}

template <bool kF32>
__device__ __forceinline__ Row8 weights8(const void *w, int64_t col)
{
    if constexpr (kF32) {
        const float *p = static_cast<const float *>(w) + col;
        const uint4 a = ld16<false>(p), b = ld16<false>(p + 4);
        return Row8{{__uint_as_float(a.x), __uint_as_float(a.y), __uint_as_float(a.z),
                     __uint_as_float(a.w), __uint_as_float(b.x), __uint_as_float(b.y),
                     __uint_as_float(b.z), __uint_as_float(b.w)}};
    } else {
        return floats(ld16<false>(static_cast<const uint16_t *>(w) + col));
    }
}

// Sum over the kWaves waves of a row, the same in all of them.  `slot` alternates so
// that one barrier a sum is enough.
template <int kWaves, class F>
__device__ __forceinline__ F row_sum(F v, F (*red)[8], int slot)
{
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) v += __shfl_xor(v, off, kWave);
    if constexpr (kWaves > 1) {
        const int wave = threadIdx.x / kWave;
        if ((threadIdx.x & (kWave - 1)) == 0) red[slot][wave] = v;
        __syncthreads();
        const int first = wave / kWaves * kWaves;
        v = red[slot][first];
#pragma unroll
        for (int i = 1; i < kWaves; ++i) v += red[slot][first + i];
    }
    return v;
}

// v^-1/2 in 64 bits: a Newton step from the 32-bit approximation doubles its bits.
__device__ __forceinline__ double inverse_root(double v)
{
    if (!(v >= 0x1p-100 && v <= 0x1p100)) return 1.0 / __builtin_sqrt(v);
    const double y = __builtin_amdgcn_rsqf((float)v);
    return y * __builtin_fma(-0.5 * v * y, y, 1.5);
}

// Largest magnitude's bits over groups of 16 lanes.
__device__ __forceinline__ uint32_t max16(uint32_t v)
{
    v = quad_max(v);
    v = max(v, (uint32_t)__shfl_xor((int)v, 4, kWave));
    return max(v, (uint32_t)__shfl_xor((int)v, 8, kWave));
}

__device__ __forceinline__ uint32_t signs_of(const float *f)
{
    uint32_t s = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) s |= (__float_as_uint(f[i]) >> 31) << (8 * i + 7);
    return s;
}

// kWaves waves on a row; a workgroup has at least four.  Seven waves to a SIMD: with
// registers for five or six 160 us (16384 x 7168, ordinary accesses), for seven 157, for
// eight, spilling, 178; held to five or four workgroups a CU 156 and 173 where 146.  (fp32
// weights with MXFP8 spill one or two registers of it: 150 us.)
template <bool kMX, int kWaves, bool kWeightF32>
__global__ __launch_bounds__(kWaves < 4 ? 256 : kWaves * 64, 7) void rmsnorm_kernel(RmsNorm a)
{
    constexpr int kThreads = kWaves < 4 ? 256 : kWaves * 64, kRows = kThreads / (kWaves * 64);
    __shared__ double red[1][8];
    const int in_row = threadIdx.x % (kWaves * 64);
    const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / (kWaves * 64);
    const bool live = row < a.rows;
    uint4 v[kVecs];
    double sum = 0;
    bool far = false;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int64_t col = (int64_t)(i * kWaves * 64 + in_row) * 8;
        v[i] = make_uint4(0, 0, 0, 0);
        if (live && col < a.cols) {
            v[i] = ld16<true>(a.x + row * a.ldx + col);
            if (a.residual) {
                const Row8 p = floats(v[i]), q = floats(ld16<true>(a.residual + row * a.ldr + col));
                Row8 s;
#pragma unroll
                for (int j = 0; j < 8; ++j) s.f[j] = p.f[j] + q.f[j];
                v[i] = bf16s(s);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int64_t col = (int64_t)(i * kWaves * 64 + in_row) * 8;
        if (a.h && live && col < a.cols) st16<true>(a.h + row * a.cols + col, v[i]);
        const Row8 f = floats(v[i]);
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) s = __builtin_fmaf(f.f[j], f.f[j], s);
        sum += s;
        far |= live && col < a.cols && !(s >= 0x1p-90f && s < __builtin_inff());
    }
    if (wave_any(far)) {  // squares that leave fp32
        sum = 0;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const Row8 f = floats(v[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = __builtin_fma((double)f.f[j], (double)f.f[j], sum);
        }
    }
    // r is held in two floats and r * weight too: y is rounded about once, so that few
    // codes and hardly a scale fall to the other side of a border.
    double root = inverse_root(row_sum<kWaves>(sum, red, 0) / (double)a.cols + (double)a.eps);
    if (a.rstd && live && in_row == 0) a.rstd[row] = (float)root;
    // A root past 2^60 either way hands its power of two to the values, which it brings near 1:
    // so neither it nor its product with a weight leaves fp32.
    int lift = 0;
    if (wave_any(root > 0 && root < __builtin_inf() && !(root >= 0x1p-60 && root <= 0x1p60))) {
        lift = __builtin_amdgcn_readfirstlane(__builtin_amdgcn_frexp_exp(root));  // a wave has one row
        root = __builtin_amdgcn_ldexp(root, -lift);
    }
    const float r = (float)root, r_low = r < __builtin_inff() ? (float)(root - (double)r) : 0.f;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int64_t col = (int64_t)(i * kWaves * 64 + in_row) * 8;
        if (i * kWaves * 512 >= a.cols) break;
        const bool in = live && col < a.cols;
        Row8 y = floats(v[i]);
        if (lift != 0) {
#pragma unroll
            for (int j = 0; j < 8; ++j) y.f[j] = __builtin_amdgcn_ldexpf(y.f[j], lift);
        }
        const Row8 w = in ? weights8<kWeightF32>(a.weight, col) : Row8{};
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float t = r * w.f[j];
            const float low = __builtin_fabsf(t) < __builtin_inff()
                                  ? __builtin_fmaf(r, w.f[j], -t) + r_low * w.f[j] : 0.f;
            y.f[j] = __builtin_fmaf(y.f[j], t, y.f[j] * low);
            if (!in) y.f[j] = 0.f;
            m = max(m, __float_as_uint(y.f[j]) & 0x7FFFFFFFu);
        }
        if (a.y && in) st16<true>(a.y + row * a.cols + col, bf16s(y));
        uint2 c;
        if constexpr (kMX) {
            m = quad_max(m);
            // What y lost when it was rounded to 32 bits counts where y has come to lie
            // on a border: then it is worked out again, seldom and in few registers.
            auto rest = [&](int j) {  // above 0: the magnitude of value j is larger than y has it
                const uint32_t pair = j < 2 ? v[i].x : j < 4 ? v[i].y : j < 6 ? v[i].z : v[i].w;
                const float x = __builtin_amdgcn_ldexpf(j & 1 ? bf16hi_to_f32(pair) : bf16lo_to_f32(pair), lift);
                const float wj = kWeightF32 ? static_cast<const float *>(a.weight)[col + j]
                                            : bf16lo_to_f32(static_cast<const uint16_t *>(a.weight)[col + j]);
                const float t = r * wj, low = __builtin_fmaf(r, wj, -t) + r_low * wj;
                const float yj = __builtin_fmaf(x, t, x * low);
                return (__builtin_fmaf(x, t, -yj) + x * low) * __builtin_copysignf(1.0f, yj);
            };
            // a largest value just below a power of two, rounded up to it, keeps the lower scale
            uint32_t below = 0;
            const bool power = (m & 0x7FFFFFu) == 0 && m != 0 && m < 0x7F800000u;
            if (wave_any(power)) {
                uint32_t reached = 0;  // some value is that power or more
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (in && (__float_as_uint(y.f[j]) & 0x7FFFFFFFu) == m && rest(j) >= 0.f) reached = 1;
                below = power && quad_max(reached) == 0;
            }
            const uint32_t e = (m >> 23) - below, s = e >= 0xFFu ? 0xFFu : e > 8u ? e - 8u : 0u;
            Row8 t;
#pragma unroll
            for (int j = 0; j < 8; ++j) t.f[j] = __builtin_amdgcn_ldexpf(y.f[j], 127 - (int)s);
            // halfway between two codes, as rounded: to the side where it was
            uint32_t halfway = ~0u;
#pragma unroll
            for (int j = 0; j < 8; ++j) halfway = min(halfway, (__float_as_uint(t.f[j]) << 12) + 0x80000000u);
            if (wave_any(halfway == 0)) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (in && s != 0xFFu && __float_as_uint(t.f[j]) << 12 == 0x80000000u) {
                        const float o = rest(j);
                        t.f[j] = __uint_as_float(__float_as_uint(t.f[j]) + (o > 0.f ? 1u : o < 0.f ? ~0u : 0u));
                    }
            }
            c.x = cvt_fp8x2_f32<true>(cvt_fp8x2_f32<false>(0u, t.f[0], t.f[1]), t.f[2], t.f[3]);
            c.y = cvt_fp8x2_f32<true>(cvt_fp8x2_f32<false>(0u, t.f[4], t.f[5]), t.f[6], t.f[7]);
            if (s == 0xFFu) c = make_uint2(0x7F7F7F7Fu | signs_of(y.f), 0x7F7F7F7Fu | signs_of(y.f + 4));
            if (in && (in_row & 3) == 0)
                static_cast<uint8_t *>(a.scale)[row * (a.cols / 32) + col / 32] = (uint8_t)s;
        } else {
            m = max16(m);
            const bool bad = m >= 0x7F800000u;
            const float S = bad ? __builtin_nanf("") : __uint_as_float(m) / 448.0f;
            const float d = S == 0.f || bad ? 1.0f : S;
            Row8 t;
            if (!wave_any(!markstein_ok(d))) {
                const float inv = 1.0f / d;
#pragma unroll
                for (int j = 0; j < 8; ++j) t.f[j] = div_markstein(y.f[j], d, inv);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) t.f[j] = y.f[j] / d;
            }
            c.x = cvt_fp8x2_f32<true>(cvt_fp8x2_f32<false>(0u, t.f[0], t.f[1]), t.f[2], t.f[3]);
            c.y = cvt_fp8x2_f32<true>(cvt_fp8x2_f32<false>(0u, t.f[4], t.f[5]), t.f[6], t.f[7]);
            if (bad) c = make_uint2(0x7F7F7F7Fu | signs_of(y.f), 0x7F7F7F7Fu | signs_of(y.f + 4));
            if (in && (in_row & 15) == 0)
                static_cast<float *>(a.scale)[row * ((a.cols + 127) / 128) + col / 128] = S;
        }
        if (in) st8<true>(a.q + row * a.cols + col, c);
    }
}

// Each workgroup takes every gridDim.x-th group of rows; what its rows give dweight
// stays in registers and leaves as one partial row.  512 workgroups: 768 took 180 us for
// 16384 x 7168 and 1024 172, where 512 take 165.
template <int kWaves, bool kWeightF32>
__global__ __launch_bounds__(kWaves < 4 ? 256 : kWaves * 64) void rmsnorm_back_kernel(RmsNormBack a)
{
    constexpr int kThreads = kWaves < 4 ? 256 : kWaves * 64, kRows = kThreads / (kWaves * 64);
    __shared__ float red[2][8];
    const int in_row = threadIdx.x % (kWaves * 64);
    Row8 w[kVecs], dw[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int64_t col = (int64_t)(i * kWaves * 64 + in_row) * 8;
        w[i] = col < a.cols ? weights8<kWeightF32>(a.weight, col) : Row8{};
        dw[i] = Row8{};
    }
    int slot = 0;
    const int64_t groups = (a.rows + kRows - 1) / kRows;
    for (int64_t g = blockIdx.x; g < groups; g += gridDim.x, slot ^= 1) {
        const int64_t row = g * kRows + threadIdx.x / (kWaves * 64);
        const bool live = row < a.rows;
        uint4 dy[kVecs], h[kVecs], dh[kVecs];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int64_t col = (int64_t)(i * kWaves * 64 + in_row) * 8;
            dy[i] = h[i] = dh[i] = make_uint4(0, 0, 0, 0);
            if (live && col < a.cols) {
                dy[i] = ld16<true>(a.dy + row * a.ld_dy + col);
                h[i] = ld16<true>(a.h + row * a.ldh + col);
                if (a.dh) dh[i] = ld16<true>(a.dh + row * a.ld_dh + col);
            }
        }
        const float r = live ? a.rstd[row] : 0.f;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const Row8 d = floats(dy[i]), x = floats(h[i]);
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float u = x.f[j] * r;
                dw[i].f[j] = __builtin_fmaf(d.f[j], u, dw[i].f[j]);
                s = __builtin_fmaf(d.f[j] * w[i].f[j], u, s);
            }
            sum += s;
        }
        const float mean = row_sum<kWaves>(sum, red, slot) / (float)a.cols;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int64_t col = (int64_t)(i * kWaves * 64 + in_row) * 8;
            const Row8 d = floats(dy[i]), x = floats(h[i]), add = floats(dh[i]);
            Row8 o;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float u = x.f[j] * r;
                o.f[j] = __builtin_fmaf(d.f[j] * w[i].f[j] - u * mean, r, add.f[j]);
            }
            if (live && col < a.cols) st16<true>(a.dx + row * a.cols + col, bf16s(o));
        }
    }
    // rows of one workgroup side by side: each leaves a partial row of its own
    float *part = a.part + ((int64_t)blockIdx.x * kRows + threadIdx.x / (kWaves * 64)) * a.cols;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int64_t col = (int64_t)(i * kWaves * 64 + in_row) * 8;
        if (col < a.cols) {
            *reinterpret_cast<float4 *>(part + col) = make_float4(dw[i].f[0], dw[i].f[1], dw[i].f[2], dw[i].f[3]);
            *reinterpret_cast<float4 *>(part + col + 4) = make_float4(dw[i].f[4], dw[i].f[5], dw[i].f[6], dw[i].f[7]);
        }
    }
}

// dweight from the partial rows: a workgroup has 64 columns, its waves every 16th row.
__global__ __launch_bounds__(1024) void rmsnorm_dweight_kernel(const float *__restrict__ part, int32_t parts,
                                                               int64_t cols, float *__restrict__ dweight)
{
    __shared__ float red[16][kWave];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int64_t col = (int64_t)blockIdx.x * kWave + lane;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    if (col < cols) {
        int p = wave;
        for (; p + 48 < parts; p += 64)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i] += part[(int64_t)(p + 16 * i) * cols + col];
        for (; p < parts; p += 16) s[0] += part[(int64_t)p * cols + col];
    }
    red[wave][lane] = (s[0] + s[1]) + (s[2] + s[3]);
    __syncthreads();
    if (wave == 0 && col < cols) {
        float v = red[0][lane];
#pragma unroll
        for (int i = 1; i < 16; ++i) v += red[i][lane];
        dweight[col] = v;
    }
}

// Waves on a row: as few as hold it.
int waves_for(int64_t cols)
{
    int w = 1;
    while ((int64_t)w * 64 * 8 * kVecs < cols) w *= 2;
    return w;
}

}  // namespace

static_assert(kRmsNormMostCols == 8 * 64 * 8 * kVecs, "8 waves hold the longest row");

int32_t rmsnorm_back_parts(int64_t rows, int64_t cols)
{
    const int w = waves_for(cols), per = w < 4 ? 4 / w : 1;
    const int64_t groups = (rows + per - 1) / per;
    return (int32_t)(groups < 512 ? groups : 512) * per;
}

hipError_t launch_rmsnorm(bool mx, const RmsNorm &a, hipStream_t stream)
{
    const int w = waves_for(a.cols), per = w < 4 ? 4 / w : 1;
    auto go = [&](auto MX, auto W, auto F) {
        constexpr int kThreads = W < 4 ? 256 : W * 64;
        const int64_t most = ((int64_t)1 << 31) / kThreads * per;  // rows of one launch, whose threads 32 bits count
        for (int64_t first = 0; first < a.rows; first += most) {
            RmsNorm b = a;
            b.rows = a.rows - first < most ? a.rows - first : most;
            b.x += first * a.ldx;
            if (a.residual) b.residual += first * a.ldr;
            b.q += first * a.cols;
            if (MX) b.scale = static_cast<uint8_t *>(a.scale) + first * (a.cols / 32);
            else b.scale = static_cast<float *>(a.scale) + first * ((a.cols + 127) / 128);
            if (a.h) b.h += first * a.cols;
            if (a.y) b.y += first * a.cols;
            if (a.rstd) b.rstd += first;
            rmsnorm_kernel<MX, W, F><<<dim3((unsigned)((b.rows + per - 1) / per)), dim3(kThreads), 0, stream>>>(b);
        }
    };
    auto by_waves = [&](auto MX, auto F) {
        switch (w) {
        case 1: go(MX, std::integral_constant<int, 1>{}, F); break;
        case 2: go(MX, std::integral_constant<int, 2>{}, F); break;
        case 4: go(MX, std::integral_constant<int, 4>{}, F); break;
        default: go(MX, std::integral_constant<int, 8>{}, F); break;
        }
    };
    if (mx) a.weight_f32 ? by_waves(std::true_type{}, std::true_type{}) : by_waves(std::true_type{}, std::false_type{});
    else a.weight_f32 ? by_waves(std::false_type{}, std::true_type{}) : by_waves(std::false_type{}, std::false_type{});
    return hipGetLastError();
}

hipError_t launch_rmsnorm_back(const RmsNormBack &a, hipStream_t stream)
{
    const int w = waves_for(a.cols), per = w < 4 ? 4 / w : 1;
    const int32_t parts = rmsnorm_back_parts(a.rows, a.cols);
    auto go = [&](auto W, auto F) {
        rmsnorm_back_kernel<W, F><<<dim3(parts / per), dim3(W < 4 ? 256 : W * 64), 0, stream>>>(a);
    };
    auto by_waves = [&](auto F) {
        switch (w) {
        case 1: go(std::integral_constant<int, 1>{}, F); break;
        case 2: go(std::integral_constant<int, 2>{}, F); break;
        case 4: go(std::integral_constant<int, 4>{}, F); break;
        default: go(std::integral_constant<int, 8>{}, F); break;
        }
    };
    if (parts > 0) {  // no rows: only dweight's zeros
        a.weight_f32 ? by_waves(std::true_type{}) : by_waves(std::false_type{});
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    rmsnorm_dweight_kernel<<<dim3((unsigned)((a.cols + 63) / 64)), dim3(1024), 0, stream>>>(a.part, parts, a.cols,
                                                                                         a.dweight);
    return hipGetLastError();
}

}  // namespace mxq
