// fp8_few.hip -- products of a few 8-bit tokens with 8-bit weights for gfx950: the
// formulas and operand layouts of fp8_tiles.hip, for where reading the weights is the
// work.
//
// A workgroup has 16 R weight rows and up to 16 T tokens; its waves cut the
// contraction, each a run of whole steps of 128, and their sums are joined in LDS in a
// fixed order.  A wave brings weights and tokens to a ring of steps of its own in LDS,
// straight from memory in whole lines, D - 1 steps ahead, and needs no barrier.
// (Loaded to registers in operand order, 16 neighbouring lanes touch 16 lines, which
// the load path takes a clock for each; and few bytes would be under way.)
//
// v_mfma_f32_16x16x128_f8f6f4: lane (p, g) = (lane % 16, lane / 16) holds of row p
// the bytes k = 16 g .. and 64 + 16 g .., the scale of its group 32 g .., and of the
// result column p in rows 4 g + 0..3.  fp32 results go through
// v_mfma_f32_16x16x32_bf16, eight bytes of a lane at a time.
//
// Bound by the weights' bytes where there are many: 512 rows of 128 groups of 2048 x 7168
// 246 to 261 us, 7.2 to 7.6 TB/s.  A single small product is latency: 1 x 2048 x 7168 takes
// 6.6 us, of which a launch is 3.9.  Then a wave waits for the scales of its tokens and
// weight rows, R + T loads one after the other (each is shifted, and so waited for, before
// the next; scale rows of less than 16 bytes come byte by byte), before it asks for the
// first weights; and its seven steps come two at a time.

#include "fp8_matmul.hpp"
#include "launch.hpp"

namespace mxq {

namespace {

constexpr int kScaleSteps = 16;  // steps whose scales a wave holds at a time

template <bool kMX, bool kExact, int kRagged, int R, int T, int W, int D>
__global__ __launch_bounds__(W * 64) void few_kernel(Fp8Matmul a)
{
    constexpr int kLoads = 2 * (R + T);          // of 8 rows, for each step
    constexpr int kSlot = kLoads * 1024;
    static_assert((D - 1) * kLoads < 64, "what vmcnt counts");
    constexpr int kOut = R * 16;                 // columns of y
    static_assert(128 % kOut == 0, "in one tile of block-FP8's scales");
    constexpr int kRing = W * D * kSlot, kJoin = W * T * 16 * kOut * 4;
    constexpr int kFar = kMX ? 0 : W * 4;        // a word of each wave
    __shared__ __align__(1024) uint8_t lds[kRing > kJoin + kFar ? kRing : kJoin + kFar];

    int group = 0;
    int32_t row0 = blockIdx.y * (T * 16), row_end = min(row0 + T * 16, a.m);
    if constexpr (kRagged == kRows) {
        if (!find_row_tile(a, T * 16, blockIdx.y, group, row0, row_end)) return;
    }
    const int32_t col0 = blockIdx.x * kOut, col_end = min(col0 + kOut, a.n);
    const int lane = threadIdx.x & 63, p = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int32_t steps = (a.k + kStep - 1) / kStep;
    const int32_t s0 = (int32_t)((int64_t)steps * wave / W), s1 = (int32_t)((int64_t)steps * (wave + 1) / W);

    const uint8_t *x = a.x + (int64_t)row0 * a.ldx;
    const uint8_t *w = a.w + (kRagged == kRows ? group * a.w_stride : 0) + (int64_t)col0 * a.ldw;
    const int xlast = row_end - row0 - 1, wlast = col_end - col0 - 1;  // rows past them repeat them
    const uint32_t chunk = (lane & 7) ^ (lane >> 4);  // as in fp8_tiles.hip
    uint32_t voff[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int r = i * 8 + (lane >> 3);
        voff[i] = (i < 2 * R ? (uint32_t)min(r, wlast) * (uint32_t)a.ldw
                             : (uint32_t)min(r - R * 16, xlast) * (uint32_t)a.ldx) + (chunk ^ (i & 1) * 4) * 16;
    }
    const __amdgpu_buffer_rsrc_t wr = buffer_at(w), xr = buffer_at(x);
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;
    auto fill = [&](int32_t s) {
        const uint32_t to = (wave * D + (s - s0) % D) * kSlot;
        const uint32_t from = (uint32_t)s * kStep;
        // k % 16 == 0; what lies past it is zero
        const uint32_t past[2] = {(int32_t)(from + chunk * 16) < a.k ? 0u : kNowhere,
                                  (int32_t)(from + (chunk ^ 4) * 16) < a.k ? 0u : kNowhere};
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            load_to_lds(i < 2 * R ? wr : xr, lds0 + to + i * 1024, voff[i] | past[i & 1], from);
    };

    // -- scales of kScaleSteps steps from s on: lane (p, g) has row p's of steps 4 g ..
    // 4 g + 3, a dword each
    uint32_t sx[T][4], sw[R][4];
    auto load4 = [&](uint32_t(&d)[4], const void *base, int64_t at, int32_t s) {  // element `at` is the row's first
        const uint8_t *row = static_cast<const uint8_t *>(base) + at * (kMX ? 1 : 4);
        const uint4 v = bytes16_of(row, (s + 4 * g) * 4, kMX ? a.k / 32 : steps * 4);
        d[0] = v.x, d[1] = v.y, d[2] = v.z, d[3] = v.w;
    };
    // Block-FP8: two scales within 2^-63 .. 2^63 have a product in fp32; are there others?
    // Zeros (all there is behind the last step) have one too.
    uint32_t least = ~0u, most = 0;
    auto note = [&](const uint32_t(&d)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            least = min(least, (d[i] << 1) - 1u);
            most = max(most, d[i] << 1);
        }
    };
    auto load_scales = [&](int32_t s) {
#pragma unroll
        for (int t = 0; t < T; ++t) {
            load4(sx[t], a.sx, (int64_t)(row0 + min(t * 16 + p, xlast)) * a.ld_sx, s);
            if constexpr (!kMX) note(sx[t]);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = col0 + min(r * 16 + p, wlast);
            load4(sw[r], a.sw, (kRagged == kRows ? group * a.sw_stride : 0) + (int64_t)(kMX ? c : c / 128) * a.ld_sw, s);
        }
        if constexpr (!kMX) note(sw[0]);  // that of all rows here
    };

    f32x4 acc[R][T];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < T; ++t) acc[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};

    const int at0 = p * kStep + ((g ^ (p >> 1)) << 4), at1 = p * kStep + (((g + 4) ^ (p >> 1)) << 4);
    auto step = [&](int32_t s, auto J) {  // step s, in place J of four of its lane group
        constexpr int j = J;
        const int from = ((s - s0) % kScaleSteps / 4) * 16 + p;  // the lane that has its scales
        const uint8_t *slot = lds + (wave * D + (s - s0) % D) * kSlot;
        uint32_t cx[T], cw[R];
#pragma unroll
        for (int t = 0; t < T; ++t) cx[t] = (uint32_t)__shfl((int)sx[t][j], from, kWave);
#pragma unroll
        for (int r = 0; r < R; ++r) cw[r] = (uint32_t)__shfl((int)sw[r][j], from, kWave);
        uint4 b[T][2];
#pragma unroll
        for (int t = 0; t < T; ++t) {
            b[t][0] = *reinterpret_cast<const uint4 *>(slot + (R + t) * 2048 + at0);
            b[t][1] = *reinterpret_cast<const uint4 *>(slot + (R + t) * 2048 + at1);
        }
        bf16x8 bb[kExact ? T : 1][2][2];
        if constexpr (kExact) {
#pragma unroll
            for (int t = 0; t < T; ++t)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    decode16(bb[t][i], b[t][i], kMX ? lifted((cx[t] >> (8 * (2 * i + (g >> 1)))) & 0xFF) : 1.0f);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint4 w0 = *reinterpret_cast<const uint4 *>(slot + r * 2048 + at0);
            const uint4 w1 = *reinterpret_cast<const uint4 *>(slot + r * 2048 + at1);
            if constexpr (kExact) {
                bf16x8 ww[2][2];
                decode16(ww[0], w0, kMX ? lifted((cw[r] >> (8 * (g >> 1))) & 0xFF) : 1.0f);
                decode16(ww[1], w1, kMX ? lifted((cw[r] >> (8 * (2 + (g >> 1)))) & 0xFF) : 1.0f);
#pragma unroll
                for (int t = 0; t < T; ++t) {
                    f32x4 q = kMX ? acc[r][t] : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        q = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ww[i / 2][i % 2], bb[t][i / 2][i % 2], q, 0, 0, 0);
                    if constexpr (kMX) {
                        acc[r][t] = q;
                    } else {
                        const float f = __uint_as_float(cx[t]) * __uint_as_float(cw[r]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[r][t][i] = __builtin_fmaf(q[i], f, acc[r][t][i]);
                    }
                }
            } else {
                const i32x8 ww = join(w0, w1);
#pragma unroll
                for (int t = 0; t < T; ++t) {
                    const i32x8 bt = join(b[t][0], b[t][1]);
                    if constexpr (kMX) {
                        acc[r][t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            ww, bt, acc[r][t], 0, 0, 0, (int)(cw[r] >> (8 * g)), 0, (int)(cx[t] >> (8 * g)));
                    } else {
                        const f32x4 q = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            ww, bt, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
                        const float f = __uint_as_float(cx[t]) * __uint_as_float(cw[r]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[r][t][i] = __builtin_fmaf(q[i], f, acc[r][t][i]);
                    }
                }
            }
        }
    };

    // every wave goes round as often as it has steps: all paths below are the wave's own
    if (s0 < s1) load_scales(s0);
    for (int32_t s = s0; s < min(s0 + D - 1, s1); ++s) fill(s);
    for (int32_t base = s0; base < s1; base += 4) {
        if (base > s0 && (base - s0) % kScaleSteps == 0) load_scales(base);
        static_for<0, 4, 1>([&](auto J) {
            const int32_t s = base + J;
            if (s < s1) {
                if (s + D - 1 < s1) {  // the slot that step s - 1 has left; its reads are in registers
                    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                    fill(s + D - 1);
                    asm volatile("s_waitcnt vmcnt(%0)" ::"n"((D - 1) * kLoads) : "memory");
                } else {
                    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
                }
                step(s, J);
            }
        });
    }

    // -- join the waves: column p is a token, rows 4 g .. are columns of y
    __syncthreads();
    float *join_at = reinterpret_cast<float *>(lds);
    uint32_t *far_at = reinterpret_cast<uint32_t *>(lds + kJoin);
    if constexpr (!kMX) far_at[wave] = wave_any(least < (64u << 24) - 1u || most > (190u << 24));
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < T; ++t)
            *reinterpret_cast<f32x4 *>(join_at + ((wave * T + t) * 16 + p) * kOut + r * 16 + 4 * g) = acc[r][t];
    __syncthreads();
    for (int e = threadIdx.x; e < T * 16 * kOut; e += W * 64) {
        const int t = e / kOut, c = e % kOut;
        float v = join_at[e];
#pragma unroll
        for (int i = 1; i < W; ++i) v += join_at[i * T * 16 * kOut + e];
        if (t > xlast || c > wlast) continue;
        if constexpr (!kMX) {
            if (unsure(v) >= kUnsure) {
                uint32_t any = 0;
#pragma unroll
                for (int i = 0; i < W; ++i) any |= far_at[i];
                const float *sxr = static_cast<const float *>(a.sx) + (int64_t)(row0 + t) * a.ld_sx;
                const float *swr = static_cast<const float *>(a.sw) + (kRagged == kRows ? group * a.sw_stride : 0) +
                                   (int64_t)((col0 + c) / 128) * a.ld_sw;
                for (int32_t i = any ? 0 : steps; i < steps; ++i)
                    if (odd_pair(__float_as_uint(sxr[i]), __float_as_uint(swr[i]))) {
                        v = block_product_again(x + (int64_t)t * a.ldx, sxr, w + (int64_t)c * a.ldw, swr, a.k);
                        break;
                    }
            }
        }
        if constexpr (kMX && kExact) {
            v *= kLowered;
            if (!__builtin_isfinite(v))
                v = mx_product_again(v, x + (int64_t)t * a.ldx, static_cast<const uint8_t *>(a.sx) + (int64_t)(row0 + t) * a.ld_sx,
                                     w + (int64_t)c * a.ldw, static_cast<const uint8_t *>(a.sw) +
                                         (kRagged == kRows ? group * a.sw_stride : 0) + (int64_t)(col0 + c) * a.ld_sw, a.k);
        }
        store_product(a.y, (int64_t)(row0 + t) * a.ldy + col0 + c, v, a.out_f32 != 0);
    }
}

template <bool kMX, int kRagged, int R, int T, int W, int D>
hipError_t launch(const Fp8Matmul &a, hipStream_t stream)
{
    const int64_t ct = (a.n + R * 16 - 1) / (R * 16);
    const int64_t rt = (a.m + T * 16 - 1) / (T * 16) + (kRagged == kRows ? a.groups : 0);
    if (ct * (W * 64) > 0xFFFFFFFF || rt > 65535) return hipErrorInvalidConfiguration;  // a grid's threads fit 32 bits
    const dim3 grid((unsigned)ct, (unsigned)rt), block(W * 64);
    if (a.out_f32) few_kernel<kMX, true, kRagged, R, T, W, D><<<grid, block, 0, stream>>>(a);
    else few_kernel<kMX, false, kRagged, R, T, W, D><<<grid, block, 0, stream>>>(a);
    return hipGetLastError();
}

// Rows to a workgroup (R x 16) so that every CU has one and none has a second turn for
// a few rows; with few rows more waves cut the contraction, and two workgroups fit a CU
// where LDS allows.  us of a call, block-FP8, for n x k = 4096 x 7168, 8192 x 8192, 16384 x
// 7168 on MI355X (below about 10 it is the host's time that counts):
//   tokens      R 1, 8 waves         R 2, 4 waves         R 4, 4 waves
//        16      9.4 12.7 25.5        9.1 13.3 22.9         -
//        32      9.6 16.5 38.7       11.0 14.3 26.8       15.2 16.6 25.4
//        64     13.1 24.1 53.3       16.5 17.9 39.2       24.3 26.3 31.0
// Just past a full turn, 33 tokens and 4097 rows: 257 workgroups of 16 rows take 17.5 us (fp32
// MXFP8 19.4), 129 of 32 rows 13.6 (15.7); 4096 rows in 256 workgroups of 16 take 10.6 (11.8).
template <bool kMX, int kRagged, int T>
hipError_t pick_rows(const Fp8Matmul &a, hipStream_t stream)
{
    const int64_t at_once = (int64_t)a.n * (kRagged == kRows ? a.groups : 1);
    if (at_once <= 16 * 256) return launch<kMX, kRagged, 1, T, 8, 2>(a, stream);
    if constexpr (T > 1 && kRagged == kDense) {
        if (at_once > 32 * 256) return launch<kMX, kRagged, 4, T, 4, 2>(a, stream);
    }
    return launch<kMX, kRagged, 2, T, 4, T == 1 ? 3 : 2>(a, stream);
}

template <bool kMX, int kRagged>
hipError_t pick(const Fp8Matmul &a, int tokens, hipStream_t stream)
{
    if constexpr (kRagged == kRows) {
        // 1, 4 and 16 rows a group, 128 groups of 2048 x 7168, us: T 1 172 255 424, 2 178 260 404;
        // longer groups take more tiles
        return tokens <= 16 ? pick_rows<kMX, kRagged, 2>(a, stream) : pick_rows<kMX, kRagged, 4>(a, stream);
    } else {
        if (tokens <= 16) return pick_rows<kMX, kRagged, 1>(a, stream);
        if (tokens <= 32) return pick_rows<kMX, kRagged, 2>(a, stream);
        if (tokens <= 48) return pick_rows<kMX, kRagged, 3>(a, stream);
        return pick_rows<kMX, kRagged, 4>(a, stream);
    }
}

}  // namespace

hipError_t launch_fp8_few(bool mx, int ragged, int tokens, const Fp8Matmul &a, hipStream_t stream)
{
    if (mx) return ragged == kDense ? pick<true, kDense>(a, tokens, stream) : pick<true, kRows>(a, tokens, stream);
    return ragged == kDense ? pick<false, kDense>(a, tokens, stream) : pick<false, kRows>(a, tokens, stream);
}

}  // namespace mxq
