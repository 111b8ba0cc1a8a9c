// fp8_tiles.hip -- products of many 8-bit tokens with 8-bit weights for gfx950.
//
//   y[r, c] = sum_k x[r, k] w[c, k]
//
// in block-FP8 (fp32 scales, x: 1 x 128, w: 128 x 128) and in MXFP8 (E8M0, both 1 x
// 32), dense, with rows grouped by expert, and with the contraction grouped (weight
// gradients).
//
// Matrix cores: v_mfma_f32_32x32x64_f8f6f4, the weights as A, the tokens as B.  Lane
// (p, h) = (lane % 32, lane / 32) holds of row p of A (of column p of B) the bytes k =
// 16 h .. 16 h + 15 and 32 + 16 h .., and of the result column p in rows 8 (i / 4) +
// 4 h + i % 4, i = 0..15: one token, four neighbouring weight rows.
//   MXFP8: lane (p, h) gives the scale of row p's group 32 h ..; the products are
//   scaled and summed in the matrix cores.
//   Block-FP8: 128 k are multiplied unscaled, from zero, and leave with one FMA an
//   element: acc += p * (sx * sw).  A lane has one token and a wave's weight rows lie in
//   one tile of 128, so the factor is one number per lane and 32 tokens.
//
// The 8-bit instruction keeps, of 8 neighbouring k, what lies above 2^-13 of their
// largest product (measured): 5e-5 of a sum's norm, a thirtieth of what rounding to bf16
// takes.  Results in fp32 (kExact) are for more than that, so there the codes are made
// bf16, without loss, and v_mfma_f32_32x32x16_bf16 multiplies: 1.5e-7, at half the rate.
//
// Bound, where the contraction is long, by the matrix cores: 4096 x 8192 x 8192 MXFP8
// 238 us (2.31 PFLOP/s; the matrix cores busy 80 % of it at 2.1 GHz), 8192 x 7168 x 7168
// block-FP8 432 to 455 us (1.85 to 1.95 PFLOP/s; 3.5 rounds of tiles cost as much as 4, and
// the FMAs with the scales run beside the products only in part).  So LDS is filled straight
// from memory, two steps deep, and what a step has to read from it is read under the last
// step's products.  Where it is short, by what does not overlap in a CU that holds one
// tile: 16384 tokens of 32 groups as the contraction of 2048 x 7168 weight gradients,
// four steps a tile, take 481 to 517 us, of which the stores alone are 181, the steps 240
// and the start of 7168 workgroups 106 (its second step is asked for only when the first is
// there: the scales loaded between the two are waited for).

#include "fp8_matmul.hpp"
#include "launch.hpp"

namespace mxq {

namespace {

struct TileGrid {
    int32_t tm, tn;  // tiles of rows (at most, if grouped) and of columns
    int32_t sm, sn;  // tiles of a block that one XCD works on at a time
    int32_t bm, bn;  // such blocks
    int32_t groups;  // that each have all tiles (kContraction, else 1)
};

// A block of sm x sn tiles, as many as an XCD has CUs, shares its rows and columns
// in that XCD's L2.  Workgroup i runs on XCD i % 8.  With several groups, which may
// differ much in length, every XCD gets as many blocks of each, and the XCDs begin
// with different ones.
__device__ __forceinline__ bool tile_of(const TileGrid &g, int32_t &tm, int32_t &tn, int32_t &group)
{
    const int32_t xcd = blockIdx.x % 8, local = blockIdx.x / 8, each = g.sm * g.sn;
    const int32_t in = local % each, turn = local / each;
    group = (turn + xcd * (g.groups / 8)) % g.groups;
    const int32_t block = turn / g.groups * 8 + (xcd + group) % 8;
    tm = block % g.bm * g.sm + in % g.sm;
    tn = block / g.bm * g.sn + in / g.sm;
    return tm < g.tm && tn < g.tn;
}

template <bool kMX, bool kExact, int kRagged, int WT, int WN, int CT, int RT>
__global__ __launch_bounds__(WT *WN * 64, 2) void tile_kernel(Fp8Matmul a, TileGrid grid)
{
    constexpr int kWaves = WT * WN, BM = WT * CT * 32, BN = WN * RT * 32;
    constexpr int kThreads = kWaves * 64, kStage = (BM + BN) * kStep;
    static_assert(BM + BN == kThreads, "one thread stages one row's scales");
    constexpr int kLoads = (BM + BN) / 8 / kWaves;  // of 8 rows, for each wave and step
    static_assert(BM / 8 % kLoads == 0, "a wave loads rows of one operand");
    constexpr int kScaled = BM + (kMX ? BN : WN);    // rows with scales in LDS (one for a wave's weight rows)
    __shared__ __align__(1024) uint8_t lds[2 * kStage];
    __shared__ __align__(16) uint32_t scales[3][4][kScaled];

    int32_t tm, tn, group;
    if (!tile_of(grid, tm, tn, group)) return;
    int32_t row0 = tm * BM, row_end = min(row0 + BM, a.m), k0 = 0, k1 = a.k;
    if constexpr (kRagged == kRows) {
        if (!find_row_tile(a, BM, tm, group, row0, row_end)) return;
    } else if constexpr (kRagged == kContraction) {
        k0 = k_offset_at(a, group);
        k1 = max(k0, k_offset_at(a, group + 1));
    }
    const int32_t col0 = tn * BN, col_end = min(col0 + BN, a.n);
    const int32_t steps = (k1 - k0 + kStep - 1) / kStep;
    const int32_t full = (k1 - k0) / kStep;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid / 64);
    const int wt = wave / WN, wn = wave % WN, p = lane & 31, h = lane >> 5;

    // -- what this wave brings to LDS: kLoads times 8 rows of x or of w
    const bool of_x = wave * kLoads * 8 < BM;
    const int first = of_x ? wave * kLoads * 8 : wave * kLoads * 8 - BM;
    const int64_t ld = __builtin_amdgcn_readfirstlane((int)(of_x ? a.ldx : a.ldw));
    const uint8_t *base = of_x ? a.x + (int64_t)row0 * a.ldx
                               : a.w + (kRagged == kRows ? group * a.w_stride : 0) +
                                     (int64_t)col0 * a.ldw;
    // rows past the last repeat it: their results are dropped
    const int last = __builtin_amdgcn_readfirstlane((of_x ? row_end - row0 : col_end - col0) - 1);
    // Row r's 16-byte piece c lies at piece c ^ (r / 2 % 8) of its line in LDS: sixteen
    // rows' pieces of one c, read together, then fall on all 64 banks.  (c ^ (r % 8), for
    // 32 banks, leaves two on each: block-FP8 8192 x 8192 x 7168 took 5 % longer.)
    const uint32_t chunk = (lane & 7) ^ (lane >> 4);  // in even loads; odd ones are four rows on: chunk ^ 4
    const uint32_t vrow = (lane >> 3) * (uint32_t)ld;
    const __amdgpu_buffer_rsrc_t rsrc = buffer_at(base);
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;
    // The i-th load of step s; a step past the last one's reads nothing.
    uint32_t piece_at[2];
    auto aim = [&](int32_t s) {  // what lies past the contraction's end is zero
        const int left = k1 - k0 - s * kStep - 16;
        piece_at[0] = chunk * 16 | ((int)(chunk * 16) > left ? kNowhere : 0u);
        piece_at[1] = (chunk ^ 4) * 16 | ((int)((chunk ^ 4) * 16) > left ? kNowhere : 0u);
    };
    auto fill_one = [&](int32_t s, int i) {
        int r = first + i * 8;
        asm volatile("" : "+s"(r));  // a few scalar operations here take no register for good
        const uint32_t in_rows = min(vrow, (uint32_t)__builtin_amdgcn_readfirstlane(max(min(last - r, 7), 0) * (int)ld));
        load_to_lds(rsrc, lds0 + (s & 1) * kStage + (wave * kLoads + i) * 1024, in_rows + piece_at[i & 1],
                    __builtin_amdgcn_readfirstlane(min(r, last) * (int)ld + k0 + s * kStep));
    };
    auto fill = [&](int32_t s) {
        aim(s);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) fill_one(s, i);
    };
    // Where the contraction ends inside 16 bytes, these are put in place by hand once
    // the last step is there otherwise.
    auto finish = [&](int32_t s) {
        if (kRagged == kContraction && (k1 & 15) != 0 && s == steps - 1) {
            const int at = (k1 - k0) % kStep & ~15;
            const int r = tid < BM ? tid : tid - BM;
            const uint8_t *row = tid < BM ? a.x + (int64_t)(row0 + min(r, row_end - row0 - 1)) * a.ldx
                                          : a.w + (int64_t)(col0 + min(r, col_end - col0 - 1)) * a.ldw;
            *reinterpret_cast<uint4 *>(lds + (s & 1) * kStage + tid * kStep + (((at >> 4) ^ (r >> 1 & 7)) << 4)) =
                first_bytes(row + (k1 & ~15), k1 & 15);
        }
    };

    // -- scales: each thread one row, four steps at a time, two such groups of steps in
    // turn.  The last group, which may be short, has a place of its own and is loaded
    // ahead of the loop: inside there is no register for its many cases.
    const int32_t last_group = (steps - 1) / 4;
    const uint8_t *scale_row;
    {
        const bool x_row = tid < BM;
        const int64_t gs = kRagged == kRows ? group * a.sw_stride : 0;
        if constexpr (kMX) {
            const int r = x_row ? row0 + min(tid, row_end - row0 - 1)
                                : col0 + min(tid - BM, col_end - col0 - 1);
            scale_row = (x_row ? static_cast<const uint8_t *>(a.sx) + (int64_t)r * a.ld_sx
                               : static_cast<const uint8_t *>(a.sw) + gs + (int64_t)r * a.ld_sw) +
                        k0 / 32;
        } else {  // a wave's weight rows lie in one tile of 128 of their scales
            const int r = x_row ? row0 + min(tid, row_end - row0 - 1)
                                : min(col0 + min(tid - BM, WN - 1) * (RT * 32), a.n - 1) / 128;
            scale_row = reinterpret_cast<const uint8_t *>(
                x_row ? static_cast<const float *>(a.sx) + (int64_t)r * a.ld_sx
                      : static_cast<const float *>(a.sw) + gs + (int64_t)r * a.ld_sw);
        }
    }
    uint32_t sreg[4];
    auto load_scales = [&](int32_t g) {  // a whole group
        if (tid < kScaled) {
            const Bytes16 v = *reinterpret_cast<const Bytes16 *>(scale_row + g * 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) sreg[i] = v.w[i];
        }
    };
    auto store_scales = [&](int place) {
        if (tid < kScaled) {
#pragma unroll
            for (int i = 0; i < 4; ++i) scales[place][i][tid] = sreg[i];
        }
    };
    auto load_last_scales = [&]() {  // zeros behind the row's end
        if (tid < kScaled) {
            const int32_t have = kMX ? (k1 - k0 + 31) / 32 : steps * 4, before = kMX ? k0 / 32 : 0;
            const uint4 v = bytes16_of(scale_row - before, before + last_group * 16, before + have);
            sreg[0] = v.x, sreg[1] = v.y, sreg[2] = v.z, sreg[3] = v.w;
        }
    };
    // where step s finds them
    auto scales_of = [&](int32_t s) { return scales[s / 4 == last_group ? 2 : s / 4 & 1][s & 3]; };

    // -- operands: lane (p, h) finds piece 2 i + h of row p's line at place ^ 32 i
    uint32_t place = p * kStep + ((h ^ (p >> 1 & 7)) << 4);
    auto piece = [&](uint32_t stage, int row, int i) {  // 16 bytes of rows row ..
        return *reinterpret_cast<const uint4 *>(lds + ((place + stage) ^ (32 * i)) + row * kStep);
    };
    auto operand = [&](uint32_t stage, int row, int t) {  // half t of the step
        return join(piece(stage, row, 2 * t), piece(stage, row, 2 * t + 1));
    };

    f32x16 acc[RT][CT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[r][c][i] = 0.f;

    // The products so far are in the accumulators here, not put off past a barrier with
    // their operands still held.
    auto settle = [&]() {
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int c = 0; c < CT; ++c) asm volatile("" : "+v"(acc[r][c]));
    };
    // Step s is multiplied while step s + 1 comes into the other half of LDS.  A barrier
    // in the middle of every step: behind it all of stage s is in registers, so its
    // place takes step s + 2, and stage s + 1 is there to be read for the next step
    // under this one's second half.  (What the last step reads ahead is not used.)
    auto turn = [&](int32_t s) {
        settle();
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        finish(s + 1);
        if ((s + 1) % 4 == 0 && (s + 1) / 4 < last_group) store_scales((s + 1) / 4 & 1);
        __syncthreads();
        if ((s + 1) % 4 == 0 && (s + 1) / 4 + 1 < last_group) load_scales((s + 1) / 4 + 1);
        aim(s + 2);
    };
    if (steps > 0) {
        fill(0);
        load_last_scales();
        store_scales(2);
        if (last_group > 0) {
            load_scales(0);
            store_scales(0);
        }
        if (1 < last_group) load_scales(1);
        if (1 < steps) {
            fill(1);
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kLoads) : "memory");
        } else {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        }
        finish(0);
        __syncthreads();
    }
    if constexpr (kExact) {
        for (int32_t s = 0; s < steps; ++s) {
            const uint32_t stage = (s & 1) * kStage;
            const uint32_t *sc = scales_of(s);
            if constexpr (kMX) {
                uint32_t sx[CT], sr[RT];
#pragma unroll
                for (int c = 0; c < CT; ++c) sx[c] = sc[(wt * CT + c) * 32 + p];
#pragma unroll
                for (int r = 0; r < RT; ++r) sr[r] = sc[BM + (wn * RT + r) * 32 + p];
                static_for<0, 4, 1>([&](auto I) {  // piece i of both halves: the step's group i
                    constexpr int i = I;
                    bf16x8 b[CT][2];
#pragma unroll
                    for (int c = 0; c < CT; ++c)
                        decode16(b[c], piece(stage, (wt * CT + c) * 32, i), lifted((sx[c] >> (8 * i)) & 0xFF));
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        bf16x8 w[2];
                        decode16(w, piece(stage, BM + (wn * RT + r) * 32, i), lifted((sr[r] >> (8 * i)) & 0xFF));
#pragma unroll
                        for (int c = 0; c < CT; ++c)
#pragma unroll
                            for (int j = 0; j < 2; ++j)
                                acc[r][c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w[j], b[c][j], acc[r][c], 0, 0, 0);
                    }
                });
            } else {
                bf16x8 b[CT][4][2];
#pragma unroll
                for (int c = 0; c < CT; ++c)
#pragma unroll
                    for (int i = 0; i < 4; ++i) decode16(b[c][i], piece(stage, (wt * CT + c) * 32, i), 1.0f);
                const float swv = __uint_as_float(sc[BM + wn]);
                float f[CT];
#pragma unroll
                for (int c = 0; c < CT; ++c) f[c] = __uint_as_float(sc[(wt * CT + c) * 32 + p]) * swv;
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    bf16x8 w[4][2];
#pragma unroll
                    for (int i = 0; i < 4; ++i) decode16(w[i], piece(stage, BM + (wn * RT + r) * 32, i), 1.0f);
#pragma unroll
                    for (int c = 0; c < CT; ++c) {
                        f32x16 q{};
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int j = 0; j < 2; ++j)
                                q = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w[i][j], b[c][i][j], q, 0, 0, 0);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            acc[r][c][i] = __builtin_fmaf(q[i], f[c], acc[r][c][i]);
                    }
                }
            }
            turn(s);
#pragma unroll
            for (int i = 0; i < kLoads; ++i) fill_one(s + 2, i);
        }
    } else if constexpr (kMX) {
        i32x8 b0[CT], b1[CT], w[RT];
        auto fetch_b = [&](i32x8(&b)[CT], int32_t s, int t) {
#pragma unroll
            for (int c = 0; c < CT; ++c) b[c] = operand((s & 1) * kStage, (wt * CT + c) * 32, t);
        };
        auto fetch_w = [&](int r, int32_t s, int t) {
            w[r] = operand((s & 1) * kStage, BM + (wn * RT + r) * 32, t);
        };
        if (steps > 0) {
            fetch_b(b0, 0, 0);
#pragma unroll
            for (int r = 0; r < RT; ++r) fetch_w(r, 0, 0);
        }
        for (int32_t s = 0; s < steps; ++s) {
            const uint32_t *sc = scales_of(s);
            int sx[CT], sr[RT];
#pragma unroll
            for (int c = 0; c < CT; ++c) sx[c] = (int)(sc[(wt * CT + c) * 32 + p] >> (8 * h));
#pragma unroll
            for (int r = 0; r < RT; ++r) sr[r] = (int)(sc[BM + (wn * RT + r) * 32 + p] >> (8 * h));
            fetch_b(b1, s, 1);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int r = 0; r < RT; ++r) {
#pragma unroll
                for (int c = 0; c < CT; ++c)
                    acc[r][c] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                        w[r], b0[c], acc[r][c], 0, 0, 0, sr[r], 0, sx[c]);
                __builtin_amdgcn_sched_barrier(0);  // into the same registers
                fetch_w(r, s, 1);
                __builtin_amdgcn_sched_barrier(0);
            }
            turn(s);
            fetch_b(b0, s + 1, 0);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int r = 0; r < RT; ++r) {
#pragma unroll
                for (int c = 0; c < CT; ++c)
                    acc[r][c] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                        w[r], b1[c], acc[r][c], 0, 0, 2, sr[r], 2, sx[c]);
                __builtin_amdgcn_sched_barrier(0);
                fetch_w(r, s + 1, 0);
                // between products, not in a row: each of these holds the wave up
#pragma unroll
                for (int i = 0; i < kLoads / RT; ++i) fill_one(s + 2, r * (kLoads / RT) + i);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    } else {
        // A step's last weight rows are multiplied behind its barrier, under the next
        // step's tokens coming to registers.
        i32x8 b0[CT][2], b1[CT][2];
        auto fetch_b = [&](i32x8(&b)[CT][2], int32_t s) {
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int t = 0; t < 2; ++t) b[c][t] = operand((s & 1) * kStage, (wt * CT + c) * 32, t);
        };
        auto step = [&](const i32x8(&b)[CT][2], i32x8(&next)[CT][2], int32_t s) {
            asm volatile("" : "+v"(place));  // its sums anew each step: few registers are left
            const uint32_t *sc = scales_of(s);
            const float swv = __uint_as_float(sc[BM + wn]);
            float f[CT];
#pragma unroll
            for (int c = 0; c < CT; ++c) f[c] = __uint_as_float(sc[(wt * CT + c) * 32 + p]) * swv;
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const i32x8 w0 = operand((s & 1) * kStage, BM + (wn * RT + r) * 32, 0);
                const i32x8 w1 = operand((s & 1) * kStage, BM + (wn * RT + r) * 32, 1);
                if (r == RT - 1) {
                    turn(s);
                    fetch_b(next, s + 1);
                    __builtin_amdgcn_sched_barrier(0);
                }
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                    f32x16 q{};
                    q = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w0, b[c][0], q, 0, 0, 0, 0, 0, 0);
                    q = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w1, b[c][1], q, 0, 0, 0, 0, 0, 0);
                    if (r == RT - 1) {
#pragma unroll
                        for (int i = 0; i < kLoads / CT; ++i) fill_one(s + 2, c * (kLoads / CT) + i);
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        acc[r][c][i] = __builtin_fmaf(q[i], f[c], acc[r][c][i]);
                }
            }
        };
        if (steps > 0) fetch_b(b0, 0);
        for (int32_t s = 0; s < steps; s += 2) {
            step(b0, b1, s);
            if (s + 1 < steps) step(b1, b0, s + 1);
        }
    }

    // -- out (what is still on its way to LDS, nothing but zeros, is let in first): a
    // wave turns 32 tokens at a time around in LDS and writes whole rows of its columns,
    // 16 bytes a lane: 256 bytes of bf16 (128 in the small tiles) or fp32.  Piece j of row
    // r lies at j ^ (r % 8).  Rows of y that are no multiple of 16 bytes are written an element
    // a lane: 8192 x 7167 x 2048 takes 168 us where 7168 columns take 132; 4096 x 8191 x 8192
    // as long as 8192.
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    constexpr int kCols = RT * 32, kSize = kExact ? 4 : 2, kRow = kCols * kSize;
    constexpr int kPieces = kRow / 16, kRowsAt = 64 / kPieces;  // pieces of a row, rows that 64 lanes write
    static_assert(kPieces >= 8 && kPieces <= 64 && kWaves * 32 * kRow <= 2 * kStage, "fits the stages");
    uint8_t *mine = lds + wave * 32 * kRow;
    const int wcol = col0 + wn * kCols, cols = min(kCols, col_end - wcol);
    uint8_t *y = static_cast<uint8_t *>(a.y) + (kRagged == kContraction ? group * a.y_stride * kSize : 0);
    const bool wide = cols == kCols && (reinterpret_cast<uintptr_t>(y) & 15) == 0 && a.ldy * kSize % 16 == 0;
#pragma unroll
    for (int c = 0; c < CT; ++c) {
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int byte = (r * 32 + 8 * i + 4 * h) * kSize;
                uint8_t *to = mine + p * kRow + (((byte >> 4) ^ (p & 7)) << 4) + (byte & 15);
                const f32x16 &v = acc[r][c];
                if constexpr (kExact) {
                    constexpr float f = kMX ? kLowered : 1.0f;
                    *reinterpret_cast<f32x4 *>(to) = f32x4{v[4 * i] * f, v[4 * i + 1] * f, v[4 * i + 2] * f, v[4 * i + 3] * f};
                } else {
                    *reinterpret_cast<uint2 *>(to) = make_uint2(bf16x2_rne(v[4 * i], v[4 * i + 1]),
                                                                bf16x2_rne(v[4 * i + 2], v[4 * i + 3]));
                }
            }
        __builtin_amdgcn_wave_barrier();
        const int32_t trow = row0 + (wt * CT + c) * 32;
        const int rows = min(32, row_end - trow);
        if constexpr (kMX && kExact) {
            static_assert(kCols == 64, "a lane has a column");
            uint32_t worst = 0;
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int i = 0; i < 16; ++i) worst = max(worst, __float_as_uint(acc[r][c][i]) << 1);
            const uint64_t look = __builtin_amdgcn_ballot_w64(worst >= 0xFF000000u && p < rows && cols > 0);
            if (look) {  // tokens and columns with a scale of NaN stay as they are
                const uint8_t *sx = static_cast<const uint8_t *>(a.sx) + (int64_t)trow * a.ld_sx + k0 / 32;
                const int64_t col = min(wcol + lane, col_end - 1);
                const uint8_t *w = a.w + (kRagged == kRows ? group * a.w_stride : 0) + col * a.ldw + k0;
                const uint8_t *sw = static_cast<const uint8_t *>(a.sw) + (kRagged == kRows ? group * a.sw_stride : 0) +
                                    col * a.ld_sw + k0 / 32;
                const int32_t groups = (k1 - k0 + 31) / 32;
                const bool in = lane < cols && !nan_scale(sw, groups);
                const uint64_t found = look & ~__builtin_amdgcn_ballot_w64(p < rows && nan_scale(sx + p * a.ld_sx, groups));
                for (uint32_t left = (uint32_t)found | (uint32_t)(found >> 32); left; left &= left - 1) {
                    const int tr = __builtin_ctz(left);
                    float *at = reinterpret_cast<float *>(mine + tr * kRow + (((lane >> 2) ^ (tr & 7)) << 4) + (lane & 3) * 4);
                    if (in && !__builtin_isfinite(*at))
                        *at = mx_product_again(*at, a.x + (int64_t)(trow + tr) * a.ldx + k0, sx + tr * a.ld_sx, w, sw, k1 - k0);
                }
                __builtin_amdgcn_wave_barrier();
            }
        }
        if constexpr (!kMX) {
            uint32_t worst = 0;
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int i = 0; i < 16; ++i) worst = max(worst, unsure(acc[r][c][i]));
            const uint64_t look = __builtin_amdgcn_ballot_w64(worst >= kUnsure && p < rows && cols > 0);
            if (look) {  // lane (p, h) looks through every other four of token p's scales
                const float *sx = static_cast<const float *>(a.sx) + (int64_t)trow * a.ld_sx;
                const float *sw = static_cast<const float *>(a.sw) + (kRagged == kRows ? group * a.sw_stride : 0) +
                                  (int64_t)(wcol / 128) * a.ld_sw;
                bool odd = false;
                if ((look >> p | look >> (p + 32)) & 1) {
#pragma unroll 4
                    for (int32_t i = h * 16; i < steps * 4; i += 32) {
                        const uint4 u = bytes16_of(reinterpret_cast<const uint8_t *>(sx + p * a.ld_sx), i, steps * 4);
                        const uint4 v = bytes16_of(reinterpret_cast<const uint8_t *>(sw), i, steps * 4);
                        odd |= odd_pair(u.x, v.x) || odd_pair(u.y, v.y) || odd_pair(u.z, v.z) || odd_pair(u.w, v.w);
                    }
                }
                const uint64_t found = __builtin_amdgcn_ballot_w64(odd);
                for (uint32_t left = (uint32_t)found | (uint32_t)(found >> 32); left; left &= left - 1) {
                    const int tr = __builtin_ctz(left);
                    for (int tc = lane; tc < cols; tc += 64) {
                        const int byte = tc * kSize;
                        uint8_t *at = mine + tr * kRow + (((byte >> 4) ^ (tr & 7)) << 4) + (byte & 15);
                        const float v = kExact ? *reinterpret_cast<const float *>(at)
                                               : __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t *>(at) << 16);
                        if (unsure(v) < kUnsure) continue;
                        const uint8_t *w = a.w + (kRagged == kRows ? group * a.w_stride : 0) + (int64_t)(wcol + tc) * a.ldw;
                        const uint8_t *x = a.x + (int64_t)(trow + tr) * a.ldx;
                        store_product(at, 0, block_product_again(x, sx + tr * a.ld_sx, w, sw, a.k), kExact);
                    }
                }
                __builtin_amdgcn_wave_barrier();
            }
        }
        if (wide) {
#pragma unroll
            for (int i = 0; i < 32 / kRowsAt; ++i) {
                const int tr = i * kRowsAt + lane / kPieces, j = lane % kPieces;
                const uint4 v = *reinterpret_cast<const uint4 *>(mine + tr * kRow + ((j ^ (tr & 7)) << 4));
                if (tr < rows)  // past the caches, which keep the operands: 2 to 4 % less time
                    st16<true>(y + ((int64_t)(trow + tr) * a.ldy + wcol) * kSize + j * 16, v);
            }
        } else if (cols > 0) {
            for (int tr = 0; tr < rows; ++tr)
                for (int tc = lane; tc < cols; tc += 64) {
                    const int byte = tc * kSize;
                    const uint8_t *from = mine + tr * kRow + (((byte >> 4) ^ (tr & 7)) << 4) + (byte & 15);
                    uint8_t *to = y + ((int64_t)(trow + tr) * a.ldy + wcol + tc) * kSize;
                    if constexpr (kExact) *reinterpret_cast<uint32_t *>(to) = *reinterpret_cast<const uint32_t *>(from);
                    else *reinterpret_cast<uint16_t *>(to) = *reinterpret_cast<const uint16_t *>(from);
                }
        }
        __builtin_amdgcn_wave_barrier();
    }
}

template <bool kMX, bool kExact, int kRagged, int WT, int WN, int CT, int RT>
hipError_t launch(const Fp8Matmul &a, hipStream_t stream)
{
    constexpr int BM = WT * CT * 32, BN = WN * RT * 32;
    TileGrid g;
    g.tm = (a.m + BM - 1) / BM + (kRagged == kRows ? a.groups : 0);
    g.tn = (a.n + BN - 1) / BN;
    auto parts = [](int32_t n, int32_t most) {  // n cut evenly into parts of at most `most`
        const int32_t cuts = (n + most - 1) / most;
        return (n + cuts - 1) / cuts;
    };
    g.sm = parts(g.tm, 8);
    g.sn = parts(g.tn, 32 / g.sm);
    if (kRagged == kContraction)  // every group's blocks are dealt to eight XCDs anew: smaller ones come out even
        while (g.sm * g.sn > 8) (g.sm > g.sn ? g.sm : g.sn) /= 2;
    g.bm = (g.tm + g.sm - 1) / g.sm;
    g.bn = (g.tn + g.sn - 1) / g.sn;
    g.groups = kRagged == kContraction ? a.groups : 1;
    const int64_t wgs = ((int64_t)g.bm * g.bn + 7) / 8 * 8 * g.sm * g.sn * g.groups;
    if (wgs * (WT * WN * 64) > 0xFFFFFFFF) return hipErrorInvalidConfiguration;  // a grid's threads fit 32 bits
    tile_kernel<kMX, kExact, kRagged, WT, WN, CT, RT>
        <<<dim3((unsigned)wgs), dim3(WT * WN * 64), 0, stream>>>(a, g);
    return hipGetLastError();
}

template <bool kMX, int kRagged>
hipError_t pick(const Fp8Matmul &a, hipStream_t stream)
{
    if (a.out_f32) return launch<kMX, true, kRagged, 2, 2, 2, 2>(a, stream);
    // 256 x 256 tiles, one to a CU, or 128 x 128, two.  us at k = 7168, MXFP8 (block-FP8 takes
    // 3 to 15 % more), by the number of large tiles that there would be:
    //             64    128    160    176    208    256    512
    //   large     97     96     90     94     95    100    208
    //   small     52     75    117    114    119    132    283
    // So the large ones are ahead from somewhere between 128 and 160 on; 192 is later than
    // that.  Rows of several groups are counted as if they were one group's.
    const int64_t big = (int64_t)((a.m + 255) / 256) * ((a.n + 255) / 256) * (kRagged == kContraction ? a.groups : 1);
    if (big >= 192) return launch<kMX, false, kRagged, 4, 2, 2, 4>(a, stream);
    return launch<kMX, false, kRagged, 2, 2, 2, 2>(a, stream);
}

}  // namespace

hipError_t launch_fp8_matmul(bool mx, int ragged, const Fp8Matmul &a, hipStream_t stream)
{
    // Up to 64 tokens the weights are the work; and while a product has few tiles, more
    // and smaller workgroups are ahead although they read the weights again for every 64.  us
    // at k = 7168, block-FP8:
    //   tokens x n      128 x 8192  128 x 16384  256 x 4096  256 x 7168  512 x 2048  1024 x 2048
    //   few tokens'         33          55           44          62          44           81
    //   tiles               48          66           47          47          47           48
    if (ragged == kDense && (a.m <= 64 || (int64_t)((a.m + 63) / 64) * a.n <= 16384))
        return launch_fp8_few(mx, ragged, a.m, a, stream);
    // Rows a group on average, us, 32 groups of 2048 x 7168 in block-FP8 and 128 of 2048 x 2048 in
    // MXFP8, whose short contraction the tiles are ahead with from few rows on:
    //                   8    16    32    48          8    16    32    48
    //   few tokens'    85    97   165   190        135   158   322   385
    //   tiles         139   144   149   147        115   119   145   173
    if (ragged == kRows && a.m <= (int64_t)32 * a.groups && a.m / 32 + a.groups < 65535)
        return launch_fp8_few(mx, ragged, (a.m - 1) / a.groups + 1, a, stream);
    if (mx)
        return ragged == kDense ? pick<true, kDense>(a, stream)
               : ragged == kRows ? pick<true, kRows>(a, stream)
                                 : pick<true, kContraction>(a, stream);
    return ragged == kDense ? pick<false, kDense>(a, stream) : pick<false, kRows>(a, stream);
}

}  // namespace mxq
