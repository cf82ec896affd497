// gfx950 kernels of the product of two coded matrices over their columns,
//     y[i, j] = sum over c of a[i, c] b[j, c],
// each element a code times its block's power of two.
//
// Codes go to LDS as they lie in memory, 128 columns a step, and from there to the matrix
// cores.  16-bit results: the scaled 8-bit instruction (32 x 32 x 64), which takes the codes
// and the exponent bytes as they are, so that a block's scale costs nothing.  Its lanes hold
// columns 16 h .. 16 h + 15 and 32 + 16 h .. of a row (h: the wave's half), the first under
// the scale that lane half 0 gives for the row, the second under that of half 1.  It adds
// products in groups of eight whose parts below 2^-13 of the group's largest are lost:
// 1.5e-5 of the result on normal data, far below a 16-bit result's rounding, but not FP32.
// FP32 results therefore convert the codes to BF16 (exact: four significant bits) on their
// way from LDS and use the BF16 instruction, whose products are exact and whose sums are FP32.
//
// LDS rows are 128 B, half the banks; 16-B unit c of row r lies at unit c ^ (r / 2 mod 8), so
// that the rows which lanes read at once fall on different banks.
#include <type_traits>

#include "block_launch.h"
#include "code_device.h"

#pragma clang fp contract(off)

namespace zs {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float code_value(uint32_t c) {
    return __builtin_amdgcn_cvt_f32_fp8(static_cast<int>(c), 0);
}

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// A pointer `bytes` past one that is the same in every lane, the base in scalar registers.
template <typename T>
__device__ __forceinline__ const GLOBAL_AS T *at_offset(const T *base, uint32_t bytes) {
    auto *b = (const GLOBAL_AS char *)(base);
    asm("" : "+s"(b));
    return (const GLOBAL_AS T *)(b + bytes);
}

// Eight codes under one scale as BF16, exact.
__device__ __forceinline__ bf16x8 codes_to_bf16(uint32_t lo, uint32_t hi, float scale) {
    u32x4 r;
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true));
    r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false));
    r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true));
    return __builtin_bit_cast(bf16x8, r);
}

// Half the scale of an exponent byte: a code of 448 under the largest scale is past BF16's
// range, its half is not.  Sums of such products are multiplied by 4 at the end (kUnhalve).
// Of what a code stands for only 2^-133, the smallest, is lost.
__device__ __forceinline__ float half_scale(uint32_t e) { return from_bits((e - 1u) << 23); }
constexpr float kUnhalve = 4.0f;

constexpr uint32_t kStep = 128;   // columns a step

struct ProductShape {
    uint64_t ldy, n;
    uint32_t m, k;
    uint32_t blocks_a, blocks_b;   // exponent bytes a row of a, and of b's blocks
    uint32_t shift_a;              // log2 of a's block
    uint32_t per_split;            // steps a split
    uint32_t tiles_m, tiles_n;
    uint32_t group_n;              // tiles a group has along n, 0: no groups
    uint64_t work;                 // work items: tiles, or places in groups
};

// Tile of work item w: tiles in groups of 32 (`group_n` along n), groups dealt to the eight
// XCDs in turn (workgroups go round them by number), so that the 32 compute units of an XCD
// share operands in its L2.  false: no such tile.
__device__ __forceinline__ bool tile_of(const ProductShape &s, uint64_t w, uint32_t *i,
                                        uint32_t *j) {
    if (s.group_n == 0) {
        *i = static_cast<uint32_t>(w / s.tiles_n);
        *j = static_cast<uint32_t>(w - static_cast<uint64_t>(*i) * s.tiles_n);
        return true;
    }
    const uint32_t group_m = 32 / s.group_n, across = (s.tiles_n + s.group_n - 1) / s.group_n;
    const uint64_t at = w >> 3, group = (at >> 5) * 8 + (w & 7);
    const uint32_t in = static_cast<uint32_t>(at & 31);
    const uint64_t gi = group / across;
    *i = static_cast<uint32_t>(gi) * group_m + in % group_m;
    *j = static_cast<uint32_t>(group - gi * across) * s.group_n + in / group_m;
    return gi * group_m < s.tiles_m && *i < s.tiles_m && *j < s.tiles_n;
}

// One BM x BN tile of y (or, SPLIT, of a split's FP32 plane); WM x WN waves.  EIGHT: the 8-bit
// instruction.  Rows past the matrix are read as its last one and not stored; columns past it
// are zeros.  k >= 16, and a tile's rows span less than 4 GiB (the launcher checks both).
template <int F, bool EIGHT, bool SPLIT, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 2) void product_tile_kernel(
    void *__restrict__ y, const uint8_t *__restrict__ qa, const uint8_t *__restrict__ ea,
    const uint8_t *__restrict__ qb, const uint8_t *__restrict__ eb, ProductShape s) {
    constexpr int kLanes = 64 * WM * WN;
    constexpr int TM = BM / WM / 32, TN = BN / WN / 32;   // 32 x 32 results a wave
    constexpr int kRows = kLanes / 8;                     // rows a pass of staging
    constexpr int PA = BM / kRows, PB = BN / kRows;
    static_assert(kLanes >= BM && BN / WN <= 128, "exponents: a lane a row, a byte a wave");
    __shared__ __align__(16) uint8_t sa[2][BM * kStep];
    __shared__ __align__(16) uint8_t sb[2][BN * kStep];
    __shared__ uint32_t se[2][BM];

    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    const uint32_t half = lane >> 5, row32 = lane & 31u;
    const uint32_t am = wave % WM * (BM / WM), bn = wave / WM * (BN / WN);
    for (uint64_t work = blockIdx.x; work < s.work; work += gridDim.x) {
        uint32_t ti, tj;
        if (!tile_of(s, work, &ti, &tj)) continue;
        const uint32_t i0 = ti * BM, j0 = tj * BN;
        const uint32_t n = static_cast<uint32_t>(s.n);
        const uint32_t all = (s.k + kStep - 1) / kStep;
        const uint32_t s0 = blockIdx.y * s.per_split;
        const uint32_t s1 = s0 + s.per_split < all ? s0 + s.per_split : all;
        const uint32_t whole = s.k / kStep;               // steps before the last, short one
        const uint8_t *const base_a = qa + static_cast<uint64_t>(i0) * s.k;
        const uint8_t *const base_b = qb + static_cast<uint64_t>(j0) * s.k;
        const uint8_t *const base_e = ea + static_cast<uint64_t>(i0) * s.blocks_a;

        // staging: this lane's unit of 16 columns and its rows
        const uint32_t unit = threadIdx.x & 7u, row0 = threadIdx.x >> 3;
        uint32_t off_a[PA], off_b[PB];
#pragma unroll
        for (int p = 0; p < PA; ++p) {
            const uint32_t r = row0 + p * kRows, last = s.m - 1 - i0;
            off_a[p] = (r < last ? r : last) * s.k + unit * 16;
        }
#pragma unroll
        for (int p = 0; p < PB; ++p) {
            const uint32_t r = row0 + p * kRows, last = n - 1 - j0;
            off_b[p] = (r < last ? r : last) * s.k + unit * 16;
        }
        const uint32_t erow = threadIdx.x < s.m - 1 - i0 ? threadIdx.x : s.m - 1 - i0;
        const uint32_t off_e = erow * s.blocks_a;
        const uint32_t jb = j0 + bn < n ? (j0 + bn) >> 7 : (n - 1) >> 7;
        const uint8_t *const row_eb = eb + static_cast<uint64_t>(jb) * s.blocks_b;
        u32x4 xa[PA], xb[PB];
        uint32_t xe, xeb;

        // The unit of 16 columns from column c of a row on, where the row ends inside it or
        // before it: the row's last 16 bytes, moved down, zeros above.
        auto tail = [&](const uint8_t *base, uint32_t row_at, uint32_t c) {
            u32x4 v{0u, 0u, 0u, 0u};
            if (c < s.k) {
                const uint32_t have = s.k - c < 16 ? s.k - c : 16u;
                v = *(const GLOBAL_AS u32x4_any *)at_offset(base, row_at + c + have - 16);
                uint64_t lo = v[0] | static_cast<uint64_t>(v[1]) << 32;
                uint64_t hi = v[2] | static_cast<uint64_t>(v[3]) << 32;
                const uint32_t by = 8 * (16 - have);
                if (by >= 64) {
                    lo = hi >> (by - 64);
                    hi = 0;
                } else if (by > 0) {
                    lo = lo >> by | hi << (64 - by);
                    hi >>= by;
                }
                v = u32x4{static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32),
                          static_cast<uint32_t>(hi), static_cast<uint32_t>(hi >> 32)};
            }
            return v;
        };
        auto load_whole = [&](uint32_t st) {
            const uint8_t *const pa = base_a + static_cast<uint64_t>(st) * kStep;
            const uint8_t *const pb = base_b + static_cast<uint64_t>(st) * kStep;
#pragma unroll
            for (int p = 0; p < PA; ++p)
                xa[p] = *(const GLOBAL_AS u32x4_any *)at_offset(pa, off_a[p]);
#pragma unroll
            for (int p = 0; p < PB; ++p)
                xb[p] = *(const GLOBAL_AS u32x4_any *)at_offset(pb, off_b[p]);
        };
        auto load_tail = [&](uint32_t st) {
            const uint32_t c = st * kStep + unit * 16;
#pragma unroll
            for (int p = 0; p < PA; ++p) xa[p] = tail(base_a, off_a[p] - unit * 16, c);
#pragma unroll
            for (int p = 0; p < PB; ++p) xb[p] = tail(base_b, off_b[p] - unit * 16, c);
        };
        // exponents of step st: a row's four bytes (one for each 32 columns; a block of 128
        // has the same in all), and the byte of this wave's block of b
        auto load_exponents = [&](uint32_t st) {
            if (s.shift_a == 7) {
                xe = *at_offset(base_e + st, off_e) * 0x01010101u;
            } else if (st * 4 + 4 <= s.blocks_a) {
                typedef uint32_t u32_any __attribute__((aligned(1)));
                xe = *(const GLOBAL_AS u32_any *)at_offset(base_e + st * 4, off_e);
            } else {
                xe = 0x7f7f7f7fu;
                for (uint32_t j = 0; st * 4 + j < s.blocks_a; ++j)
                    xe = (xe & ~(0xffu << (8 * j))) |
                         static_cast<uint32_t>(*at_offset(base_e + st * 4 + j, off_e)) << (8 * j);
            }
            xeb = row_eb[st];
        };
        auto load = [&](uint32_t st) {
            if (st < whole)
                load_whole(st);
            else
                load_tail(st);
            load_exponents(st);
        };
        auto place = [](uint32_t r, uint32_t c) { return r * kStep + ((c ^ ((r >> 1) & 7u)) << 4); };
        auto stage = [&](uint32_t buf) {
#pragma unroll
            for (int p = 0; p < PA; ++p)
                *reinterpret_cast<u32x4 *>(&sa[buf][place(row0 + p * kRows, unit)]) = xa[p];
#pragma unroll
            for (int p = 0; p < PB; ++p)
                *reinterpret_cast<u32x4 *>(&sb[buf][place(row0 + p * kRows, unit)]) = xb[p];
            if (kLanes == BM || threadIdx.x < BM) se[buf][threadIdx.x] = xe;
        };

        f32x16 acc[TM][TN];
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
        uint32_t wa[TM], wb = 127u;       // exponents of the step in hand

        // MFMA step kk (64 columns) of buffer buf
        auto fragment = [&](const uint8_t *t, uint32_t r, int kk) {
            const u32x4 lo = *reinterpret_cast<const u32x4 *>(&t[place(r, kk * 4 + half)]);
            const u32x4 hi = *reinterpret_cast<const u32x4 *>(&t[place(r, kk * 4 + 2 + half)]);
            i32x8 v;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] = static_cast<int>(lo[j]);
                v[4 + j] = static_cast<int>(hi[j]);
            }
            return v;
        };
        auto multiply = [&](auto KK, uint32_t buf) {
            constexpr int kk = decltype(KK)::value;
            i32x8 a[TM], b[TN];
#pragma unroll
            for (int i = 0; i < TM; ++i) a[i] = fragment(sa[buf], am + i * 32 + row32, kk);
#pragma unroll
            for (int j = 0; j < TN; ++j) b[j] = fragment(sb[buf], bn + j * 32 + row32, kk);
            if constexpr (EIGHT) {
#pragma unroll
                for (int j = 0; j < TN; ++j)
#pragma unroll
                    for (int i = 0; i < TM; ++i)
                        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                            a[i], b[j], acc[i][j], 0, 0, kk * 2,
                            static_cast<int>(wa[i] >> (8 * half)), 0, static_cast<int>(wb));
            } else {
                const float scale_b = half_scale(wb);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    bf16x8 c[TN];
#pragma unroll
                    for (int j = 0; j < TN; ++j)
                        c[j] = codes_to_bf16(static_cast<uint32_t>(b[j][2 * q]),
                                             static_cast<uint32_t>(b[j][2 * q + 1]), scale_b);
#pragma unroll
                    for (int i = 0; i < TM; ++i) {
                        const bf16x8 d = codes_to_bf16(static_cast<uint32_t>(a[i][2 * q]),
                                                       static_cast<uint32_t>(a[i][2 * q + 1]),
                                                       half_scale((wa[i] >> (8 * (kk * 2 + q / 2))) & 0xffu));
#pragma unroll
                        for (int j = 0; j < TN; ++j)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(d, c[j], acc[i][j],
                                                                                0, 0, 0);
                    }
                }
            }
        };

        uint32_t eb_next = 127u;
        if (s0 < s1) {
            load(s0);
            stage(0);
            eb_next = xeb;
            if (s0 + 1 < s1) load(s0 + 1);
            __syncthreads();
        }
        for (uint32_t st = s0; st < s1; ++st) {
            const uint32_t buf = (st - s0) & 1u;
            wb = eb_next;
#pragma unroll
            for (int i = 0; i < TM; ++i) wa[i] = se[buf][am + i * 32 + row32];
            if (st + 1 < s1) {
                stage(buf ^ 1u);
                eb_next = xeb;
                if (st + 2 < s1) load(st + 2);
            }
            multiply(std::integral_constant<int, 0>{}, buf);
            multiply(std::integral_constant<int, 1>{}, buf);
            __syncthreads();
        }

        if constexpr (!EIGHT) {
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j)
#pragma unroll
                    for (int r = 0; r < 16; ++r) acc[i][j][r] = acc[i][j][r] * kUnhalve;
        }
        // result register r of a lane: row 8 (r / 4) + 4 half + r mod 4, column lane mod 32
        if constexpr (!SPLIT && F != 2) {
            // each wave turns 32 rows at a time through its part of LDS into whole lines
            constexpr uint32_t W = BN / WN, kPerRow = W / 8, kAtOnce = 64 / kPerRow;
            constexpr uint32_t kSwap = W >= 64 ? 32 : 0;
            static_assert(WM * WN * 32 * W * 2 <= 2 * BM * kStep, "room for 32 rows a wave");
            uint16_t *const mine = reinterpret_cast<uint16_t *>(&sa[0][0]) + wave * (32 * W);
            const uint32_t c = lane % kPerRow * 8, col = j0 + bn + c;
#pragma unroll
            for (int i = 0; i < TM; ++i) {
#pragma unroll
                for (int j = 0; j < TN; ++j)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        mine[(8 * (r / 4) + 4 * half + r % 4) * W +
                             ((j * 32 + row32) ^ (half * kSwap))] = from_f32<F>(acc[i][j][r]);
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
                for (uint32_t r0 = 0; r0 < 32; r0 += kAtOnce) {
                    const uint32_t r = r0 + lane / kPerRow, row = i0 + am + i * 32 + r;
                    if (row >= s.m || col >= n) continue;
                    const uint16_t *v = &mine[r * W + (c ^ (((r >> 2) & 1u) * kSwap))];
                    uint16_t *d = static_cast<uint16_t *>(y) + row * s.ldy + col;
                    if (col + 8 <= n) {
                        *reinterpret_cast<u32x4_any *>(d) = *reinterpret_cast<const u32x4 *>(v);
                    } else {
                        for (uint32_t t = 0; t < n - col; ++t) d[t] = v[t];
                    }
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
            }
        } else {
            float *const out = static_cast<float *>(y) +
                               (SPLIT ? blockIdx.y * (static_cast<uint64_t>(s.m) * s.n) : 0ull);
            const uint64_t ld = SPLIT ? s.n : s.ldy;
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const uint32_t row = i0 + am + i * 32 + 8 * (r / 4) + 4 * half + r % 4;
                    if (row >= s.m) continue;
#pragma unroll
                    for (int j = 0; j < TN; ++j) {
                        const uint32_t col = j0 + bn + j * 32 + row32;
                        if (col < n) out[row * ld + col] = acc[i][j][r];
                    }
                }
        }
        __syncthreads();   // the next tile writes LDS
    }
}

// y = the sum of `splits` planes of m x n FP32 values, in split order.
template <int F>
__global__ __launch_bounds__(kThreads) void product_join_kernel(elem_t<F> *__restrict__ y,
                                                               uint64_t ldy,
                                                               const float *__restrict__ part,
                                                               uint64_t m, uint64_t n,
                                                               uint32_t splits) {
    const uint64_t total = m * n;
    for (uint64_t at = static_cast<uint64_t>(blockIdx.x) * kThreads + threadIdx.x; at < total;
         at += static_cast<uint64_t>(gridDim.x) * kThreads) {
        float sum = part[at];
        for (uint32_t p = 1; p < splits; ++p) sum = sum + part[p * total + at];
        const uint64_t i = at / n;
        y[i * ldy + (at - i * n)] = from_f32<F>(sum);
    }
}

// One result a lane, element by element: for the few products whose rows are too short for
// the tiles.
template <int F>
__global__ __launch_bounds__(kThreads) void product_plain_kernel(
    elem_t<F> *__restrict__ y, const uint8_t *__restrict__ qa, const uint8_t *__restrict__ ea,
    const uint8_t *__restrict__ qb, const uint8_t *__restrict__ eb, ProductShape s) {
    const uint64_t total = s.m * s.n;
    for (uint64_t at = static_cast<uint64_t>(blockIdx.x) * kThreads + threadIdx.x; at < total;
         at += static_cast<uint64_t>(gridDim.x) * kThreads) {
        const uint64_t i = at / s.n, j = at - i * s.n;
        float sum = 0.0f;
        for (uint32_t c = 0; c < s.k; ++c) {
            const int e = static_cast<int>(ea[i * s.blocks_a + (c >> s.shift_a)]) +
                          static_cast<int>(eb[(j >> 7) * s.blocks_b + (c >> 7)]) - 254;
            const float p = code_value(qa[i * s.k + c]) * code_value(qb[j * s.k + c]);
            sum = sum + __builtin_amdgcn_ldexpf(p, e);
        }
        y[i * s.ldy + j] = from_f32<F>(sum);
    }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void zero_matrix_kernel(T *__restrict__ y, uint64_t ldy,
                                                              uint64_t cols, uint64_t total) {
    for (uint64_t at = static_cast<uint64_t>(blockIdx.x) * kThreads + threadIdx.x; at < total;
         at += static_cast<uint64_t>(gridDim.x) * kThreads) {
        const uint64_t i = at / cols;
        y[i * ldy + (at - i * cols)] = T(0);
    }
}

uint32_t capped(uint64_t n) {
    const uint64_t cap = max_blocks();
    return static_cast<uint32_t>(n < cap ? n : cap);
}

// Tile and splits of a call, by its extents alone (so the workspace and the order of the
// sums do not depend on the device).
struct Plan {
    uint32_t tile;        // rows of a and of b
    uint32_t splits;
    uint32_t per_split;   // steps of 128 columns
};

constexpr uint64_t kFill = 256;              // compute units of the chip
constexpr uint64_t kMaxLength = 1ull << 24;  // a tile's rows stay below 2^32 bytes

struct TileCost {
    uint32_t tile, step, ends;   // ns: a step of 128 columns, a tile's start and end
};
constexpr TileCost kTiles[3] = {{256, 1100, 8000}, {128, 500, 4000}, {64, 300, 2500}};

Plan plan_of(uint64_t m, uint64_t n, uint64_t k) {
    const uint64_t steps = (k + kStep - 1) / kStep;
    const uint64_t plane_ns = m * n / 1000;
    Plan best{0, 1, 0};
    uint64_t best_ns = ~0ull;
    for (const TileCost &c : kTiles) {
        const uint64_t tiles = ((m + c.tile - 1) / c.tile) * ((n + c.tile - 1) / c.tile);
        for (uint64_t s = 1; s <= 64 && s <= steps && (s == 1 || tiles * s <= 2 * kFill); ++s) {
            const uint64_t per = (steps + s - 1) / s, used = (steps + per - 1) / per;
            if (used != s) continue;
            const uint64_t rounds = (tiles * s + kFill - 1) / kFill;
            uint64_t ns = rounds * (per * c.step + c.ends);
            if (s > 1) ns += 5000 + s * (plane_ns + 150);
            if (ns < best_ns) {
                best_ns = ns;
                best = Plan{c.tile, static_cast<uint32_t>(s), static_cast<uint32_t>(per)};
            }
        }
    }
    return best;
}

bool tiled(uint64_t k) { return k >= 16 && k < kMaxLength; }

template <int F, bool EIGHT, bool SPLIT>
hipError_t tiles_of(const ProductArgs &a, const ProductShape &s, const Plan &p,
                    hipStream_t stream) {
    const dim3 grid(capped(s.work), p.splits);
    void *out = SPLIT ? a.workspace : a.y;
#define ZS_TILE(B, WM, WN)                                                                   \
    product_tile_kernel<F, EIGHT, SPLIT, B, B, WM, WN>                                       \
        <<<grid, 64 * WM * WN, 0, stream>>>(out, a.qa, a.ea, a.qb, a.eb, s)
    if (p.tile == 256)
        ZS_TILE(256, 4, 2);
    else if (p.tile == 128)
        ZS_TILE(128, 2, 2);
    else
        ZS_TILE(64, 2, 2);
#undef ZS_TILE
    return hipGetLastError();
}

template <int F>
hipError_t product_as(const ProductArgs &a, hipStream_t stream) {
    auto *const y = static_cast<elem_t<F> *>(a.y);
    const Plan p = plan_of(a.m, a.n, a.k);
    const uint64_t tiles_m = (a.m + p.tile - 1) / p.tile, tiles_n = (a.n + p.tile - 1) / p.tile;
    ProductShape s{a.ldy,
                   a.n,
                   static_cast<uint32_t>(a.m),
                   static_cast<uint32_t>(a.k),
                   static_cast<uint32_t>((a.k + a.a_block - 1) / a.a_block),
                   static_cast<uint32_t>((a.k + ZERO_BLOCK - 1) / ZERO_BLOCK),
                   a.a_block == ZERO_BLOCK ? 7u : 5u,
                   p.per_split,
                   static_cast<uint32_t>(tiles_m),
                   static_cast<uint32_t>(tiles_n),
                   0,
                   tiles_m * tiles_n};
    if (!tiled(a.k)) {
        product_plain_kernel<F><<<capped((a.m * a.n + kThreads - 1) / kThreads), kThreads, 0,
                                  stream>>>(y, a.qa, a.ea, a.qb, a.eb, s);
        return hipGetLastError();
    }
    // groups where they leave few places empty (empty ones cost the XCDs' balance)
    for (uint32_t gn = 8; gn > 0 && s.group_n == 0 && s.work >= kFill; gn /= 2) {
        const uint64_t gm = 32 / gn;
        const uint64_t groups = ((tiles_m + gm - 1) / gm) * ((tiles_n + gn - 1) / gn);
        const uint64_t places = (groups + 7) / 8 * 8 * 32;
        if (places * 8 <= s.work * 9) {
            s.group_n = gn;
            s.work = places;
        }
    }
    if (p.splits == 1) return tiles_of<F, F != 2, false>(a, s, p, stream);
    const hipError_t e = tiles_of<F, F != 2, true>(a, s, p, stream);
    if (e != hipSuccess) return e;
    product_join_kernel<F><<<capped((a.m * a.n + kThreads - 1) / kThreads), kThreads, 0, stream>>>(
        y, a.ldy, static_cast<const float *>(a.workspace), a.m, a.n, p.splits);
    return hipGetLastError();
}

}  // namespace

uint64_t product_workspace(uint64_t m, uint64_t n, uint64_t k) {
    if (!tiled(k)) return 0;
    const Plan p = plan_of(m, n, k);
    return p.splits == 1 ? 0 : 4 * m * n * p.splits;
}

hipError_t launch_product(const ProductArgs &a, int fmt, hipStream_t stream) {
    if (fmt == 0) return product_as<0>(a, stream);
    if (fmt == 1) return product_as<1>(a, stream);
    return product_as<2>(a, stream);
}

hipError_t launch_zero_matrix(void *y, uint64_t ldy, int fmt, uint64_t rows, uint64_t cols,
                              hipStream_t stream) {
    const uint64_t total = rows * cols;
    const uint32_t grid = capped((total + kThreads - 1) / kThreads);
    if (fmt == 2)
        zero_matrix_kernel<<<grid, kThreads, 0, stream>>>(static_cast<uint32_t *>(y), ldy, cols,
                                                          total);
    else
        zero_matrix_kernel<<<grid, kThreads, 0, stream>>>(static_cast<uint16_t *>(y), ldy, cols,
                                                          total);
    return hipGetLastError();
}

}  // namespace zs
