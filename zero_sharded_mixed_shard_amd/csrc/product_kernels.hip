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
// What bounds the large tiles: the matrix cores, at the clock that their power leaves (8192^3
// BF16: busy in 64% of the cycles, 425 us, 2.59 PFLOP/s), and between a workgroup's tiles their
// results, which all compute units store at once (16384 x 8192 x 4096: 448 us, 2.45 PFLOP/s).
// These are means over calls in a row; the first twenty after an idle time take 460 to 650 while
// the clock settles, so that the mean of sixty from there is 483.  Codes of full spread take 2%
// longer.  The library's FP8 product, in turn with these on one card: 340 and 365 us.  FP32
// results of the latter extents 883 us (1.25 PFLOP/s).  1 x 8192 x 8192 15.6 us (4.3 TB/s of
// codes), 61 x 50257 x 768 FP32 13.
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

__device__ __forceinline__ uint32_t uniform(uint32_t x) {
    return static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(x)));
}

// A pointer `bytes` past one that is the same in every lane, the base in scalar registers.
// (readfirstlane: what the compiler knows to be the same costs nothing, and of the rest it
// loses sight in divisions and loops.)
template <typename T>
__device__ __forceinline__ const GLOBAL_AS T *at_offset(const T *base, uint32_t bytes) {
    const uint64_t p = reinterpret_cast<uint64_t>(base);
    const uint64_t u = uniform(static_cast<uint32_t>(p)) |
                       static_cast<uint64_t>(uniform(static_cast<uint32_t>(p >> 32))) << 32;
    auto *b = (const GLOBAL_AS char *)(u);
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

// The scale of an exponent byte below the largest: BF16 holds all that a code stands for under
// it, from 2^-133, its smallest number, on.  Codes of 256 and more under the largest byte are
// past its end: results that such blocks have a part in are made element by element (see
// store_plain).
constexpr uint32_t kTopByte = 247;
__device__ __forceinline__ float bf16_scale(uint32_t e) { return from_bits(e << 23); }
// Not zero: some byte of a word is 247 or more (bit 7 is set, and the rest is 119 or more).
__device__ __forceinline__ uint32_t top_bytes(uint32_t w) {
    return ((w & 0x7f7f7f7fu) + 0x09090909u) & w & 0x80808080u;
}

// Order of a scheduling region that holds M MFMAs, R LDS reads, W LDS writes and G memory
// reads: each kind dealt evenly between the MFMAs.
template <int I, int M, int R, int W, int G>
__device__ __forceinline__ void deal() {
    if constexpr (I < M) {
        constexpr int kTo = I + 1;
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        if constexpr (R * kTo / M > R * I / M)
            __builtin_amdgcn_sched_group_barrier(0x100, R * kTo / M - R * I / M, 0);
        if constexpr (W * kTo / M > W * I / M)
            __builtin_amdgcn_sched_group_barrier(0x200, W * kTo / M - W * I / M, 0);
        if constexpr (G * kTo / M > G * I / M)
            __builtin_amdgcn_sched_group_barrier(0x020, G * kTo / M - G * I / M, 0);
        deal<I + 1, M, R, W, G>();
    }
}
template <bool EIGHT, int M, int R, int W, int G>
__device__ __forceinline__ void interleave() {
    if constexpr (EIGHT) deal<0, M, R, W, G>();
    __builtin_amdgcn_sched_barrier(0);
}

constexpr uint32_t kStep = 128;   // columns a step

struct ProductShape {
    uint64_t ldy, n;
    uint32_t m, k;
    uint32_t blocks_a, blocks_b;   // exponent bytes a row of a, and of b's blocks
    uint32_t shift_a;              // log2 of a's block
    uint32_t per_split;            // steps a split
    uint32_t tiles_n;
    uint64_t work;                 // tiles, along n first (grouped by XCD they took the same time)
};

// Columns c0 to c1 of one result.  Summed in FP64, where products are exact and 2^31 of them lose
// nothing that FP32 shows (a single FP32 sum of 2^24 ones and more stays at 2^24).
__device__ __forceinline__ float plain_sum(const uint8_t *__restrict__ qa,
                                           const uint8_t *__restrict__ ea,
                                           const uint8_t *__restrict__ qb,
                                           const uint8_t *__restrict__ eb, const ProductShape &s,
                                           uint64_t i, uint64_t j, uint32_t c0, uint32_t c1) {
    double sum = 0.0;
    for (uint32_t c = c0; c < c1; ++c) {
        const int e = static_cast<int>(ea[i * s.blocks_a + (c >> s.shift_a)]) +
                      static_cast<int>(eb[(j >> 7) * s.blocks_b + (c >> 7)]) - 254;
        const float p = code_value(qa[i * s.k + c]) * code_value(qb[j * s.k + c]);
        sum = sum + __builtin_amdgcn_ldexp(static_cast<double>(p), e);
    }
    return static_cast<float>(sum);
}

// BM x BN tiles of y (or, SPLIT, of a split's FP32 plane); WM x WN waves.  EIGHT: the 8-bit
// instruction.  A32: a's blocks are of 32 columns.  RAGGED: the last step is short.  Rows past
// the matrix are read as its last one and not stored; columns past it are zeros.  k >= 16, and a
// tile's rows span less than 4 GiB (the launcher checks both).
//
// b's rows are the matrix instruction's rows and a's its columns, so that a lane holds four
// neighbours of a row of y.
template <int F, bool EIGHT, bool SPLIT, bool A32, bool RAGGED, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, BM == 256 ? 1 : BM == 64 && !EIGHT ? 4 : 2)
void product_tile_kernel(
    void *__restrict__ y, const uint8_t *__restrict__ qa, const uint8_t *__restrict__ ea,
    const uint8_t *__restrict__ qb, const uint8_t *__restrict__ eb, ProductShape s) {
    constexpr int kLanes = 64 * WM * WN;
    constexpr int TM = BM / WM / 32, TN = BN / WN / 32;   // 32 x 32 results a wave
    constexpr int kRows = kLanes / 8;                     // rows a pass of staging
    constexpr int PA = BM / kRows, PB = BN / kRows;
    static_assert(kLanes >= BM && BN / WN <= 128, "exponents: a lane a row, a byte a wave");
    static_assert(kRows % 16 == 0, "a lane's rows share its unit's place");
    __shared__ __align__(16) uint8_t sa[2][BM * kStep];
    __shared__ __align__(16) uint8_t sb[2][BN * kStep];
    __shared__ uint32_t se[2][kLanes];   // (of the first BM rows; the rest is not read)
    // CHAIN: a workgroup's tiles are one long run of steps: the next tile's first ones are
    // requested, staged and read into registers as the last ones of this are multiplied, and
    // its results are stored beside them, through LDS of their own.
    constexpr bool CHAIN = BM == 256;
    constexpr uint32_t kTurn = 32 * 128;   // bytes a wave turns at a time: 32 rows of a line
    __shared__ __align__(16) uint8_t sc[CHAIN ? WM * WN * kTurn : 16];

    const uint32_t lane = threadIdx.x & 63u;
    const uint32_t wave =
        static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6));
    const uint32_t half = lane >> 5, row32 = lane & 31u;
    const uint32_t am = wave % WM * (BM / WM), bn = wave / WM * (BN / WN);
    const uint32_t n = static_cast<uint32_t>(s.n);
    const uint32_t whole = s.k / kStep;               // steps before the last, short one
    const uint32_t all = whole + (RAGGED ? 1 : 0);
    const uint32_t s0 = blockIdx.y * s.per_split;
    const uint32_t s1 = s0 + s.per_split < all ? s0 + s.per_split : all;

    // Staging: this lane's unit of 16 columns and its rows.  LDS places: rows that a lane
    // visits are multiples of 16 apart, so that its unit's place in a row is the same in all of
    // them and the rest are constant offsets.
    const uint32_t unit = threadIdx.x & 7u, row0 = threadIdx.x >> 3;
    const uint32_t put = row0 * kStep + ((unit ^ ((row0 >> 1) & 7u)) << 4);
    uint32_t get[4];   // unit 4 kk + 2 x + half of a row, at 2 kk + x
#pragma unroll
    for (int c = 0; c < 4; ++c)
        get[c] = row32 * kStep + (((2u * c + half) ^ ((row32 >> 1) & 7u)) << 4);

    struct Tile {
        uint32_t i0, j0;   // its first row and column
    };
    auto tile_at = [&](uint64_t w) {
        const uint64_t i = w / s.tiles_n;
        return Tile{uniform(static_cast<uint32_t>(i)) * BM,
                    uniform(static_cast<uint32_t>(w - i * s.tiles_n)) * BN};
    };

    // what is requested: step `ask` of tile `from`
    Tile from{0, 0};
    uint32_t ask = s0;
    uint32_t off_a[PA], off_b[PB], off_e = 0;
    u32x4 xa[PA], xb[PB];
    uint32_t xe = 0, xeb = 0;
    auto aim = [&]() {
        const uint32_t last_a = s.m - 1 - from.i0, last_b = n - 1 - from.j0;
#pragma unroll
        for (int p = 0; p < PA; ++p) {
            const uint32_t r = row0 + p * kRows;
            off_a[p] = (r < last_a ? r : last_a) * s.k + (RAGGED ? 0u : unit * 16);
        }
#pragma unroll
        for (int p = 0; p < PB; ++p) {
            const uint32_t r = row0 + p * kRows;
            off_b[p] = (r < last_b ? r : last_b) * s.k + (RAGGED ? 0u : unit * 16);
        }
        off_e = (threadIdx.x < last_a ? threadIdx.x : last_a) * s.blocks_a;
    };
    auto base_a = [&]() { return qa + static_cast<uint64_t>(uniform(from.i0)) * s.k; };
    auto base_b = [&]() { return qb + static_cast<uint64_t>(uniform(from.j0)) * s.k; };
    auto base_e = [&]() { return ea + static_cast<uint64_t>(uniform(from.i0)) * s.blocks_a; };
    auto byte_b = [&](uint32_t st) {
        const uint32_t j = uniform(from.j0) + bn;
        return eb[static_cast<uint64_t>((j < n ? j : n - 1) >> 7) * s.blocks_b + st];
    };
    // A short step's unit that the row ends in or before is read as the row's last 16 columns
    // (and moved down by trim() before it is staged), so that requests do not branch: what
    // comes from two branches is waited for where they meet.
    auto column = [&](uint32_t st) {
        const uint32_t c = st * kStep + unit * 16;
        return c + 16 <= s.k ? c : s.k - 16;
    };
    auto load_a = [&](uint32_t st) {
        const uint8_t *const p0 =
            base_a() + (RAGGED ? 0ull : static_cast<uint64_t>(uniform(st)) * kStep);
        const uint32_t c = RAGGED ? column(st) : 0u;
#pragma unroll
        for (int p = 0; p < PA; ++p)
            xa[p] = *(const GLOBAL_AS u32x4_any *)at_offset(p0, off_a[p] + c);
    };
    auto load_b = [&](uint32_t st) {
        const uint8_t *const p0 =
            base_b() + (RAGGED ? 0ull : static_cast<uint64_t>(uniform(st)) * kStep);
        const uint32_t c = RAGGED ? column(st) : 0u;
#pragma unroll
        for (int p = 0; p < PB; ++p)
            xb[p] = *(const GLOBAL_AS u32x4_any *)at_offset(p0, off_b[p] + c);
    };
    // exponents of step st: a row's four bytes (one for each 32 columns; a block of 128 has the
    // same in all; past the row's end the last), and the byte of this wave's block of b
    auto load_exponents = [&](uint32_t st) {
        typedef uint32_t u32_any __attribute__((aligned(1)));
        if constexpr (A32 && RAGGED) {
            const uint8_t *const p0 = base_e();
            const uint32_t last = s.blocks_a - 1, i = st * 4;
            xe = *at_offset(p0 + (i < last ? i : last), off_e);
#pragma unroll
            for (uint32_t j = 1; j < 4; ++j)
                xe |= static_cast<uint32_t>(*at_offset(p0 + (i + j < last ? i + j : last), off_e))
                      << (8 * j);
        } else if constexpr (A32) {
            xe = *(const GLOBAL_AS u32_any *)at_offset(base_e() + uniform(st) * 4, off_e);
        } else {
            xe = *at_offset(base_e() + uniform(st), off_e) * 0x01010101u;
        }
        xeb = byte_b(uniform(st));
    };
    uint32_t held = 0;   // the step that the staging registers hold
    auto load = [&](uint32_t st) {
        load_a(st);
        load_b(st);
        load_exponents(st);
        held = st;
    };
    // 16 columns moved down by `by`, zeros above
    auto move_down = [](u32x4 v, uint32_t by) {
        uint64_t lo = v[0] | static_cast<uint64_t>(v[1]) << 32;
        uint64_t hi = v[2] | static_cast<uint64_t>(v[3]) << 32;
        if (by >= 16) {
            lo = hi = 0;
        } else if (by >= 8) {
            lo = hi >> (8 * by - 64);
            hi = 0;
        } else if (by > 0) {
            lo = lo >> (8 * by) | hi << (64 - 8 * by);
            hi >>= 8 * by;
        }
        return u32x4{static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32),
                     static_cast<uint32_t>(hi), static_cast<uint32_t>(hi >> 32)};
    };
    auto trim = [&]() {
        if (!RAGGED || uniform(held) != whole) return;
        const uint32_t by = whole * kStep + unit * 16 - column(whole);
#pragma unroll
        for (int p = 0; p < PA; ++p) xa[p] = move_down(xa[p], by);
#pragma unroll
        for (int p = 0; p < PB; ++p) xb[p] = move_down(xb[p], by);
    };
    auto stage_a = [&](uint32_t buf) {
#pragma unroll
        for (int p = 0; p < PA; ++p)
            *reinterpret_cast<u32x4 *>(&sa[buf][put + p * (kRows * kStep)]) = xa[p];
        se[buf][threadIdx.x] = xe;
    };
    auto stage_b = [&](uint32_t buf) {
#pragma unroll
        for (int p = 0; p < PB; ++p)
            *reinterpret_cast<u32x4 *>(&sb[buf][put + p * (kRows * kStep)]) = xb[p];
    };

    // One request further: the next step, or the next tile's first one; nothing is left: the
    // last step again, which nothing reads.
    uint64_t asked = 0;
    auto advance = [&]() {
        if (ask + 1 < s1) {
            ++ask;
        } else if (CHAIN && asked + gridDim.x < s.work) {
            asked += gridDim.x;
            from = tile_at(asked);
            ask = s0;
            aim();
        }
    };

    f32x16 acc[TM][TN];
            // Fragments of MFMA step kk (64 columns), and their products
            constexpr int H = TN / 2;
            i32x8 a[2][TM], b[TN == 1 ? 2 : TN];
            uint32_t wa[TM], wb = 127u;
            auto fragment = [&](const uint8_t *t, int i, int kk) {
                const u32x4 lo = *reinterpret_cast<const u32x4 *>(&t[get[2 * kk] + i * (32 * kStep)]);
                const u32x4 hi =
                    *reinterpret_cast<const u32x4 *>(&t[get[2 * kk + 1] + i * (32 * kStep)]);
                i32x8 v;
    #pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[j] = static_cast<int>(lo[j]);
                    v[4 + j] = static_cast<int>(hi[j]);
                }
                return v;
            };
            auto read_a = [&](int f, uint32_t buf, int kk) {
    #pragma unroll
                for (int i = 0; i < TM; ++i) a[f][i] = fragment(&sa[buf][am * kStep], i, kk);
            };
            auto read_b = [&](int from, int to, uint32_t buf, int kk) {
    #pragma unroll
                for (int j = from; j < to; ++j)
                    b[TN == 1 ? kk : j] = fragment(&sb[buf][bn * kStep], j, kk);
            };
            auto read_exponents = [&](uint32_t buf) {
    #pragma unroll
                for (int i = 0; i < TM; ++i)
                    wa[i] = se[buf][am + i * 32 + row32] >> (EIGHT ? 8 * half : 0);
            };
            auto times = [&](auto KK, int from, int to) {
                constexpr int kk = decltype(KK)::value;
                if constexpr (EIGHT) {
    #pragma unroll
                    for (int j = from; j < to; ++j)
    #pragma unroll
                        for (int i = 0; i < TM; ++i)
                            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                                b[TN == 1 ? kk : j], a[kk][i], acc[i][j], 0, 0, 0,
                                static_cast<int>(wb), kk * 2, static_cast<int>(wa[i]));
                } else {
                    const float scale_b = bf16_scale(wb);
    #pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        bf16x8 d[TM];
    #pragma unroll
                        for (int i = 0; i < TM; ++i)
                            d[i] = codes_to_bf16(static_cast<uint32_t>(a[kk][i][2 * q]),
                                                 static_cast<uint32_t>(a[kk][i][2 * q + 1]),
                                                 bf16_scale((wa[i] >> (8 * (kk * 2 + q / 2))) & 0xffu));
    #pragma unroll
                        for (int j = from; j < to; ++j) {
                            const i32x8 &v = b[TN == 1 ? kk : j];
                            const bf16x8 c = codes_to_bf16(static_cast<uint32_t>(v[2 * q]),
                                                           static_cast<uint32_t>(v[2 * q + 1]),
                                                           scale_b);
    #pragma unroll
                            for (int i = 0; i < TM; ++i)
                                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(c, d[i], acc[i][j],
                                                                                    0, 0, 0);
                        }
                    }
                }
            };
            constexpr std::integral_constant<int, 0> k0{};
            constexpr std::integral_constant<int, 1> k1{};

    // A step.  Four scheduling regions, each half an MFMA step's products; a wave's LDS reads,
    // LDS writes and requests are dealt between its MFMAs.  Fragments are a region ahead: those
    // of b's first half and of a for the next MFMA step, those of b's second half as the first
    // half is multiplied.  The barrier stands where every wave has this buffer's last fragments
    // in registers and its share of the next buffer written.
    constexpr int B1 = TN > 1 ? H : 1;
    uint32_t eb_next = 127u, buf = 0;
    auto begin = [&]() {
        load(ask);
        trim();
        advance();
        stage_a(0);
        stage_b(0);
        eb_next = xeb;
        load(ask);
        __syncthreads();
        buf = 0;
        read_exponents(0);
        read_a(0, 0, 0);
        read_b(0, B1, 0, 0);
    };

    for (uint64_t work = blockIdx.x; work < s.work; work += gridDim.x) {
        const Tile tile = tile_at(work);
        if (!CHAIN || work == blockIdx.x) {
            asked = work;
            from = tile;
            ask = s0;
            aim();
            begin();
        }
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
        // of this lane's rows of a: A32, not zero where a block has the largest byte; else their
        // largest word (four times a byte); and the largest byte of b's blocks
        uint32_t top = 0, top_b = 0;
#pragma unroll 1
        for (uint32_t at = s0; at < s1; ++at) {
            trim();
            advance();   // (up here: with a branch behind them the products are moved past it)
            wb = eb_next;
            eb_next = xeb;
            if constexpr (!EIGHT) {
#pragma unroll
                for (int i = 0; i < TM; ++i)
                    if constexpr (A32)
                        top |= top_bytes(wa[i]);
                    else
                        top = wa[i] > top ? wa[i] : top;
                top_b = wb > top_b ? wb : top_b;
            }
            if constexpr (TN > 1) read_b(H, TN, buf, 0);
            read_a(1, buf, 1);
            if constexpr (TN == 1) read_b(0, 1, buf, 1);
            stage_a(buf ^ 1u);
            load_a(ask);
            load_exponents(ask);
            if constexpr (TN > 1) {
                times(k0, 0, H);
                interleave<EIGHT, TM * H, 2 * (TN - H) + 2 * TM, PA + 1, PA + 2>();
                read_b(0, H, buf, 1);
            }
            stage_b(buf ^ 1u);
            load_b(ask);
            held = ask;
            times(k0, H, TN);
            interleave<EIGHT, TM * (TN - H), 2 * H, PB, PB>();
            if constexpr (TN > 1) {
                read_b(H, TN, buf, 1);
                times(k1, 0, H);
                interleave<EIGHT, TM * H, 2 * (TN - H), 0, 0>();
            }
            __syncthreads();
            read_a(0, buf ^ 1u, 0);
            read_b(0, B1, buf ^ 1u, 0);
            times(k1, H, TN);
            interleave<EIGHT, TM * (TN - H), 2 * B1 + 2 * TM, 0, 0>();
            read_exponents(buf ^ 1u);
            buf ^= 1u;
        }
        if constexpr (!CHAIN) __syncthreads();   // LDS is free
        if constexpr (BM == 256) {
            // The results stay in the accumulation registers until they are stored: what leaves
            // a loop is else copied to vector registers all at once, which spills.  (The waits
            // are a matrix instruction's, should one be in flight.)
            asm volatile("s_nop 15\n\ts_nop 15");
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) asm volatile("" : "+a"(acc[i][j]));
        }
        // Result register r of a lane: row lane mod 32, columns 8 (r / 4) + 4 half + r mod 4.
        // Each wave turns 32 rows at a time through its part of LDS into whole lines; unit c of
        // four columns of row r lies at c ^ 2 (r mod 16) (and the same lower bits), so that the
        // lanes of a write fall on different banks.
        using T = elem_t<SPLIT ? 2 : F>;
        constexpr uint32_t W = BN / WN, kBytes = sizeof(T);
        constexpr uint32_t kPart = W * kBytes <= 128 ? W : 128 / kBytes;   // columns at a time
        constexpr uint32_t kUnits = kPart / 4, kLine = kPart * kBytes / 16, kAtOnce = 64 / kLine;
        constexpr uint32_t kMask = kUnits / 2 < 16 ? kUnits / 2 - 1 : 15;
        static_assert(32 * kPart * kBytes <= kTurn && WM * WN * kTurn <= 2 * BM * kStep, "room");
        uint8_t *const mine = (CHAIN ? sc : &sa[0][0]) + wave * kTurn;
        T *const out = static_cast<T *>(y) +
                       (SPLIT ? blockIdx.y * (static_cast<uint64_t>(s.m) * s.n) : 0ull);
        const uint64_t ld = SPLIT ? s.n : s.ldy;
        const uint32_t turn = (row32 & kMask) * 2;
        // store_plain: what a block of the largest byte makes of a sum may be past FP32
        if constexpr (!EIGHT) {
            if (__any((A32 ? top != 0 : top >> 24 >= kTopByte) || top_b >= kTopByte)) {
                const uint32_t end = s1 * kStep < s.k ? s1 * kStep : s.k;
#pragma unroll 1
                for (uint32_t at = lane; at < BM / WM * W; at += 64) {
                    const uint32_t row = tile.i0 + am + at / W, col = tile.j0 + bn + at % W;
                    if (row < s.m && col < n)
                        out[row * ld + col] =
                            from_f32<F>(plain_sum(qa, ea, qb, eb, s, row, col, s0 * kStep, end));
                }
                if constexpr (!CHAIN) __syncthreads();   // the next tile writes LDS
                continue;
            }
        }
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (uint32_t part = 0; part < W / kPart; ++part) {
#pragma unroll
                for (uint32_t j = part * (kPart / 32); j < (part + 1) * (kPart / 32); ++j)
#pragma unroll
                    for (uint32_t r = 0; r < 16; r += 4) {
                        const uint32_t u = ((j % (kPart / 32)) * 8 + r / 2 + half) ^ turn;
                        float v[4];
#pragma unroll
                        for (uint32_t t = 0; t < 4; ++t)
                            v[t] = acc[i][j][r + t];
                        if constexpr (kBytes == 2)
                            *reinterpret_cast<u32x2 *>(mine + row32 * (kPart * 2) + u * 8) =
                                u32x2{pack2<F>(v[0], v[1]), pack2<F>(v[2], v[3])};
                        else
                            *reinterpret_cast<f32x4 *>(mine + row32 * (kPart * 4) + u * 16) =
                                f32x4{v[0], v[1], v[2], v[3]};
                    }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
                const uint32_t c = lane % kLine;   // 16 B of a line
#pragma unroll
                for (uint32_t r0 = 0; r0 < 32; r0 += kAtOnce) {
                    const uint32_t r = r0 + lane / kLine, row = tile.i0 + am + i * 32 + r;
                    const uint32_t col = tile.j0 + bn + part * kPart + c * (16 / kBytes);
                    const uint32_t at = kBytes == 2 ? c ^ (r & kMask) : c ^ ((r & kMask) * 2);
                    const u32x4 v = *reinterpret_cast<const u32x4 *>(
                        mine + r * (kPart * kBytes) + at * 16);
                    if (row >= s.m || col >= n) continue;
                    T *d = out + row * ld + col;
                    if (col + 16 / kBytes <= n) {
                        __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any *>(d));
                    } else {
#pragma unroll
                        for (uint32_t t = 0; t < 16 / kBytes; ++t)
                            if (col + t < n) {
                                if constexpr (kBytes == 2)
                                    d[t] = static_cast<uint16_t>(v[t / 2] >> (16 * (t % 2)));
                                else
                                    d[t] = from_bits(v[t]);
                            }
                    }
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
            }
        if constexpr (!CHAIN) __syncthreads();   // the next tile writes LDS
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

// One result a lane, element by element: for the few products whose rows are too short or too
// long for the tiles.
template <int F>
__global__ __launch_bounds__(kThreads) void product_plain_kernel(
    elem_t<F> *__restrict__ y, const uint8_t *__restrict__ qa, const uint8_t *__restrict__ ea,
    const uint8_t *__restrict__ qb, const uint8_t *__restrict__ eb, ProductShape s) {
    const uint64_t total = s.m * s.n;
    for (uint64_t at = static_cast<uint64_t>(blockIdx.x) * kThreads + threadIdx.x; at < total;
         at += static_cast<uint64_t>(gridDim.x) * kThreads) {
        const uint64_t i = at / s.n, j = at - i * s.n;
        y[i * s.ldy + j] = from_f32<F>(plain_sum(qa, ea, qb, eb, s, i, j, 0, s.k));
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

// Measured on MI355X, in ns: a step of 128 columns of a tile that has a compute unit to itself,
// its share of one where several run side by side (`resident` at most), and a tile's start and
// end.  The large tile uses each operand most but fills and drains slowly; a small one starts
// quickly and is bound by latency.
struct TileCost {
    uint32_t tile, resident, alone, shared, ends;
};
constexpr TileCost kTiles[3] = {
    {256, 1, 1500, 1500, 9000}, {128, 2, 620, 500, 4000}, {64, 4, 400, 240, 3000}};

// The tile and splits of least estimated time; splits cost the join's launch and its planes,
// written and read.  The costs are those of 16-bit results; FP32 ones, whose steps take longer,
// share them.  Over ten shapes of 1 to 2048 rows, 768 to 50257 columns and 768 to 8192 summed
// ones the choice was within 5% of the best of every tile with 1 to 16 splits, for either kind of
// results, but for 16 x 4096 x 4096 (8 splits: 10.0 us, FP32 11.0; 4 splits: 8.3 and 9.7).
// 1024 x 1024 x 8192, for example, takes 24 us in 128 x 128 tiles and 4 splits (FP32 28), 28 in
// 64 x 64 and 2 (FP32 32), 38 in 256 x 256 and 8; 1 x 8192 x 8192 15.6 us in 64 x 64 and 4 (FP32
// 18), 30 in one.
Plan plan_of(uint64_t m, uint64_t n, uint64_t k) {
    const uint64_t steps = (k + kStep - 1) / kStep;
    Plan best{0, 1, 0};
    uint64_t best_ns = ~0ull;
    for (const TileCost &c : kTiles) {
        const uint64_t tiles = ((m + c.tile - 1) / c.tile) * ((n + c.tile - 1) / c.tile);
        for (uint64_t s = 1; s <= 64 && s <= steps && (s == 1 || tiles * s <= 4 * kFill); ++s) {
            const uint64_t per = (steps + s - 1) / s, used = (steps + per - 1) / per;
            if (used != s) continue;
            const uint64_t each = (tiles * s + kFill - 1) / kFill;   // of a compute unit
            const uint64_t beside = each < c.resident ? each : c.resident;
            const uint64_t step =
                beside * c.shared > c.alone ? beside * c.shared : c.alone;
            uint64_t ns = (each + c.resident - 1) / c.resident * (per * step + c.ends);
            if (s > 1) ns += 2500 + s * (m * n / 625);   // 8 B a result at 5 TB/s
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
    // workgroups that fill the chip once, each with its tiles in turn
    const uint64_t fill = kFill * (p.tile == 256 ? 1 : p.tile == 128 ? 2 : 4);
    const dim3 grid(capped(s.work < fill ? s.work : fill), p.splits);
    void *out = SPLIT ? a.workspace : a.y;
    const bool a32 = a.a_block == ZERO_ACT_BLOCK, ragged = a.k % kStep != 0;
#define ZS_FORM(A32, RAGGED, B, WM, WN)                                                      \
    product_tile_kernel<F, EIGHT, SPLIT, A32, RAGGED, B, B, WM, WN>                          \
        <<<grid, 64 * WM * WN, 0, stream>>>(out, a.qa, a.ea, a.qb, a.eb, s)
#define ZS_TILE(B, WM, WN)                                                                   \
    do {                                                                                     \
        if (a32 && ragged)                                                                   \
            ZS_FORM(true, true, B, WM, WN);                                                  \
        else if (a32)                                                                        \
            ZS_FORM(true, false, B, WM, WN);                                                 \
        else if (ragged)                                                                     \
            ZS_FORM(false, true, B, WM, WN);                                                 \
        else                                                                                 \
            ZS_FORM(false, false, B, WM, WN);                                                \
    } while (0)
    if (p.tile == 256)
        ZS_TILE(256, 2, 2);
    else if (p.tile == 128)
        ZS_TILE(128, 2, 2);
    else
        ZS_TILE(64, 2, 2);
#undef ZS_TILE
#undef ZS_FORM
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
                   static_cast<uint32_t>(tiles_n),
                   tiles_m * tiles_n};
    if (!tiled(a.k)) {
        product_plain_kernel<F><<<capped((a.m * a.n + kThreads - 1) / kThreads), kThreads, 0,
                                  stream>>>(y, a.qa, a.ea, a.qb, a.eb, s);
        return hipGetLastError();
    }
    if (p.splits == 1) return tiles_of<F, F != 2, false>(a, s, p, stream);
    // (planes are FP32 whatever the format: one set of kernels for both 16-bit ones)
    const hipError_t e = tiles_of<F == 0 ? 1 : F, F != 2, true>(a, s, p, stream);
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
