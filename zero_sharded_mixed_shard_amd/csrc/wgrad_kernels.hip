// gfx950 kernels of the weight gradient G[o, i] = sum over t of dy[t, o] v[t, i],
// v the values of an 8-bit activation checkpoint.
//
// The reduction runs over the tokens, the slow axis of both operands, while an
// MFMA lane wants eight consecutive reduction steps of one row.  Both tiles are
// staged in LDS as they lie in memory ([token][column]) and read with the
// transposing LDS read (four tokens of one column a lane and instruction).
// Codes become 16-bit floats on their way into LDS, where a row's exponent is the
// same for eight neighbours: one convert makes two exact values (code * 2^k has
// four significant bits), so products are exact and only the FP32 sum rounds.
//
// LDS columns are permuted in units of 16 (32 B): unit u of token t sits at
// u ^ 2 (t mod 4), so the four token rows that 16 lanes read at once, and the
// next 16 lanes' rows, fall on different banks (64-column tiles, whose rows are half
// the banks: u ^ (t & 2)).  Measured bank conflicts: none.
//
// The loop keeps one step of global loads in registers and two steps in LDS:
// step s multiplies buffer s mod 2 while step s+1 is written to the other and
// step s+2 is on its way from memory, with one barrier a step.
//
// Few tiles: the tokens are split over several blocks of a tile, which write FP32
// partial products; a second kernel adds them in split order.
//
// What bounds it: the matrix cores, at the clock that their power leaves.  16384 x 8192 x 4096
// BF16 takes 1.56e6 cycles, the cores busy in 67% of them: 866 to 890 us repeated alone (1.24
// to 1.27 PFLOP/s, about 1.78 GHz), 966 us on average (891 to 1025, as 4096 x 8192) among other
// operators.
// FP32 results 885 us; added to the FP32 accumulator 998 us, as an epilogue of its own reads
// and writes it in the accumulators' layout.  The 256 x 256 tile spills 27 vector registers
// with 16-bit results and 48 with FP32 ones, around the loop and not in its steady part.
#include "grad_device.h"

#pragma clang fp contract(off)

namespace zs {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

template <int F>
__device__ __forceinline__ f32x16 mfma(s16x8 a, s16x8 b, f32x16 c) {
    if constexpr (F == 0)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                      __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Eight codes of one block (exponent byte eb) as eight 16-bit floats.
template <int F>
__device__ __forceinline__ u32x4 codes_to_16(u32x2 c, uint32_t eb) {
    const float s = from_bits(eb << 23);
    u32x4 r;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if constexpr (F == 0) {
            r[2 * h] = __builtin_bit_cast(uint32_t,
                                          __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[h], s, false));
            r[2 * h + 1] = __builtin_bit_cast(
                uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[h], s, true));
        } else {
            r[2 * h] = __builtin_bit_cast(
                uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[h], s, false));
            r[2 * h + 1] = __builtin_bit_cast(
                uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[h], s, true));
        }
    }
    return r;
}

// Four tokens of one column: lanes 4r .. 4r+3 of each 16 address row r's 16 columns.
__device__ __forceinline__ s16x4 read_tr(const uint16_t *p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) s16x4 *)(p));
}

// A pointer `bytes` past one that is the same in every lane: the base is kept in
// scalar registers, so an access needs no address registers of its own.
template <bool WIDE> struct Offset { using T = uint32_t; };
template <> struct Offset<true> { using T = uint64_t; };
template <typename T, typename O>
__device__ __forceinline__ const GLOBAL_AS T *at_offset(const T *base, O bytes) {
    auto *b = (const GLOBAL_AS char *)(base);
    if constexpr (sizeof(O) == 4) asm("" : "+s"(b));
    return (const GLOBAL_AS T *)(b + bytes);
}

// Order of a scheduling region that holds M MFMAs, R LDS reads, V other vector
// operations, W LDS writes and G memory reads: each kind dealt evenly between the MFMAs.
template <int I, int M, int R, int V, int W, int G>
__device__ __forceinline__ void deal() {
    if constexpr (I < M) {
        constexpr int kFrom = I, kTo = I + 1;
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        if constexpr (R * kTo / M > R * kFrom / M)
            __builtin_amdgcn_sched_group_barrier(0x100, R * kTo / M - R * kFrom / M, 0);
        if constexpr (V * kTo / M > V * kFrom / M)
            __builtin_amdgcn_sched_group_barrier(0x002, V * kTo / M - V * kFrom / M, 0);
        if constexpr (W * kTo / M > W * kFrom / M)
            __builtin_amdgcn_sched_group_barrier(0x200, W * kTo / M - W * kFrom / M, 0);
        if constexpr (G * kTo / M > G * kFrom / M)
            __builtin_amdgcn_sched_group_barrier(0x020, G * kTo / M - G * kFrom / M, 0);
        deal<I + 1, M, R, V, W, G>();
    }
}
template <int M, int R, int V, int W, int G>
__device__ __forceinline__ void interleave() {
    deal<0, M, R, V, W, G>();
}

enum class Out { k16, k32, kAdd32 };   // 16-bit result, FP32 result, added to FP32

struct GradShape {
    uint64_t lddy;
    uint32_t tokens, n_out, n_in, blocks_in;   // blocks_in: exponent bytes a row
    uint32_t per_split;                        // tokens a split (whole steps)
    uint32_t tiles_out, tiles_in;
    uint32_t group_i;                          // tiles a group has along n_in, 0: no groups
    uint64_t work;                             // work items: tiles, or places in groups
};

// Tile of work item w: tiles in groups of `group_o` x `group_i` (32), groups dealt to
// the eight XCDs in turn (workgroups go round them by number), so that the 32 compute
// units of an XCD share operands in its L2 (4 x 8 tiles 943 us, 8 x 4 952 us, ungrouped
// 1003 us at 16384 x 8192 x 4096, same clock).  false: no such tile.
__device__ __forceinline__ bool tile_of(const GradShape &g, uint64_t w, uint32_t *o, uint32_t *i) {
    if (g.group_i == 0) {
        *o = static_cast<uint32_t>(w / g.tiles_in);
        *i = static_cast<uint32_t>(w - static_cast<uint64_t>(*o) * g.tiles_in);
        return true;
    }
    const uint32_t group_o = 32 / g.group_i, groups_in = (g.tiles_in + g.group_i - 1) / g.group_i;
    const uint64_t k = w >> 3, group = (k >> 5) * 8 + (w & 7);
    const uint32_t at = static_cast<uint32_t>(k & 31);
    const uint64_t go = group / groups_in;
    *o = static_cast<uint32_t>(go) * group_o + at % group_o;
    *i = static_cast<uint32_t>(group - go * groups_in) * g.group_i + at / group_o;
    return go * group_o < g.tiles_out && *o < g.tiles_out && *i < g.tiles_in;
}

// One BM x BN tile of G over one split of the tokens; WM x WN waves.
//
// Ragged edges.  A thread stages groups of eight columns.  The last group of a row
// is read eight columns back from the row's end, so it never leaves the row; its
// columns are the row's last eight, and the epilogue stores only those that no
// other group holds.  Groups past the row's end read the same columns and store
// nothing.  TINY (n_out or n_in below 8): element by element.  Tokens past the end
// of the split are read as its last token and replaced by zeros.
template <int F, Out O, int BM, int BN, int WM, int WN, int kStep, bool TINY>
__global__ __launch_bounds__(64 * WM * WN, 2) void weight_grad_kernel(
    void *__restrict__ out, const uint16_t *__restrict__ dy, const uint8_t *__restrict__ q,
    const uint8_t *__restrict__ e, GradShape g) {
    constexpr int kThreads = 64 * WM * WN;
    constexpr int TM = BM / WM / 32, TN = BN / WN / 32;     // 32x32 results a wave
    constexpr int kRowsA = kThreads * 8 / BM, kRowsB = kThreads * 8 / BN;  // rows a pass
    constexpr int PA = kStep / kRowsA, PB = kStep / kRowsB;                // passes a step
    constexpr int KK = kStep / 16;                                         // MFMA steps a step
    // two buffers of each tile; arrays of their own, so that the compiler may move reads of
    // one over writes of the other (one array for both: 3% slower)
    __shared__ __align__(16) uint16_t sa[2][kStep * BM];
    __shared__ __align__(16) uint16_t sb[2][kStep * BN];

    for (uint64_t work = blockIdx.x; work < g.work; work += gridDim.x) {
        const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
        uint32_t tile_o, tile_i;
        if (!tile_of(g, work, &tile_o, &tile_i)) continue;
        const uint32_t o0 = tile_o * BM, i0 = tile_i * BN;
        const uint64_t t_first = static_cast<uint64_t>(blockIdx.y) * g.per_split;
        const uint32_t t_begin = static_cast<uint32_t>(t_first < g.tokens ? t_first : g.tokens);
        const uint32_t t_end = static_cast<uint32_t>(
            t_first + g.per_split < g.tokens ? t_first + g.per_split : g.tokens);
        const uint32_t steps = (t_end - t_begin + kStep - 1) / kStep;

        // staging: this thread's eight columns and first row of each tile
        const uint32_t ca = threadIdx.x % (BM / 8) * 8, ra = threadIdx.x / (BM / 8);
        const uint32_t cb = threadIdx.x % (BN / 8) * 8, rb = threadIdx.x / (BN / 8);
        const uint32_t na = TINY ? (o0 + ca < g.n_out ? g.n_out - o0 - ca : 0u) : 8u;
        const uint32_t nb = TINY ? (i0 + cb < g.n_in ? g.n_in - i0 - cb : 0u) : 8u;
        const uint32_t col_a = TINY || o0 + ca + 8 <= g.n_out ? o0 + ca : g.n_out - 8;
        const uint32_t col_b = TINY || i0 + cb + 8 <= g.n_in ? i0 + cb : g.n_in - 8;
        const uint32_t blk_b = (i0 + cb < g.n_in ? i0 + cb : g.n_in - 1) / ZERO_ACT_BLOCK;
        // offsets of a lane from a row's start that is the same in every lane: 32 bits
        // (the launcher checks that kStep rows stay below 4 GiB; TINY takes any)
        using Off = typename Offset<TINY>::T;
        u32x4 xa[PA];
        u32x2 xb[PB];
        uint32_t eb[PB];
        auto get_a = [&](const uint16_t *row, Off off) {
            const GLOBAL_AS uint16_t *s = at_offset(row, off * 2);
            if constexpr (!TINY) return *(const GLOBAL_AS u32x4_any *)(s);
            u32x4 r{0u, 0u, 0u, 0u};
#pragma unroll
            for (uint32_t j = 0; j < 8; ++j)
                if (j < na) r[j / 2] |= static_cast<uint32_t>(s[j]) << (16 * (j % 2));
            return r;
        };
        auto get_b = [&](const uint8_t *row, Off off) {
            const GLOBAL_AS uint8_t *s = at_offset(row, off);
            if constexpr (!TINY) return *(const GLOBAL_AS u32x2_any *)(s);
            u32x2 r{0u, 0u};
#pragma unroll
            for (uint32_t j = 0; j < 8; ++j)
                if (j < nb) r[j / 4] |= static_cast<uint32_t>(s[j]) << (8 * (j % 4));
            return r;
        };
        const Off off_a = static_cast<Off>(ra) * static_cast<Off>(g.lddy) + col_a;
        const Off off_b = static_cast<Off>(rb) * g.n_in + col_b;
        const Off off_e = static_cast<Off>(rb) * g.blocks_in + blk_b;
        // step s into registers: a whole step, or (load_last) the last, perhaps short, one
        auto load_a = [&](uint32_t s) {
            const uint16_t *row = dy + static_cast<uint64_t>(t_begin + s * kStep) * g.lddy;
#pragma unroll
            for (int p = 0; p < PA; ++p)
                xa[p] = get_a(row + static_cast<uint64_t>(p * kRowsA) * g.lddy, off_a);
        };
        auto load_b = [&](uint32_t s) {
            const uint64_t t0 = t_begin + s * kStep;
#pragma unroll
            for (int p = 0; p < PB; ++p) {
                xb[p] = get_b(q + (t0 + p * kRowsB) * g.n_in, off_b);
                eb[p] = *at_offset(e + (t0 + p * kRowsB) * g.blocks_in, off_e);
            }
        };
        auto load_last = [&](uint32_t s) {
            const uint32_t t0 = t_begin + s * kStep, last = t_end - 1 - t0;
#pragma unroll
            for (int p = 0; p < PA; ++p) {
                const uint32_t t = ra + p * kRowsA, u = t < last ? t : last;
                xa[p] = get_a(dy + static_cast<uint64_t>(t0) * g.lddy,
                              static_cast<Off>(u) * static_cast<Off>(g.lddy) + col_a);
                if (t > last) xa[p] = u32x4{0u, 0u, 0u, 0u};
            }
#pragma unroll
            for (int p = 0; p < PB; ++p) {
                const uint32_t t = rb + p * kRowsB, u = t < last ? t : last;
                xb[p] = get_b(q + static_cast<uint64_t>(t0) * g.n_in,
                              static_cast<Off>(u) * g.n_in + col_b);
                eb[p] = *at_offset(e + static_cast<uint64_t>(t0) * g.blocks_in,
                                   static_cast<Off>(u) * g.blocks_in + blk_b);
                if (t > last) xb[p] = u32x2{0u, 0u};
            }
        };
        auto load = [&](uint32_t s) {
            if (s + 1 == steps) {
                load_last(s);
            } else {
                load_a(s);
                load_b(s);
            }
        };
        // LDS place of eight columns c of row r in a tile of `width` columns
        auto place = [](uint32_t r, uint32_t c, uint32_t width) {
            const uint32_t turn = width >= 128 ? (r & 3u) << 1 : r & 2u;
            return r * width + (((c >> 4) ^ turn) << 4) + (c & 15u);
        };
        auto stage_a = [&](uint32_t buf) {
#pragma unroll
            for (int p = 0; p < PA; ++p)
                *reinterpret_cast<u32x4 *>(&sa[buf][place(ra + p * kRowsA, ca, BM)]) = xa[p];
        };
        auto stage_b = [&](uint32_t buf) {
#pragma unroll
            for (int p = 0; p < PB; ++p)
                *reinterpret_cast<u32x4 *>(&sb[buf][place(rb + p * kRowsB, cb, BN)]) =
                    codes_to_16<F>(xb[p], eb[p]);
        };

        // reading: lane (half, group of 16, j) reads row 8 half + j/4 (+4), columns
        // 16 group + 4 (j mod 4) of a 32-column unit
        const uint32_t half = lane >> 5, grp = (lane >> 4) & 1u, j = lane & 15u;
        const uint32_t am = wave % WM * (BM / WM), bn = wave / WM * (BN / WN);
        uint32_t pa[TM], pb[TN];
#pragma unroll
        for (int m = 0; m < TM; ++m)
            pa[m] = place(half * 8 + (j >> 2), am + m * 32 + grp * 16 + (j & 3u) * 4, BM);
#pragma unroll
        for (int n = 0; n < TN; ++n)
            pb[n] = place(half * 8 + (j >> 2), bn + n * 32 + grp * 16 + (j & 3u) * 4, BN);
        s16x8 a[2][TM], b[2][TN];
        auto read = [&](int f, uint32_t buf, int kk) {
#pragma unroll
            for (int m = 0; m < TM; ++m) {
                const s16x4 lo = read_tr(&sa[buf][pa[m] + kk * 16 * BM]);
                const s16x4 hi = read_tr(&sa[buf][pa[m] + (kk * 16 + 4) * BM]);
                a[f][m] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
            }
#pragma unroll
            for (int n = 0; n < TN; ++n) {
                const s16x4 lo = read_tr(&sb[buf][pb[n] + kk * 16 * BN]);
                const s16x4 hi = read_tr(&sb[buf][pb[n] + (kk * 16 + 4) * BN]);
                b[f][n] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
            }
        };

        f32x16 acc[TM][TN];
#pragma unroll
        for (int m = 0; m < TM; ++m)
#pragma unroll
            for (int n = 0; n < TN; ++n)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[m][n][r] = 0.0f;

        auto multiply = [&](int f) {
#pragma unroll
            for (int m = 0; m < TM; ++m)
#pragma unroll
                for (int n = 0; n < TN; ++n) acc[m][n] = mfma<F>(a[f][m], b[f][n], acc[m][n]);
        };

        if (steps > 0) {
            load(0);
            stage_a(0);
            stage_b(0);
            if (steps > 1) load(1);
            __syncthreads();
            read(0, 0, 0);
        }
        // A step: fragments one MFMA step ahead; the next step's tiles go to LDS beside the
        // first two MFMA steps, and the ones after that are requested from memory as their
        // registers become free.  The barrier stands where every wave has this buffer's last
        // fragments in registers and its share of the next buffer written: behind it the next
        // buffer may be read and this one be overwritten.
        //
        // Steady state, free of branches so that each MFMA step is one scheduling region: a
        // wave's LDS reads, conversions, LDS writes and requests are dealt between its MFMAs.
        // (The checkpoint first, then dy: 952 us; the other way round 985 us.)
        constexpr int kMfma = TM * TN, kReads = 2 * (TM + TN);
        auto steady = [&](uint32_t s, uint32_t buf) {
            static_assert(KK >= 4 && KK % 2 == 0,
                          "staging takes two MFMA steps, fragments alternate");
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) {
                if (kk + 1 == KK) __syncthreads();
                read((kk + 1) & 1, kk + 1 == KK ? buf ^ 1u : buf, (kk + 1) % KK);
                multiply(kk & 1);
                if (kk == 0) {
                    stage_b(buf ^ 1u);
                    load_b(s + 2);
                    interleave<kMfma, kReads, 12 * PB, PB, 2 * PB>();
                } else if (kk == 1) {
                    stage_a(buf ^ 1u);
                    load_a(s + 2);
                    interleave<kMfma, kReads, 0, PA, PA>();
                } else {
                    interleave<kMfma, kReads, 0, 0, 0>();
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        auto step = [&](uint32_t s, uint32_t buf) {
            const bool more = s + 1 < steps;
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) {
                if (kk + 1 < KK) {
                    read((kk + 1) & 1, buf, kk + 1);
                } else {
                    __syncthreads();
                    if (more) read(0, buf ^ 1u, 0);
                }
                if (kk == 0 && more) {
                    stage_a(buf ^ 1u);
                    stage_b(buf ^ 1u);
                    if (s + 2 < steps) load(s + 2);
                }
                multiply(kk & 1);
            }
        };
        uint32_t s = 0;
        for (; s + 4 < steps; s += 2) {   // steps s + 2 and s + 3 are whole
            steady(s, 0);
            steady(s + 1, 1);
        }
        for (; s < steps; ++s) step(s, s & 1u);

        // the lane again, opaque: what the stores need is worked out here and not kept in
        // registers (or spilled) from before the loop
        uint32_t el = lane;
        asm volatile("" : "+v"(el));
        const uint32_t eh = el >> 5;
        // result register r of a lane: row 8 (r/4) + 4 half + r%4, column lane mod 32;
        // positions of the last group stand for the row's last eight columns
        auto column = [](uint32_t at, uint32_t first, uint32_t n) {   // ~0: not this one's to store
            const uint32_t c = first + at;
            if (TINY || first + (at | 7u) < n) return c < n ? c : ~0u;
            const uint32_t group = c & ~7u;
            if (group >= n) return ~0u;
            const uint32_t real = n - 8 + (c & 7u);
            return real >= group ? real : ~0u;
        };
        if constexpr (O == Out::k16 && !TINY) {
            // Stored as they lie, a wave's 16-bit results are 64-B pieces of 128-B lines (1.8
            // times the bytes moved, a tenth of the time at 2048 tokens).  Each wave turns 32
            // rows at a time through LDS (its own part: every wave is past the last barrier,
            // behind which nothing is read) into rows of 16-B groups.  Units of 32 columns are
            // swapped in every second four rows, so that the two halves of a wave write
            // different banks.
            constexpr uint32_t W = BN / WN, kPerRow = W / 8, kRows = 64 / kPerRow;
            constexpr uint32_t kSwap = W >= 64 ? 32 : 0;
            static_assert(WM * WN * 32 * W <= 2 * kStep * BM, "room for 32 rows a wave");
            uint16_t *const mine = &sa[0][0] + wave * (32 * W);
            const uint32_t c = el % kPerRow * 8, group = i0 + bn + c;
#pragma unroll
            for (int m = 0; m < TM; ++m) {
#pragma unroll
                for (int n = 0; n < TN; ++n)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        mine[(8 * (r / 4) + 4 * eh + r % 4) * W +
                             ((n * 32 + (el & 31u)) ^ (eh * kSwap))] = from_f32<F>(acc[m][n][r]);
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
                for (uint32_t r0 = 0; r0 < 32; r0 += kRows) {
                    const uint32_t r = r0 + el / kPerRow;
                    const uint32_t row = column(am + m * 32 + r, o0, g.n_out);
                    if (row == ~0u || group >= g.n_in) continue;
                    const uint16_t *v = &mine[r * W + (c ^ (((r >> 2) & 1u) * kSwap))];
                    uint16_t *d =
                        static_cast<uint16_t *>(out) + static_cast<uint64_t>(row) * g.n_in;
                    if (group + 8 <= g.n_in) {
                        *reinterpret_cast<u32x4_any *>(d + group) =
                            *reinterpret_cast<const u32x4 *>(v);
                    } else {   // the row's last eight columns, those from `group` on
                        for (uint32_t k = group - (g.n_in - 8); k < 8; ++k)
                            d[g.n_in - 8 + k] = v[k];
                    }
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
            }
            __syncthreads();   // the next tile writes LDS
            continue;
        }
        const uint64_t plane = static_cast<uint64_t>(g.n_out) * g.n_in;
#pragma unroll
        for (int n = 0; n < TN; ++n) {
            const uint32_t col = column(bn + n * 32 + (el & 31u), i0, g.n_in);
#pragma unroll
            for (int m = 0; m < TM; ++m) {
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    __builtin_amdgcn_sched_barrier(0);
                    const uint32_t row = column(am + m * 32 + 8 * (r / 4) + 4 * eh + r % 4, o0,
                                                g.n_out);
                    if (row != ~0u && col != ~0u) {
                        const uint64_t at = static_cast<uint64_t>(row) * g.n_in + col;
                        if constexpr (O == Out::k16) {
                            static_cast<uint16_t *>(out)[at] = from_f32<F>(acc[m][n][r]);
                        } else {
                            float *d = static_cast<float *>(out) + blockIdx.y * plane + at;
                            *d = O == Out::kAdd32 ? *d + acc[m][n][r] : acc[m][n][r];
                        }
                    }
                }
            }
        }
        __syncthreads();   // the next tile writes LDS
    }
}

// dw = (dw +) the sum of `splits` planes of n FP32 values, in split order.
constexpr int kJoinThreads = 256;
template <int F, Out O>
__global__ __launch_bounds__(kJoinThreads) void join_splits_kernel(
    void *__restrict__ dw, const float *__restrict__ part, uint64_t n, uint32_t splits) {
    const uint64_t stride = static_cast<uint64_t>(gridDim.x) * kJoinThreads;
    for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * kJoinThreads + threadIdx.x; i < n;
         i += stride) {
        float s = part[i];
        for (uint32_t k = 1; k < splits; ++k) s = s + part[k * n + i];
        if constexpr (O == Out::k16)
            static_cast<uint16_t *>(dw)[i] = from_f32<F>(s);
        else
            static_cast<float *>(dw)[i] = O == Out::kAdd32 ? static_cast<float *>(dw)[i] + s : s;
    }
}

template <typename T>
__global__ __launch_bounds__(kJoinThreads) void zero_fill_kernel(T *__restrict__ d, uint64_t n) {
    const uint64_t stride = static_cast<uint64_t>(gridDim.x) * kJoinThreads;
    for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * kJoinThreads + threadIdx.x; i < n;
         i += stride)
        d[i] = T(0);
}

uint32_t capped_blocks(uint64_t n) {
    const uint64_t b = (n + kJoinThreads - 1) / kJoinThreads, cap = max_blocks();
    return static_cast<uint32_t>(b < cap ? b : cap);
}

// Tile and splits of a call, by its extents alone (so the workspace and the order
// of the sums do not depend on the device).
struct Plan {
    uint32_t tile;        // 256, 128 or 64 columns of each operand
    uint32_t splits;
    uint32_t per_split;
};

constexpr uint64_t kFill = 256;   // compute units of the chip
constexpr uint64_t kMaxStride = 1ull << 24;   // a step's rows stay below 2^32 bytes
constexpr uint64_t kSplitUnit = 128;          // tokens: whole steps of every tile

// Measured on MI355X, one tile a compute unit, in ns: 64 tokens of a tile, and a
// tile's start and end.  The large tile reuses each operand most but needs many tiles
// and many tokens; a small one starts quickly and is bound by latency.
struct TileCost {
    uint32_t tile, step, ends;
};
constexpr TileCost kTiles[3] = {{256, 1900, 15000}, {128, 660, 4000}, {64, 310, 2000}};

// The tile and splits of least estimated time: rounds of 256 tiles, and for split
// tokens the join's launch, its partial products (about 8 TB/s out of the caches) and
// its walk over the splits.  Over fourteen shapes of 200 to 16384 tokens and 64 to
// 50257 columns the choice was within 12% of the best of every tile with 1 to 64
// splits; for 16384 x 768 x 768, for example, 128 x 128 tiles in 6 splits take 44 us,
// 64 x 64 in 3 53 us and 256 x 256 in 16 55 us, and for 1024 x 768 x 768 64 x 64
// tiles 9 us, 128 x 128 17 us.
Plan plan_of(uint64_t tokens, uint64_t n_out, uint64_t n_in) {
    const uint64_t units = (tokens + kSplitUnit - 1) / kSplitUnit;
    const uint64_t plane_ns = n_out * n_in / 1000;          // 4 B written and read: 8 B a result
    Plan best{0, 1, 0};
    uint64_t best_ns = ~0ull;
    for (const TileCost &c : kTiles) {
        const uint64_t n = ((n_out + c.tile - 1) / c.tile) * ((n_in + c.tile - 1) / c.tile);
        for (uint64_t s = 1; s <= 64 && s <= units && (s == 1 || n * s <= 2 * kFill); ++s) {
            const uint64_t per = (units + s - 1) / s, used = (units + per - 1) / per;
            if (used != s) continue;
            const uint64_t rounds = (n * s + kFill - 1) / kFill;
            uint64_t ns = rounds * (per * (kSplitUnit / 64) * c.step + c.ends);
            if (s > 1) ns += 5000 + s * (plane_ns + 150);
            if (ns < best_ns) {
                best_ns = ns;
                best = Plan{c.tile, static_cast<uint32_t>(s),
                            static_cast<uint32_t>(per * kSplitUnit)};
            }
        }
    }
    return best;
}

template <int F, Out O>
hipError_t tiles_of(void *out, const uint16_t *dy, const uint8_t *q, const uint8_t *e,
                    const GradShape &g, const Plan &p, bool tiny, hipStream_t stream) {
    const uint64_t cap = max_blocks();
    const dim3 grid(static_cast<uint32_t>(g.work < cap ? g.work : cap), p.splits);
#define ZS_TILE(B, WM, WN, STEP, TINY)                                                    \
    weight_grad_kernel<F, O, B, B, WM, WN, STEP, TINY>                                    \
        <<<grid, 64 * WM * WN, 0, stream>>>(out, dy, q, e, g)
    if (tiny)
        ZS_TILE(64, 2, 2, 64, true);
    else if (p.tile == 256)
        ZS_TILE(256, 4, 2, 64, false);
    else if (p.tile == 128)
        ZS_TILE(128, 2, 2, 64, false);
    else
        ZS_TILE(64, 2, 2, 128, false);
#undef ZS_TILE
    return hipGetLastError();
}

template <int F, Out O>
hipError_t grad_as(void *dw, const uint16_t *dy, const uint8_t *q, const uint8_t *e,
                   const GradShape &g, const Plan &p, bool tiny, void *workspace,
                   hipStream_t stream) {
    if (p.splits == 1) return tiles_of<F, O>(dw, dy, q, e, g, p, tiny, stream);
    const hipError_t err = tiles_of<F, Out::k32>(workspace, dy, q, e, g, p, tiny, stream);
    if (err != hipSuccess) return err;
    const uint64_t n = static_cast<uint64_t>(g.n_out) * g.n_in;
    join_splits_kernel<F, O><<<capped_blocks(n), kJoinThreads, 0, stream>>>(
        dw, static_cast<const float *>(workspace), n, p.splits);
    return hipGetLastError();
}

}  // namespace

uint64_t weight_grad_workspace(uint64_t tokens, uint64_t n_out, uint64_t n_in) {
    const Plan p = plan_of(tokens, n_out, n_in);
    return p.splits == 1 ? 0 : 4 * n_out * n_in * p.splits;
}

hipError_t launch_weight_grad(void *dw, bool dw32, bool first, const uint16_t *dy, uint64_t lddy,
                              int fmt, const uint8_t *q, const uint8_t *e, uint64_t tokens,
                              uint64_t n_out, uint64_t n_in, void *workspace,
                              hipStream_t stream) {
    const Plan p = plan_of(tokens, n_out, n_in);
    // Element by element (TINY), the price of extents and strides that hardly occur: 1024
    // tokens, 2304 x 768, rows of dy 2^24 elements apart 77 us, eight elements less 18; 8192 x
    // 4096 1160 and 95; 16384 tokens, 7 x 4096 196 us, 8 x 4096 34.
    const bool tiny = n_out < 8 || n_in < 8 || n_in >= kMaxStride || lddy >= kMaxStride;
    const uint64_t b = tiny ? 64 : p.tile;
    const uint64_t tiles_in = (n_in + b - 1) / b, tiles_out = (n_out + b - 1) / b;
    GradShape g{lddy,
                static_cast<uint32_t>(tokens),
                static_cast<uint32_t>(n_out),
                static_cast<uint32_t>(n_in),
                static_cast<uint32_t>((n_in + ZERO_ACT_BLOCK - 1) / ZERO_ACT_BLOCK),
                p.per_split,
                static_cast<uint32_t>(tiles_out),
                static_cast<uint32_t>(tiles_in),
                0,
                tiles_in * tiles_out};
    // Groups where they leave few places empty (empty ones cost the XCDs' balance: with
    // 432 tiles in 768 places a 1023 x 2304 x 768 call took 20.7 us, ungrouped 13.5).
    for (uint32_t gi = 8; gi > 0 && g.group_i == 0 && g.work >= kFill; gi /= 2) {
        const uint64_t go = 32 / gi;
        const uint64_t groups = ((tiles_out + go - 1) / go) * ((tiles_in + gi - 1) / gi);
        const uint64_t places = (groups + 7) / 8 * 8 * 32;
        if (places * 8 <= g.work * 9) {
            g.group_i = gi;
            g.work = places;
        }
    }
#define ZS_GRAD(F, O) return grad_as<F, O>(dw, dy, q, e, g, p, tiny, workspace, stream)
    if (fmt == 0) {
        if (!dw32) ZS_GRAD(0, Out::k16);
        if (first) ZS_GRAD(0, Out::k32);
        ZS_GRAD(0, Out::kAdd32);
    }
    if (!dw32) ZS_GRAD(1, Out::k16);
    if (first) ZS_GRAD(1, Out::k32);
    ZS_GRAD(1, Out::kAdd32);
#undef ZS_GRAD
}

hipError_t launch_zero_fill(void *dw, int elem_bytes, uint64_t n, hipStream_t stream) {
    if (elem_bytes == 4)
        zero_fill_kernel<<<capped_blocks(n), kJoinThreads, 0, stream>>>(
            static_cast<uint32_t *>(dw), n);
    else
        zero_fill_kernel<<<capped_blocks(n), kJoinThreads, 0, stream>>>(
            static_cast<uint16_t *>(dw), n);
    return hipGetLastError();
}

}  // namespace zs
