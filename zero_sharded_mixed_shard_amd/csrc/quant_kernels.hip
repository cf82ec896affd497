// gfx950 kernels of matrices in 8-bit codes with a power of two for each block of 128:
// writing one from blocks of a row or 128 x 128 blocks (these with the transposed codes in
// the same pass), and reading one back.
//
// Mathematics as for the activation checkpoints: the exponent byte comes from the largest
// finite magnitude's FP32 bits, multiplying by 2^-k is exact, and the hardware's e4m3
// convert does the one rounding, to nearest even.
//
// Blocks of a row: sixteen neighbouring lanes hold a block, eight elements each, and its
// maximum takes four exchanges inside the sixteen (a DPP row).
//
// Square blocks: a workgroup holds one in registers, eight rows by eight columns a lane, so
// that x is read once.  A lane transposes its 8 x 8 codes in registers (byte permutes) and
// the block goes through LDS into whole lines of the transposed codes.  Eight-byte units of
// an LDS line are permuted by the writing lanes' column group, so that a wave's writes fall
// on all of its 32 banks.
//
// These kernels are streams over HBM.  BF16 16384 x 8192: blocks of a row 68 us (5.9 TB/s),
// square ones 68, with the transposed codes 111 (4.8: their rows are written in pieces of 128 B),
// reading back 71.  Rows of odd length (16384 x 8191) start at any byte: 89, 168, 211 and 96 us.
#include "block_device.h"
#include "code_device.h"

#pragma clang fp contract(off)

namespace zs {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 2;   // groups of eight elements a lane keeps in flight

// Maximum over the sixteen lanes of a DPP row: quad permutes 1,0,3,2 and 2,3,0,1, then the
// half row and the row mirrored.
__device__ __forceinline__ uint32_t row_max(uint32_t a) {
    uint32_t b = __builtin_amdgcn_update_dpp(0u, a, 0xB1, 0xf, 0xf, true);
    a = a > b ? a : b;
    b = __builtin_amdgcn_update_dpp(0u, a, 0x4E, 0xf, 0xf, true);
    a = a > b ? a : b;
    b = __builtin_amdgcn_update_dpp(0u, a, 0x141, 0xf, 0xf, true);
    a = a > b ? a : b;
    b = __builtin_amdgcn_update_dpp(0u, a, 0x140, 0xf, 0xf, true);
    return a > b ? a : b;
}

// The same of finite values only.
__device__ __forceinline__ uint32_t finite_magnitude8(const float x[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t a = bits(x[j]) & 0x7fffffffu;
        m = a < 0x7f800000u && a > m ? a : m;
    }
    return m;
}

// Eight elements of a row from column col on; past the row's end zeros.
template <int F>
__device__ __forceinline__ void load_group(const elem_t<F> *row, uint64_t col, uint64_t cols,
                                           float out[8]) {
    if (col + 8 <= cols)
        widen8<F>(load8<F>(row + col), out);
    else
        load_some<F>(row + col, col < cols ? static_cast<uint32_t>(cols - col) : 0u, out);
}

__device__ __forceinline__ uint32_t group_size(uint64_t col, uint64_t cols) {
    return col >= cols ? 0u : cols - col < 8 ? static_cast<uint32_t>(cols - col) : 8u;
}

template <int F>
__global__ __launch_bounds__(kThreads) void quant_row_kernel(
    uint8_t *__restrict__ q, uint8_t *__restrict__ e, const elem_t<F> *__restrict__ x,
    uint64_t ldx, uint64_t cols, FastDiv nb, uint64_t n_groups) {
    constexpr uint64_t kTile = kThreads * kUnroll;
    for (uint64_t t0 = blockIdx.x * kTile; t0 < n_groups; t0 += gridDim.x * kTile) {
        float v[kUnroll][8];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const uint64_t g = t0 + u * kThreads + threadIdx.x;
            if (g < n_groups) {
                const uint64_t b = g >> 4, row = div_by(b, nb);
                load_group<F>(x + row * ldx, (b - row * nb.d) * ZERO_BLOCK + (g & 15) * 8, cols,
                              v[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const uint64_t g = t0 + u * kThreads + threadIdx.x;
            if (g < n_groups) {   // n_groups is a multiple of 16: whole blocks take part
                const uint64_t b = g >> 4, row = div_by(b, nb);
                const uint64_t col = (b - row * nb.d) * ZERO_BLOCK + (g & 15) * 8;
                uint32_t m = magnitude8(v[u]);
                const bool rare = __any(m > bits(kTop<F>));
                if (rare) m = finite_magnitude8(v[u]);
                const uint32_t eb = block_exponent(row_max(m));
                const u32x2 c = rare ? encode8<F, true>(v[u], eb) : encode8<F, false>(v[u], eb);
                store_codes(q + row * cols + col, group_size(col, cols), c);
                if ((g & 15) == 0) e[b] = static_cast<uint8_t>(eb);
            }
        }
    }
}

// Four rows of four bytes as four columns.
__device__ __forceinline__ void transpose4(uint32_t a, uint32_t b, uint32_t c, uint32_t d,
                                           uint32_t out[4]) {
    const uint32_t ab = __builtin_amdgcn_perm(b, a, 0x05010400u);   // a0 b0 a1 b1
    const uint32_t ab2 = __builtin_amdgcn_perm(b, a, 0x07030602u);  // a2 b2 a3 b3
    const uint32_t cd = __builtin_amdgcn_perm(d, c, 0x05010400u);
    const uint32_t cd2 = __builtin_amdgcn_perm(d, c, 0x07030602u);
    out[0] = __builtin_amdgcn_perm(cd, ab, 0x05040100u);
    out[1] = __builtin_amdgcn_perm(cd, ab, 0x07060302u);
    out[2] = __builtin_amdgcn_perm(cd2, ab2, 0x05040100u);
    out[3] = __builtin_amdgcn_perm(cd2, ab2, 0x07060302u);
}

// One 128 x 128 block a workgroup; lane (tr, tc) of 16 x 16 holds rows 8 tr .. 8 tr + 7 of
// columns 8 tc .. 8 tc + 7, as they lie in memory (widened twice, for the maximum and for the
// codes: held as FP32 they take the registers of every second workgroup).  NARROW: rows of
// less than eight columns.
template <int F, bool TRANSPOSED, bool NARROW>
__global__ __launch_bounds__(kThreads) void quant_square_kernel(
    uint8_t *__restrict__ q, uint8_t *__restrict__ e, uint8_t *__restrict__ qt,
    uint8_t *__restrict__ et, const elem_t<F> *__restrict__ x, uint64_t ldx, uint64_t rows,
    uint64_t cols, FastDiv nb, uint64_t n_blocks) {
    __shared__ uint32_t part[2][kThreads / 64];
    __shared__ __align__(16) u32x2 turned[TRANSPOSED ? 128 * 16 : 1];
    const uint32_t tr = threadIdx.x >> 4, tc = threadIdx.x & 15u, wave = threadIdx.x >> 6;
    uint32_t parity = 0;
    for (uint64_t blk = blockIdx.x; blk < n_blocks; blk += gridDim.x, parity ^= 1u) {
        const uint64_t br = div_by(blk, nb), bc = blk - br * nb.d;
        const uint64_t r0 = br * ZERO_BLOCK + tr * 8, c0 = bc * ZERO_BLOCK + tc * 8;
        const uint32_t n = group_size(c0, cols);
        Raw8<F> raw[8];
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            const elem_t<F> *row = x + (r0 + p < rows ? r0 + p : rows - 1) * ldx;
            if constexpr (NARROW) {
                float v[8];
                load_some<F>(row + c0, n, v);
                raw[p] = narrow8<F>(v);
            } else {
                raw[p] = raw_group<F>(row, static_cast<uint32_t>(c0),
                                      static_cast<uint32_t>(cols));
            }
        }
        if (!NARROW && n - 1u < 7u) {
#pragma unroll
            for (int p = 0; p < 8; ++p) move_down<F>(raw[p], n);
        }
        if (n == 0 || r0 + 8 > rows) {
#pragma unroll
            for (int p = 0; p < 8; ++p)
                if (n == 0 || r0 + p >= rows) raw[p] = Raw8<F>{};
        }
        uint32_t m = 0;
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            float v[8];
            widen8<F>(raw[p], v);
            const uint32_t a = magnitude8(v);
            m = a > m ? a : m;
        }
        const bool rare = __any(m > bits(kTop<F>));
        if (rare) {   // the block's scale goes by its finite elements
            m = 0;
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                float v[8];
                widen8<F>(raw[p], v);
                const uint32_t a = finite_magnitude8(v);
                m = a > m ? a : m;
            }
        }
        m = row_max(m);
#pragma unroll
        for (int j = 16; j < 64; j += 16) {
            const uint32_t a = static_cast<uint32_t>(
                __builtin_amdgcn_readlane(static_cast<int>(m), j));
            m = a > m ? a : m;
        }
        m = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(m)));
        // two sets of partial maxima in turn: a wave that is a block ahead does not
        // overwrite what another still reads
        if ((threadIdx.x & 63u) == 0) part[parity][wave] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kThreads / 64; ++w) m = part[parity][w] > m ? part[parity][w] : m;
        const uint32_t eb = block_exponent(m);
        u32x2 c[8];
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            float v[8];
            asm volatile("" : "+v"(raw[p].v[0]));   // widened anew, not kept from above
            widen8<F>(raw[p], v);
            c[p] = rare ? encode8<F, true>(v, eb) : encode8<F, false>(v, eb);
        }
#pragma unroll
        for (int p = 0; p < 8; ++p)
            if (r0 + p < rows) store_codes(q + (r0 + p) * cols + c0, n, c[p]);
        if (threadIdx.x == 0) e[blk] = static_cast<uint8_t>(eb);
        if constexpr (TRANSPOSED) {
            const uint64_t tall = (rows + ZERO_BLOCK - 1) / ZERO_BLOCK;
            if (threadIdx.x == 0) et[bc * tall + br] = static_cast<uint8_t>(eb);
            // unit tr of column 8 tc + j lies at unit tr ^ tc of its line
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t lo[4], hi[4];
                transpose4(c[0][h], c[1][h], c[2][h], c[3][h], lo);
                transpose4(c[4][h], c[5][h], c[6][h], c[7][h], hi);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    turned[(tc * 8 + h * 4 + j) * 16 + (tr ^ tc)] = u32x2{lo[j], hi[j]};
            }
            __syncthreads();
            const uint32_t pair = threadIdx.x & 7u;   // sixteen rows of the block
            const uint64_t row = br * ZERO_BLOCK + pair * 16;
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const uint32_t col = (threadIdx.x >> 3) + 32 * p, turn = col >> 3;
                const u32x2 a = turned[col * 16 + ((2 * pair) ^ turn)];
                const u32x2 b = turned[col * 16 + ((2 * pair + 1) ^ turn)];
                const uint64_t to = bc * ZERO_BLOCK + col;
                if (to < cols && row < rows) {
                    uint8_t *d = qt + to * rows + row;
                    if (row + 16 <= rows) {
                        __builtin_nontemporal_store(u32x4{a[0], a[1], b[0], b[1]},
                                                    reinterpret_cast<u32x4_any *>(d));
                    } else {
                        store_codes(d, group_size(row, rows), a);
                        store_codes(d + 8, group_size(row + 8, rows), b);
                    }
                }
            }
            __syncthreads();   // the next block writes the lines
        }
    }
}

template <int F>
__global__ __launch_bounds__(kThreads) void block_load_kernel(
    elem_t<F> *__restrict__ x, uint64_t ldx, const uint8_t *__restrict__ q,
    const uint8_t *__restrict__ e, uint32_t row_shift, uint64_t cols, uint64_t nb, FastDiv per_row,
    uint64_t n_groups) {
    constexpr uint64_t kTile = kThreads * kUnroll;
    for (uint64_t t0 = blockIdx.x * kTile; t0 < n_groups; t0 += gridDim.x * kTile) {
        u32x2 c[kUnroll];
        uint32_t eb[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const uint64_t g = t0 + u * kThreads + threadIdx.x;
            if (g < n_groups) {
                const uint64_t row = div_by(g, per_row), col = (g - row * per_row.d) * 8;
                c[u] = load_codes(q + row * cols + col, group_size(col, cols));
                eb[u] = e[(row >> row_shift) * nb + (col >> 7)];
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const uint64_t g = t0 + u * kThreads + threadIdx.x;
            if (g < n_groups) {
                const uint64_t row = div_by(g, per_row), col = (g - row * per_row.d) * 8;
                float r[8];
                decode8(c[u], eb[u], r);
                const uint32_t n = group_size(col, cols);
                if (n == 8)
                    store8<F>(x + row * ldx + col, r);
                else
                    store_some<F>(x + row * ldx + col, n, r);
            }
        }
    }
}

uint32_t grid_of(uint64_t blocks) {
    const uint64_t cap = max_blocks();
    return static_cast<uint32_t>(blocks < cap ? blocks : cap);
}

uint32_t grid_of_groups(uint64_t groups) {
    const uint64_t tile = static_cast<uint64_t>(kThreads) * kUnroll;
    return grid_of((groups + tile - 1) / tile);
}

template <int F>
hipError_t quant_as(uint8_t *q, uint8_t *e, uint8_t *qt, uint8_t *et, const void *x, uint64_t ldx,
                    bool square, uint64_t rows, uint64_t cols, hipStream_t stream) {
    const auto *xt = static_cast<const elem_t<F> *>(x);
    const uint64_t nb = (cols + ZERO_BLOCK - 1) / ZERO_BLOCK;
    const FastDiv div = fast_div(static_cast<uint32_t>(nb));
    if (!square) {
        const uint64_t groups = rows * nb * 16;
        quant_row_kernel<F><<<grid_of_groups(groups), kThreads, 0, stream>>>(q, e, xt, ldx, cols,
                                                                            div, groups);
    } else {
        const uint64_t blocks = nb * ((rows + ZERO_BLOCK - 1) / ZERO_BLOCK);
#define ZS_SQUARE(TRANSPOSED, NARROW)                                                        \
    quant_square_kernel<F, TRANSPOSED, NARROW><<<grid_of(blocks), kThreads, 0, stream>>>(    \
        q, e, qt, et, xt, ldx, rows, cols, div, blocks)
        if (cols < 8 && qt != nullptr)
            ZS_SQUARE(true, true);
        else if (cols < 8)
            ZS_SQUARE(false, true);
        else if (qt != nullptr)
            ZS_SQUARE(true, false);
        else
            ZS_SQUARE(false, false);
#undef ZS_SQUARE
    }
    return hipGetLastError();
}

template <int F>
hipError_t load_as(void *x, uint64_t ldx, const uint8_t *q, const uint8_t *e, bool square,
                   uint64_t rows, uint64_t cols, hipStream_t stream) {
    const uint64_t per_row = (cols + 7) / 8, groups = rows * per_row;
    block_load_kernel<F><<<grid_of_groups(groups), kThreads, 0, stream>>>(
        static_cast<elem_t<F> *>(x), ldx, q, e, square ? 7u : 0u, cols,
        (cols + ZERO_BLOCK - 1) / ZERO_BLOCK, fast_div(static_cast<uint32_t>(per_row)), groups);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_block_quant(uint8_t *q, uint8_t *e, uint8_t *qt, uint8_t *et, const void *x,
                              uint64_t ldx, int fmt, bool square, uint64_t rows, uint64_t cols,
                              hipStream_t stream) {
    if (fmt == 0) return quant_as<0>(q, e, qt, et, x, ldx, square, rows, cols, stream);
    if (fmt == 1) return quant_as<1>(q, e, qt, et, x, ldx, square, rows, cols, stream);
    return quant_as<2>(q, e, qt, et, x, ldx, square, rows, cols, stream);
}

hipError_t launch_block_load(void *x, uint64_t ldx, int fmt, const uint8_t *q, const uint8_t *e,
                             bool square, uint64_t rows, uint64_t cols, hipStream_t stream) {
    if (fmt == 0) return load_as<0>(x, ldx, q, e, square, rows, cols, stream);
    if (fmt == 1) return load_as<1>(x, ldx, q, e, square, rows, cols, stream);
    return load_as<2>(x, ldx, q, e, square, rows, cols, stream);
}

}  // namespace zs
