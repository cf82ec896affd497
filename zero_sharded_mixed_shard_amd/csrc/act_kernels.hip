// gfx950 kernels of the 8-bit activation checkpoints: writing one (with the
// activation function's forward pass), reading one back, and the activation
// function's backward pass from one.
//
// Mathematics.  A block of 32 neighbours of a row shares 2^k, the smallest
// with amax <= 448 * 2^k.  With amax = f * 2^x, 1 <= f < 2, and
// 448 = 1.75 * 2^8, that is k = x - 8 for f <= 1.75 and x - 7 above: the
// exponent byte is the biased exponent of amax minus 8, plus one if its
// significand bits exceed those of 1.75, held at 3 (k = -124).  Multiplying by
// 2^-k is exact (k is in [-124, 120], and FP32 denormals are kept), so the
// hardware's e4m3 convert does the only rounding, to nearest even.
//
// Layout.  Four neighbouring lanes hold a block, eight elements each: one 16-B
// access of 16-bit data a lane, 8 B of codes, and the block's maximum takes two
// exchanges inside the four lanes.  When every view is contiguous and cols is a
// multiple of 32 the matrix is treated as one long row; otherwise the row of a
// block comes from one multiplication (FastDiv), and the last group of a row
// is done element by element.
//
// These kernels are streams over HBM.  16384 x 8192 BF16: writing a checkpoint 64 us, reading
// it back 66 to 69 us (6.4 and 6.0 TB/s); with the GELU the forward pass 103 us and the
// backward pass 109 us (6.6 and 6.2 TB/s).  127 x 1601 FP32: 4 us each, the launch.
#include "grad_device.h"

#pragma clang fp contract(off)

namespace zs {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 2;   // groups of eight elements a lane keeps in flight

// Largest magnitude a checkpoint written from format F stands for.
template <int F> constexpr float kTop = F == 0 ? 61440.0f : 0x1.ep127f;

// Element positions of group g (eight elements) of a matrix whose rows hold
// nb.d blocks: FLAT: the matrix is one row.
template <bool FLAT>
struct Group {
    uint64_t row, blk;   // block blk (from the row's first) of row row
    uint64_t col;
    uint32_t n;          // elements of the row in the group, 0..8
    __device__ __forceinline__ Group(uint64_t g, const FastDiv &nb, uint64_t cols) {
        const uint64_t b = g >> 2;
        row = FLAT ? 0 : div_by(b, nb);
        blk = FLAT ? b : b - row * nb.d;
        col = blk * 32 + (g & 3) * 8;
        n = FLAT ? 8u : (col >= cols ? 0u : cols - col < 8 ? static_cast<uint32_t>(cols - col) : 8u);
    }
};

// Activation functions, act(x) = x s(t) with s(t) = 1 / (1 + e^-t).
//
// FP32 data: with e = e^-|t|, q = e / (1 + e) = s(-|t|) and r = 1 / (1 + e) = s(|t|),
//     act(x)  = x - x q  for t > 0,  x q  otherwise
//     act'(x) = 1 + q (x t' r - 1)  for t > 0,  q (x t' r + 1)  otherwise.
// e never overflows and reaches zero with t on both sides (e^-t held at the range's end left
// a slope of x 2^-125), and where the result is large the evaluation's error is scaled by the
// small q: one rounding remains.  16384 x 8192 FP32: GELU forward 224 us, backward 226 us.
//
// For 16-bit data the constants are folded into one polynomial, e^-t = 2^(x (a + b x^2)),
// and the hardware's 2^x and reciprocal (each within an ulp, zero for subnormals, which
// costs up to 2^-117 absolute) do, as the result is rounded to 16 bits.  The arithmetic is
// what bounds the GELU kernels once the memory streams well: about twenty VALU operations
// and two quarter-rate ones an element.
constexpr float kGeluC = 0.7978845608028654f;   // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;
constexpr float kLog2e = 1.4426950408889634f;

// t of FP32 data
template <int ACT>
__device__ __forceinline__ float inner(float x) {
    return ACT == ZERO_ACT_SILU ? x : 2.0f * kGeluC * (x + kGeluA * x * x * x);
}

// e^-t of 16-bit data
template <int ACT>
__device__ __forceinline__ float exp_neg_t(float x) {
    if constexpr (ACT == ZERO_ACT_SILU) {
        return __builtin_amdgcn_exp2f(x * -kLog2e);
    } else {
        constexpr float a = -2.0f * kGeluC * kLog2e, b = a * kGeluA;
        return __builtin_amdgcn_exp2f(x * __builtin_fmaf(b, x * x, a));
    }
}

template <int F, int ACT>
__device__ __forceinline__ float act_value(float x) {
    if constexpr (F == 2) {
        const float t = inner<ACT>(x), e = expf(-__builtin_fabsf(t));
        const float q = e / (1.0f + e);
        // the factor of q held at the largest number, so that infinity less nothing is infinity
        const float h = x < 0x1.fffffep127f ? x : 0x1.fffffep127f;
        return t > 0.0f ? __builtin_fmaf(-h, q, x) : x * q;
    } else {
        return x * __builtin_amdgcn_rcpf(1.0f + exp_neg_t<ACT>(x));
    }
}

// act'(x).  Past |x| = 20 the GELU's slope is 0 or 1; t' is taken from x held there, which
// keeps it finite.  A NaN gets through q or s(t).
// 16-bit: s(t) (1 + x t' (1 - s(t))); the difference's error (2^-24, next to x t' of at most
// some dozens where it matters) is far below the rounding to come.
template <int F, int ACT>
__device__ __forceinline__ float act_slope(float x) {
    float xt = x;   // x t'
    if constexpr (ACT == ZERO_ACT_GELU) {
        constexpr float a = 2.0f * kGeluC, b = 3.0f * a * kGeluA;
        const float h = __builtin_amdgcn_fmed3f(x, -20.0f, 20.0f);
        xt = h * __builtin_fmaf(b, h * h, a);
    }
    if constexpr (F == 2) {
        const float t = inner<ACT>(x), e = expf(-__builtin_fabsf(t));
        const float r = 1.0f / (1.0f + e), q = e * r;
        const bool up = t > 0.0f;
        return __builtin_fmaf(q, __builtin_fmaf(xt, r, up ? -1.0f : 1.0f), up ? 1.0f : 0.0f);
    } else {
        const float s = __builtin_amdgcn_rcpf(1.0f + exp_neg_t<ACT>(x));
        return s * __builtin_fmaf(xt, 1.0f - s, 1.0f);
    }
}

// Maximum over the four lanes of a block (quad permutes 1,0,3,2 and 2,3,0,1).
__device__ __forceinline__ uint32_t quad_max(uint32_t a) {
    uint32_t b = __builtin_amdgcn_update_dpp(0u, a, 0xB1, 0xf, 0xf, true);
    a = a > b ? a : b;
    b = __builtin_amdgcn_update_dpp(0u, a, 0x4E, 0xf, 0xf, true);
    return a > b ? a : b;
}

// Codes of eight values of a block whose exponent byte is eb.  RARE: some value of
// the wave is not finite or lies above the largest a checkpoint stands for.
template <int F, bool RARE>
__device__ __forceinline__ u32x2 encode8(const float x[8], uint32_t eb) {
    const float inv = from_bits((254u - eb) << 23);   // 2^-k
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float c = x[j];
        if constexpr (RARE) {
            c = c > kTop<F> ? kTop<F> : c;
            c = c < -kTop<F> ? -kTop<F> : c;
            const bool bad = (bits(x[j]) & 0x7fffffffu) >= 0x7f800000u;
            v[j] = bad ? from_bits(0x7fc00000u) : c * inv;
        } else {
            v[j] = c * inv;
        }
    }
    u32x2 r;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h], v[4 * h + 1], 0, false);
        r[h] = static_cast<uint32_t>(
            __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2], v[4 * h + 3], w, true));
    }
    return r;
}

// Largest magnitude of eight values as FP32 bits; a NaN or infinity counts as such.
__device__ __forceinline__ uint32_t magnitude8(const float x[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t a = bits(x[j]) & 0x7fffffffu;
        m = a > m ? a : m;
    }
    return m;
}

// The values eight codes stand for: code * 2^(eb - 127), exact in FP32.
__device__ __forceinline__ void decode8(u32x2 c, uint32_t eb, float out[8]) {
    const int k = static_cast<int>(eb) - 127;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(c[h]), false);
        const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(c[h]), true);
        out[4 * h] = __builtin_amdgcn_ldexpf(lo.x, k);
        out[4 * h + 1] = __builtin_amdgcn_ldexpf(lo.y, k);
        out[4 * h + 2] = __builtin_amdgcn_ldexpf(hi.x, k);
        out[4 * h + 3] = __builtin_amdgcn_ldexpf(hi.y, k);
    }
}

__device__ __forceinline__ u32x2 load_codes(const uint8_t *p, uint32_t n) {
    if (n == 8) return __builtin_nontemporal_load(reinterpret_cast<const u32x2_any *>(p));
    u32x2 r{0u, 0u};
#pragma unroll
    for (uint32_t j = 0; j < 8; ++j)
        if (j < n) r[j / 4] |= static_cast<uint32_t>(p[j]) << (8 * (j % 4));
    return r;
}

__device__ __forceinline__ void store_codes(uint8_t *p, uint32_t n, u32x2 c) {
    if (n == 8) {
        __builtin_nontemporal_store(c, reinterpret_cast<u32x2_any *>(p));
        return;
    }
#pragma unroll
    for (uint32_t j = 0; j < 8; ++j)
        if (j < n) p[j] = static_cast<uint8_t>(c[j / 4] >> (8 * (j % 4)));
}

// y may be x: every lane reads its elements before it writes them.
template <int F, int ACT, bool FLAT>
__global__ __launch_bounds__(kThreads) void act_save_kernel(
    uint8_t *__restrict__ q, uint8_t *__restrict__ e, elem_t<F> *y, uint64_t ldy,
    const elem_t<F> *x, uint64_t ldx, uint64_t cols, FastDiv nb, uint64_t n_groups) {
    constexpr uint64_t kTile = kThreads * kUnroll;
    for (uint64_t t0 = blockIdx.x * kTile; t0 < n_groups; t0 += gridDim.x * kTile) {
        float v[kUnroll][8];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const uint64_t g = t0 + u * kThreads + threadIdx.x;
            if (g < n_groups) {
                const Group<FLAT> p(g, nb, cols);
                const elem_t<F> *s = x + p.row * ldx + p.col;
                if (p.n == 8)
                    widen8<F>(load8<F>(s), v[u]);
                else
                    load_some<F>(s, p.n, v[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const uint64_t g = t0 + u * kThreads + threadIdx.x;
            if (g < n_groups) {   // n_groups is a multiple of 4: whole blocks take part
                const Group<FLAT> p(g, nb, cols);
                uint32_t m = magnitude8(v[u]);
                const bool rare = __any(m > bits(kTop<F>));
                if (rare) {   // the block's scale goes by its finite elements
                    m = 0;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t a = bits(v[u][j]) & 0x7fffffffu;
                        m = a < 0x7f800000u && a > m ? a : m;
                    }
                }
                m = quad_max(m);
                const int b0 = static_cast<int>(m >> 23) - 8 + ((m & 0x7fffffu) > 0x600000u ? 1 : 0);
                const uint32_t eb = static_cast<uint32_t>(b0 < 3 ? 3 : b0);
                const u32x2 c = rare ? encode8<F, true>(v[u], eb) : encode8<F, false>(v[u], eb);
                store_codes(q + p.row * cols + p.col, p.n, c);
                if ((g & 3) == 0) e[g >> 2] = static_cast<uint8_t>(eb);
                if constexpr (ACT != ZERO_ACT_NONE) {
                    float r[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) r[j] = act_value<F, ACT>(v[u][j]);
                    elem_t<F> *d = y + p.row * ldy + p.col;
                    if (p.n == 8)
                        store8<F>(d, r);
                    else
                        store_some<F>(d, p.n, r);
                }
            }
        }
    }
}

// ACT == NONE: x = the checkpoint's values (dy is not used).  Otherwise
// dx = dy * act'(value); dx may be dy.
template <int F, int ACT, bool FLAT>
__global__ __launch_bounds__(kThreads) void act_read_kernel(
    elem_t<F> *dx, uint64_t lddx, const elem_t<F> *dy, uint64_t lddy,
    const uint8_t *__restrict__ q, const uint8_t *__restrict__ e, uint64_t cols, FastDiv nb,
    uint64_t n_groups) {
    constexpr uint64_t kTile = kThreads * kUnroll;
    for (uint64_t t0 = blockIdx.x * kTile; t0 < n_groups; t0 += gridDim.x * kTile) {
        float v[kUnroll][8];
        u32x2 c[kUnroll];
        uint32_t eb[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const uint64_t g = t0 + u * kThreads + threadIdx.x;
            if (g < n_groups) {
                const Group<FLAT> p(g, nb, cols);
                c[u] = load_codes(q + p.row * cols + p.col, p.n);
                eb[u] = e[g >> 2];
                if constexpr (ACT != ZERO_ACT_NONE) {
                    const elem_t<F> *s = dy + p.row * lddy + p.col;
                    if (p.n == 8)
                        widen8<F>(load8<F>(s), v[u]);
                    else
                        load_some<F>(s, p.n, v[u]);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const uint64_t g = t0 + u * kThreads + threadIdx.x;
            if (g < n_groups) {
                const Group<FLAT> p(g, nb, cols);
                float r[8];
                decode8(c[u], eb[u], r);
                if constexpr (ACT != ZERO_ACT_NONE) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) r[j] = v[u][j] * act_slope<F, ACT>(r[j]);
                }
                elem_t<F> *d = dx + p.row * lddx + p.col;
                if (p.n == 8)
                    store8<F>(d, r);
                else
                    store_some<F>(d, p.n, r);
            }
        }
    }
}

// Blocks of a row, and the groups of the whole matrix.  flat: one long row of
// whole blocks.
struct Shape {
    bool flat;
    FastDiv nb;
    uint64_t groups;
    uint32_t grid;
};

Shape shape_of(uint64_t rows, uint64_t cols, bool contiguous) {
    Shape s;
    const uint64_t nb = (cols + ZERO_ACT_BLOCK - 1) / ZERO_ACT_BLOCK;
    s.flat = contiguous && cols % ZERO_ACT_BLOCK == 0;
    s.nb = fast_div(static_cast<uint32_t>(nb));
    s.groups = rows * nb * 4;
    const uint64_t tile = static_cast<uint64_t>(kThreads) * kUnroll;
    const uint64_t blocks = (s.groups + tile - 1) / tile, cap = max_blocks();
    s.grid = static_cast<uint32_t>(blocks < cap ? blocks : cap);
    return s;
}

template <int F, int ACT>
hipError_t save_as(uint8_t *q, uint8_t *e, void *y, uint64_t ldy, const void *x, uint64_t ldx,
                   uint64_t rows, uint64_t cols, hipStream_t stream) {
    const Shape s = shape_of(rows, cols, ldx == cols && (ACT == ZERO_ACT_NONE || ldy == cols));
    auto *yt = static_cast<elem_t<F> *>(y);
    auto *xt = static_cast<const elem_t<F> *>(x);
    if (s.flat)
        act_save_kernel<F, ACT, true><<<s.grid, kThreads, 0, stream>>>(q, e, yt, ldy, xt, ldx,
                                                                      cols, s.nb, s.groups);
    else
        act_save_kernel<F, ACT, false><<<s.grid, kThreads, 0, stream>>>(q, e, yt, ldy, xt, ldx,
                                                                       cols, s.nb, s.groups);
    return hipGetLastError();
}

template <int F, int ACT>
hipError_t read_as(void *dx, uint64_t lddx, const void *dy, uint64_t lddy, const uint8_t *q,
                   const uint8_t *e, uint64_t rows, uint64_t cols, hipStream_t stream) {
    const Shape s = shape_of(rows, cols, lddx == cols && (ACT == ZERO_ACT_NONE || lddy == cols));
    auto *dt = static_cast<elem_t<F> *>(dx);
    auto *st = static_cast<const elem_t<F> *>(dy);
    if (s.flat)
        act_read_kernel<F, ACT, true><<<s.grid, kThreads, 0, stream>>>(dt, lddx, st, lddy, q, e,
                                                                      cols, s.nb, s.groups);
    else
        act_read_kernel<F, ACT, false><<<s.grid, kThreads, 0, stream>>>(dt, lddx, st, lddy, q, e,
                                                                       cols, s.nb, s.groups);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_act_save(uint8_t *q, uint8_t *e, void *y, uint64_t ldy, const void *x,
                           uint64_t ldx, int fmt, int act, uint64_t rows, uint64_t cols,
                           hipStream_t stream) {
#define ZS_SAVE(F, A) \
    if (fmt == F && act == A) return save_as<F, A>(q, e, y, ldy, x, ldx, rows, cols, stream);
    ZS_SAVE(0, 0) ZS_SAVE(0, 1) ZS_SAVE(0, 2)
    ZS_SAVE(1, 0) ZS_SAVE(1, 1) ZS_SAVE(1, 2)
    ZS_SAVE(2, 0) ZS_SAVE(2, 1) ZS_SAVE(2, 2)
#undef ZS_SAVE
    return hipErrorInvalidValue;
}

hipError_t launch_act_load(void *x, uint64_t ldx, int fmt, const uint8_t *q, const uint8_t *e,
                           uint64_t rows, uint64_t cols, hipStream_t stream) {
    if (fmt == 0) return read_as<0, 0>(x, ldx, nullptr, 0, q, e, rows, cols, stream);
    if (fmt == 1) return read_as<1, 0>(x, ldx, nullptr, 0, q, e, rows, cols, stream);
    return read_as<2, 0>(x, ldx, nullptr, 0, q, e, rows, cols, stream);
}

hipError_t launch_act_backward(void *dx, uint64_t lddx, const void *dy, uint64_t lddy, int fmt,
                               int act, const uint8_t *q, const uint8_t *e, uint64_t rows,
                               uint64_t cols, hipStream_t stream) {
#define ZS_BACK(F, A) \
    if (fmt == F && act == A) return read_as<F, A>(dx, lddx, dy, lddy, q, e, rows, cols, stream);
    ZS_BACK(0, 1) ZS_BACK(0, 2) ZS_BACK(1, 1) ZS_BACK(1, 2) ZS_BACK(2, 1) ZS_BACK(2, 2)
#undef ZS_BACK
    return hipErrorInvalidValue;
}

}  // namespace zs
