// gfx950 kernels of the step between two blocks, for each row
//     n = post(f),  u = s r + gate * drop(n),  h = pre(u)
// and of its backward pass.
//
// Mathematics.  With z = (x - mean) rho the normalised row and g the gradient of z, a norm
// passes back rho (g - [mean(g)] - z mean(g z)) (the bracket for the layer norm only).  So
// a row of the backward pass needs two pairs of sums, one after the other:
//     g2 = w2 dh        c = mean(g2 u^), [mean(g2)]     G' = du + rho2 (g2 - [..] - u^ c)
//     G = drop(G')      g1 = w1 gate G   the same of f^  df = rho1 (g1 - [..] - f^ c)
// and the parameters' gradients need four sums over the rows for each column, whatever the
// kinds of norm: sum dh u^, sum dh, A = sum G f^ and B = sum G; the gate's is w1 A + b1 B, the
// post norm's gate A and gate B.
//
// What bounds it: HBM, with the arithmetic close behind.  16384 x 8192, norms of the mean
// square on both sides and a gate, means over calls in a row: all BF16 172 to 199 us forward in
// different runs (6.2 to 5.4 TB/s) and 274 backward (5.9), the stream in FP32 293 and 464 (5.5
// and 5.2); all FP32 415 and 630 (5.2 and 5.1).  Rows walked over several times in memory took
// 367 and 672, and 398 and 965 (the latter before their requests stood a row ahead); rows past
// 16384 columns still are (4096 x 20480 BF16 212 and 446, half and a third of HBM's rate).  64 x
// 768 FP16: 5.5 us forward, the launch and two sums; 1023 x 768 backward 13 and 4 for the join.
//
// Sums of squares are taken around the mean (two passes over a row that is on chip); rows
// whose sum leaves FP32's middle are summed again scaled by 2^-80.
#include "block_device.h"

#pragma clang fp contract(off)

namespace zs {
namespace {

constexpr int kWideThreads = 256;

// Sum over a wave, the same in every lane: four steps inside the sixteen lanes of a DPP
// row (quad permutes, then the half row and the row mirrored), then the four rows' sums.
__device__ __forceinline__ float wave_total(float x) {
#define ZS_STEP(C) \
    x = x + from_bits(__builtin_amdgcn_update_dpp(0u, bits(x), C, 0xf, 0xf, true))
    ZS_STEP(0xB1);
    ZS_STEP(0x4E);
    ZS_STEP(0x141);
    ZS_STEP(0x140);
#undef ZS_STEP
    const int b = static_cast<int>(bits(x));
    const float a0 = from_bits(static_cast<uint32_t>(__builtin_amdgcn_readlane(b, 0)));
    const float a1 = from_bits(static_cast<uint32_t>(__builtin_amdgcn_readlane(b, 16)));
    const float a2 = from_bits(static_cast<uint32_t>(__builtin_amdgcn_readlane(b, 32)));
    const float a3 = from_bits(static_cast<uint32_t>(__builtin_amdgcn_readlane(b, 48)));
    return (a0 + a1) + (a2 + a3);
}

// mean and 1 / sqrt(mean of squares around it + eps) of a row of `cols` values; total(op) is
// the sum of op(x) over the row.  Only a row that is not finite or whose sum of squares is
// 2^120 and more takes the scaled sums.
template <typename Total>
__device__ __forceinline__ void row_stats(int kind, float cols, float eps, Total &&total,
                                          float *mean, float *rho) {
    float m = 0.0f;
    if (kind == ZERO_NORM_LAYER) m = total([](float x) { return x; }) / cols;
    float ss = total([m](float x) { return (x - m) * (x - m); });
    if (ss < 0x1p120f) {
        *mean = m;
        *rho = 1.0f / sqrtf(ss / cols + eps);
        return;
    }
    constexpr float k = 0x1p-80f;
    m = kind == ZERO_NORM_LAYER ? total([](float x) { return x * k; }) / cols : 0.0f;
    ss = total([m](float x) { return (x * k - m) * (x * k - m); });
    const float v = ss / cols + eps * k * k;
    *mean = m * 0x1p80f;
    *rho = 1.0f / sqrtf(v < 0x1p-120f ? 0x1p-120f : v) * k;   // equal values: no quotient by 0
}

// Eight values of a parameter from column col on: `other` where there is none.
template <int F>
__device__ __forceinline__ void load_param(const void *p, uint32_t col, uint32_t n, float other,
                                           float out[8]) {
    if (p == nullptr) {
#pragma unroll
        for (int j = 0; j < 8; ++j) out[j] = other;
        return;
    }
    const elem_t<F> *s = static_cast<const elem_t<F> *>(p) + col;
    if (n == 8)
        widen8<F>(load8_cached<F>(s), out);
    else
        load_some<F>(s, n, out);
}

template <int F>
__device__ __forceinline__ void load_row(const elem_t<F> *row, uint32_t col, uint32_t n,
                                         float out[8]) {
    if (n == 8)
        widen8<F>(load8_cached<F>(row + col), out);
    else
        load_some<F>(row + col, n, out);
}

template <int F>
__device__ __forceinline__ void store_row(elem_t<F> *row, uint32_t col, uint32_t n,
                                          const float v[8]) {
    if (n == 8)
        store8<F>(row + col, v);
    else
        store_some<F>(row + col, n, v);
}

// What a kernel is told of the step (pointers that may be null are checked for it).
struct Step {
    uint64_t rows;
    uint32_t cols;
    int post, pre;
    float eps, res_scale;
    const void *w1, *b1, *gate, *w2, *b2;
    Mask mask;
};

// gate * drop(n) of eight values f of a row, n = (f - mean) rho w1 + b1.
template <int F>
__device__ __forceinline__ void branch8(const Step &s, const MaskKey &key, uint32_t row,
                                        uint32_t col, uint32_t n, float mean, float rho,
                                        float v[8]) {
    float w[8], b[8], g[8];
    load_param<F>(s.w1, col, n, 1.0f, w);
    load_param<F>(s.b1, col, n, 0.0f, b);
    load_param<F>(s.gate, col, n, 1.0f, g);
    const uint32_t keep = s.mask.threshold != 0 ? key.keep8(row, col >> 3) : 0xffu;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float x = s.post != ZERO_NORM_NONE ? (v[j] - mean) * rho : v[j];
        x = (x * w[j] + b[j]) * g[j];
        v[j] = (keep >> j) & 1u ? x * s.mask.factor : 0.0f;
    }
}

// ---- rows of any length: a workgroup walks a row several times -------------------------

// Sum over the workgroup, the same in every lane; `slots` is used in two halves in turn, so
// that one barrier a sum is enough.
struct BlockTotal {
    float *slots;
    uint32_t turn = 0;
    __device__ __forceinline__ float operator()(float x) {
        constexpr uint32_t W = kWideThreads / 64;
        float *mine = slots + (turn ^= 1u) * W;
        x = wave_total(x);
        if ((threadIdx.x & 63u) == 0) mine[threadIdx.x >> 6] = x;
        __syncthreads();
        float t = mine[0];
#pragma unroll
        for (uint32_t w = 1; w < W; ++w) t = t + mine[w];
        return t;
    }
};

template <int F, int R>
__global__ __launch_bounds__(kWideThreads) void wide_forward_kernel(
    Step s, elem_t<R> *u, uint64_t ldu, elem_t<F> *h, uint64_t ldh, float *stats,
    const elem_t<R> *r, uint64_t ldr, const elem_t<F> *f, uint64_t ldf) {
    __shared__ float slots[2 * kWideThreads / 64];
    BlockTotal block{slots};
    const MaskKey key(s.mask);
    const float cols = static_cast<float>(s.cols);
    constexpr uint32_t kStride = kWideThreads * 8;
    for (uint64_t row = blockIdx.x; row < s.rows; row += gridDim.x) {
        float mean1 = 0.0f, rho1 = 1.0f, mean2 = 0.0f, rho2 = 1.0f;
        // the sum of op over the row of values that get(col, n, v) gives
        auto total_of = [&](auto &&get, auto &&op) {
            float sum = 0.0f;
            for (uint64_t c = threadIdx.x * 8u; c < s.cols; c += kStride) {
                const uint32_t col = static_cast<uint32_t>(c);
                const uint32_t n = s.cols - col < 8 ? s.cols - col : 8u;
                float v[8];
                get(col, n, v);
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j) sum = sum + (j < n ? op(v[j]) : 0.0f);
            }
            return block(sum);
        };
        auto get_f = [&](uint32_t col, uint32_t n, float v[8]) {
            load_row<F>(f + row * ldf, col, n, v);
        };
        if (s.post != ZERO_NORM_NONE)
            row_stats(s.post, cols, s.eps, [&](auto &&op) { return total_of(get_f, op); },
                      &mean1, &rho1);
        auto get_u = [&](uint32_t col, uint32_t n, float v[8]) {
            load_row<R>(r + row * ldr, col, n, v);
            if (f == nullptr) return;
            float b[8];
            load_row<F>(f + row * ldf, col, n, b);
            branch8<F>(s, key, static_cast<uint32_t>(row), col, n, mean1, rho1, b);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = s.res_scale * v[j] + b[j];
        };
        if (s.pre != ZERO_NORM_NONE)
            row_stats(s.pre, cols, s.eps, [&](auto &&op) { return total_of(get_u, op); },
                      &mean2, &rho2);
        for (uint64_t c = threadIdx.x * 8u; c < s.cols; c += kStride) {
            const uint32_t col = static_cast<uint32_t>(c);
            const uint32_t n = s.cols - col < 8 ? s.cols - col : 8u;
            float v[8], w[8], b[8];
            get_u(col, n, v);
            if (u != nullptr) store_row<R>(u + row * ldu, col, n, v);
            if (h == nullptr) continue;
            load_param<F>(s.w2, col, n, 1.0f, w);
            load_param<F>(s.b2, col, n, 0.0f, b);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = (v[j] - mean2) * rho2 * w[j] + b[j];
            store_row<F>(h + row * ldh, col, n, v);
        }
        if (stats != nullptr && threadIdx.x == 0) {
            float *d = stats + row * 4;
            d[0] = mean1;
            d[1] = rho1;
            d[2] = mean2;
            d[3] = rho2;
        }
    }
}

// What the backward kernels read of a row and write of it.
template <int F, int R>
struct Back {
    const elem_t<F> *dh, *f;   // nullable
    const elem_t<R> *du, *u;   // du nullable
    elem_t<F> *df;
    elem_t<R> *dr;
    uint64_t lddh, ldf, lddu, ldu, lddf, lddr;
    const float *stats;
};

// A row's four statistics and the four means of its backward pass.
struct RowMeans {
    float mean1, rho1, mean2, rho2;
    float zg2, g2, zg1, g1;
};

// u^ and dh of eight columns.
template <int F, int R>
__device__ __forceinline__ void pre8(const Back<F, R> &p, uint64_t row, uint32_t col, uint32_t n,
                                     const RowMeans &m, float dh[8], float uhat[8]) {
    if (p.dh == nullptr) {
#pragma unroll
        for (int j = 0; j < 8; ++j) dh[j] = uhat[j] = 0.0f;
        return;
    }
    load_row<F>(p.dh + row * p.lddh, col, n, dh);
    load_row<R>(p.u + row * p.ldu, col, n, uhat);
#pragma unroll
    for (int j = 0; j < 8; ++j) uhat[j] = (uhat[j] - m.mean2) * m.rho2;
}

// G' of eight columns from dh and u^; w2: the pre norm's weight there.
template <int F, int R>
__device__ __forceinline__ void stream8(const Back<F, R> &p, uint64_t row, uint32_t col,
                                        uint32_t n, const RowMeans &m, const float dh[8],
                                        const float uhat[8], const float w2[8], float out[8]) {
    float du[8];
    if (p.du != nullptr) {
        load_row<R>(p.du + row * p.lddu, col, n, du);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) du[j] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        out[j] = p.dh == nullptr ? du[j]
                                 : du[j] + m.rho2 * ((w2[j] * dh[j] - m.g2) - uhat[j] * m.zg2);
}

// G = drop(G') in place, and f^ (f itself without a post norm) of eight columns.
template <int F, int R>
__device__ __forceinline__ void post8(const Step &s, const MaskKey &key, const Back<F, R> &p,
                                      uint64_t row, uint32_t col, uint32_t n, const RowMeans &m,
                                      float G[8], float fhat[8]) {
    load_row<F>(p.f + row * p.ldf, col, n, fhat);
    const uint32_t keep =
        s.mask.threshold != 0 ? key.keep8(static_cast<uint32_t>(row), col >> 3) : 0xffu;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        G[j] = (keep >> j) & 1u ? G[j] * s.mask.factor : 0.0f;
        if (s.post != ZERO_NORM_NONE) fhat[j] = (fhat[j] - m.mean1) * m.rho1;
    }
}

// A row's means, to means[row][4].
template <int F, int R>
__global__ __launch_bounds__(kWideThreads) void wide_means_kernel(Step s, Back<F, R> p,
                                                                 float *__restrict__ means) {
    __shared__ float slots[2 * kWideThreads / 64];
    BlockTotal block{slots};
    const MaskKey key(s.mask);
    const float cols = static_cast<float>(s.cols);
    constexpr uint32_t kStride = kWideThreads * 8;
    for (uint64_t row = blockIdx.x; row < s.rows; row += gridDim.x) {
        const float *st = p.stats + row * 4;
        RowMeans m{st[0], st[1], st[2], st[3], 0.0f, 0.0f, 0.0f, 0.0f};
        float zg = 0.0f, g = 0.0f;
        if (s.pre != ZERO_NORM_NONE) {
            for (uint64_t c = threadIdx.x * 8u; c < s.cols; c += kStride) {
                const uint32_t col = static_cast<uint32_t>(c);
                const uint32_t n = s.cols - col < 8 ? s.cols - col : 8u;
                float dh[8], uhat[8], w2[8];
                pre8(p, row, col, n, m, dh, uhat);
                load_param<F>(s.w2, col, n, 1.0f, w2);
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j) {
                    const float x = j < n ? w2[j] * dh[j] : 0.0f;
                    g = g + x;
                    zg = zg + (j < n ? x * uhat[j] : 0.0f);
                }
            }
            m.zg2 = block(zg) / cols;
            if (s.pre == ZERO_NORM_LAYER) m.g2 = block(g) / cols;
        }
        if (s.post != ZERO_NORM_NONE) {
            zg = g = 0.0f;
            for (uint64_t c = threadIdx.x * 8u; c < s.cols; c += kStride) {
                const uint32_t col = static_cast<uint32_t>(c);
                const uint32_t n = s.cols - col < 8 ? s.cols - col : 8u;
                float dh[8], uhat[8], G[8], fhat[8], w[8];
                pre8(p, row, col, n, m, dh, uhat);
                load_param<F>(s.w2, col, n, 1.0f, w);
                stream8(p, row, col, n, m, dh, uhat, w, G);
                post8(s, key, p, row, col, n, m, G, fhat);
                float gate[8];
                load_param<F>(s.w1, col, n, 1.0f, w);
                load_param<F>(s.gate, col, n, 1.0f, gate);
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j) {
                    const float x = j < n ? w[j] * (gate[j] * G[j]) : 0.0f;
                    g = g + x;
                    zg = zg + (j < n ? x * fhat[j] : 0.0f);
                }
            }
            m.zg1 = block(zg) / cols;
            if (s.post == ZERO_NORM_LAYER) m.g1 = block(g) / cols;
        }
        if (threadIdx.x == 0) {
            float *d = means + row * 4;
            d[0] = m.zg2;
            d[1] = m.g2;
            d[2] = m.zg1;
            d[3] = m.g1;
        }
    }
}

// The n (0 to 8) columns of a group that are the lane's, zeros past them; ragged: the row's
// length is no multiple of eight.
template <int F>
__device__ __forceinline__ void widen_some(Raw8<F> &r, bool ragged, uint32_t n, float out[8]) {
    if (ragged) {
        if (n - 1u < 7u) move_down<F>(r, n);
    }
    if (n != 0) {
        widen8<F>(r, out);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) out[j] = 0.0f;
    }
}

// df, dr and the four column sums over the rows of part blockIdx.y, to
// part[blockIdx.y][4][cols].  A lane owns eight columns; the next row's are on their way while
// it works on this one's (read without a branch where rows have eight columns at least, see
// below).  df may be dh, and dr du: a lane reads its elements before it writes them.
template <int F, int R, bool NARROW>
__global__ __launch_bounds__(kWideThreads) void wide_backward_kernel(
    Step s, Back<F, R> p, const float *__restrict__ means, float *__restrict__ part,
    uint64_t rows_per_part) {
    const MaskKey key(s.mask);
    const uint64_t first = blockIdx.y * rows_per_part;
    const uint64_t last = first + rows_per_part < s.rows ? first + rows_per_part : s.rows;
    const bool pre = s.pre != ZERO_NORM_NONE, post = s.post != ZERO_NORM_NONE;
    const bool ragged = s.cols % 8 != 0;
    constexpr uint64_t kStride = kWideThreads * 8;
    for (uint64_t c = blockIdx.x * kStride + threadIdx.x * 8u; c < s.cols;
         c += gridDim.x * kStride) {
        const uint32_t col = static_cast<uint32_t>(c);
        const uint32_t n = s.cols - col < 8 ? s.cols - col : 8u;
        float w1[8], w2[8], gate[8], sums[4][8] = {};
        load_param<F>(s.w1, col, n, 1.0f, w1);
        load_param<F>(s.w2, col, n, 1.0f, w2);
        load_param<F>(s.gate, col, n, 1.0f, gate);
        Raw8<F> raw_dh, raw_f;
        Raw8<R> raw_u, raw_du;
        auto fetch = [&](uint64_t t) {
            const elem_t<F> *dh = pre ? p.dh + t * p.lddh : p.f + t * p.ldf;
            const elem_t<R> *u = pre ? p.u + t * p.ldu : p.du + t * p.lddu;
            const elem_t<F> *f = p.f != nullptr ? p.f + t * p.ldf : dh;
            const elem_t<R> *du = p.du != nullptr ? p.du + t * p.lddu : u;
            if constexpr (!NARROW) {
                raw_dh = raw_group<F>(dh, col, s.cols);
                raw_u = raw_group<R>(u, col, s.cols);
                raw_f = raw_group<F>(f, col, s.cols);
                raw_du = raw_group<R>(du, col, s.cols);
            } else {
                float v[8];
                load_some<F>(dh + col, n, v);
                raw_dh = narrow8<F>(v);
                load_some<R>(u + col, n, v);
                raw_u = narrow8<R>(v);
                load_some<F>(f + col, n, v);
                raw_f = narrow8<F>(v);
                load_some<R>(du + col, n, v);
                raw_du = narrow8<R>(v);
            }
        };
        if (first < last) fetch(first);
        for (uint64_t row = first; row < last; ++row) {
            const float *st = p.stats + row * 4, *mn = means + row * 4;
            const float mean1 = st[0], rho1 = st[1], mean2 = st[2], rho2 = st[3];
            const float zg2 = mn[0], g2 = mn[1], zg1 = mn[2], g1 = mn[3];
            float dh[8], z[8], G[8], fh[8], out[8];
            const bool move = ragged && !NARROW;
            widen_some<F>(raw_dh, move, n, dh);
            widen_some<R>(raw_u, move, n, z);
            widen_some<F>(raw_f, move, n, fh);
            widen_some<R>(raw_du, move, n, G);
            fetch(row + 1 < last ? row + 1 : row);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (p.du == nullptr) G[j] = 0.0f;
                if (pre) {
                    z[j] = (z[j] - mean2) * rho2;
                    sums[0][j] = __builtin_fmaf(dh[j], z[j], sums[0][j]);
                    sums[1][j] = sums[1][j] + dh[j];
                    const float g = w2[j] * dh[j];
                    G[j] = __builtin_fmaf(rho2, __builtin_fmaf(-zg2, z[j], g - g2), G[j]);
                }
                out[j] = product32(s.res_scale, G[j]);
            }
            if (p.f != nullptr) {
                const uint32_t keep = s.mask.threshold != 0
                                          ? key.keep8(static_cast<uint32_t>(row), col >> 3)
                                          : 0xffu;
                float df[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    G[j] = (keep >> j) & 1u ? G[j] * s.mask.factor : 0.0f;
                    if (post) fh[j] = (fh[j] - mean1) * rho1;
                    sums[2][j] = __builtin_fmaf(G[j], fh[j], sums[2][j]);
                    sums[3][j] = sums[3][j] + G[j];
                    const float x = product32(gate[j], G[j]);
                    df[j] = post ? product32(rho1, __builtin_fmaf(-zg1, fh[j], w1[j] * x - g1))
                                 : x;
                }
                store_row<F>(p.df + row * p.lddf, col, n, df);
            }
            store_row<R>(p.dr + row * p.lddr, col, n, out);
        }
        float *d = part + blockIdx.y * 4ull * s.cols + col;
#pragma unroll
        for (int k = 0; k < 4; ++k) store_row<2>(d + static_cast<uint64_t>(k) * s.cols, 0, n, sums[k]);
    }
}

// ---- rows that stay on chip ---------------------------------------------------------------
//
// A row is held by W waves, V groups of eight columns a lane.  Rows of up to 64 x 8 V columns
// take one wave each (no barriers) and several waves a workgroup; longer ones a workgroup each.
//
// The next row's data is on its way while this one is worked on, each operand requested anew
// as soon as its registers are free: what a row needs first is asked for half a row before
// what it needs last, so the memory is never waited for with nothing in flight (all requests
// at one point: 244 and 348 us forward and backward at 16384 x 8192 BF16).  So that the waits
// are exact, rows are read without a branch: lanes without columns read the row's last eight,
// and an operand that is not there is read from another one's place.

constexpr int kRowWaves = 16;   // most waves of a workgroup

// Sums over a row's W waves, the same in every lane.  The waves' sums go through LDS, in two
// halves in turn, so that one barrier a sum is enough; W == 1 needs neither.
struct RowTotal {
    float (*slots)[2][kRowWaves];   // [turn][value][wave]
    uint32_t waves, wave, lane, turn;
    __device__ __forceinline__ RowTotal(float (*p)[2][kRowWaves], uint32_t w)
        : slots(p), waves(w),
          wave(static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6))),
          lane(threadIdx.x & 63u), turn(0) {}
    __device__ __forceinline__ float join(uint32_t which) const {
        float x = (lane & 15u) < waves ? slots[turn][which][lane & 15u] : 0.0f;
#define ZS_STEP(C) \
    x = x + from_bits(__builtin_amdgcn_update_dpp(0u, bits(x), C, 0xf, 0xf, true))
        ZS_STEP(0xB1);
        ZS_STEP(0x4E);
        ZS_STEP(0x141);
        ZS_STEP(0x140);
#undef ZS_STEP
        return x;
    }
    __device__ __forceinline__ float operator()(float x) {
        x = wave_total(x);
        if (waves == 1) return x;
        turn ^= 1u;
        if (lane == 0) slots[turn][0][wave] = x;
        __syncthreads();
        return join(0);
    }
    __device__ __forceinline__ void operator()(float *x, float *y) {
        *x = wave_total(*x);
        *y = wave_total(*y);
        if (waves == 1) return;
        turn ^= 1u;
        if (lane == 0) {
            slots[turn][0][wave] = *x;
            slots[turn][1][wave] = *y;
        }
        __syncthreads();
        *x = join(0);
        *y = join(1);
    }
};

// This lane's groups of a row: group v holds columns col(v) .. col(v) + n(v) - 1.
template <int V>
struct LaneColumns {
    uint32_t at, step, cols;
    __device__ __forceinline__ LaneColumns(uint32_t lane_of_row, uint32_t lanes, uint32_t c)
        : at(lane_of_row * 8), step(lanes * 8), cols(c) {}
    __device__ __forceinline__ uint32_t col(int v) const { return at + v * step; }
    __device__ __forceinline__ uint32_t n(int v) const {
        const uint32_t c = col(v);
        return c >= cols ? 0u : cols - c < 8 ? cols - c : 8u;
    }
};

// What the columns of a lane are multiplied with and shifted by: HELD in registers over all
// its rows, or read again for each (where the registers do not suffice).  A parameter that is
// not there costs nothing: the branch on it is the same in every lane.
template <int F, int V, bool HELD>
struct Held {
    const void *p;
    const void *q;         // nullable: a second factor
    float other;
    float v[HELD ? V : 1][8];
    __device__ __forceinline__ Held(const void *first, const void *second, float o)
        : p(first), q(second), other(o) {}
    __device__ __forceinline__ bool there() const { return p != nullptr || q != nullptr; }
    __device__ __forceinline__ void read(int i, uint32_t col, uint32_t n) {
        load_param<F>(p, col, n, other, v[i]);
        if (q == nullptr) return;
        float w[8];
        load_param<F>(q, col, n, 1.0f, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * w[j];
    }
    __device__ __forceinline__ void hold(const LaneColumns<V> &m) {
        if constexpr (HELD) {
            if (!there()) return;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (m.n(i) != 0) read(i, m.col(i), m.n(i));
        }
    }
    // group i's eight values; only where there() is
    __device__ __forceinline__ const float *at(const LaneColumns<V> &m, int i) {
        if constexpr (HELD) return v[i];
        read(0, m.col(i), m.n(i));
        return v[0];
    }
};

// waves: of a row (W).  A workgroup of W == 1 takes blockDim.x / 64 rows at once.
template <int F, int R, int V>
__global__ __launch_bounds__(64 * kRowWaves) void row_forward_kernel(
    Step s, uint32_t waves, elem_t<R> *u, uint64_t ldu, elem_t<F> *h, uint64_t ldh, float *stats,
    const elem_t<R> *r, uint64_t ldr, const elem_t<F> *f, uint64_t ldf) {
    constexpr bool kHeld = V == 1;
    __shared__ float slots[2][2][kRowWaves];
    RowTotal total(slots, waves);
    const MaskKey key(s.mask);
    const float cols = static_cast<float>(s.cols);
    const uint32_t at_once = waves == 1 ? blockDim.x >> 6 : 1u;
    const LaneColumns<V> mine(waves == 1 ? total.lane : threadIdx.x, waves * 64, s.cols);
    const uint64_t stride = static_cast<uint64_t>(gridDim.x) * at_once;
    uint64_t row = static_cast<uint64_t>(blockIdx.x) * at_once + (waves == 1 ? total.wave : 0u);

    const bool branch = f != nullptr, ragged = s.cols % 8 != 0;
    const void *const at_f = branch ? static_cast<const void *>(f) : r;   // (only read)
    Raw8<R> raw_r[V];
    Raw8<F> raw_f[V];
    auto fetch_r = [&](uint64_t t) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            raw_r[v] = raw_group<R>(r + t * ldr, mine.col(v), s.cols);
    };
    auto fetch_f = [&](uint64_t t) {
        const auto *base = static_cast<const elem_t<F> *>(at_f) + (branch ? t * ldf : 0);
#pragma unroll
        for (int v = 0; v < V; ++v) raw_f[v] = raw_group<F>(base, mine.col(v), s.cols);
    };
    if (row < s.rows) {
        fetch_f(row);
        fetch_r(row);
    }
    Held<F, V, kHeld> w1(s.w1 != nullptr ? s.w1 : s.gate, s.w1 != nullptr ? s.gate : nullptr, 1.0f);
    Held<F, V, kHeld> b1(s.b1, s.b1 != nullptr ? s.gate : nullptr, 0.0f);
    Held<F, V, kHeld> w2(s.w2, nullptr, 1.0f), b2(s.b2, nullptr, 0.0f);
    w1.hold(mine);
    b1.hold(mine);
    w2.hold(mine);
    b2.hold(mine);
    for (; row < s.rows; row += stride) {
        const uint64_t next = row + stride < s.rows ? row + stride : row;
        float x[V][8], b[V][8];
#pragma unroll
        for (int v = 0; v < V; ++v) widen_some<F>(raw_f[v], ragged, mine.n(v), b[v]);
        fetch_f(next);
        // the sum of op over the row of the values y
        auto total_of = [&](float (*y)[8], auto &&op) {
            float sum = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const uint32_t n = mine.n(v);
                if (n == 8) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum = sum + op(y[v][j]);
                } else if (n != 0) {
#pragma unroll
                    for (uint32_t j = 0; j < 7; ++j) sum = sum + (j < n ? op(y[v][j]) : 0.0f);
                }
            }
            return total(sum);
        };
        float mean1 = 0.0f, rho1 = 1.0f, mean2 = 0.0f, rho2 = 1.0f;
        if (s.post != ZERO_NORM_NONE)
            row_stats(s.post, cols, s.eps, [&](auto &&op) { return total_of(b, op); }, &mean1,
                      &rho1);
#pragma unroll
        for (int v = 0; v < V; ++v) widen_some<R>(raw_r[v], ragged, mine.n(v), x[v]);
        fetch_r(next);
        if (branch) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const uint32_t n = mine.n(v);
                if (n == 0) continue;
                if (s.post == ZERO_NORM_LAYER) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) b[v][j] = b[v][j] - mean1;
                }
                if (s.post != ZERO_NORM_NONE) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) b[v][j] = b[v][j] * rho1;
                }
                if (w1.there()) {
                    const float *w = w1.at(mine, v);
#pragma unroll
                    for (int j = 0; j < 8; ++j) b[v][j] = b[v][j] * w[j];
                }
                if (b1.there()) {
                    const float *c = b1.at(mine, v);
#pragma unroll
                    for (int j = 0; j < 8; ++j) b[v][j] = b[v][j] + c[j];
                }
                if (s.mask.threshold != 0) {
                    const uint32_t keep =
                        key.keep8(static_cast<uint32_t>(row), mine.col(v) >> 3);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        b[v][j] = (keep >> j) & 1u ? b[v][j] * s.mask.factor : 0.0f;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    x[v][j] = __builtin_fmaf(s.res_scale, x[v][j], b[v][j]);
                store_row<R>(u + row * ldu, mine.col(v), n, x[v]);
            }
        }
        if (s.pre != ZERO_NORM_NONE) {
            row_stats(s.pre, cols, s.eps, [&](auto &&op) { return total_of(x, op); }, &mean2,
                      &rho2);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const uint32_t n = mine.n(v);
                if (n == 0) continue;
                if (s.pre == ZERO_NORM_LAYER) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[v][j] = x[v][j] - mean2;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) x[v][j] = x[v][j] * rho2;
                if (w2.there()) {
                    const float *w = w2.at(mine, v);
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[v][j] = product32(x[v][j], w[j]);
                }
                if (b2.there()) {
                    const float *c = b2.at(mine, v);
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[v][j] = x[v][j] + c[j];
                }
                store_row<F>(h + row * ldh, mine.col(v), n, x[v]);
            }
        }
        if (stats != nullptr && mine.at == 0)
            *reinterpret_cast<u32x4_any *>(stats + row * 4) =
                u32x4{bits(mean1), bits(rho1), bits(mean2), bits(rho2)};
    }
}

// Rows part * at_once + wave, further on by parts * at_once; the sums of a part's rows to
// part[part][4][cols].  BIAS: the two sums that biases need as well.
template <int F, int R, int V, int WAVES, bool BIAS>
__global__ __launch_bounds__(64 * WAVES) void row_backward_kernel(
    Step s, uint32_t waves, Back<F, R> p, float *__restrict__ part, uint32_t parts) {
    // Rows of more than 8192 columns: sum dh u^ and sum G f^ of a lane's columns are kept in LDS
    // and factors read again for each row, or the registers would not suffice (16 waves of 128).
    constexpr bool kLong = V == 2 && WAVES == 16, kHeld = !kLong;
    __shared__ float slots[2][2][kRowWaves];
    __shared__ __align__(16) float kept[kLong ? 2 : 1][kLong ? kRowWaves * 1024 : 4];
    // [rows at once][columns in whole groups], W == 1 only
    extern __shared__ __align__(16) float joined[];
    RowTotal total(slots, waves);
    const MaskKey key(s.mask);
    const float cols = static_cast<float>(s.cols);
    const uint32_t at_once = waves == 1 ? blockDim.x >> 6 : 1u;
    const LaneColumns<V> mine(waves == 1 ? total.lane : threadIdx.x, waves * 64, s.cols);
    const uint64_t stride = static_cast<uint64_t>(parts) * at_once;
    const bool pre = s.pre != ZERO_NORM_NONE, post = s.post != ZERO_NORM_NONE;
    const bool ragged = s.cols % 8 != 0;
    const bool layer1 = s.post == ZERO_NORM_LAYER, layer2 = s.pre == ZERO_NORM_LAYER;
    Held<F, V, kHeld> w1(s.w1 != nullptr ? s.w1 : s.gate, s.w1 != nullptr ? s.gate : nullptr, 1.0f);
    Held<F, V, kHeld> w2(s.w2, nullptr, 1.0f);
    w1.hold(mine);
    w2.hold(mine);
    for (uint32_t q = blockIdx.x; q < parts; q += gridDim.x) {
        uint64_t row = static_cast<uint64_t>(q) * at_once + (waves == 1 ? total.wave : 0u);
        // sum dh u^, sum dh, sum G f^, sum G
        float sums[4][V][8] = {};
        if constexpr (kLong) {
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int j = 0; j < 8; j += 4)
                        *reinterpret_cast<f32x4 *>(&kept[k][mine.col(v) + j]) =
                            f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        // sums[k] + x y of group v (k: 0 or 2)
        auto add = [&](int k, int v, const float *x, const float *y) {
            if constexpr (kLong) {
                float *d = &kept[k / 2][mine.col(v)];
#pragma unroll
                for (int j = 0; j < 8; j += 4) {
                    f32x4 t = *reinterpret_cast<f32x4 *>(d + j);
#pragma unroll
                    for (int i = 0; i < 4; ++i) t[i] = __builtin_fmaf(x[j + i], y[j + i], t[i]);
                    *reinterpret_cast<f32x4 *>(d + j) = t;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    sums[k][v][j] = __builtin_fmaf(x[j], y[j], sums[k][v][j]);
            }
        };
        Raw8<F> raw_dh[V], raw_f[V];
        Raw8<R> raw_u[V], raw_du[V];
        auto fetch_pre = [&](uint64_t t) {
            const elem_t<F> *a = pre ? p.dh + t * p.lddh : p.f + t * p.ldf;
            const elem_t<R> *b = pre ? p.u + t * p.ldu : p.du + t * p.lddu;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                raw_dh[v] = raw_group<F>(a, mine.col(v), s.cols);
                raw_u[v] = raw_group<R>(b, mine.col(v), s.cols);
            }
        };
        auto fetch_post = [&](uint64_t t) {
            const elem_t<F> *a = p.f != nullptr ? p.f + t * p.ldf : p.dh + t * p.lddh;
            const elem_t<R> *b = p.du != nullptr ? p.du + t * p.lddu : p.u + t * p.ldu;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                raw_f[v] = raw_group<F>(a, mine.col(v), s.cols);
                raw_du[v] = raw_group<R>(b, mine.col(v), s.cols);
            }
        };
        if (row < s.rows) {
            fetch_pre(row);
            fetch_post(row);
        }
        for (; row < s.rows; row += stride) {
            const uint64_t next = row + stride < s.rows ? row + stride : row;
            const float *st = p.stats + row * 4;
            const float mean1 = st[0], rho1 = st[1], mean2 = st[2], rho2 = st[3];
            // g: w2 dh; z: u^; columns past the row's end have zeros in g (G below), which
            // keeps them out of every sum
            float g[V][8], z[V][8], G[V][8], fh[V][8];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (!pre) continue;
                widen_some<F>(raw_dh[v], ragged, mine.n(v), g[v]);
                widen_some<R>(raw_u[v], ragged, mine.n(v), z[v]);
            }
            fetch_pre(next);
            float zg2 = 0.0f, sg2 = 0.0f;
            if (pre) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    if (mine.n(v) == 0) continue;
                    if (layer2) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) z[v][j] = z[v][j] - mean2;
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        z[v][j] = z[v][j] * rho2;
                        if constexpr (BIAS) sums[1][v][j] = sums[1][v][j] + g[v][j];
                    }
                    add(0, v, g[v], z[v]);
                    if (w2.there()) {
                        const float *w = w2.at(mine, v);
#pragma unroll
                        for (int j = 0; j < 8; ++j) g[v][j] = g[v][j] * w[j];
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) zg2 = __builtin_fmaf(g[v][j], z[v][j], zg2);
                    if (layer2) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) sg2 = sg2 + g[v][j];
                    }
                }
                if (layer2) {
                    total(&zg2, &sg2);
                    sg2 = sg2 / cols;
                } else {
                    zg2 = total(zg2);
                }
                zg2 = zg2 / cols;
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                widen_some<F>(raw_f[v], ragged, mine.n(v), fh[v]);
                widen_some<R>(raw_du[v], ragged, mine.n(v), G[v]);
                if (p.du == nullptr) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) G[v][j] = 0.0f;
                }
            }
            fetch_post(next);
            if (pre) {
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        G[v][j] = __builtin_fmaf(
                            rho2, __builtin_fmaf(-zg2, z[v][j], g[v][j] - sg2), G[v][j]);
            }
            float zg = 0.0f, sg = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const uint32_t n = mine.n(v);
                if (n == 0) continue;
                float out[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) out[j] = product32(s.res_scale, G[v][j]);
                store_row<R>(p.dr + row * p.lddr, mine.col(v), n, out);
                if (p.f == nullptr) continue;
                if (n != 8) {   // (g - sg is not zero there)
#pragma unroll
                    for (uint32_t j = 1; j < 8; ++j) G[v][j] = j < n ? G[v][j] : 0.0f;
                }
                if (s.mask.threshold != 0) {
                    const uint32_t keep =
                        key.keep8(static_cast<uint32_t>(row), mine.col(v) >> 3);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        G[v][j] = (keep >> j) & 1u ? G[v][j] * s.mask.factor : 0.0f;
                }
                if (layer1) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) fh[v][j] = fh[v][j] - mean1;
                }
                if (post) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) fh[v][j] = fh[v][j] * rho1;
                }
                add(2, v, G[v], fh[v]);
                if constexpr (BIAS) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) sums[3][v][j] = sums[3][v][j] + G[v][j];
                }
                if (w1.there()) {
                    const float *w = w1.at(mine, v);
#pragma unroll
                    for (int j = 0; j < 8; ++j) G[v][j] = product32(G[v][j], w[j]);
                }
                if (post) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) zg = __builtin_fmaf(G[v][j], fh[v][j], zg);
                }
                if (layer1) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) sg = sg + G[v][j];
                }
            }
            if (post) {
                if (layer1) {
                    total(&zg, &sg);
                    sg = sg / cols;
                } else {
                    zg = total(zg);
                }
                zg = zg / cols;
            }
            if (p.f != nullptr) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const uint32_t n = mine.n(v);
                    if (n == 0) continue;
                    if (post) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            G[v][j] = product32(rho1,
                                                __builtin_fmaf(-zg, fh[v][j], G[v][j] - sg));
                    }
                    store_row<F>(p.df + row * p.lddf, mine.col(v), n, G[v]);
                }
            }
        }
        // sum k of this part: of one wave's rows (W > 1: of the workgroup's), or of its waves'
        // in their order
#pragma unroll
        for (int k = 0; k < 4; k += BIAS ? 1 : 2) {
            float *d = part + (static_cast<uint64_t>(q) * 4 + k) * s.cols;
            if (at_once == 1) {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (mine.n(v) != 0)
                        store_row<2>(d, mine.col(v), mine.n(v),
                                     kLong && k % 2 == 0 ? &kept[k / 2][mine.col(v)] : sums[k][v]);
                continue;
            }
            // (whole groups, in lines of whole groups)
            const uint32_t line = (s.cols + 7) & ~7u;
            __syncthreads();
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (mine.n(v) == 0) continue;
                f32x4 *t = reinterpret_cast<f32x4 *>(&joined[total.wave * line + mine.col(v)]);
                t[0] = f32x4{sums[k][v][0], sums[k][v][1], sums[k][v][2], sums[k][v][3]};
                t[1] = f32x4{sums[k][v][4], sums[k][v][5], sums[k][v][6], sums[k][v][7]};
            }
            __syncthreads();
            for (uint32_t c = threadIdx.x; c < s.cols; c += blockDim.x) {
                float x = joined[c];
                if (at_once == 8) {
#pragma unroll
                    for (uint32_t w = 1; w < 8; ++w) x = x + joined[w * line + c];
                } else {
                    for (uint32_t w = 1; w < at_once; ++w) x = x + joined[w * line + c];
                }
                d[c] = x;
            }
        }
    }
}

// ---- the parameters' gradients -----------------------------------------------------------

struct Grads {
    void *w1, *b1, *gate, *w2, *b2;   // nullable
    bool first;
};

// G of a column, stored or added.
template <typename T, int G>
__device__ __forceinline__ void put_grad(void *d, uint32_t col, float v, bool first) {
    if (d == nullptr) return;
    T *t = static_cast<T *>(d) + col;
    if constexpr (G == 2)
        *t = first ? v : *t + v;
    else
        *t = from_f32<G>(v);
}

// The parts' four sums of a column: kJoinParts shares of the parts, each added in order by a
// lane that has eight of them in flight, the shares joined in order, a lane a sum, and the
// gradients made from them.  BIAS: all four sums are there, else the first and the third.
// G: the gradients' format.
constexpr uint32_t kJoinCols = 32, kJoinParts = 32;
template <int F, int G, bool BIAS>
__global__ __launch_bounds__(kJoinCols *kJoinParts) void join_grads_kernel(
    Grads g, const float *__restrict__ part, uint32_t parts, uint32_t cols, const void *w1,
    const void *b1, const void *gate) {
    __shared__ float slots[4][kJoinParts][kJoinCols];
    const uint32_t lane_col = threadIdx.x % kJoinCols, share = threadIdx.x / kJoinCols;
    const uint32_t per = (parts + kJoinParts - 1) / kJoinParts;
    const uint32_t from = share * per < parts ? share * per : parts;
    const uint32_t to = from + per < parts ? from + per : parts;
    for (uint64_t c0 = static_cast<uint64_t>(blockIdx.x) * kJoinCols; c0 < cols;
         c0 += static_cast<uint64_t>(gridDim.x) * kJoinCols) {
        const uint64_t col = c0 + lane_col;
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (col < cols) {
#pragma unroll 8
            for (uint32_t k = from; k < to; ++k)
#pragma unroll
                for (int i = 0; i < 4; i += BIAS ? 1 : 2)
                    sum[i] = sum[i] + part[(static_cast<uint64_t>(k) * 4 + i) * cols + col];
        }
#pragma unroll
        for (int i = 0; i < 4; i += BIAS ? 1 : 2) slots[i][share][lane_col] = sum[i];
        __syncthreads();
        if (share < 4 && (BIAS || share % 2 == 0)) {
            float x = slots[share][0][lane_col];
#pragma unroll
            for (uint32_t k = 1; k < kJoinParts; ++k) x = x + slots[share][k][lane_col];
            slots[share][0][lane_col] = x;
        }
        __syncthreads();
        if (share == 0 && col < cols) {
#pragma unroll
            for (int i = 0; i < 4; i += BIAS ? 1 : 2) sum[i] = slots[i][0][lane_col];
            const uint32_t c = static_cast<uint32_t>(col);
            float one[8], bias[8], gt[8];
            load_param<F>(w1, c, 1, 1.0f, one);
            load_param<F>(b1, c, 1, 0.0f, bias);
            load_param<F>(gate, c, 1, 1.0f, gt);
            using T = elem_t<G>;
            put_grad<T, G>(g.w2, c, sum[0], g.first);
            put_grad<T, G>(g.b2, c, sum[1], g.first);
            put_grad<T, G>(g.w1, c, product32(gt[0], sum[2]), g.first);
            put_grad<T, G>(g.b1, c, product32(gt[0], sum[3]), g.first);
            put_grad<T, G>(g.gate, c, one[0] * sum[2] + bias[0] * sum[3], g.first);
        }
        __syncthreads();
    }
}

template <int F, int G>
void join_grads(const Grads &g, const ResidualArgs &a, const float *part, uint32_t parts,
                bool bias_sums, uint32_t blocks, hipStream_t stream) {
    if (bias_sums)
        join_grads_kernel<F, G, true><<<blocks, kJoinCols * kJoinParts, 0, stream>>>(
            g, part, parts, a.cols, a.w1, a.b1, a.gate);
    else
        join_grads_kernel<F, G, false><<<blocks, kJoinCols * kJoinParts, 0, stream>>>(
            g, part, parts, a.cols, a.w1, a.b1, a.gate);
}

Step step_of(const ResidualArgs &a) {
    return Step{a.rows, a.cols, a.post, a.pre, a.eps, a.res_scale,
                a.w1, a.b1, a.gate, a.w2, a.b2, a.mask};
}

uint32_t capped(uint64_t n) {
    const uint64_t cap = max_blocks();
    return static_cast<uint32_t>(n < cap ? n : cap);
}

// How rows of these extents are held: by the extents alone, so that the workspace and the
// order of the sums do not depend on the device.
struct RowPlan {
    int groups;         // V, 0: rows are too long to stay on chip
    uint32_t waves;     // W
    uint32_t at_once;   // rows a workgroup takes at once
    uint32_t parts;     // workgroups that sum over rows
};

constexpr uint64_t kUnits = 256;   // compute units of the chip

uint32_t waves_of(uint64_t cols, int groups) {
    const uint64_t span = 512u * groups;
    return static_cast<uint32_t>((cols + span - 1) / span);
}

// How much a lane of the backward pass holds: 16-bit data with two sums, with four or beside an
// FP32 stream, or FP32 data and four sums beside an FP32 stream.
enum class Load { kLight, kMiddle, kHeavy };
template <int F, int R>
constexpr Load load_of(bool bias_sums) {
    if (F == 2 || (R == 2 && bias_sums)) return Load::kHeavy;
    return R == 2 || bias_sums ? Load::kMiddle : Load::kLight;
}

// The backward pass: rows of one wave up to 1024 columns, so that a workgroup joins eight rows'
// sums before it writes them (1023 x 768 FP16, four sums: 17.4 us; in parts of four rows 22.6
// where these took 19); up to 8192 columns rows of several waves, one group a lane (16 waves of
// 128 registers), or two for what is heavy (8 of 256: 16384 x 8192 FP32, four sums, 652 us
// against 948, two sums 630 against 728).  For the rest the two were alike when this was chosen;
// at 16384 x 8192 one group now takes 276 us and two 278 where it is light, 471 and 458 with an
// FP32 stream, 309 and 284 with four sums and a mask.  Up to 16384 columns two groups of 16
// waves for what is light (8192 x 12288 BF16: 340 us, walked over in memory 494; with a mask 465
// and 506; 8193 columns 362 and 416); the rest spills there (with an FP32 stream 818, walked over
// 669).  As many parts as fill the chip once, fewer where a wave would have less than four rows
// (each part is joined afterwards: 4000 x 512 FP16, four sums, 34 us in 500 parts, 24 in 256).
RowPlan backward_plan(uint64_t rows, uint64_t cols, Load load) {
    const uint64_t per = (rows + kUnits - 1) / kUnits;
    RowPlan p{0, 1, 1, static_cast<uint32_t>((rows + per - 1) / per)};
    if (cols > (load == Load::kLight ? 16384u : 8192u) || cols < 8) return p;
    p.groups =
        cols > 8192 || (cols > 512 && (cols <= 1024 || load == Load::kHeavy)) ? 2 : 1;
    p.waves = waves_of(cols, p.groups);
    if (p.waves == 1) p.at_once = static_cast<uint32_t>(rows < 8 ? rows : 8);
    const uint64_t resident = (p.groups == 1 ? 16 : 8) / (p.waves * p.at_once);
    uint64_t most = kUnits * (resident > 1 ? resident : 1);
    const uint64_t need = (rows + p.at_once - 1) / p.at_once;
    while (most > kUnits && need < 4 * most) most = most / 2 > kUnits ? most / 2 : kUnits;
    p.parts = static_cast<uint32_t>(need < most ? need : most);
    return p;
}

template <int F, int R>
hipError_t forward_as(const ResidualArgs &a, hipStream_t stream) {
    const Step s = step_of(a);
    auto *u = static_cast<elem_t<R> *>(a.u_out);
    auto *h = static_cast<elem_t<F> *>(a.h);
    const auto *r = static_cast<const elem_t<R> *>(a.r);
    const auto *f = static_cast<const elem_t<F> *>(a.f);
    if (a.cols > 16384 || a.cols < 8) {
        wide_forward_kernel<F, R><<<capped(a.rows), kWideThreads, 0, stream>>>(
            s, u, a.ldu, h, a.ldh, a.stats, r, a.ldr, f, a.ldf);
        return hipGetLastError();
    }
    const int groups = a.cols <= 8192 ? 1 : 2;
    const uint32_t waves = waves_of(a.cols, groups);
    const uint64_t per = (a.rows + kUnits - 1) / kUnits;
    const uint32_t at_once = waves == 1 ? static_cast<uint32_t>(per < 8 ? per : 8) : 1u;
    const uint32_t threads = 64 * waves * at_once;
    // workgroups that fill the chip once: 16 waves a compute unit (of 128 registers each)
    const uint64_t resident = 16 / (waves * at_once);
    const uint64_t need = (a.rows + at_once - 1) / at_once;
    const uint64_t most = kUnits * (resident > 1 ? resident : 1);
    const uint32_t grid = capped(need < most ? need : most);
    if (groups == 1)
        row_forward_kernel<F, R, 1><<<grid, threads, 0, stream>>>(
            s, waves, u, a.ldu, h, a.ldh, a.stats, r, a.ldr, f, a.ldf);
    else
        row_forward_kernel<F, R, 2><<<grid, threads, 0, stream>>>(
            s, waves, u, a.ldu, h, a.ldh, a.stats, r, a.ldr, f, a.ldf);
    return hipGetLastError();
}

template <int F, int R, bool BIAS>
hipError_t rows_backward(const Step &s, const RowPlan &plan, const Back<F, R> &p, float *part,
                         hipStream_t stream) {
    const uint32_t threads = 64 * plan.waves * plan.at_once, grid = capped(plan.parts);
    const size_t lds = plan.at_once > 1 ? sizeof(float) * plan.at_once * ((s.cols + 7) & ~7u) : 0;
    constexpr Load kLoad = load_of<F, R>(BIAS);
#define ZS_ROWS(V, WAVES)                                                                    \
    row_backward_kernel<F, R, V, WAVES, BIAS><<<grid, threads, lds, stream>>>(               \
        s, plan.waves, p, part, plan.parts)
    if (plan.groups == 1)
        ZS_ROWS(1, kLoad == Load::kHeavy ? 8 : 16);
    else if (kLoad != Load::kLight || plan.waves <= 8)
        ZS_ROWS(2, 8);
    else
        ZS_ROWS(2, kLoad == Load::kLight ? 16 : 8);
#undef ZS_ROWS
    return hipGetLastError();
}

template <int F, int R>
hipError_t backward_as(const ResidualArgs &a, hipStream_t stream) {
    const Step s = step_of(a);
    const Back<F, R> p{static_cast<const elem_t<F> *>(a.dh), static_cast<const elem_t<F> *>(a.f),
                       static_cast<const elem_t<R> *>(a.du), static_cast<const elem_t<R> *>(a.u),
                       static_cast<elem_t<F> *>(a.df), static_cast<elem_t<R> *>(a.dr),
                       a.lddh, a.ldf, a.lddu, a.ldu, a.lddf, a.lddr, a.stats};
    float *part = static_cast<float *>(a.workspace);
    bool bias_sums = a.db1 != nullptr || a.db2 != nullptr ||
                     (a.dgate != nullptr && a.b1 != nullptr);
    const RowPlan plan = backward_plan(a.rows, a.cols, load_of<F, R>(bias_sums));
    hipError_t e;
    if (plan.groups == 0) {
        bias_sums = true;
        float *means = part + static_cast<uint64_t>(plan.parts) * 4 * a.cols;
        wide_means_kernel<F, R><<<capped(a.rows), kWideThreads, 0, stream>>>(s, p, means);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
        const dim3 grid(capped((a.cols + kWideThreads * 8ull - 1) / (kWideThreads * 8ull)),
                        plan.parts);
        const uint64_t per = (a.rows + plan.parts - 1) / plan.parts;
        if (a.cols < 8)
            wide_backward_kernel<F, R, true><<<grid, kWideThreads, 0, stream>>>(s, p, means, part,
                                                                                per);
        else
            wide_backward_kernel<F, R, false><<<grid, kWideThreads, 0, stream>>>(s, p, means, part,
                                                                                 per);
        e = hipGetLastError();
    } else {
        e = bias_sums ? rows_backward<F, R, true>(s, plan, p, part, stream)
                      : rows_backward<F, R, false>(s, plan, p, part, stream);
    }
    if (e != hipSuccess) return e;
    const Grads g{a.dw1, a.db1, a.dgate, a.dw2, a.db2, a.first};
    if (!a.dw1 && !a.db1 && !a.dgate && !a.dw2 && !a.db2) return hipSuccess;
    const uint32_t blocks = capped((a.cols + kJoinCols - 1) / kJoinCols);
    if (a.grad32)
        join_grads<F, 2>(g, a, part, plan.parts, bias_sums, blocks, stream);
    else
        join_grads<F, F>(g, a, part, plan.parts, bias_sums, blocks, stream);
    return hipGetLastError();
}

}  // namespace

uint64_t residual_workspace(uint64_t rows, uint64_t cols) {
    uint64_t bytes = 0;
    for (const Load load : {Load::kLight, Load::kMiddle, Load::kHeavy}) {
        const RowPlan p = backward_plan(rows, cols, load);
        const uint64_t n = (p.parts * cols + (p.groups == 0 ? rows : 0)) * 16;
        bytes = n > bytes ? n : bytes;
    }
    return bytes;
}

hipError_t launch_residual_forward(const ResidualArgs &a, hipStream_t stream) {
    if (a.fmt == 0) return a.res32 ? forward_as<0, 2>(a, stream) : forward_as<0, 0>(a, stream);
    if (a.fmt == 1) return a.res32 ? forward_as<1, 2>(a, stream) : forward_as<1, 1>(a, stream);
    return forward_as<2, 2>(a, stream);
}

hipError_t launch_residual_backward(const ResidualArgs &a, hipStream_t stream) {
    if (a.fmt == 0) return a.res32 ? backward_as<0, 2>(a, stream) : backward_as<0, 0>(a, stream);
    if (a.fmt == 1) return a.res32 ? backward_as<1, 2>(a, stream) : backward_as<1, 1>(a, stream);
    return backward_as<2, 2>(a, stream);
}

}  // namespace zs
