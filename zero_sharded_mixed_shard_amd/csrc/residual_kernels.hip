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
    const float v = ss / cols;
    *mean = m * 0x1p80f;
    *rho = 1.0f / sqrtf(v < 0x1p-120f ? 0x1p-120f : v) * k;   // eps k^2 is far below v; a NaN stays
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
__device__ __forceinline__ void pre8(const Step &s, const Back<F, R> &p, uint64_t row,
                                     uint32_t col, uint32_t n, const RowMeans &m, float dh[8],
                                     float uhat[8]) {
    if (p.dh == nullptr) {
#pragma unroll
        for (int j = 0; j < 8; ++j) dh[j] = uhat[j] = 0.0f;
        return;
    }
    load_row<F>(p.dh + row * p.lddh, col, n, dh);
    load_row<R>(p.u + row * p.ldu, col, n, uhat);
#pragma unroll
    for (int j = 0; j < 8; ++j) uhat[j] = (uhat[j] - m.mean2) * m.rho2;
    (void)s;
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
                pre8(s, p, row, col, n, m, dh, uhat);
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
                pre8(s, p, row, col, n, m, dh, uhat);
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

// df, dr and the four column sums over the rows of part blockIdx.y, to
// part[blockIdx.y][4][cols].  A lane owns eight columns.  df may be dh, and dr du: a lane
// reads its elements before it writes them.
template <int F, int R>
__global__ __launch_bounds__(kWideThreads) void wide_backward_kernel(
    Step s, Back<F, R> p, const float *__restrict__ means, float *__restrict__ part,
    uint64_t rows_per_part) {
    const MaskKey key(s.mask);
    const uint64_t first = blockIdx.y * rows_per_part;
    const uint64_t last = first + rows_per_part < s.rows ? first + rows_per_part : s.rows;
    constexpr uint64_t kStride = kWideThreads * 8;
    for (uint64_t c = blockIdx.x * kStride + threadIdx.x * 8u; c < s.cols;
         c += gridDim.x * kStride) {
        const uint32_t col = static_cast<uint32_t>(c);
        const uint32_t n = s.cols - col < 8 ? s.cols - col : 8u;
        float w1[8], w2[8], gate[8], sums[4][8] = {};
        load_param<F>(s.w1, col, n, 1.0f, w1);
        load_param<F>(s.w2, col, n, 1.0f, w2);
        load_param<F>(s.gate, col, n, 1.0f, gate);
        for (uint64_t row = first; row < last; ++row) {
            const float *st = p.stats + row * 4, *mn = means + row * 4;
            const RowMeans m{st[0], st[1], st[2], st[3], mn[0], mn[1], mn[2], mn[3]};
            float dh[8], uhat[8], G[8], fhat[8], out[8];
            pre8(s, p, row, col, n, m, dh, uhat);
            stream8(p, row, col, n, m, dh, uhat, w2, G);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                sums[0][j] = sums[0][j] + dh[j] * uhat[j];
                sums[1][j] = sums[1][j] + dh[j];
                out[j] = product32(s.res_scale, G[j]);
            }
            if (p.f != nullptr) {
                float df[8];
                post8(s, key, p, row, col, n, m, G, fhat);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    sums[2][j] = sums[2][j] + G[j] * fhat[j];
                    sums[3][j] = sums[3][j] + G[j];
                    const float x = gate[j] * G[j];
                    df[j] = s.post == ZERO_NORM_NONE
                                ? product32(gate[j], G[j])
                                : product32(m.rho1, (w1[j] * x - m.g1) - fhat[j] * m.zg1);
                }
                store_row<F>(p.df + row * p.lddf, col, n, df);
            }
            store_row<R>(p.dr + row * p.lddr, col, n, out);
        }
        float *d = part + blockIdx.y * 4ull * s.cols + col;
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (uint32_t j = 0; j < 8; ++j)
                if (j < n) d[static_cast<uint64_t>(k) * s.cols + j] = sums[k][j];
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

// The parts' four sums of a column, added in the parts' order by kJoinParts lanes (each its
// share), those joined in order, and the gradients made from them.  G: the gradients' format.
constexpr uint32_t kJoinCols = 16, kJoinParts = 16;
template <int F, int G>
__global__ __launch_bounds__(kJoinCols *kJoinParts) void join_grads_kernel(
    Grads g, const float *__restrict__ part, uint32_t parts, uint32_t cols, const void *w1,
    const void *b1, const void *gate) {
    __shared__ float slots[4][kJoinParts][kJoinCols];
    const uint32_t lane_col = threadIdx.x % kJoinCols, share = threadIdx.x / kJoinCols;
    const uint32_t per = (parts + kJoinParts - 1) / kJoinParts;
    for (uint64_t c0 = static_cast<uint64_t>(blockIdx.x) * kJoinCols; c0 < cols;
         c0 += static_cast<uint64_t>(gridDim.x) * kJoinCols) {
        const uint64_t col = c0 + lane_col;
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (col < cols) {
            const uint32_t from = share * per, to = from + per < parts ? from + per : parts;
            for (uint32_t k = from; k < to; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sum[i] = sum[i] + part[(static_cast<uint64_t>(k) * 4 + i) * cols + col];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) slots[i][share][lane_col] = sum[i];
        __syncthreads();
        if (share == 0 && col < cols) {
            for (uint32_t k = 1; k < kJoinParts; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) sum[i] = sum[i] + slots[i][k][lane_col];
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

Step step_of(const ResidualArgs &a) {
    return Step{a.rows, a.cols, a.post, a.pre, a.eps, a.res_scale,
                a.w1, a.b1, a.gate, a.w2, a.b2, a.mask};
}

uint32_t capped(uint64_t n) {
    const uint64_t cap = max_blocks();
    return static_cast<uint32_t>(n < cap ? n : cap);
}

// Parts of the rows in the column sums: by the extents alone.
constexpr uint64_t kParts = 256;
uint64_t rows_per_part(uint64_t rows) { return (rows + kParts - 1) / kParts; }
uint64_t parts_of(uint64_t rows) {
    const uint64_t per = rows_per_part(rows);
    return (rows + per - 1) / per;
}

template <int F, int R>
hipError_t forward_as(const ResidualArgs &a, hipStream_t stream) {
    wide_forward_kernel<F, R><<<capped(a.rows), kWideThreads, 0, stream>>>(
        step_of(a), static_cast<elem_t<R> *>(a.u_out), a.ldu, static_cast<elem_t<F> *>(a.h), a.ldh,
        a.stats, static_cast<const elem_t<R> *>(a.r), a.ldr, static_cast<const elem_t<F> *>(a.f),
        a.ldf);
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
    const uint64_t parts = parts_of(a.rows), per = rows_per_part(a.rows);
    float *means = part + parts * 4 * a.cols;
    wide_means_kernel<F, R><<<capped(a.rows), kWideThreads, 0, stream>>>(s, p, means);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const dim3 grid(capped((a.cols + kWideThreads * 8ull - 1) / (kWideThreads * 8ull)),
                    static_cast<uint32_t>(parts));
    wide_backward_kernel<F, R><<<grid, kWideThreads, 0, stream>>>(s, p, means, part, per);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    const Grads g{a.dw1, a.db1, a.dgate, a.dw2, a.db2, a.first};
    if (!a.dw1 && !a.db1 && !a.dgate && !a.dw2 && !a.db2) return hipSuccess;
    const uint32_t blocks = capped((a.cols + kJoinCols - 1) / kJoinCols);
    if (a.grad32)
        join_grads_kernel<F, 2><<<blocks, kJoinCols * kJoinParts, 0, stream>>>(
            g, part, static_cast<uint32_t>(parts), a.cols, a.w1, a.b1, a.gate);
    else
        join_grads_kernel<F, F><<<blocks, kJoinCols * kJoinParts, 0, stream>>>(
            g, part, static_cast<uint32_t>(parts), a.cols, a.w1, a.b1, a.gate);
    return hipGetLastError();
}

}  // namespace

uint64_t residual_workspace(uint64_t rows, uint64_t cols) {
    return (parts_of(rows) * cols + rows) * 16;
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
