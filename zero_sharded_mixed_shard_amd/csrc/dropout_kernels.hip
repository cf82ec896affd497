// gfx950 kernel of dropout with a mask that is never stored.
//
// The mask of eight neighbouring columns is one Philox4x32 block (ten rounds; Salmon,
// Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011): 16 bits an
// element, so that an element costs two and a half of the block's twenty wide products, which
// run beside the memory's traffic.  16 bits put the probability on a grid of 2^-16, which the
// factor of what stays goes by, so the mean is kept.
//
// Bound by HBM: BF16 16384 x 8192 89 us (6.1 TB/s), FP32 198 (5.4); FP16 61 x 769 the launch.
#include "block_device.h"

#pragma clang fp contract(off)

namespace zs {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 2;   // groups of eight elements a lane keeps in flight

// y may be x: every lane reads its elements before it writes them.
template <int F>
__global__ __launch_bounds__(kThreads) void dropout_kernel(elem_t<F> *y, uint64_t ldy,
                                                          const elem_t<F> *x, uint64_t ldx,
                                                          uint64_t cols, FastDiv per_row,
                                                          uint64_t n_groups, Mask mask) {
    constexpr uint64_t kTile = kThreads * kUnroll;
    const MaskKey key(mask);
    for (uint64_t t0 = blockIdx.x * kTile; t0 < n_groups; t0 += gridDim.x * kTile) {
        float v[kUnroll][8];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const uint64_t g = t0 + u * kThreads + threadIdx.x;
            if (g < n_groups) {
                const uint64_t row = div_by(g, per_row), col = (g - row * per_row.d) * 8;
                const elem_t<F> *s = x + row * ldx + col;
                if (col + 8 <= cols)
                    widen8<F>(load8<F>(s), v[u]);
                else
                    load_some<F>(s, static_cast<uint32_t>(cols - col), v[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const uint64_t g = t0 + u * kThreads + threadIdx.x;
            if (g < n_groups) {
                const uint64_t row = div_by(g, per_row), group = g - row * per_row.d;
                const uint64_t col = group * 8;
                const uint32_t keep = key.keep8(static_cast<uint32_t>(row),
                                                static_cast<uint32_t>(group));
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[u][j] = (keep >> j) & 1u ? product32(v[u][j], mask.factor) : 0.0f;
                elem_t<F> *d = y + row * ldy + col;
                if (col + 8 <= cols)
                    store8<F>(d, v[u]);
                else
                    store_some<F>(d, static_cast<uint32_t>(cols - col), v[u]);
            }
        }
    }
}

template <int F>
hipError_t dropout_as(void *y, uint64_t ldy, const void *x, uint64_t ldx, uint64_t rows,
                      uint64_t cols, const Mask &mask, hipStream_t stream) {
    const uint64_t per_row = (cols + 7) / 8, groups = rows * per_row;
    const uint64_t tile = static_cast<uint64_t>(kThreads) * kUnroll;
    const uint64_t blocks = (groups + tile - 1) / tile, cap = max_blocks();
    dropout_kernel<F><<<static_cast<uint32_t>(blocks < cap ? blocks : cap), kThreads, 0, stream>>>(
        static_cast<elem_t<F> *>(y), ldy, static_cast<const elem_t<F> *>(x), ldx, cols,
        fast_div(static_cast<uint32_t>(per_row)), groups, mask);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_dropout(void *y, uint64_t ldy, const void *x, uint64_t ldx, int fmt,
                          uint64_t rows, uint64_t cols, const Mask &mask, hipStream_t stream) {
    if (fmt == 0) return dropout_as<0>(y, ldy, x, ldx, rows, cols, mask, stream);
    if (fmt == 1) return dropout_as<1>(y, ldy, x, ldx, rows, cols, mask, stream);
    return dropout_as<2>(y, ldy, x, ldx, rows, cols, mask, stream);
}

}  // namespace zs
