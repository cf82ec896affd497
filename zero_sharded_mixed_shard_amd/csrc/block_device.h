// Device helpers of the kernels around a block's linear layers: the dropout mask, and groups
// of eight of a row of any length read without a branch.
#pragma once

#include "block_launch.h"
#include "grad_device.h"

namespace zs {
namespace {

// Four words of the Philox4x32 block of a counter, ten rounds.
__device__ __forceinline__ u32x4 philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3,
                                        uint32_t k0, uint32_t k1) {
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = static_cast<uint64_t>(c0) * 0xD2511F53u;
        const uint64_t b = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
        const uint32_t n0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ (k0 + r * 0x9E3779B9u);
        const uint32_t n2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ (k1 + r * 0xBB67AE85u);
        c0 = n0;
        c1 = static_cast<uint32_t>(b);
        c2 = n2;
        c3 = static_cast<uint32_t>(a);
    }
    return u32x4{c0, c1, c2, c3};
}

// Eight columns of a row from col on, read without a branch: where the row ends inside or
// before them, its last eight (the row has eight at least).
template <int F>
__device__ __forceinline__ Raw8<F> raw_group(const elem_t<F> *row, uint32_t col, uint32_t cols) {
    return load8<F>(row + (col + 8 <= cols ? col : cols - 8));
}

// Eight values of format F as raw bits.
template <int F>
__device__ __forceinline__ Raw8<F> narrow8(const float v[8]) {
    Raw8<F> r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (F == 2) {
            r.v[0][j] = bits(v[j]);
            r.v[1][j] = bits(v[4 + j]);
        } else {
            r.v[0][j] = pack2<F>(v[2 * j], v[2 * j + 1]);
        }
    }
    return r;
}

// What was read as the row's last eight, moved down to the n (1 to 7) that are the lane's,
// zeros above.
template <int F>
__device__ __forceinline__ void move_down(Raw8<F> &r, uint32_t n) {
    constexpr int kWords = F == 2 ? 8 : 4;
    uint32_t w[kWords];
#pragma unroll
    for (int j = 0; j < kWords; ++j) w[j] = r.v[j / 4][j % 4];
    const uint32_t by = 8 - n;   // elements
    if constexpr (F != 2) {
        if (by & 1u) {
#pragma unroll
            for (int j = 0; j < kWords; ++j)
                w[j] = w[j] >> 16 | (j + 1 < kWords ? w[j + 1] << 16 : 0u);
        }
    }
#pragma unroll
    for (int k = F == 2 ? 1 : 2; k < 8; k *= 2) {
        const int words = F == 2 ? k : k / 2;
        if (by & static_cast<uint32_t>(k)) {
#pragma unroll
            for (int j = 0; j < kWords; ++j) w[j] = j + words < kWords ? w[j + words] : 0u;
        }
    }
#pragma unroll
    for (int j = 0; j < kWords; ++j) r.v[j / 4][j % 4] = w[j];
}

// A call's key and offset, the same in every lane.
struct MaskKey {
    uint32_t k0, k1, o0, o1, threshold;
    __device__ __forceinline__ explicit MaskKey(const Mask &m)
        : k0(static_cast<uint32_t>(m.seed)), k1(static_cast<uint32_t>(m.seed >> 32)),
          threshold(m.threshold) {
        const uint64_t o = m.offset + (m.d_offset != nullptr ? *m.d_offset : 0ull);
        o0 = static_cast<uint32_t>(o);
        o1 = static_cast<uint32_t>(o >> 32);
    }
    // Bit j: column 8 group + j of the row stays.
    __device__ __forceinline__ uint32_t keep8(uint32_t row, uint32_t group) const {
        const u32x4 w = philox(group, row, o0, o1, k0, k1);
        uint32_t keep = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            keep |= (w[j] & 0xffffu) >= threshold ? 1u << (2 * j) : 0u;
            keep |= (w[j] >> 16) >= threshold ? 2u << (2 * j) : 0u;
        }
        return keep;
    }
};

}  // namespace
}  // namespace zs
