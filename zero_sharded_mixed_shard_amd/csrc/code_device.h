// Device helpers of the kernels that write and read 8-bit codes with a power of two
// for each block: rounding to codes, reading them, groups of eight at any address.
#pragma once

#include "grad_device.h"

#pragma clang fp contract(off)

namespace zs {
namespace {

// Largest magnitude a checkpoint written from format F stands for.
template <int F> constexpr float kTop = F == 0 ? 61440.0f : 0x1.ep127f;

// Exponent byte of a block whose largest finite magnitude has FP32 bits m: that of the
// smallest 2^k with amax <= 448 * 2^k, k >= -124.
__device__ __forceinline__ uint32_t block_exponent(uint32_t m) {
    const int b0 = static_cast<int>(m >> 23) - 8 + ((m & 0x7fffffu) > 0x600000u ? 1 : 0);
    return static_cast<uint32_t>(b0 < 3 ? 3 : b0);
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

}  // namespace
}  // namespace zs
