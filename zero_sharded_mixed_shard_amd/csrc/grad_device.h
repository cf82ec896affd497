// Device helpers of the gradient operators' kernels: formats, groups of eight
// elements at any element alignment, e4m3 codes, wave reductions.
//
// Format codes: 0 FP16, 1 BF16, 2 FP32.  Global memory takes unaligned vector
// accesses on gfx950, so one 16-B access serves a matrix that starts anywhere
// in a flat buffer; aligned addresses keep their full rate.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "grad_launch.h"

namespace zs {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// the same at any address: how the groups below are read and written
typedef u32x2 u32x2_any __attribute__((aligned(1)));
typedef u32x4 u32x4_any __attribute__((aligned(1)));

// Global memory by type: a pointer that went through an empty asm statement (to keep it
// in scalar registers) is not known to be global any more, and would be read by flat
// instructions.
#define GLOBAL_AS __attribute__((address_space(1)))

template <int F> struct Elem { using T = uint16_t; };
template <> struct Elem<2> { using T = float; };
template <int F> using elem_t = typename Elem<F>::T;

template <int F>
__device__ __forceinline__ float to_f32(elem_t<F> x) {
    if constexpr (F == 0)
        return static_cast<float>(__builtin_bit_cast(_Float16, x));
    else if constexpr (F == 1)
        return __builtin_bit_cast(float, static_cast<uint32_t>(x) << 16);
    else
        return x;
}

template <int F>
__device__ __forceinline__ elem_t<F> from_f32(float f) {
    if constexpr (F == 0)
        return __builtin_bit_cast(uint16_t, static_cast<_Float16>(f));  // RNE
    else if constexpr (F == 1)
        return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));    // RNE
    else
        return f;
}

__device__ __forceinline__ uint32_t bits(float f) { return __builtin_bit_cast(uint32_t, f); }
__device__ __forceinline__ float from_bits(uint32_t b) { return __builtin_bit_cast(float, b); }

template <int F>
__device__ __forceinline__ void unpack2(uint32_t w, float *out) {
    if constexpr (F == 1) {
        out[0] = from_bits(w << 16);
        out[1] = from_bits(w & 0xffff0000u);
    } else {
        out[0] = to_f32<F>(static_cast<uint16_t>(w & 0xffffu));
        out[1] = to_f32<F>(static_cast<uint16_t>(w >> 16));
    }
}

template <int F>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    return static_cast<uint32_t>(from_f32<F>(a)) | (static_cast<uint32_t>(from_f32<F>(b)) << 16);
}

// Eight elements as raw bits (16 or 32 bytes).
template <int F> struct Raw8 {
    u32x4 v[F == 2 ? 2 : 1];
};

template <int F>
__device__ __forceinline__ Raw8<F> load8(const elem_t<F> *p) {
    Raw8<F> r;
    const u32x4_any *s = reinterpret_cast<const u32x4_any *>(p);
    r.v[0] = __builtin_nontemporal_load(s);
    if constexpr (F == 2) r.v[1] = __builtin_nontemporal_load(s + 1);
    return r;
}

// The same for data that other lanes read too: kept in the caches.
template <int F>
__device__ __forceinline__ Raw8<F> load8_cached(const elem_t<F> *p) {
    Raw8<F> r;
    const u32x4_any *s = reinterpret_cast<const u32x4_any *>(p);
    r.v[0] = s[0];
    if constexpr (F == 2) r.v[1] = s[1];
    return r;
}

template <int F>
__device__ __forceinline__ void widen8(const Raw8<F> &r, float out[8]) {
    if constexpr (F == 2) {
#pragma unroll
        for (int j = 0; j < 8; ++j) out[j] = from_bits(r.v[j / 4][j % 4]);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) unpack2<F>(r.v[0][j], out + 2 * j);
    }
}

template <int F>
__device__ __forceinline__ void store8(elem_t<F> *p, const float v[8]) {
    u32x4_any *d = reinterpret_cast<u32x4_any *>(p);
    if constexpr (F == 2) {
        d[0] = u32x4{bits(v[0]), bits(v[1]), bits(v[2]), bits(v[3])};
        d[1] = u32x4{bits(v[4]), bits(v[5]), bits(v[6]), bits(v[7])};
    } else {
        __builtin_nontemporal_store(u32x4{pack2<F>(v[0], v[1]), pack2<F>(v[2], v[3]),
                                          pack2<F>(v[4], v[5]), pack2<F>(v[6], v[7])}, d);
    }
}

// n of eight elements (n < 8): the rest reads as zero and is not written.
template <int F>
__device__ __forceinline__ void load_some(const elem_t<F> *p, uint32_t n, float out[8]) {
#pragma unroll
    for (uint32_t j = 0; j < 8; ++j) out[j] = j < n ? to_f32<F>(p[j]) : 0.0f;
}
template <int F>
__device__ __forceinline__ void store_some(elem_t<F> *p, uint32_t n, const float v[8]) {
#pragma unroll
    for (uint32_t j = 0; j < 8; ++j)
        if (j < n) p[j] = from_f32<F>(v[j]);
}

// a * b rounded to FP32: hides the product from the mixed-precision multiply that
// would round it straight to FP16, so that 16-bit and FP32 results come from the
// same FP32 value.
__device__ __forceinline__ float product32(float a, float b) {
    float p = a * b;
    asm volatile("" : "+v"(p));
    return p;
}

__device__ __forceinline__ uint64_t div_by(uint64_t n, const FastDiv &f) {
    return __umul64hi(n << 2, f.m) >> f.s;
}

// e^x by the hardware's 2^x: the product x log2 e rounds once, so the relative
// error is below 2^-22 + |x| 2^-24.  Used where the result is rounded to 16 bits
// or its terms matter only while x is small.
__device__ __forceinline__ float exp_fast(float x) {
    return __builtin_amdgcn_exp2f(x * 1.44269504088896340736f);
}

}  // namespace
}  // namespace zs
