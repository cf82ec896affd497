// gfx950 kernels of the clipped policy loss with a KL term.
//
// A row's softmax needs its maximum and sum before any gradient can be written,
// so a plain pass structure reads the logits twice.  Here one block takes a row
// and keeps its logits in registers (raw 16-B vectors, up to kMaxVec a lane:
// 196,608 16-bit logits at 1024 lanes): every logit is read once and every
// gradient written once, which is the floor of 2 + 2 bytes an element.  Longer
// rows (and the loss without gradients) take a running maximum and sum over one
// pass and, for the gradients, read the row again.
//
// Rows start anywhere: vectors are taken at the 16-B boundaries of the row, the
// first and last partial ones element by element (outside the row a vector
// holds -inf, which adds nothing).  dlogits may be logits: all of a row is in
// registers before any of it is written, and the two-pass form writes an
// element after its last read.
#include "grad_device.h"

#pragma clang fp contract(off)

namespace zs {
namespace {

constexpr float kInf = __builtin_inff();

template <int F> constexpr int kPer = F == 2 ? 4 : 8;   // logits of a 16-B vector

// ex = e^(z - m): FP32 logits take the accurate form, 16-bit ones the hardware's
// 2^x (gradients are rounded to 16 bits, and a term's share of the sum falls
// with the same factor as its relative error grows).
template <int F>
__device__ __forceinline__ float exp_from(float z, float m) {
    if constexpr (F == 2)
        return expf(z - m);
    else
        return exp_fast(z - m);
}

template <int F>
__device__ __forceinline__ void widen_vec(const u32x4 &w, float out[kPer<F>]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (F == 2)
            out[j] = from_bits(w[j]);
        else
            unpack2<F>(w[j], out + 2 * j);
    }
}

// Hides that the vectors' values are those already widened once, so that the
// raw 16-bit form stays in registers rather than its FP32 form (twice as many).
__device__ __forceinline__ void keep_raw(u32x4 &w) { asm volatile("" : "+v"(w)); }

// -inf in every element of a vector
template <int F>
__device__ __forceinline__ u32x4 neg_inf_vec() {
    const uint32_t w = F == 2 ? 0xff800000u : F == 1 ? 0xff80ff80u : 0xfc00fc00u;
    return u32x4{w, w, w, w};
}

// Vector j of a row: elements j*K - shift .. +K-1 of the row, shift the elements
// between the 16-B boundary below the row's start and that start.
template <int F>
__device__ __forceinline__ u32x4 row_vec(const elem_t<F> *row, uint32_t shift, uint32_t vocab,
                                         uint32_t j) {
    constexpr int K = kPer<F>;
    const int64_t e0 = static_cast<int64_t>(j) * K - shift;
    if (e0 >= 0 && e0 + K <= vocab)
        return __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(row + e0));
    u32x4 r = neg_inf_vec<F>();
#pragma unroll
    for (int i = 0; i < K; ++i) {
        const int64_t e = e0 + i;
        if (e >= 0 && e < vocab) {
            if constexpr (F == 2) {
                r[i] = bits(row[e]);
            } else {
                const uint32_t h = row[e];
                const uint32_t old = r[i / 2];
                r[i / 2] = i % 2 ? (old & 0xffffu) | (h << 16) : (old & 0xffff0000u) | h;
            }
        }
    }
    return r;
}

template <int F>
__device__ __forceinline__ void store_row_vec(elem_t<F> *row, uint32_t shift, uint32_t vocab,
                                              uint32_t j, const float v[kPer<F>]) {
    constexpr int K = kPer<F>;
    const int64_t e0 = static_cast<int64_t>(j) * K - shift;
    if (e0 >= 0 && e0 + K <= vocab) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = F == 2 ? bits(v[i]) : pack2<F == 2 ? 0 : F>(v[2 * i % K], v[(2 * i + 1) % K]);
        __builtin_nontemporal_store(w, reinterpret_cast<u32x4_any *>(row + e0));
        return;
    }
#pragma unroll
    for (int i = 0; i < K; ++i) {
        const int64_t e = e0 + i;
        if (e >= 0 && e < vocab) row[e] = from_f32<F>(v[i]);
    }
}

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor(x, o));
    return x;
}
__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) x = x + __shfl_xor(x, o);
    return x;
}

// The same over the block; red: one slot a wave, free for reuse on return.
template <int T, bool MAX>
__device__ __forceinline__ float block_reduce(float x, float *red) {
    x = MAX ? wave_max(x) : wave_sum(x);
    if constexpr (T == 64) return x;
    if ((threadIdx.x & 63u) == 0) red[threadIdx.x >> 6] = x;
    __syncthreads();
    float r = red[0];
#pragma unroll
    for (int w = 1; w < T / 64; ++w) r = MAX ? fmaxf(r, red[w]) : r + red[w];
    __syncthreads();
    return r;
}

// What a row's gradient needs, the same in every lane.
struct RowGrad {
    float m;        // the row's largest logit
    float scale;    // -S w g / sum
    float hit;      // S w g, added at the target
};

// The row's loss from its maximum and sum; lane 0 writes token_loss and logp.
__device__ __forceinline__ RowGrad finish_row(const PolicyArgs &a, uint64_t t, float m, float sum,
                                              float z_target, float w) {
    const float logp = z_target - m - logf(sum);
    const float A = a.advantage[t];
    const float r = a.old_logp != nullptr ? expf(logp - a.old_logp[t]) : 1.0f;
    const float lo = 1.0f - a.clip_low, hi = 1.0f + a.clip_high;
    float rc = r < lo ? lo : r;
    rc = rc > hi ? hi : rc;
    const float p0 = -(r * A), p1 = -(rc * A);
    float L = p0 >= p1 || p0 != p0 ? p0 : p1;      // the larger; NaN stays
    const bool cut = (A > 0.0f && r > hi) || (A < 0.0f && r < lo);
    float g = cut ? 0.0f : p0;
    if (a.ref_logp != nullptr && a.kl_coef != 0.0f) {
        // e^d - d - 1 without cancellation near d = 0: expm1(d) - d
        const float d = a.ref_logp[t] - logp, em = expm1f(d);
        L = L + a.kl_coef * (em - d);
        g = g - a.kl_coef * em;
    }
    if (threadIdx.x == 0) {
        a.token_loss[t] = L;
        a.logp[t] = logp;
    }
    const float S = a.loss_scale_dev != nullptr ? *a.loss_scale_dev : a.loss_scale;
    const float c = S * (w * g);
    return RowGrad{m, -c / sum, c};
}

// The target's logit, NaN for a target outside the vocabulary (at: its index,
// ~0 then).
template <int F>
__device__ __forceinline__ float target_logit(const PolicyArgs &a, const elem_t<F> *row,
                                              uint64_t t, uint32_t *at) {
    const int64_t v = a.targets64 ? static_cast<const int64_t *>(a.targets)[t]
                                  : static_cast<const int32_t *>(a.targets)[t];
    const bool in = v >= 0 && static_cast<uint64_t>(v) < a.vocab;
    *at = in ? static_cast<uint32_t>(v) : 0xffffffffu;
    return in ? to_f32<F>(row[v]) : __builtin_nanf("");
}

template <int F>
__host__ __device__ __forceinline__ uint32_t shift_of(const elem_t<F> *row) {
    return static_cast<uint32_t>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(elem_t<F>));
}

// Row t's gradient is zero everywhere.
template <int F, int T>
__device__ __forceinline__ void skip_row(const PolicyArgs &a, uint64_t t) {
    if (threadIdx.x == 0) {
        a.token_loss[t] = 0.0f;
        a.logp[t] = 0.0f;
    }
    if (a.dlogits == nullptr) return;
    auto *d = static_cast<elem_t<F> *>(a.dlogits) + t * a.ldd;
    const uint32_t V = static_cast<uint32_t>(a.vocab), shift = shift_of<F>(d);
    const uint32_t n_vec = static_cast<uint32_t>((static_cast<uint64_t>(shift) + V + kPer<F> - 1) /
                                                 kPer<F>);
    const float zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (uint32_t j = threadIdx.x; j < n_vec; j += T) store_row_vec<F>(d, shift, V, j, zero);
}

// Gradients of vector j from its logits.
template <int F>
__device__ __forceinline__ void grad_vec(elem_t<F> *d, uint32_t shift, uint32_t V, uint32_t j,
                                         const u32x4 &w, const RowGrad &g, uint32_t target) {
    constexpr int K = kPer<F>;
    float z[K];
    widen_vec<F>(w, z);
    const int64_t e0 = static_cast<int64_t>(j) * K - shift;
#pragma unroll
    for (int i = 0; i < K; ++i) {
        const float p = exp_from<F>(z[i], g.m) * g.scale;
        z[i] = e0 + i == static_cast<int64_t>(target) ? p + g.hit : p;
    }
    store_row_vec<F>(d, shift, V, j, z);
}

// One row a block of T lanes, its logits in registers: N vectors a lane.
template <int F, int T, int N>
__global__ __launch_bounds__(T) void policy_row_kernel(PolicyArgs a) {
    constexpr int K = kPer<F>;
    __shared__ float red[T / 64];
    const uint32_t V = static_cast<uint32_t>(a.vocab);
    for (uint64_t t = blockIdx.x; t < a.rows; t += gridDim.x) {
        const float weight = a.weight[t];
        if (weight == 0.0f) {
            skip_row<F, T>(a, t);
            continue;
        }
        const auto *row = static_cast<const elem_t<F> *>(a.logits) + t * a.ld;
        const uint32_t shift = shift_of<F>(row);
        const uint32_t n_vec =
            static_cast<uint32_t>((static_cast<uint64_t>(shift) + V + K - 1) / K);
        u32x4 x[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t j = i * T + threadIdx.x;
            x[i] = j < n_vec ? row_vec<F>(row, shift, V, j) : neg_inf_vec<F>();
        }
        uint32_t target;
        const float zt = target_logit<F>(a, row, t, &target);
        float m = -kInf;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float z[K];
            widen_vec<F>(x[i], z);
#pragma unroll
            for (int k = 0; k < K; ++k) m = fmaxf(m, z[k]);
        }
        m = block_reduce<T, true>(m, red);
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float z[K];
            keep_raw(x[i]);
            widen_vec<F>(x[i], z);
#pragma unroll
            for (int k = 0; k < K; ++k) s = s + exp_from<F>(z[k], m);
        }
        s = block_reduce<T, false>(s, red);
        const RowGrad g = finish_row(a, t, m, s, zt, weight);
        auto *d = static_cast<elem_t<F> *>(a.dlogits) + t * a.ldd;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t j = i * T + threadIdx.x;
            keep_raw(x[i]);
            if (j < n_vec) grad_vec<F>(d, shift, V, j, x[i], g, target);
        }
    }
}

// One row a block of T lanes in one pass for the loss (running maximum and sum a
// lane) and, with dlogits, a second for the gradients.
template <int F, int T>
__global__ __launch_bounds__(T) void policy_long_kernel(PolicyArgs a) {
    constexpr int K = kPer<F>;
    __shared__ float red[T / 64];
    const uint32_t V = static_cast<uint32_t>(a.vocab);
    for (uint64_t t = blockIdx.x; t < a.rows; t += gridDim.x) {
        const float weight = a.weight[t];
        if (weight == 0.0f) {
            skip_row<F, T>(a, t);
            continue;
        }
        const auto *row = static_cast<const elem_t<F> *>(a.logits) + t * a.ld;
        const uint32_t shift = shift_of<F>(row);
        const uint32_t n_vec =
            static_cast<uint32_t>((static_cast<uint64_t>(shift) + V + K - 1) / K);
        uint32_t target;
        const float zt = target_logit<F>(a, row, t, &target);
        float m = -kInf, s = 0.0f;
        for (uint32_t j = threadIdx.x; j < n_vec; j += T) {
            float z[K];
            widen_vec<F>(row_vec<F>(row, shift, V, j), z);
            float vm = z[0];
#pragma unroll
            for (int k = 1; k < K; ++k) vm = fmaxf(vm, z[k]);
            if (vm > m) {            // the sum so far in units of the new maximum
                s = m == -kInf ? s : s * exp_from<F>(m, vm);
                m = vm;
            }
            // nothing but -inf so far adds nothing; a NaN still reaches the sum
            const float base = m == -kInf ? 0.0f : m;
#pragma unroll
            for (int k = 0; k < K; ++k) s = s + exp_from<F>(z[k], base);
        }
        const float rm = block_reduce<T, true>(m, red);
        s = block_reduce<T, false>(m == -kInf ? s : s * exp_from<F>(m, rm), red);
        const RowGrad g = finish_row(a, t, rm, s, zt, weight);
        if (a.dlogits == nullptr) continue;
        auto *d = static_cast<elem_t<F> *>(a.dlogits) + t * a.ldd;
        for (uint32_t j = threadIdx.x; j < n_vec; j += T)
            grad_vec<F>(d, shift, V, j, row_vec<F>(row, shift, V, j), g, target);
    }
}

// loss = sum of weight * token_loss in FP64: each lane its stride of rows, then
// a tree over the lanes.  Rows of weight zero add nothing.
constexpr int kSumThreads = 1024;
__global__ __launch_bounds__(kSumThreads) void policy_sum_kernel(
    float *__restrict__ loss, const float *__restrict__ token_loss,
    const float *__restrict__ weight, uint64_t rows) {
    __shared__ double red[kSumThreads];
    double s = 0.0;
    for (uint64_t t = threadIdx.x; t < rows; t += kSumThreads) {
        const float w = weight[t];
        if (w != 0.0f) s += static_cast<double>(w) * static_cast<double>(token_loss[t]);
    }
    red[threadIdx.x] = s;
    for (int o = kSumThreads / 2; o > 0; o >>= 1) {
        __syncthreads();
        if (static_cast<int>(threadIdx.x) < o) red[threadIdx.x] += red[threadIdx.x + o];
    }
    if (threadIdx.x == 0) *loss = static_cast<float>(red[0]);
}

constexpr uint64_t kMaxGrid = 1ull << 21;   // 1024-lane blocks: below 2^32 lanes a launch
constexpr int kMaxVec = 24;   // vectors a lane of a 1024-lane block holds

template <int F>
hipError_t policy_rows(const PolicyArgs &a, hipStream_t stream) {
    uint64_t cap = max_blocks();
    if (cap > kMaxGrid) cap = kMaxGrid;
    const uint32_t grid = static_cast<uint32_t>(a.rows < cap ? a.rows : cap);
    // vectors of a row: rows share the first one's phase when their stride is whole
    // vectors, and may have any otherwise
    constexpr uint64_t K = kPer<F>;
    const uint64_t shift = a.ld % K == 0 ? shift_of<F>(static_cast<const elem_t<F> *>(a.logits))
                                         : K - 1;
    const uint64_t n_vec = (shift + a.vocab + K - 1) / K;
#define ZS_ROW(T, N)                                                                 \
    if (n_vec <= static_cast<uint64_t>(T) * (N)) {                                   \
        policy_row_kernel<F, T, N><<<grid, T, 0, stream>>>(a);                       \
        return hipGetLastError();                                                    \
    }
    if (a.dlogits != nullptr) {
        ZS_ROW(64, 2)
        ZS_ROW(64, 4)
        ZS_ROW(256, 4)
        ZS_ROW(256, 8)
        ZS_ROW(1024, 4)
        ZS_ROW(1024, 8)
        ZS_ROW(1024, 16)
        ZS_ROW(1024, kMaxVec)
    }
#undef ZS_ROW
    if (n_vec <= 64 * 4)
        policy_long_kernel<F, 64><<<grid, 64, 0, stream>>>(a);
    else
        policy_long_kernel<F, 1024><<<grid, 1024, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_policy_loss(const PolicyArgs &a, int fmt, hipStream_t stream) {
    if (a.rows > 0) {
        const hipError_t e = fmt == 0   ? policy_rows<0>(a, stream)
                             : fmt == 1 ? policy_rows<1>(a, stream)
                                        : policy_rows<2>(a, stream);
        if (e != hipSuccess) return e;
    }
    policy_sum_kernel<<<1, kSumThreads, 0, stream>>>(a.loss, a.token_loss, a.weight, a.rows);
    return hipGetLastError();
}

}  // namespace zs
