// gfx950 kernels of the clipped policy loss with a KL term.
//
// A row's softmax needs its maximum and sum before any gradient can be written,
// so a plain pass structure reads the logits twice.  Here one block takes a row
// and holds its logits on chip (raw 16-B vectors in registers, for the longest
// rows part of them in LDS): every logit is read once and every gradient written
// once, which is the floor of 2 + 2 bytes an element.  Block sizes are such that
// two or more rows share a compute unit, so that one row's loads and stores run
// under another's arithmetic.  Rows too long for that (and the loss without
// gradients) take a running maximum and sum over one pass and, for the gradients,
// read the row again.
//
// The arithmetic matters next to the memory: an element takes a packed maximum,
// two fused multiply-adds and two 2^x.  e^(z - m) is taken as 2^(z log2 e - c) with
// c = m log2 e rounded: that rounding scales every term and the sum alike, and the
// log-probability is formed with the same c, so it cancels.  A row whose maximum is
// not within 2^20 (where the scaling stays below 2^0.1), infinities and NaN among them,
// is read again and takes (z - m) log2 e.
//
// Rows start anywhere: vectors are taken at the 16-B boundaries of the row, and the
// fewer than 2 * 8 elements before the first and after the last whole vector one a
// lane (lanes without a vector or an element hold -inf, which adds nothing).  dlogits
// may be logits: all of a row is on chip before any of it is written, and the forms that
// read a row twice write an element after its last read.
#include "grad_device.h"

#pragma clang fp contract(off)

namespace zs {
namespace {

constexpr float kInf = __builtin_inff();

template <int F> constexpr int kPer = F == 2 ? 4 : 8;   // logits of a 16-B vector

constexpr float kLog2e = 1.44269504088896340736f;

// e^(z - m): with c = m log2 e folded in, and by the difference.
struct Folded {
    float c;
    __device__ __forceinline__ float operator()(float z) const {
        return __builtin_amdgcn_exp2f(__builtin_fmaf(z, kLog2e, -c));
    }
};
struct Plain {
    float m;
    __device__ __forceinline__ float operator()(float z) const {
        return __builtin_amdgcn_exp2f((z - m) * kLog2e);
    }
};
constexpr float kFoldLimit = 0x1p20f;

// The largest logit, from the bit patterns: non-negative floats order like signed
// integers, and among negative ones the largest has the smallest unsigned pattern.
// Both are tracked, two 16-bit logits an instruction.  A positive NaN ends up as the
// maximum and a negative one reaches the sum, so either way the row becomes NaN.
typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

template <int F>
struct MaxBits {
    u32x2 most{F == 2 ? 0x80000000u : 0x80008000u, 0u}, least{0xffffffffu, 0u};
    __device__ __forceinline__ void take(uint32_t w) {
        if constexpr (F == 2) {
            const int a = static_cast<int>(most.x), b = static_cast<int>(w);
            most.x = static_cast<uint32_t>(a > b ? a : b);
            least.x = least.x < w ? least.x : w;
        } else {
            most.x = __builtin_bit_cast(
                uint32_t, __builtin_elementwise_max(__builtin_bit_cast(s16x2, most.x),
                                                    __builtin_bit_cast(s16x2, w)));
            least.x = __builtin_bit_cast(
                uint32_t, __builtin_elementwise_min(__builtin_bit_cast(u16x2, least.x),
                                                    __builtin_bit_cast(u16x2, w)));
        }
    }
    // as FP32, NaN where a positive NaN was seen
    __device__ __forceinline__ float value() const {
        if constexpr (F == 2) {
            return from_bits(static_cast<int>(most.x) >= 0 ? most.x : least.x);
        } else {
            const s16x2 m = __builtin_bit_cast(s16x2, most.x);
            const u16x2 l = __builtin_bit_cast(u16x2, least.x);
            const short hi = m.x > m.y ? m.x : m.y;
            const unsigned short lo = l.x < l.y ? l.x : l.y;
            return to_f32<F == 2 ? 0 : F>(hi >= 0 ? static_cast<uint16_t>(hi) : lo);
        }
    }
};

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

// A row as whole vectors from its first 16-B boundary, and at most one edge element
// a lane: lane l < head holds element l, lane K + l element tail + l of the rest.
template <int F>
struct Row {
    static constexpr uint32_t K = kPer<F>;
    uint32_t head, n_vec;    // elements before the vectors, whole vectors
    uint32_t edge;           // lane l's edge element, ~0 if none
    __device__ __forceinline__ Row(const elem_t<F> *row, uint32_t V, uint32_t l) {
        const uint32_t to_vec =
            static_cast<uint32_t>((16 - reinterpret_cast<uintptr_t>(row) % 16) % 16 /
                                  sizeof(elem_t<F>));
        head = to_vec < V ? to_vec : V;
        n_vec = (V - head) / K;
        const uint32_t tail = head + n_vec * K;
        edge = l < head ? l : l >= K && l < 2 * K && tail + (l - K) < V ? tail + (l - K) : ~0u;
    }
};

// Vector first + l of a row, `first` the same in every lane (so it goes into the
// scalar part of the address), l the lane's own.
template <int F>
__device__ __forceinline__ u32x4 vec_at(const elem_t<F> *row, uint32_t head, uint32_t first,
                                        uint32_t l) {
    auto *base = (const GLOBAL_AS char *)(row + head) + static_cast<uint64_t>(first) * 16;
    asm volatile("" : "+s"(base));   // a scalar base: no address registers a vector
    return __builtin_nontemporal_load((const GLOBAL_AS u32x4 *)(base + l * 16));
}

template <int F>
__device__ __forceinline__ void store_vec_at(elem_t<F> *row, uint32_t head, uint32_t first,
                                             uint32_t l, const float v[kPer<F>]) {
    constexpr int K = kPer<F>;
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = F == 2 ? bits(v[i]) : pack2<F == 2 ? 0 : F>(v[2 * i % K], v[(2 * i + 1) % K]);
    auto *base = (GLOBAL_AS char *)(row + head) + static_cast<uint64_t>(first) * 16;
    asm volatile("" : "+s"(base));
    __builtin_nontemporal_store(w, (GLOBAL_AS u32x4_any *)(base + l * 16));
}

// The larger, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) { return a > b || a != a ? a : b; }

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) x = max_nan(x, __shfl_xor(x, o));
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
    for (int w = 1; w < T / 64; ++w) r = MAX ? max_nan(r, red[w]) : r + red[w];
    __syncthreads();
    return r;
}

// A value that no kernel of this call writes, at an address that is the same in every
// lane: a scalar load, whose result waits in scalar registers until it is needed.
template <typename T>
__device__ __forceinline__ T uniform_load(const T *p) {
    return *(const __attribute__((address_space(4))) T *)(p);
}

// A row's own inputs, requested before its logits so that nothing waits for them later:
// 16384 x 50257 BF16 rows 647 -> 604 us, 400000 x 1024 523 -> 417 us (each repeated alone; among
// other operators the first takes 591 to 704, 653 on average).
struct RowIn {
    float advantage, old_logp, ref_logp, loss_scale;
    int64_t target;
    __device__ __forceinline__ RowIn(const PolicyArgs &a, uint64_t t) {
        advantage = uniform_load(a.advantage + t);
        old_logp = a.old_logp != nullptr ? uniform_load(a.old_logp + t) : 0.0f;
        ref_logp = a.ref_logp != nullptr ? uniform_load(a.ref_logp + t) : 0.0f;
        loss_scale = a.loss_scale_dev != nullptr ? uniform_load(a.loss_scale_dev) : a.loss_scale;
        target = a.targets64 ? uniform_load(static_cast<const int64_t *>(a.targets) + t)
                             : uniform_load(static_cast<const int32_t *>(a.targets) + t);
    }
    // In scalar registers up to here: nothing made from them is held beside the row.
    __device__ __forceinline__ void arrive() {
        asm volatile("" : "+s"(advantage), "+s"(old_logp), "+s"(ref_logp), "+s"(loss_scale));
    }
};

// What a row's gradient needs, the same in every lane.
struct RowGrad {
    float scale;    // -S w g / sum
    float hit;      // S w g, added at the target
};

// e^d - 1 - d and e^d - 1.  Up to |d| = 1 the first by its own series (the first term left
// out is below 2^-31 of the sum), and the second as d more: a difference of the two would
// lose d's digits twice as the policy comes near its reference (all of them at d = 1e-6).
// Beyond, differences, which cancel no more than two bits.  Written out because it is live
// beside the whole row: the library's form would push logits out of registers.
struct ExpTail {
    float tail, minus_1;
};
__device__ __forceinline__ ExpTail exp_tail(float d) {
    if (!(__builtin_fabsf(d) <= 1.0f)) {
        const float em = exp_fast(d) - 1.0f;
        return ExpTail{em - d, em};
    }
    float s = 1.0f;
#pragma unroll
    for (int n = 12; n >= 3; --n) s = __builtin_fmaf(d * (1.0f / n), s, 1.0f);
    const float t = d * d * 0.5f * s;
    return ExpTail{t, d + t};
}
__device__ __forceinline__ float exp_near(float x) {
    return __builtin_fabsf(x) <= 1.0f ? 1.0f + exp_tail(x).minus_1 : exp_fast(x);
}

// ln(x) for x of normal FP32 range, to about 2^-25 absolute next to the exact multiple
// of ln 2: x = 2^k f, f in [0.7, 1.42), ln f = 2 atanh((f - 1) / (f + 1)) by its series
// (the first term left out is below 2^-30).  Anything else as the hardware's logarithm
// has it (0, infinity, NaN).
__device__ __forceinline__ double log_of(float x) {
    if (!(x >= 0x1p-126f && x < kInf))
        return static_cast<double>(__builtin_amdgcn_logf(x));
    int k = __builtin_amdgcn_frexp_expf(x);
    float f = __builtin_amdgcn_frexp_mantf(x);     // [0.5, 1)
    if (f < 0.70710678f) {
        f = f + f;
        k = k - 1;
    }
    const float q = (f - 1.0f) / (f + 1.0f), q2 = q * q;
    float p = 1.0f / 11.0f;
    p = __builtin_fmaf(p, q2, 1.0f / 9.0f);
    p = __builtin_fmaf(p, q2, 1.0f / 7.0f);
    p = __builtin_fmaf(p, q2, 1.0f / 5.0f);
    p = __builtin_fmaf(p, q2, 1.0f / 3.0f);
    const float ln_f = 2.0f * __builtin_fmaf(q * q2, p, q);
    return static_cast<double>(k) * 0.693147180559945309417 + static_cast<double>(ln_f);
}

// The row's loss from its maximum m and the sum of its terms, which hold a factor
// 2^rest; lane 0 writes token_loss and logp.  Losses of both signs cancel in the total,
// so the log-probability and its distances to the old and the reference one are taken in
// FP64: rest = m log2 e - c is known exactly from one fused operation, and what is left
// is the sum's own error.
__device__ __forceinline__ RowGrad finish_row(const PolicyArgs &a, RowIn in, uint64_t t,
                                              float m, float rest, float sum, float z_target,
                                              float w, uint32_t lane) {
    in.arrive();
    const double lp = (static_cast<double>(z_target) - static_cast<double>(m)) -
                      (log_of(sum) - static_cast<double>(rest) * 0.693147180559945309417);
    const float logp = static_cast<float>(lp);
    const float A = in.advantage;
    float r = 1.0f;
    if (a.old_logp != nullptr)
        r = exp_near(static_cast<float>(lp - static_cast<double>(in.old_logp)));
    const float lo = 1.0f - a.clip_low, hi = 1.0f + a.clip_high;
    float rc = r < lo ? lo : r;
    rc = rc > hi ? hi : rc;
    const float p0 = -(r * A), p1 = -(rc * A);
    float L = p0 >= p1 || p0 != p0 ? p0 : p1;      // the larger; NaN stays
    const bool cut = (A > 0.0f && r > hi) || (A < 0.0f && r < lo);
    float g = cut ? 0.0f : p0;
    if (a.ref_logp != nullptr && a.kl_coef != 0.0f) {
        const float d = static_cast<float>(static_cast<double>(in.ref_logp) - lp);
        const ExpTail x = exp_tail(d);
        L = L + a.kl_coef * x.tail;
        g = g - a.kl_coef * x.minus_1;
    }
    if (lane == 0) {
        a.token_loss[t] = L;
        a.logp[t] = logp;
    }
    const float h = in.loss_scale * (w * g);
    return RowGrad{-h / sum, h};
}

// The target's logit, NaN for a target outside the vocabulary (at: its index,
// ~0 then).
template <int F>
__device__ __forceinline__ float target_logit(const PolicyArgs &a, const elem_t<F> *row,
                                              int64_t v, uint32_t *at) {
    const bool in = v >= 0 && static_cast<uint64_t>(v) < a.vocab;
    *at = in ? static_cast<uint32_t>(v) : 0xffffffffu;
    return in ? to_f32<F>(row[v]) : __builtin_nanf("");
}

// This lane's place in the group of T lanes that has its row.
template <int T>
__device__ __forceinline__ uint32_t lane_of() {
    return T == 64 ? threadIdx.x & 63u : threadIdx.x;
}

// Row t's gradient is zero everywhere.
template <int F, int T>
__device__ __forceinline__ void skip_row(const PolicyArgs &a, uint64_t t) {
    const uint32_t lane = lane_of<T>();
    if (lane == 0) {
        a.token_loss[t] = 0.0f;
        a.logp[t] = 0.0f;
    }
    if (a.dlogits == nullptr) return;
    auto *d = static_cast<elem_t<F> *>(a.dlogits) + t * a.ldd;
    const Row<F> r(d, static_cast<uint32_t>(a.vocab), lane);
    const float zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (uint32_t j = 0; j + lane < r.n_vec; j += T)
        store_vec_at<F>(d, r.head, j, lane, zero);
    if (r.edge != ~0u) d[r.edge] = from_f32<F>(0.0f);
}

// Gradients of vector first + lane from its logits.
template <int F, typename Exp>
__device__ __forceinline__ void grad_vec(elem_t<F> *d, uint32_t head, uint32_t first,
                                         uint32_t lane, const u32x4 &w, const Exp &exp_of,
                                         const RowGrad &g, uint32_t target) {
    constexpr uint32_t K = kPer<F>;
    float z[K];
    widen_vec<F>(w, z);
#pragma unroll
    for (uint32_t i = 0; i < K; ++i) z[i] = exp_of(z[i]) * g.scale;
    // the target's place among the vectors (it wraps to none for an edge element)
    const uint32_t at = target - head;
    if (at / K - first == lane) {
#pragma unroll
        for (uint32_t i = 0; i < K; ++i) z[i] = at % K == i ? z[i] + g.hit : z[i];
    }
    store_vec_at<F>(d, head, first, lane, z);
}

template <int F, typename Exp>
__device__ __forceinline__ void grad_edge(elem_t<F> *d, uint32_t edge, float z, const Exp &exp_of,
                                          const RowGrad &g, uint32_t target) {
    if (edge == ~0u) return;
    const float p = exp_of(z) * g.scale;
    d[edge] = from_f32<F>(edge == target ? p + g.hit : p);
}

// Row t by reading it again, once its maximum m is known: the sum, then the gradients.
// Everything else is made anew from t, so that nothing is held for it beside a row on chip.
template <int F, int T>
__device__ __forceinline__ void reread_row(const PolicyArgs &a, uint64_t t, float m, float *red) {
    uint32_t lane = lane_of<T>();
    asm volatile("" : "+v"(lane));
    const RowIn in(a, t);
    const auto *row = static_cast<const elem_t<F> *>(a.logits) + t * a.ld;
    const Row<F> r(row, static_cast<uint32_t>(a.vocab), lane);
    uint32_t target;
    const float zt = target_logit<F>(a, row, in.target, &target);
    const float ze = r.edge != ~0u ? to_f32<F>(row[r.edge]) : -kInf;
    const Plain exp_of{m};
    float s = r.edge != ~0u ? exp_of(ze) : 0.0f;
    for (uint32_t j = 0; j + lane < r.n_vec; j += T) {
        float z[kPer<F>];
        widen_vec<F>(vec_at<F>(row, r.head, j, lane), z);
#pragma unroll
        for (int k = 0; k < kPer<F>; ++k) s = s + exp_of(z[k]);
    }
    s = block_reduce<T, false>(s, red);
    const RowGrad g = finish_row(a, in, t, m, 0.0f, s, zt, uniform_load(a.weight + t), lane);
    auto *d = static_cast<elem_t<F> *>(a.dlogits) + t * a.ldd;
    for (uint32_t j = 0; j + lane < r.n_vec; j += T)
        grad_vec<F>(d, r.head, j, lane, vec_at<F>(row, r.head, j, lane), exp_of, g, target);
    grad_edge<F>(d, r.edge, ze, exp_of, g, target);
}

// A block of 64 lanes a row would be bound by the rate at which blocks start: rows
// that one wave holds share a block of kShare waves.
constexpr int kShare = 4;
template <int T> constexpr int kBlock = T == 64 ? 64 * kShare : T;
template <int T>
__device__ __forceinline__ uint64_t first_row() {
    if constexpr (T == 64)
        return static_cast<uint64_t>(blockIdx.x) * kShare +
               __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    else
        return blockIdx.x;
}
template <int T>
__device__ __forceinline__ uint64_t row_stride() {
    return static_cast<uint64_t>(gridDim.x) * (T == 64 ? kShare : 1);
}

// One row a group of T lanes (a block, or one of the waves of a block), its logits on
// chip: N vectors a lane in registers and L in LDS.
// Four waves a SIMD leave 128 registers a lane.  The longest rows spill 33 to 39 of them
// around the row's scalar part; three waves a SIMD with more vectors a lane (384 lanes x
// (31 + 12)) measured a third slower, as the arithmetic then hides less.  8192 x 131072
// BF16: 815 us, 5.3 TB/s.
template <int F, int T, int N, int L>
__global__ __launch_bounds__(kBlock<T>, 4) void policy_row_kernel(PolicyArgs a) {
    constexpr int B = 3;                  // vectors on their way to LDS at once
    static_assert(L % B == 0, "whole batches");
    __shared__ float red[kBlock<T> / 64];
    __shared__ u32x4 held[L > 0 ? L : 1][T];
    const uint32_t V = static_cast<uint32_t>(a.vocab);
    for (uint64_t t = first_row<T>(); t < a.rows; t += row_stride<T>()) {
        uint32_t lane = lane_of<T>();  // of the group; opaque, so that nothing made from it
        asm volatile("" : "+v"(lane)); // is held in registers from row to row
        const float weight = uniform_load(a.weight + t);
        if (weight == 0.0f) {
            skip_row<F, T>(a, t);
            continue;
        }
        const RowIn in(a, t);
        const auto *row = static_cast<const elem_t<F> *>(a.logits) + t * a.ld;
        const Row<F> r(row, V, lane);
        // lane holds vector i * T + lane; n_vec is hidden between the passes, so that their
        // lane masks are not kept (in registers the logits need)
        uint32_t n_vec = r.n_vec;
        auto on = [&](int i) { return static_cast<uint32_t>(i) * T + lane < n_vec; };
        auto fetch = [&](int i) {
            u32x4 w = neg_inf_vec<F>();
            if (on(i)) w = vec_at<F>(row, r.head, i * T, lane);
            return w;
        };
        MaxBits<F> most;
        auto take = [&](const u32x4 &w) {
#pragma unroll
            for (int k = 0; k < 4; ++k) most.take(w[k]);
        };
        u32x4 x[N];
#pragma unroll
        for (int i = 0; i < L; i += B) {
            u32x4 y[B];
#pragma unroll
            for (int b = 0; b < B; ++b) y[b] = fetch(N + i + b);
#pragma unroll
            for (int b = 0; b < B; ++b) {
                take(y[b]);
                held[i + b][lane] = y[b];   // read by the same lane only
            }
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = fetch(i);
        uint32_t target;
        const float zt = target_logit<F>(a, row, in.target, &target);
        const float ze = r.edge != ~0u ? to_f32<F>(row[r.edge]) : -kInf;
#pragma unroll
        for (int i = 0; i < N; ++i) take(x[i]);
        const float m = block_reduce<T, true>(max_nan(most.value(), ze), red);
        if (!(__builtin_fabsf(m) <= kFoldLimit)) {   // the same in every lane of the row
            reread_row<F, T>(a, t, m, red);
            continue;
        }
        const Folded exp_of{m * kLog2e};
        float s = exp_of(ze);
        auto add = [&](const u32x4 &w) {
            float z[kPer<F>];
            widen_vec<F>(w, z);
#pragma unroll
            for (int k = 0; k < kPer<F>; ++k) s = s + exp_of(z[k]);
        };
#pragma unroll
        for (int i = 0; i < N; ++i) {
            keep_raw(x[i]);
            add(x[i]);
        }
        // one LDS vector at a time: read ahead, they would push the row out of registers
#pragma unroll
        for (int i = 0; i < L; ++i) {
            __builtin_amdgcn_sched_barrier(0);
            add(held[i][lane]);
        }
        s = block_reduce<T, false>(s, red);
        // beside the longest rows even these scalars cost a spill: asked for again there
        const RowGrad g = finish_row(a, N > 16 ? RowIn(a, t) : in, t, m,
                                     __builtin_fmaf(m, kLog2e, -exp_of.c), s, zt, weight, lane);
        auto *d = static_cast<elem_t<F> *>(a.dlogits) + t * a.ldd;
        asm volatile("" : "+s"(n_vec));
#pragma unroll
        for (int i = 0; i < N; ++i) {
            keep_raw(x[i]);
            if (on(i)) grad_vec<F>(d, r.head, i * T, lane, x[i], exp_of, g, target);
        }
#pragma unroll
        for (int i = 0; i < L; ++i) {
            __builtin_amdgcn_sched_barrier(0);
            if (on(N + i))
                grad_vec<F>(d, r.head, (N + i) * T, lane, held[i][lane], exp_of, g, target);
        }
        grad_edge<F>(d, r.edge, ze, exp_of, g, target);
    }
}

// One row a block of T lanes in one pass for the loss (running maximum and sum a
// lane) and, with dlogits, a second for the gradients: 3.3 to 3.5 TB/s of the logits read
// once and the gradients written once, where the rows on chip reach 5.  The loss alone, BF16:
// 400000 x 1024 263 us, 32768 x 8192 504 (1.1 TB/s: a vector a lane, between two reductions of
// the block), 8192 x 131072 537, 2048 x 262144 245 (4.4 TB/s).
template <int F, int T>
__global__ __launch_bounds__(kBlock<T>) void policy_long_kernel(PolicyArgs a) {
    constexpr int K = kPer<F>;
    __shared__ float red[kBlock<T> / 64];
    const uint32_t V = static_cast<uint32_t>(a.vocab);
    const uint32_t lane = lane_of<T>();
    for (uint64_t t = first_row<T>(); t < a.rows; t += row_stride<T>()) {
        const float weight = a.weight[t];
        if (weight == 0.0f) {
            skip_row<F, T>(a, t);
            continue;
        }
        const RowIn in(a, t);
        const auto *row = static_cast<const elem_t<F> *>(a.logits) + t * a.ld;
        const Row<F> r(row, V, lane);
        uint32_t target;
        const float zt = target_logit<F>(a, row, in.target, &target);
        const float ze = r.edge != ~0u ? to_f32<F>(row[r.edge]) : -kInf;
        // the running maximum and the sum in its units; nothing but -inf so far adds nothing.
        // The edge element's term is 1 in its own units (NaN if it is infinite or NaN)
        float m = ze;
        float s = m == -kInf ? 0.0f : Plain{m}(ze);
        for (uint32_t j = 0; j + lane < r.n_vec; j += T) {
            const u32x4 w = vec_at<F>(row, r.head, j, lane);
            MaxBits<F> most;
#pragma unroll
            for (int k = 0; k < 4; ++k) most.take(w[k]);
            const float vm = max_nan(most.value(), m);
            if (vm != m) {           // the sum so far in units of the new maximum
                s = m == -kInf ? s : s * Plain{vm}(m);
                m = vm;
            }
            const Plain exp_of{m == -kInf ? 0.0f : m};
            float z[K];
            widen_vec<F>(w, z);
#pragma unroll
            for (int k = 0; k < K; ++k) s = s + exp_of(z[k]);
        }
        const float rm = block_reduce<T, true>(m, red);
        const Plain exp_of{rm};
        s = block_reduce<T, false>(m == -kInf ? s : s * exp_of(m), red);
        if (rm == -kInf) s = __builtin_nanf("");   // nothing left to choose from
        const RowGrad g = finish_row(a, in, t, rm, 0.0f, s, zt, weight, lane);
        if (a.dlogits == nullptr) continue;
        auto *d = static_cast<elem_t<F> *>(a.dlogits) + t * a.ldd;
        for (uint32_t j = 0; j + lane < r.n_vec; j += T)
            grad_vec<F>(d, r.head, j, lane, vec_at<F>(row, r.head, j, lane), exp_of, g,
                        target);
        grad_edge<F>(d, r.edge, ze, exp_of, g, target);
    }
}

// loss = sum of weight * token_loss in FP64: each lane its stride of rows, then
// a tree over the lanes.  Rows of weight zero add nothing.  One block, bound by the latency of
// its loads: 3 us for 61 rows, 9 for 16384, 128 for 400000.
constexpr int kSumThreads = 1024;
__global__ __launch_bounds__(kSumThreads) void policy_sum_kernel(
    float *__restrict__ loss, const float *__restrict__ token_loss,
    const float *__restrict__ weight, uint64_t rows) {
    __shared__ double red[kSumThreads];
    constexpr int U = 8;   // rows in flight a lane
    double s = 0.0;
    for (uint64_t t0 = threadIdx.x; t0 < rows; t0 += U * kSumThreads) {
        float w[U], l[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint64_t t = t0 + u * kSumThreads;
            w[u] = t < rows ? weight[t] : 0.0f;
            l[u] = t < rows ? token_loss[t] : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (w[u] != 0.0f) s += static_cast<double>(w[u]) * static_cast<double>(l[u]);
    }
    red[threadIdx.x] = s;
    for (int o = kSumThreads / 2; o > 0; o >>= 1) {
        __syncthreads();
        if (static_cast<int>(threadIdx.x) < o) red[threadIdx.x] += red[threadIdx.x + o];
    }
    if (threadIdx.x == 0) *loss = static_cast<float>(red[0]);
}

constexpr uint64_t kMaxGrid = 1ull << 21;   // 1024-lane blocks: below 2^32 lanes a launch

template <int F>
hipError_t policy_rows(const PolicyArgs &a, hipStream_t stream) {
    const uint64_t n_vec = a.vocab / kPer<F>;   // whole vectors of a row at most
#define ZS_LAUNCH(kernel, T)                                                          \
    do {                                                                              \
        const uint64_t per = T == 64 ? kShare : 1, want = (a.rows + per - 1) / per;   \
        const uint64_t cap = max_blocks() < kMaxGrid ? max_blocks() : kMaxGrid;       \
        kernel<<<static_cast<uint32_t>(want < cap ? want : cap), kBlock<T>, 0,        \
                 stream>>>(a);                                                        \
        return hipGetLastError();                                                     \
    } while (0)
#define ZS_ROW(T, N, L) \
    if (n_vec <= static_cast<uint64_t>(T) * (N + L)) ZS_LAUNCH((policy_row_kernel<F, T, N, L>), T)
    if (a.dlogits != nullptr) {
        ZS_ROW(64, 2, 0);
        ZS_ROW(64, 4, 0);
        ZS_ROW(256, 4, 0);
        ZS_ROW(256, 8, 0);
        ZS_ROW(256, 16, 0);
        ZS_ROW(512, 16, 0);
        ZS_ROW(512, 16, 9);   // without spills: 8192 x 98304 598 us, with 24 in registers 649
        ZS_ROW(512, 23, 9);
        ZS_ROW(1024, 23, 9);
    }
    if (n_vec <= 64 * 4) ZS_LAUNCH((policy_long_kernel<F, 64>), 64);
    ZS_LAUNCH((policy_long_kernel<F, 1024>), 1024);
#undef ZS_ROW
#undef ZS_LAUNCH
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
