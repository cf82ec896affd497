// Internal interface between the C-ABI layer of zero_shard_grad.h (grad_api.cpp)
// and its gfx950 kernels.  Not installed.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "launch.h"
#include "zero_shard_grad.h"

namespace zs {

// Division by a fixed 32-bit divisor d >= 1 of any numerator below 2^62, by one
// high product: with s = ceil(log2 d) and m = floor(2^(62+s) / d) + 1, the
// error m*d - 2^(62+s) is in (0, d], at most 2^s, so floor(n*m / 2^(62+s)) is
// floor(n/d) for every n < 2^62.  m < 2^63 + 1 fits 64 bits; the product's
// high word is the quotient shifted by s - 2, so the kernel computes
// mulhi(n << 2, m) >> s.
struct FastDiv {
    uint64_t m;
    uint32_t d, s;
};

inline FastDiv fast_div(uint32_t d) {
    FastDiv f{0, d, 0};
    while ((1ull << f.s) < d) ++f.s;
    f.m = static_cast<uint64_t>((static_cast<unsigned __int128>(1) << (62 + f.s)) / d) + 1;
    return f;
}

// ---- activation checkpoints (act_kernels.hip) ----
// Every count is non-zero and every argument checked; fmt is a zero_dtype value.
hipError_t launch_act_save(uint8_t *q, uint8_t *e, void *y, uint64_t ldy, const void *x,
                           uint64_t ldx, int fmt, int act, uint64_t rows, uint64_t cols,
                           hipStream_t stream);
hipError_t launch_act_load(void *x, uint64_t ldx, int fmt, const uint8_t *q, const uint8_t *e,
                           uint64_t rows, uint64_t cols, hipStream_t stream);
hipError_t launch_act_backward(void *dx, uint64_t lddx, const void *dy, uint64_t lddy, int fmt,
                               int act, const uint8_t *q, const uint8_t *e, uint64_t rows,
                               uint64_t cols, hipStream_t stream);

// ---- weight gradient (wgrad_kernels.hip) ----
// Bytes of workspace for these extents (tokens, n_out and n_in non-zero).
uint64_t weight_grad_workspace(uint64_t tokens, uint64_t n_out, uint64_t n_in);
hipError_t launch_weight_grad(void *dw, bool dw32, bool first, const uint16_t *dy, uint64_t lddy,
                              int fmt, const uint8_t *q, const uint8_t *e, uint64_t tokens,
                              uint64_t n_out, uint64_t n_in, void *workspace, hipStream_t stream);
// dw[0, n) = 0 (fill kernel).
hipError_t launch_zero_fill(void *dw, int elem_bytes, uint64_t n, hipStream_t stream);

// ---- embedding (embed_kernels.hip) ----
hipError_t launch_embed_lookup(void *out, uint64_t ldo, const void *table, int fmt,
                               const void *ids, bool ids64, uint64_t tokens, uint64_t vocab,
                               uint64_t width, float scale, hipStream_t stream);
uint64_t embed_grad_workspace(uint64_t tokens, uint64_t vocab, uint64_t width);
hipError_t launch_embed_grad(void *dw, bool dw32, bool first, const uint16_t *dy, uint64_t lddy,
                             int fmt, const void *ids, bool ids64, uint64_t tokens,
                             uint64_t vocab, uint64_t width, float scale, void *workspace,
                             hipStream_t stream);

// ---- policy loss (policy_kernels.hip) ----
struct PolicyArgs {
    float *loss, *token_loss, *logp;
    void *dlogits;             // nullable
    const void *logits;
    uint64_t ldd, ld;
    const void *targets;
    bool targets64;
    const float *old_logp;     // nullable
    const float *ref_logp;     // nullable
    const float *advantage, *weight;
    uint64_t rows, vocab;
    float clip_low, clip_high, kl_coef, loss_scale;
    const float *loss_scale_dev;  // nullable: replaces loss_scale
};
hipError_t launch_policy_loss(const PolicyArgs &a, int fmt, hipStream_t stream);

}  // namespace zs
