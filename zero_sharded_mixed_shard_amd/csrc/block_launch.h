// Internal interface between the C-ABI layer of zero_shard_block.h
// (block_api.cpp) and its gfx950 kernels.  Not installed.
#pragma once

#include "grad_launch.h"
#include "zero_shard_block.h"

namespace zs {

// Every extent is non-zero and every argument checked; fmt is a zero_dtype value.

// ---- codes in blocks of 128 (quant_kernels.hip) ----
hipError_t launch_block_quant(uint8_t *q, uint8_t *e, uint8_t *qt, uint8_t *et, const void *x,
                              uint64_t ldx, int fmt, bool square, uint64_t rows, uint64_t cols,
                              hipStream_t stream);
hipError_t launch_block_load(void *x, uint64_t ldx, int fmt, const uint8_t *q, const uint8_t *e,
                             bool square, uint64_t rows, uint64_t cols, hipStream_t stream);

// ---- their product (product_kernels.hip) ----
struct ProductArgs {
    void *y;
    const uint8_t *qa, *ea, *qb, *eb;
    uint64_t ldy, m, n, k;
    uint32_t a_block;
    void *workspace;
};
uint64_t product_workspace(uint64_t m, uint64_t n, uint64_t k);
hipError_t launch_product(const ProductArgs &a, int fmt, hipStream_t stream);
// y[rows, cols] = 0
hipError_t launch_zero_matrix(void *y, uint64_t ldy, int fmt, uint64_t rows, uint64_t cols,
                              hipStream_t stream);

// ---- dropout (dropout_kernels.hip) ----
// The mask of a call: what stays has bits >= threshold and is multiplied by factor.
struct Mask {
    uint32_t threshold;        // t, 0 to 65536
    float factor;
    uint64_t seed, offset;
    const uint64_t *d_offset;  // nullable: added to offset
};
hipError_t launch_dropout(void *y, uint64_t ldy, const void *x, uint64_t ldx, int fmt,
                          uint64_t rows, uint64_t cols, const Mask &mask, hipStream_t stream);

// ---- the step between two blocks (residual_kernels.hip) ----
struct ResidualArgs {
    uint64_t rows;
    uint32_t cols;
    int fmt;                   // of f, h and the parameters
    bool res32;                // the residual stream is FP32 where fmt is not
    int post, pre;             // zero_norm
    const void *w1, *b1, *gate, *w2, *b2;   // nullable
    float eps, res_scale;
    Mask mask;
    const void *f;             // nullable
    uint64_t ldf;
    float *stats;              // written (nullable) or read
    // forward
    const void *r;
    void *u_out, *h;
    uint64_t ldr, ldu, ldh;
    // backward
    const void *u, *dh, *du;   // du nullable; dh null iff pre is NONE
    void *df, *dr;             // df null iff f is
    uint64_t lddh, lddu, lddf, lddr;
    void *dw1, *db1, *dgate, *dw2, *db2;    // nullable
    bool grad32, first;
    void *workspace;
};
hipError_t launch_residual_forward(const ResidualArgs &a, hipStream_t stream);
hipError_t launch_residual_backward(const ResidualArgs &a, hipStream_t stream);
uint64_t residual_workspace(uint64_t rows, uint64_t cols);

}  // namespace zs
