/*
 * zero_shard_block.h -- C ABI of the operators around the linear layers of a
 * transformer block, on an MI355X (gfx950): the layers' products in 8 bits, the
 * step between two blocks (norms, gate, residual scale) forward and backward,
 * and dropout.  They stand between the operators of zero_shard_grad.h: a norm's
 * output becomes a checkpoint or codes, a product reads those, the activation
 * and weight gradient kernels do the rest of the layer.
 *
 * Conventions: those of zero_shard_grad.h (matrices by row stride, any
 * element-aligned pointer, no overlaps except where a function says so, sums in
 * an order that the arguments fix, workspaces and what two calls may share).
 */
#ifndef ZERO_SHARD_BLOCK_H_
#define ZERO_SHARD_BLOCK_H_

#include "zero_shard_grad.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------------
 * Matrices in 8 bits with one power of two for each block of 128.
 *
 * Codes and exponent bytes are those of the activation checkpoints (the value
 * is code * 2^(e - 127); e is 3 to 247; the scale is the smallest 2^k,
 * k >= -124, with max|x| <= 448 * 2^k over the block's finite elements;
 * magnitudes above 15/16 of the power of two that ends the format are held
 * there; an infinity or NaN is kept as NaN and does not disturb its block).
 * What differs is the block:
 *   ZERO_BLOCKS_ROW     128 neighbours of a row (activations and gradients):
 *                       e[rows, ceil(cols/128)];
 *   ZERO_BLOCKS_SQUARE  128 x 128 (weights): e[ceil(rows/128), ceil(cols/128)].
 * The last blocks of a row or column may be shorter.  q[rows, cols] and e are
 * contiguous.
 * ------------------------------------------------------------------------- */
#define ZERO_BLOCK 128

typedef enum { ZERO_BLOCKS_ROW = 0, ZERO_BLOCKS_SQUARE = 1 } zero_blocks;

/*
 * zero_block_quant -- the codes and exponents of x, and with square blocks also
 * those of its transpose (the codes transposed; the same blocks).
 *   q   device, rows*cols bytes;  e  device, as above.
 *   qt  device, cols*rows bytes, or NULL;  et  device, the exponents
 *       transposed, NULL exactly where qt is.  Square blocks only.
 *   x   device, format dt (F16, BF16 or F32), row stride ldx.
 *   rows == 0 or cols == 0: no-op.
 *   Errors: ZERO_EDTYPE; ZERO_EINVAL for a bad `blocks`, a NULL or misaligned
 *   pointer, one of qt and et without the other or without square blocks,
 *   ldx < cols, an extent past its limit, or an overlap; ZERO_EHIP.
 */
int zero_block_quant(uint8_t *q, uint8_t *e, uint8_t *qt, uint8_t *et, const void *x,
                     uint64_t ldx, zero_dtype dt, zero_blocks blocks, uint64_t rows,
                     uint64_t cols, void *stream);

/*
 * zero_block_load -- x = the values that codes stand for, rounded once to dt
 * (exact where dt is the format they were written from, or holds it).
 *   Errors: as zero_block_quant.
 */
int zero_block_load(void *x, uint64_t ldx, zero_dtype dt, const uint8_t *q, const uint8_t *e,
                    zero_blocks blocks, uint64_t rows, uint64_t cols, void *stream);

/*
 * zero_block_product -- the product of two coded matrices over their columns:
 *     y[i, j] = sum over c of a[i, c] * b[j, c]
 * a[m, k] in blocks of a row, b[n, k] in square ones.  With a = x's codes and
 * b = W's it is the linear layer y = x W^T; with dy's codes and W's transposed
 * ones it is the input gradient dx = dy W.
 *   y   device, format dt (F16, BF16 or F32), row stride ldy.
 *   qa, ea  codes of a, exponents [m, ceil(k/a_block)], contiguous.  a_block
 *       is ZERO_BLOCK, or ZERO_ACT_BLOCK for an activation checkpoint.
 *   qb, eb  codes of b, exponents [ceil(n/128), ceil(k/128)], contiguous.
 *   Products are exact.  dt == ZERO_F32: summed in FP32 (in FP64, and many times
 *   slower, in tiles where a block has exponent byte 247, values of 1.75 * 2^127
 *   and more).  16-bit dt: rounded
 *   once from FP32 sums whose matrix instructions drop, from each product of a
 *   group of eight, what lies 2^-13 and more below the group's largest (an
 *   error of at most 2^-10 of the sum of magnitudes, typically 1.5e-5 of the
 *   result).  Codes of NaN give NaN in their row or column of y.
 *   workspace  device, workspace_bytes >= zero_block_product_workspace's
 *       answer, 16-byte aligned; may be NULL if that is 0.  Its contents
 *       before the call do not matter.
 *   m == 0 or n == 0: no-op.  k == 0: y = 0.  k below 16, or of 2^24 and more,
 *   is summed in FP64, and many times slower.
 *   Errors: ZERO_EDTYPE; ZERO_EINVAL for an a_block other than those two, a
 *   NULL or misaligned pointer, ldy < n, a small or misaligned workspace, an
 *   extent past its limit, or an overlap; ZERO_EHIP.
 */
int zero_block_product(void *y, uint64_t ldy, zero_dtype dt, const uint8_t *qa, const uint8_t *ea,
                       uint32_t a_block, const uint8_t *qb, const uint8_t *eb, uint64_t m,
                       uint64_t n, uint64_t k, void *workspace, uint64_t workspace_bytes,
                       void *stream);

/* zero_block_product_workspace -- bytes zero_block_product needs for these
 * extents, whatever the formats.  Host only.  Errors: ZERO_EINVAL for an extent
 * past its limit or a NULL bytes. */
int zero_block_product_workspace(uint64_t m, uint64_t n, uint64_t k, uint64_t *bytes);

/* ---------------------------------------------------------------------------
 * Dropout.
 *
 * The mask is a function of (seed, offset, row, column), computed where it is
 * needed and never stored: Philox4x32 with ten rounds (Salmon, Moraes, Dror and
 * Shaw, 2011) of the counter
 *     (column / 8, row, offset mod 2^32, offset / 2^32)
 * under the key (seed mod 2^32, seed / 2^32) gives eight columns 16 bits each,
 * word (column mod 8) / 2, its low half for even columns.  An element stays
 * where its bits are >= t = rint(65536 p), halves to even, and is multiplied by
 * the FP32 quotient 65536 / (65536 - t); so the probability in force is
 * t / 65536.  A dropped element becomes 0 whatever it was.
 * Calls that are to differ (layers, steps, ranks) take offsets that differ.
 * With d_offset the value it points to, read on the device when the kernel
 * runs, is added to offset (mod 2^64): a captured graph draws a new mask each
 * replay if the program advances that value.
 * ------------------------------------------------------------------------- */

/*
 * zero_dropout -- y = x with its mask applied, in FP32, rounded once to dt.
 * The same call with dy for x is the backward pass.  p == 0 copies, p == 1
 * (and t == 65536) clears.
 *   y, x  device, format dt (F16, BF16 or F32); y may be exactly x.
 *   d_offset  device, one value, 8-byte aligned, or NULL.
 *   rows == 0 or cols == 0: no-op.
 *   Errors: ZERO_EDTYPE; ZERO_EINVAL for a p outside [0, 1], a NULL or
 *   misaligned pointer, a row stride < cols, an extent past its limit, or an
 *   overlap; ZERO_EHIP.
 */
int zero_dropout(void *y, uint64_t ldy, const void *x, uint64_t ldx, zero_dtype dt, uint64_t rows,
                 uint64_t cols, float p, uint64_t seed, uint64_t offset, const uint64_t *d_offset,
                 void *stream);

/* ---------------------------------------------------------------------------
 * The step between two blocks.
 *
 * With f the output of a block, r the residual stream before it, for each row:
 *     n = post(f)                         norm after the block, or f itself
 *     u = res_scale * r + gate * drop(n)  the residual stream after it
 *     h = pre(u)                          norm before the next block
 * where a norm of kind ZERO_NORM_RMS is x / sqrt(mean(x^2) + eps), of kind
 * ZERO_NORM_LAYER (x - mean(x)) / sqrt(mean((x - mean(x))^2) + eps), times its
 * weight, plus its bias; gate is a factor for each column; drop is
 * zero_dropout's mask and factor.  FP32 throughout (u is rounded to res_dt once
 * on its way out; h comes from u before that).  f == NULL: no block lies
 * before, and h = pre(r).
 * ------------------------------------------------------------------------- */
typedef enum { ZERO_NORM_NONE = 0, ZERO_NORM_RMS = 1, ZERO_NORM_LAYER = 2 } zero_norm;

/* What both passes are told alike. */
typedef struct zero_residual {
    uint64_t rows, cols;
    zero_dtype dt;           /* of f, h, their gradients, and the parameters */
    zero_dtype res_dt;       /* of r, u and their gradients: dt or ZERO_F32 */
    zero_norm post, pre;
    /* device, cols values of format dt each, or NULL (weights and gate 1, biases 0) */
    const void *post_weight, *post_bias, *gate, *pre_weight, *pre_bias;
    float eps;               /* of both norms, 2^-80 at least and finite */
    float res_scale;         /* finite */
    float p;                 /* dropout probability; 0: none */
    uint64_t seed, offset;   /* of the mask, as zero_dropout's */
    const uint64_t *d_offset;
} zero_residual;

/* Where the parameters' gradients go: cols values each, contiguous; NULL: not
 * wanted. */
typedef struct zero_residual_grads {
    void *post_weight, *post_bias, *gate, *pre_weight, *pre_bias;
} zero_residual_grads;

/*
 * zero_residual_norm -- u, h and what the backward pass needs of each row.
 *   u      device, res_dt; may be exactly r.  NULL iff f is NULL.
 *   h      device, dt.  NULL iff pre is ZERO_NORM_NONE.
 *   stats  device FP32, [rows, 4] contiguous: mean and reciprocal deviation of
 *          f, then of u (0 and 1 for a norm that is not there; the mean is 0
 *          for ZERO_NORM_RMS); or NULL.
 *   r      device, res_dt.   f  device, dt, or NULL; then post is
 *          ZERO_NORM_NONE, pre is not, gate is NULL, res_scale 1 and p 0.
 *   rows == 0 or cols == 0: no-op.
 *   Errors: ZERO_EDTYPE for a bad dt or a res_dt that is neither dt nor
 *   ZERO_F32; ZERO_EINVAL for a bad norm, a parameter of a norm that is not
 *   there, eps, res_scale or p outside its range, a NULL or misaligned
 *   pointer, a row stride < cols, an extent past its limit, or an overlap;
 *   ZERO_EHIP.
 */
int zero_residual_norm(void *u, uint64_t ldu, void *h, uint64_t ldh, float *stats, const void *r,
                       uint64_t ldr, const void *f, uint64_t ldf, const zero_residual *block,
                       void *stream);

/*
 * zero_residual_norm_backward -- gradients of r, f and the parameters:
 *     g  = du + pre's Jacobian^T (pre_weight * dh)
 *     dr = res_scale * g
 *     df = post's Jacobian^T (post_weight * gate * drop(g))
 * and over the rows, with u^ and f^ the normalised rows (f itself without a
 * post norm), G = drop(g):
 *     pre_weight: sum dh u^      pre_bias: sum dh
 *     post_weight: gate * sum G f^     post_bias: gate * sum G
 *     gate: post_weight * sum G f^ + post_bias * sum G
 *   df     device, dt; may be exactly dh.  NULL iff f is.
 *   dr     device, res_dt; may be exactly du.
 *   grads  a gradient may be asked for only where its parameter is given.
 *   grad_dt, first  as zero_weight_grad's dw_dt and first: dt with first
 *          non-zero, or ZERO_F32 stored or added.
 *   dh     device, dt.  NULL iff pre is ZERO_NORM_NONE.
 *   du     device, res_dt: what comes down the residual stream; NULL: zero
 *          (not where pre is ZERO_NORM_NONE).
 *   f, u   as the forward pass had and left them (f == NULL: u is its r).
 *          With a 16-bit res_dt u^ is made from the rounded u, where h came from
 *          the sum before: off by u's rounding over the row's deviation.  Near
 *          zero that is the rounding of any 16-bit value, but rows that lie far
 *          from zero for their deviation lose by it: with a mean of ten
 *          deviations pre_weight's gradient (of a layer norm) is off by 1.8% of
 *          its norm in BF16 and 0.2% in FP16, with a hundred by 14% and 1.8%
 *          (dr by 0.04% and 0.3%, BF16).  A stream in FP32 has none of this; nor
 *          has a norm in a call of its own (pre ZERO_NORM_NONE here, then f ==
 *          NULL with this u for r), where both passes see the rounded row.
 *   stats  the forward pass's.
 *   workspace  device, workspace_bytes >= zero_residual_norm_workspace's
 *          answer, 16-byte aligned; may be NULL if that is 0.
 *   rows == 0: the parameters' gradients are 0 when first, else no-op.
 *   cols == 0: no-op.
 *   Errors: as zero_residual_norm; ZERO_EDTYPE also for a grad_dt that is
 *   neither dt nor ZERO_F32; ZERO_EINVAL also for first == 0 with another
 *   grad_dt than ZERO_F32 and for a small or misaligned workspace.
 */
int zero_residual_norm_backward(void *df, uint64_t lddf, void *dr, uint64_t lddr,
                                const zero_residual_grads *grads, zero_dtype grad_dt,
                                int32_t first, const void *dh, uint64_t lddh, const void *du,
                                uint64_t lddu, const void *f, uint64_t ldf, const void *u,
                                uint64_t ldu, const float *stats, const zero_residual *block,
                                void *workspace, uint64_t workspace_bytes, void *stream);

/* zero_residual_norm_workspace -- bytes zero_residual_norm_backward needs for
 * these extents, whatever else it is told.  Host only.  Errors: ZERO_EINVAL. */
int zero_residual_norm_workspace(uint64_t rows, uint64_t cols, uint64_t *bytes);

#ifdef __cplusplus
}
#endif

#endif /* ZERO_SHARD_BLOCK_H_ */
