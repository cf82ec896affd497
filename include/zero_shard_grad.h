/*
 * zero_shard_grad.h -- C ABI of the operators that make a rank's gradients, on
 * an MI355X (gfx950).  They stand before the overflow check and the step of
 * zero_shard.h: the policy loss multiplies in the loss scale S, the weight and
 * embedding gradients land in the flat gradient buffer (16-bit, or the FP32
 * accumulator), and the activations that the backward pass needs are kept in
 * 8 bits meanwhile.
 *
 * Conventions: those of zero_shard.h (return codes, zero_strerror, the caller
 * owns every buffer, work is enqueued on `stream` of the current device and
 * the call returns without synchronising, calls are thread-safe and keep
 * nothing between calls, argument errors are found before anything is
 * enqueued), and
 *   - A matrix of `rows` rows and `cols` columns has unit column stride and a
 *     row stride ("ld", in elements) of at least cols.  Where no ld is given
 *     the matrix is contiguous.  Only its rows*cols elements are touched: the
 *     gap between rows, and what follows the last row, stay as they were.
 *   - Any element-aligned pointer is accepted (2 bytes for 16-bit formats, 4
 *     for FP32 and int32, 8 for int64), so a matrix may start anywhere in a
 *     flat buffer.
 *   - Matrices of one call may not overlap, except where a function says so;
 *     overlaps are rejected with ZERO_EINVAL.  (Two matrices with the same row
 *     stride in bytes may interleave: columns [0, a) and [a, b) of one buffer.
 *     Otherwise a matrix counts as all bytes from its first element to its
 *     last, the gaps between its rows included.)
 *   - Extents (rows, columns, tokens, vocabulary, ...) are at most
 *     ZERO_MAX_EXTENT, and a matrix spans less than 2^56 bytes.
 *   - Results are repeatable bit for bit: every sum is taken in an order that
 *     the arguments fix, and no floating-point atomics are used.
 *   - Two calls that overlap in time need workspaces of their own, and so do
 *     two captured graphs that may run at once.
 */
#ifndef ZERO_SHARD_GRAD_H_
#define ZERO_SHARD_GRAD_H_

#include "zero_shard.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ZERO_MAX_EXTENT 0x7fffffffull /* largest rows, cols, tokens, vocabulary */

/* Format of token ids. */
typedef enum { ZERO_I32 = 0, ZERO_I64 = 1 } zero_itype;

/* ---------------------------------------------------------------------------
 * Activation checkpoints in 8 bits.
 *
 * A checkpoint of x[rows, cols] is q[rows, cols], one e4m3 code an element
 * (1 sign, 4 exponent, 3 mantissa bits; largest 448, no infinity), and
 * e[rows, ceil(cols/32)], one exponent byte for each block of 32 neighbours of
 * a row (the last block of a row may be shorter), both contiguous: 33/32 bytes
 * an element instead of 2 or 4.  The value an element stands for is
 *     code * 2^(e - 127)
 * (e is 3 to 247 as written here; other bytes have no defined value).
 * Writing takes for each block the smallest k >= -124 with
 * max|x| <= 448 * 2^k over the block's finite elements, e = k + 127, and
 * rounds x / 2^k to nearest even.  The block scale is a power of two, so
 * neither the division nor reading back rounds: the one rounding is the
 * code's, at most 2^-4 of the value (or 2^(k-10) absolute for the smallest).
 * Magnitudes above 15/16 * 2^16 (FP16) or 15/16 * 2^128 (BF16, FP32) are held
 * at that value, which keeps them inside the same 2^-4.  So every value a
 * checkpoint stands for is a finite number of the format it was written from,
 * exactly (for FP32: of BF16 too).  An infinity or NaN is kept as NaN, so
 * that gradients made from it still raise the overflow check; it does not
 * disturb its block's other elements.
 * ------------------------------------------------------------------------- */
#define ZERO_ACT_BLOCK 32

typedef enum {
    ZERO_ACT_NONE = 0, /* the identity: only the checkpoint is written */
    ZERO_ACT_GELU = 1, /* x * s(2u), u = sqrt(2/pi) * (x + 0.044715 x^3), s(t) = 1/(1+e^-t):
                          the tanh form 0.5 x (1 + tanh u) */
    ZERO_ACT_SILU = 2  /* x * s(x) */
} zero_act;

/*
 * zero_act_save -- write the checkpoint (q, e) of x and, with an activation
 * function, y = act(x) computed from x itself (FP32, rounded once to dt), in
 * one pass: the forward pass of an activation that keeps its input in 8 bits.
 *   q   device, rows*cols bytes; e  device, rows*ceil(cols/32) bytes.
 *   x   device, format dt (F16, BF16 or F32), row stride ldx.
 *   y   device, format dt, row stride ldy; required iff act != ZERO_ACT_NONE,
 *       otherwise NULL.  y may be exactly x (same pointer and stride).
 *   rows == 0 or cols == 0: no-op.
 *   Errors: ZERO_EDTYPE; ZERO_EINVAL for a bad act, a NULL or misaligned
 *   pointer, a y with ZERO_ACT_NONE, ldx or ldy < cols, an extent past its
 *   limit, or an overlap; ZERO_EHIP.
 */
int zero_act_save(uint8_t *q, uint8_t *e, void *y, uint64_t ldy, const void *x, uint64_t ldx,
                  zero_dtype dt, zero_act act, uint64_t rows, uint64_t cols, void *stream);

/*
 * zero_act_load -- x = the values a checkpoint stands for, rounded once to dt
 * (exact where dt is the format it was written from, or holds it).
 *   Errors: as zero_act_save.
 */
int zero_act_load(void *x, uint64_t ldx, zero_dtype dt, const uint8_t *q, const uint8_t *e,
                  uint64_t rows, uint64_t cols, void *stream);

/*
 * zero_act_backward -- dx = dy * act'(v), v the value the checkpoint stands
 * for, in FP32, rounded once to dt.  dx may be exactly dy.
 *   Errors: as zero_act_save; ZERO_EINVAL also for ZERO_ACT_NONE.
 */
int zero_act_backward(void *dx, uint64_t lddx, const void *dy, uint64_t lddy, zero_dtype dt,
                      zero_act act, const uint8_t *q, const uint8_t *e, uint64_t rows,
                      uint64_t cols, void *stream);

/*
 * zero_weight_grad -- weight gradient of a linear layer y = x W^T whose input
 * x[tokens, n_in] is kept as a checkpoint:
 *     G[o, i] = sum over t of dy[t, o] * v[t, i]
 * products exact, sums FP32.  dw is the layer's place in the flat gradient
 * buffer, [n_out, n_in] contiguous:
 *   dw_dt == dt (16-bit):  dw = G rounded once; first must be non-zero.
 *   dw_dt == ZERO_F32:     dw = G when first is non-zero, dw + G (one FP32
 *                          addition) otherwise, as zero_grad_accumulate.
 *   dy   device, 16-bit format dt, [tokens, n_out], row stride lddy.
 *   q, e the checkpoint; written from FP16 activations for dt == ZERO_F16 and
 *        from BF16 or FP32 ones for ZERO_BF16 (a value that FP16 does not hold
 *        is rounded to it, to infinity past its range).
 *   workspace  device, workspace_bytes >= zero_weight_grad_workspace's answer,
 *        16-byte aligned; may be NULL if that is 0.  Its contents before the
 *        call do not matter.
 *   tokens == 0: dw = 0 when first, else no-op.  n_out or n_in == 0: no-op.
 *   Row strides or n_in of 2^24 elements and more, and extents below 8, are
 *   correct but several times slower.
 *   Errors: ZERO_EDTYPE for a dt that is not 16-bit or a dw_dt that is neither
 *   dt nor ZERO_F32; ZERO_EINVAL as above, for first == 0 with a 16-bit dw and
 *   for a small or misaligned workspace; ZERO_EHIP.
 */
int zero_weight_grad(void *dw, zero_dtype dw_dt, int32_t first, const void *dy, uint64_t lddy,
                     zero_dtype dt, const uint8_t *q, const uint8_t *e, uint64_t tokens,
                     uint64_t n_out, uint64_t n_in, void *workspace, uint64_t workspace_bytes,
                     void *stream);

/* zero_weight_grad_workspace -- bytes zero_weight_grad needs for these extents,
 * whatever the formats.  Host only.  Errors: ZERO_EINVAL for an extent past its
 * limit or a NULL bytes. */
int zero_weight_grad_workspace(uint64_t tokens, uint64_t n_out, uint64_t n_in, uint64_t *bytes);

/* ---------------------------------------------------------------------------
 * Embedding.
 * ------------------------------------------------------------------------- */

/*
 * zero_embed_lookup -- out[t, :] = scale * table[ids[t], :], in FP32, rounded
 * once to dt; zeros where ids[t] is outside [0, vocab) (a padding position).
 *   out    device, format dt (F16, BF16 or F32), [tokens, width], row stride ldo.
 *   table  device, format dt, [vocab, width] contiguous (its place in w16).
 *   ids    device, tokens ids of format it, contiguous.
 *   tokens == 0 or width == 0: no-op.  vocab == 0: every id is outside.
 *   Errors: ZERO_EDTYPE for a bad dt or it; ZERO_EINVAL; ZERO_EHIP.
 */
int zero_embed_lookup(void *out, uint64_t ldo, const void *table, zero_dtype dt, const void *ids,
                      zero_itype it, uint64_t tokens, uint64_t vocab, uint64_t width, float scale,
                      void *stream);

/*
 * zero_embed_grad -- gradient of that lookup with respect to the table:
 *     G[v, :] = scale * (sum over t with ids[t] == v of dy[t, :])
 * the sum in FP32 over the tokens sorted by id, equal ids by position, in an
 * order that the ids fix.  dw is the table's place in the flat gradient buffer,
 * [vocab, width] contiguous:
 *   dw_dt == dt (16-bit):  dw = G rounded once, zeros for ids that do not
 *                          occur; first must be non-zero.
 *   dw_dt == ZERO_F32:     dw = G when first is non-zero; otherwise dw + G (one
 *                          FP32 addition) in the rows whose id occurs, and the
 *                          others are not touched.
 *   dy   device, 16-bit format dt, [tokens, width], row stride lddy.
 *   ids  as for the lookup; positions outside [0, vocab) are ignored (their
 *        dy is not read).
 *   workspace  as for zero_weight_grad (zero_embed_grad_workspace).
 *   vocab == 0 or width == 0: no-op.
 *   Errors: as zero_weight_grad; ZERO_EDTYPE also for a bad it.
 */
int zero_embed_grad(void *dw, zero_dtype dw_dt, int32_t first, const void *dy, uint64_t lddy,
                    zero_dtype dt, const void *ids, zero_itype it, uint64_t tokens,
                    uint64_t vocab, uint64_t width, float scale, void *workspace,
                    uint64_t workspace_bytes, void *stream);

/* zero_embed_grad_workspace -- bytes zero_embed_grad needs for these extents,
 * whatever the formats.  Host only.  Errors: ZERO_EINVAL. */
int zero_embed_grad_workspace(uint64_t tokens, uint64_t vocab, uint64_t width, uint64_t *bytes);

/* ---------------------------------------------------------------------------
 * Policy loss.
 * ------------------------------------------------------------------------- */

/*
 * zero_policy_loss -- clipped policy loss with a KL term over `rows` sampled
 * tokens, and its gradient times the loss scale.  For row t with logits z, the
 * sampled token a = targets[t], advantage A and weight w:
 *     logp  = z[a] - log(sum over v of e^z[v])
 *     r     = e^(logp - old_logp)          (1 where old_logp is NULL: on policy)
 *     d     = ref_logp - logp              (0 where ref_logp is NULL)
 *     L     = max(-r A, -clamp(r, 1 - clip_low, 1 + clip_high) A)
 *             + kl_coef * (e^d - d - 1)
 *     loss  = sum over t of w L            (FP64, in a fixed order, rounded once)
 *     dlogits[v] = S w g ([v == a] - e^(z[v]) / sum)
 *     g     = kl_coef * (1 - e^d) - (0 where the clamp cuts r off, r A elsewhere)
 * where the clamp cuts off for A > 0 and r > 1 + clip_high, and for A < 0 and
 * r < 1 - clip_low.  FP32 throughout, dlogits rounded once to dt.  The caller
 * puts any averaging into w (a mask divided by the token count).
 *   A row with w == 0 is skipped: its logits, target and other inputs may hold
 *   anything, its token_loss and logp become 0 and its dlogits zeros.  In any
 *   other row a target outside [0, vocab) gives NaN in the row and the loss,
 *   as do infinities and NaN by the formulas (logits of -inf stand for
 *   excluded tokens and get a zero gradient), so that the overflow check sees
 *   them.
 *   loss        device FP32, one value.
 *   token_loss  device FP32, rows values: L.   logp  device FP32, rows values.
 *   dlogits     device, format dt, row stride ldd, or NULL for the loss only;
 *               may be exactly logits.
 *   logits      device, format dt (F16, BF16 or F32), [rows, vocab], row stride ld.
 *   targets     device, rows ids of format it.
 *   old_logp, ref_logp  device FP32, rows values, or NULL.
 *   advantage, weight   device FP32, rows values.
 *   clip_low in [0, 1], clip_high >= 0 (infinity: no cut), kl_coef finite (0:
 *   ref_logp has no effect, whatever it holds), loss_scale > 0 and finite.
 *   rows == 0: loss = 0.
 *   Errors: ZERO_EDTYPE for a bad dt or it; ZERO_EINVAL for vocab == 0 with
 *   rows > 0, a NULL ref_logp with kl_coef != 0, and as above; ZERO_EHIP.
 */
int zero_policy_loss(float *loss, float *token_loss, float *logp, void *dlogits, uint64_t ldd,
                     const void *logits, uint64_t ld, zero_dtype dt, const void *targets,
                     zero_itype it, const float *old_logp, const float *ref_logp,
                     const float *advantage, const float *weight, uint64_t rows, uint64_t vocab,
                     float clip_low, float clip_high, float kl_coef, float loss_scale,
                     void *stream);

/*
 * zero_policy_loss_dev -- zero_policy_loss with S read from
 * d_ctl->scaler.loss_scale on the device, for the device-resident sequence
 * (zero_overflow_check_dev, zero_scaler_update_dev and zero_adam_step_dev
 * follow).  d_ctl is read only and may not overlap an output.
 */
int zero_policy_loss_dev(float *loss, float *token_loss, float *logp, void *dlogits, uint64_t ldd,
                         const void *logits, uint64_t ld, zero_dtype dt, const void *targets,
                         zero_itype it, const float *old_logp, const float *ref_logp,
                         const float *advantage, const float *weight, uint64_t rows,
                         uint64_t vocab, float clip_low, float clip_high, float kl_coef,
                         const zero_device_ctl *d_ctl, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* ZERO_SHARD_GRAD_H_ */
