// C-ABI entry points of zero_shard_block.h: argument checks and dispatch.
//
// Every check runs before anything is enqueued.  No C++ exception crosses the
// boundary (nothing here allocates or throws).
#include <hip/hip_runtime_api.h>

#include <cmath>

#include "block_launch.h"
#include "views.h"

using namespace zs;

namespace {

constexpr View kNone{nullptr, 0, 0, 0};

uint64_t blocks_of(uint64_t n, uint64_t block) { return (n + block - 1) / block; }

bool is_blocks(zero_blocks b) { return b == ZERO_BLOCKS_ROW || b == ZERO_BLOCKS_SQUARE; }

View codes(const uint8_t *q, uint64_t rows, uint64_t cols) { return vec(q, rows * cols, 1); }
View exponents(const uint8_t *e, zero_blocks blocks, uint64_t rows, uint64_t cols) {
    const uint64_t tall = blocks == ZERO_BLOCKS_SQUARE ? blocks_of(rows, ZERO_BLOCK) : rows;
    return vec(e, tall * blocks_of(cols, ZERO_BLOCK), 1);
}

}  // namespace

extern "C" int zero_block_quant(uint8_t *q, uint8_t *e, uint8_t *qt, uint8_t *et, const void *x,
                                uint64_t ldx, zero_dtype dt, zero_blocks blocks, uint64_t rows,
                                uint64_t cols, void *stream) {
    if (!is_any(dt)) return ZERO_EDTYPE;
    if (!is_blocks(blocks) || !extent(rows) || !extent(cols)) return ZERO_EINVAL;
    if ((qt == nullptr) != (et == nullptr)) return ZERO_EINVAL;
    if (qt != nullptr && blocks != ZERO_BLOCKS_SQUARE) return ZERO_EINVAL;
    if (rows == 0 || cols == 0) return ZERO_OK;
    const uint64_t b = bytes_of(dt);
    if (q == nullptr || e == nullptr || !matrix_ok(x, rows, cols, ldx, b)) return ZERO_EINVAL;
    const View out[4] = {codes(q, rows, cols), exponents(e, blocks, rows, cols),
                         qt != nullptr ? codes(qt, cols, rows) : kNone,
                         qt != nullptr ? exponents(et, blocks, cols, rows) : kNone};
    const View in[1] = {mat(x, rows, cols, ldx, b)};
    if (!apart(out, 4, in, 1)) return ZERO_EINVAL;
    return done(launch_block_quant(q, e, qt, et, x, ldx, static_cast<int>(dt),
                                   blocks == ZERO_BLOCKS_SQUARE, rows, cols,
                                   static_cast<hipStream_t>(stream)),
                "zero_block_quant launch");
}

extern "C" int zero_block_load(void *x, uint64_t ldx, zero_dtype dt, const uint8_t *q,
                               const uint8_t *e, zero_blocks blocks, uint64_t rows, uint64_t cols,
                               void *stream) {
    if (!is_any(dt)) return ZERO_EDTYPE;
    if (!is_blocks(blocks) || !extent(rows) || !extent(cols)) return ZERO_EINVAL;
    if (rows == 0 || cols == 0) return ZERO_OK;
    const uint64_t b = bytes_of(dt);
    if (q == nullptr || e == nullptr || !matrix_ok(x, rows, cols, ldx, b)) return ZERO_EINVAL;
    const View out[1] = {mat(x, rows, cols, ldx, b)};
    const View in[2] = {codes(q, rows, cols), exponents(e, blocks, rows, cols)};
    if (!apart(out, 1, in, 2)) return ZERO_EINVAL;
    return done(launch_block_load(x, ldx, static_cast<int>(dt), q, e,
                                  blocks == ZERO_BLOCKS_SQUARE, rows, cols,
                                  static_cast<hipStream_t>(stream)),
                "zero_block_load launch");
}

extern "C" int zero_block_product_workspace(uint64_t m, uint64_t n, uint64_t k, uint64_t *bytes) {
    if (bytes == nullptr || !extent(m) || !extent(n) || !extent(k)) return ZERO_EINVAL;
    *bytes = m == 0 || n == 0 || k == 0 ? 0 : product_workspace(m, n, k);
    return ZERO_OK;
}

extern "C" int zero_block_product(void *y, uint64_t ldy, zero_dtype dt, const uint8_t *qa,
                                  const uint8_t *ea, uint32_t a_block, const uint8_t *qb,
                                  const uint8_t *eb, uint64_t m, uint64_t n, uint64_t k,
                                  void *workspace, uint64_t workspace_bytes, void *stream) {
    if (!is_any(dt)) return ZERO_EDTYPE;
    if (a_block != ZERO_BLOCK && a_block != ZERO_ACT_BLOCK) return ZERO_EINVAL;
    if (!extent(m) || !extent(n) || !extent(k)) return ZERO_EINVAL;
    if (m == 0 || n == 0) return ZERO_OK;
    const uint64_t b = bytes_of(dt);
    if (!matrix_ok(y, m, n, ldy, b)) return ZERO_EINVAL;
    if (k == 0)
        return done(launch_zero_matrix(y, ldy, static_cast<int>(dt), m, n,
                                       static_cast<hipStream_t>(stream)),
                    "zero_block_product launch");
    if (qa == nullptr || ea == nullptr || qb == nullptr || eb == nullptr) return ZERO_EINVAL;
    const uint64_t need = product_workspace(m, n, k);
    if (workspace_ok(workspace, workspace_bytes, need) != ZERO_OK) return ZERO_EINVAL;
    const View out[2] = {mat(y, m, n, ldy, b), vec(workspace, need, 1)};
    const View in[4] = {codes(qa, m, k), vec(ea, m * blocks_of(k, a_block), 1), codes(qb, n, k),
                        exponents(eb, ZERO_BLOCKS_SQUARE, n, k)};
    if (!apart(out, 2, in, 4)) return ZERO_EINVAL;
    const ProductArgs a{y, qa, ea, qb, eb, ldy, m, n, k, a_block, workspace};
    return done(launch_product(a, static_cast<int>(dt), static_cast<hipStream_t>(stream)),
                "zero_block_product launch");
}

namespace {

bool mask_ok(float p, const uint64_t *d_offset) {
    return p >= 0.0f && p <= 1.0f && aligned(d_offset, 8);
}

Mask mask_of(float p, uint64_t seed, uint64_t offset, const uint64_t *d_offset) {
    // p 2^16 is exact in FP32 (down to where it rounds to 0), rintf rounds halves to even
    const uint32_t t = static_cast<uint32_t>(std::rint(p * 65536.0f));
    const float factor = t < 65536 ? 65536.0f / static_cast<float>(65536 - t) : 0.0f;
    return Mask{t, factor, seed, offset, d_offset};
}

View offset_view(const uint64_t *d_offset) { return vec(d_offset, d_offset != nullptr ? 1 : 0, 8); }

}  // namespace

extern "C" int zero_dropout(void *y, uint64_t ldy, const void *x, uint64_t ldx, zero_dtype dt,
                            uint64_t rows, uint64_t cols, float p, uint64_t seed, uint64_t offset,
                            const uint64_t *d_offset, void *stream) {
    if (!is_any(dt)) return ZERO_EDTYPE;
    if (!mask_ok(p, d_offset) || !extent(rows) || !extent(cols)) return ZERO_EINVAL;
    if (rows == 0 || cols == 0) return ZERO_OK;
    const uint64_t b = bytes_of(dt);
    if (!matrix_ok(y, rows, cols, ldy, b) || !matrix_ok(x, rows, cols, ldx, b))
        return ZERO_EINVAL;
    const View out = mat(y, rows, cols, ldy, b), in = mat(x, rows, cols, ldx, b);
    if (meet(out, in) && !same(y, ldy, x, ldx)) return ZERO_EINVAL;
    if (meet(out, offset_view(d_offset))) return ZERO_EINVAL;
    return done(launch_dropout(y, ldy, x, ldx, static_cast<int>(dt), rows, cols,
                               mask_of(p, seed, offset, d_offset),
                               static_cast<hipStream_t>(stream)),
                "zero_dropout launch");
}

namespace {

bool is_norm(zero_norm n) {
    return n == ZERO_NORM_NONE || n == ZERO_NORM_RMS || n == ZERO_NORM_LAYER;
}

// What both passes check of the block's description.  Parameters are looked at by
// their pointers only where there is a column.
int block_ok(const zero_residual *b, bool have_f) {
    if (b == nullptr) return ZERO_EINVAL;
    if (!is_any(b->dt) || (b->res_dt != b->dt && b->res_dt != ZERO_F32)) return ZERO_EDTYPE;
    if (!is_norm(b->post) || !is_norm(b->pre) || !extent(b->rows) || !extent(b->cols))
        return ZERO_EINVAL;
    if (!(b->eps >= 0x1p-80f) || !std::isfinite(b->eps) || !std::isfinite(b->res_scale) ||
        !mask_ok(b->p, b->d_offset))
        return ZERO_EINVAL;
    if (b->post == ZERO_NORM_NONE && (b->post_weight != nullptr || b->post_bias != nullptr))
        return ZERO_EINVAL;
    if (b->pre == ZERO_NORM_NONE && (b->pre_weight != nullptr || b->pre_bias != nullptr))
        return ZERO_EINVAL;
    if (!have_f && (b->post != ZERO_NORM_NONE || b->pre == ZERO_NORM_NONE || b->gate != nullptr ||
                    b->res_scale != 1.0f || b->p != 0.0f))
        return ZERO_EINVAL;
    const void *params[5] = {b->post_weight, b->post_bias, b->gate, b->pre_weight, b->pre_bias};
    for (const void *p : params)
        if (!aligned(p, bytes_of(b->dt))) return ZERO_EINVAL;
    return ZERO_OK;
}

View param(const void *p, const zero_residual *b, zero_dtype dt) {
    return vec(p, p != nullptr ? b->cols : 0, bytes_of(dt));
}

ResidualArgs args_of(const zero_residual *b) {
    ResidualArgs a{};
    a.rows = b->rows;
    a.cols = static_cast<uint32_t>(b->cols);
    a.fmt = static_cast<int>(b->dt);
    a.res32 = b->res_dt == ZERO_F32 && b->dt != ZERO_F32;
    a.post = static_cast<int>(b->post);
    a.pre = static_cast<int>(b->pre);
    a.w1 = b->post_weight;
    a.b1 = b->post_bias;
    a.gate = b->gate;
    a.w2 = b->pre_weight;
    a.b2 = b->pre_bias;
    a.eps = b->eps;
    a.res_scale = b->res_scale;
    a.mask = mask_of(b->p, b->seed, b->offset, b->d_offset);
    return a;
}

}  // namespace

extern "C" int zero_residual_norm(void *u, uint64_t ldu, void *h, uint64_t ldh, float *stats,
                                  const void *r, uint64_t ldr, const void *f, uint64_t ldf,
                                  const zero_residual *block, void *stream) {
    // an empty matrix may come without its pointer, so nothing is read from there being none
    const bool empty = block != nullptr && (block->rows == 0 || block->cols == 0);
    const int rc = block_ok(block, f != nullptr || empty);
    if (rc != ZERO_OK) return rc;
    const uint64_t rows = block->rows, cols = block->cols;
    if (empty) return ZERO_OK;
    if ((u != nullptr) != (f != nullptr) || (h != nullptr) != (block->pre != ZERO_NORM_NONE))
        return ZERO_EINVAL;
    const uint64_t b = bytes_of(block->dt), rb = bytes_of(block->res_dt);
    if (!matrix_ok(r, rows, cols, ldr, rb) ||
        (f != nullptr && (!matrix_ok(f, rows, cols, ldf, b) || !matrix_ok(u, rows, cols, ldu, rb))) ||
        (h != nullptr && !matrix_ok(h, rows, cols, ldh, b)) || !aligned(stats, 4))
        return ZERO_EINVAL;
    const View vr = mat(r, rows, cols, ldr, rb);
    const View out[3] = {f != nullptr ? mat(u, rows, cols, ldu, rb) : kNone,
                         h != nullptr ? mat(h, rows, cols, ldh, b) : kNone,
                         vec(stats, stats != nullptr ? rows * 4 : 0, 4)};
    const View in[7] = {f != nullptr ? mat(f, rows, cols, ldf, b) : kNone,
                        param(block->post_weight, block, block->dt),
                        param(block->post_bias, block, block->dt),
                        param(block->gate, block, block->dt),
                        param(block->pre_weight, block, block->dt),
                        param(block->pre_bias, block, block->dt),
                        offset_view(block->d_offset)};
    if (!apart(out, 3, in, 7) || meet(out[1], vr) || meet(out[2], vr)) return ZERO_EINVAL;
    if (meet(out[0], vr) && !same(u, ldu, r, ldr)) return ZERO_EINVAL;
    ResidualArgs a = args_of(block);
    a.f = f;
    a.ldf = ldf;
    a.stats = stats;
    a.r = r;
    a.u_out = u;
    a.h = h;
    a.ldr = ldr;
    a.ldu = ldu;
    a.ldh = ldh;
    return done(launch_residual_forward(a, static_cast<hipStream_t>(stream)),
                "zero_residual_norm launch");
}

extern "C" int zero_residual_norm_workspace(uint64_t rows, uint64_t cols, uint64_t *bytes) {
    if (bytes == nullptr || !extent(rows) || !extent(cols)) return ZERO_EINVAL;
    *bytes = rows == 0 || cols == 0 ? 0 : residual_workspace(rows, cols);
    return ZERO_OK;
}

extern "C" int zero_residual_norm_backward(
    void *df, uint64_t lddf, void *dr, uint64_t lddr, const zero_residual_grads *grads,
    zero_dtype grad_dt, int32_t first, const void *dh, uint64_t lddh, const void *du, uint64_t lddu,
    const void *f, uint64_t ldf, const void *u, uint64_t ldu, const float *stats,
    const zero_residual *block, void *workspace, uint64_t workspace_bytes, void *stream) {
    const bool empty = block != nullptr && (block->rows == 0 || block->cols == 0);
    const int rc = block_ok(block, f != nullptr || empty);
    if (rc != ZERO_OK) return rc;
    if (!grad_format_ok(grad_dt, block->dt)) return ZERO_EDTYPE;
    if (grad_dt != ZERO_F32 && first == 0) return ZERO_EINVAL;
    if (block->cols == 0) return ZERO_OK;
    if (!empty &&
        ((df != nullptr) != (f != nullptr) || (dh != nullptr) != (block->pre != ZERO_NORM_NONE) ||
         (dh == nullptr && du == nullptr)))
        return ZERO_EINVAL;
    zero_residual_grads none{};
    const zero_residual_grads &g = grads != nullptr ? *grads : none;
    const uint64_t rows = block->rows, cols = block->cols;
    const uint64_t b = bytes_of(block->dt), rb = bytes_of(block->res_dt), gb = bytes_of(grad_dt);
    void *const asked[5] = {g.post_weight, g.post_bias, g.gate, g.pre_weight, g.pre_bias};
    const void *const given[5] = {block->post_weight, block->post_bias, block->gate,
                                  block->pre_weight, block->pre_bias};
    for (int i = 0; i < 5; ++i)
        if (!aligned(asked[i], gb) || (asked[i] != nullptr && given[i] == nullptr))
            return ZERO_EINVAL;
    View out[8] = {kNone, kNone, kNone};
    for (int i = 0; i < 5; ++i) out[3 + i] = param(asked[i], block, grad_dt);
    const uint64_t need = rows == 0 ? 0 : residual_workspace(rows, cols);
    View in[10];
    for (int i = 0; i < 5; ++i) in[i] = param(given[i], block, block->dt);
    in[5] = offset_view(block->d_offset);
    in[6] = in[7] = in[8] = in[9] = kNone;
    View vdh = kNone, vdu = kNone;
    if (rows > 0) {
        if (!matrix_ok(dr, rows, cols, lddr, rb) || !matrix_ok(u, rows, cols, ldu, rb) ||
            (f != nullptr &&
             (!matrix_ok(f, rows, cols, ldf, b) || !matrix_ok(df, rows, cols, lddf, b))) ||
            (dh != nullptr && !matrix_ok(dh, rows, cols, lddh, b)) ||
            (du != nullptr && !matrix_ok(du, rows, cols, lddu, rb)) || stats == nullptr ||
            !aligned(stats, 4))
            return ZERO_EINVAL;
        if (workspace_ok(workspace, workspace_bytes, need) != ZERO_OK) return ZERO_EINVAL;
        out[0] = mat(dr, rows, cols, lddr, rb);
        out[1] = f != nullptr ? mat(df, rows, cols, lddf, b) : kNone;
        out[2] = vec(workspace, need, 1);
        in[6] = mat(u, rows, cols, ldu, rb);
        in[7] = f != nullptr ? mat(f, rows, cols, ldf, b) : kNone;
        in[8] = vec(stats, rows * 4, 4);
        vdh = dh != nullptr ? mat(dh, rows, cols, lddh, b) : kNone;
        vdu = du != nullptr ? mat(du, rows, cols, lddu, rb) : kNone;
    }
    if (!apart(out, 8, in, 9)) return ZERO_EINVAL;
    for (int i = 0; i < 8; ++i) {
        if (meet(out[i], vdh) && !(i == 1 && same(df, lddf, dh, lddh))) return ZERO_EINVAL;
        if (meet(out[i], vdu) && !(i == 0 && same(dr, lddr, du, lddu))) return ZERO_EINVAL;
    }
    if (rows == 0) {
        for (void *p : asked) {
            if (p == nullptr || first == 0) continue;
            const int r0 = done(launch_zero_fill(p, static_cast<int>(gb), cols,
                                                 static_cast<hipStream_t>(stream)),
                                "zero_residual_norm_backward launch");
            if (r0 != ZERO_OK) return r0;
        }
        return ZERO_OK;
    }
    ResidualArgs a = args_of(block);
    a.f = f;
    a.ldf = ldf;
    a.stats = const_cast<float *>(stats);
    a.u = u;
    a.ldu = ldu;
    a.dh = dh;
    a.lddh = lddh;
    a.du = du;
    a.lddu = lddu;
    a.df = df;
    a.lddf = lddf;
    a.dr = dr;
    a.lddr = lddr;
    a.dw1 = g.post_weight;
    a.db1 = g.post_bias;
    a.dgate = g.gate;
    a.dw2 = g.pre_weight;
    a.db2 = g.pre_bias;
    a.grad32 = grad_dt == ZERO_F32;
    a.first = first != 0;
    a.workspace = workspace;
    return done(launch_residual_backward(a, static_cast<hipStream_t>(stream)),
                "zero_residual_norm_backward launch");
}
