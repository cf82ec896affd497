// C-ABI entry points of zero_shard_grad.h: argument checks and dispatch.
//
// Every check runs before anything is enqueued.  No C++ exception crosses the
// boundary (nothing here allocates or throws).
#include <hip/hip_runtime_api.h>

#include <cmath>

#include "grad_launch.h"
#include "zero_shard_grad.h"

namespace {

bool aligned(const void *p, uint64_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

uint64_t bytes_of(zero_dtype dt) { return dt == ZERO_F32 ? 4 : 2; }
bool is_16(zero_dtype dt) { return dt == ZERO_F16 || dt == ZERO_BF16; }
bool is_any(zero_dtype dt) { return is_16(dt) || dt == ZERO_F32; }
bool is_id(zero_itype it) { return it == ZERO_I32 || it == ZERO_I64; }

constexpr uint64_t kMaxBytes = 1ull << 56;

// A matrix view in bytes: rows of `width` bytes, `stride` bytes apart.
struct View {
    const void *p;
    uint64_t rows, width, stride;
    // bytes from the first element to the end of the last row
    uint64_t span() const { return rows == 0 || width == 0 ? 0 : (rows - 1) * stride + width; }
};

View vec(const void *p, uint64_t n, uint64_t elem) { return View{p, 1, n * elem, n * elem}; }

// Extents at most ZERO_MAX_EXTENT, ld at least cols, and a span below 2^56 bytes.
bool matrix_ok(const void *p, uint64_t rows, uint64_t cols, uint64_t ld, uint64_t elem) {
    if (p == nullptr || !aligned(p, elem)) return false;
    if (ld < cols || ld >= kMaxBytes / 8) return false;
    const unsigned __int128 span =
        (static_cast<unsigned __int128>(rows - 1) * ld + cols) * elem;
    return span < kMaxBytes;
}

View mat(const void *p, uint64_t rows, uint64_t cols, uint64_t ld, uint64_t elem) {
    return View{p, rows, cols * elem, ld * elem};
}

// Some byte belongs to both.  Two matrices of one stride whose columns do not
// meet are apart although their spans cross.
bool meet(const View &a, const View &b) {
    const uint64_t na = a.span(), nb = b.span();
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    if (na == 0 || nb == 0 || x >= y + nb || y >= x + na) return false;
    if (a.rows > 1 && b.rows > 1 && a.stride == b.stride) {
        const View &lo = x <= y ? a : b, &hi = x <= y ? b : a;
        const uint64_t d = (x <= y ? y - x : x - y) % a.stride;   // hi's column after lo's
        if (d >= lo.width && d + hi.width <= a.stride) return false;
    }
    return true;
}

// Every output apart from every other view.
bool apart(const View *out, int n_out, const View *in, int n_in) {
    for (int i = 0; i < n_out; ++i) {
        for (int j = i + 1; j < n_out; ++j)
            if (meet(out[i], out[j])) return false;
        for (int j = 0; j < n_in; ++j)
            if (meet(out[i], in[j])) return false;
    }
    return true;
}

bool extent(uint64_t n) { return n <= ZERO_MAX_EXTENT; }

int done(hipError_t e, const char *what) { return e == hipSuccess ? ZERO_OK : zs::fail_hip(e, what); }

uint64_t act_blocks(uint64_t cols) { return (cols + ZERO_ACT_BLOCK - 1) / ZERO_ACT_BLOCK; }

View codes(const uint8_t *q, uint64_t rows, uint64_t cols) { return vec(q, rows * cols, 1); }
View exponents(const uint8_t *e, uint64_t rows, uint64_t cols) {
    return vec(e, rows * act_blocks(cols), 1);
}

bool same(const void *a, uint64_t lda, const void *b, uint64_t ldb) { return a == b && lda == ldb; }

}  // namespace

extern "C" int zero_act_save(uint8_t *q, uint8_t *e, void *y, uint64_t ldy, const void *x,
                             uint64_t ldx, zero_dtype dt, zero_act act, uint64_t rows,
                             uint64_t cols, void *stream) {
    if (!is_any(dt)) return ZERO_EDTYPE;
    if (act != ZERO_ACT_NONE && act != ZERO_ACT_GELU && act != ZERO_ACT_SILU) return ZERO_EINVAL;
    if (!extent(rows) || !extent(cols)) return ZERO_EINVAL;
    if (act == ZERO_ACT_NONE && y != nullptr) return ZERO_EINVAL;
    if (rows == 0 || cols == 0) return ZERO_OK;
    const uint64_t b = bytes_of(dt);
    if (q == nullptr || e == nullptr || !matrix_ok(x, rows, cols, ldx, b)) return ZERO_EINVAL;
    View out[3] = {codes(q, rows, cols), exponents(e, rows, cols), View{nullptr, 0, 0, 0}};
    const View in[1] = {mat(x, rows, cols, ldx, b)};
    if (act != ZERO_ACT_NONE) {
        if (!matrix_ok(y, rows, cols, ldy, b)) return ZERO_EINVAL;
        out[2] = mat(y, rows, cols, ldy, b);
        if (meet(out[2], in[0]) && !same(y, ldy, x, ldx)) return ZERO_EINVAL;
        if (meet(out[2], out[0]) || meet(out[2], out[1])) return ZERO_EINVAL;
    }
    if (!apart(out, 2, in, 1)) return ZERO_EINVAL;
    return done(zs::launch_act_save(q, e, y, ldy, x, ldx, static_cast<int>(dt),
                                    static_cast<int>(act), rows, cols,
                                    static_cast<hipStream_t>(stream)),
                "zero_act_save launch");
}

extern "C" int zero_act_load(void *x, uint64_t ldx, zero_dtype dt, const uint8_t *q,
                             const uint8_t *e, uint64_t rows, uint64_t cols, void *stream) {
    if (!is_any(dt)) return ZERO_EDTYPE;
    if (!extent(rows) || !extent(cols)) return ZERO_EINVAL;
    if (rows == 0 || cols == 0) return ZERO_OK;
    const uint64_t b = bytes_of(dt);
    if (q == nullptr || e == nullptr || !matrix_ok(x, rows, cols, ldx, b)) return ZERO_EINVAL;
    const View out[1] = {mat(x, rows, cols, ldx, b)};
    const View in[2] = {codes(q, rows, cols), exponents(e, rows, cols)};
    if (!apart(out, 1, in, 2)) return ZERO_EINVAL;
    return done(zs::launch_act_load(x, ldx, static_cast<int>(dt), q, e, rows, cols,
                                    static_cast<hipStream_t>(stream)),
                "zero_act_load launch");
}

extern "C" int zero_act_backward(void *dx, uint64_t lddx, const void *dy, uint64_t lddy,
                                 zero_dtype dt, zero_act act, const uint8_t *q, const uint8_t *e,
                                 uint64_t rows, uint64_t cols, void *stream) {
    if (!is_any(dt)) return ZERO_EDTYPE;
    if (act != ZERO_ACT_GELU && act != ZERO_ACT_SILU) return ZERO_EINVAL;
    if (!extent(rows) || !extent(cols)) return ZERO_EINVAL;
    if (rows == 0 || cols == 0) return ZERO_OK;
    const uint64_t b = bytes_of(dt);
    if (q == nullptr || e == nullptr || !matrix_ok(dx, rows, cols, lddx, b) ||
        !matrix_ok(dy, rows, cols, lddy, b))
        return ZERO_EINVAL;
    const View out[1] = {mat(dx, rows, cols, lddx, b)};
    const View in[2] = {codes(q, rows, cols), exponents(e, rows, cols)};
    if (!apart(out, 1, in, 2)) return ZERO_EINVAL;
    if (meet(out[0], mat(dy, rows, cols, lddy, b)) && !same(dx, lddx, dy, lddy))
        return ZERO_EINVAL;
    return done(zs::launch_act_backward(dx, lddx, dy, lddy, static_cast<int>(dt),
                                        static_cast<int>(act), q, e, rows, cols,
                                        static_cast<hipStream_t>(stream)),
                "zero_act_backward launch");
}

namespace {

// The gradient's place in the flat buffer, and its format against dy's.
int grad_target(const void *dw, zero_dtype dw_dt, int32_t first, zero_dtype dt, uint64_t rows,
                uint64_t cols) {
    if (!is_16(dt) || (dw_dt != dt && dw_dt != ZERO_F32)) return ZERO_EDTYPE;
    if (dw_dt != ZERO_F32 && first == 0) return ZERO_EINVAL;
    if (rows == 0 || cols == 0) return ZERO_OK;
    return matrix_ok(dw, rows, cols, cols, bytes_of(dw_dt)) ? ZERO_OK : ZERO_EINVAL;
}

int workspace_ok(const void *workspace, uint64_t have, uint64_t need) {
    if (need == 0) return ZERO_OK;
    return workspace != nullptr && aligned(workspace, 16) && have >= need ? ZERO_OK : ZERO_EINVAL;
}

// No tokens: the gradient is zero.
int zero_grad(void *dw, zero_dtype dw_dt, int32_t first, uint64_t n, void *stream,
              const char *what) {
    if (first == 0) return ZERO_OK;
    return done(zs::launch_zero_fill(dw, static_cast<int>(bytes_of(dw_dt)), n,
                                     static_cast<hipStream_t>(stream)),
                what);
}

}  // namespace

extern "C" int zero_weight_grad_workspace(uint64_t tokens, uint64_t n_out, uint64_t n_in,
                                          uint64_t *bytes) {
    if (bytes == nullptr || !extent(tokens) || !extent(n_out) || !extent(n_in))
        return ZERO_EINVAL;
    *bytes = tokens == 0 || n_out == 0 || n_in == 0 ? 0
                                                    : zs::weight_grad_workspace(tokens, n_out, n_in);
    return ZERO_OK;
}

extern "C" int zero_weight_grad(void *dw, zero_dtype dw_dt, int32_t first, const void *dy,
                                uint64_t lddy, zero_dtype dt, const uint8_t *q, const uint8_t *e,
                                uint64_t tokens, uint64_t n_out, uint64_t n_in, void *workspace,
                                uint64_t workspace_bytes, void *stream) {
    if (!is_16(dt)) return ZERO_EDTYPE;
    if (!extent(tokens) || !extent(n_out) || !extent(n_in)) return ZERO_EINVAL;
    const int rc = grad_target(dw, dw_dt, first, dt, n_out, n_in);
    if (rc != ZERO_OK) return rc;
    if (n_out == 0 || n_in == 0) return ZERO_OK;
    if (tokens == 0)
        return zero_grad(dw, dw_dt, first, n_out * n_in, stream, "zero_weight_grad launch");
    if (q == nullptr || e == nullptr || !matrix_ok(dy, tokens, n_out, lddy, 2)) return ZERO_EINVAL;
    const uint64_t need = zs::weight_grad_workspace(tokens, n_out, n_in);
    if (workspace_ok(workspace, workspace_bytes, need) != ZERO_OK) return ZERO_EINVAL;
    const View out[2] = {vec(dw, n_out * n_in, bytes_of(dw_dt)), vec(workspace, need, 1)};
    const View in[3] = {mat(dy, tokens, n_out, lddy, 2), codes(q, tokens, n_in),
                        exponents(e, tokens, n_in)};
    if (!apart(out, 2, in, 3)) return ZERO_EINVAL;
    return done(zs::launch_weight_grad(dw, dw_dt == ZERO_F32, first != 0,
                                       static_cast<const uint16_t *>(dy), lddy,
                                       static_cast<int>(dt), q, e, tokens, n_out, n_in, workspace,
                                       static_cast<hipStream_t>(stream)),
                "zero_weight_grad launch");
}

extern "C" int zero_embed_lookup(void *out, uint64_t ldo, const void *table, zero_dtype dt,
                                 const void *ids, zero_itype it, uint64_t tokens, uint64_t vocab,
                                 uint64_t width, float scale, void *stream) {
    if (!is_any(dt) || !is_id(it)) return ZERO_EDTYPE;
    if (!extent(tokens) || !extent(vocab) || !extent(width)) return ZERO_EINVAL;
    if (tokens == 0 || width == 0) return ZERO_OK;
    const uint64_t b = bytes_of(dt), ib = it == ZERO_I64 ? 8 : 4;
    if (!matrix_ok(out, tokens, width, ldo, b) || ids == nullptr || !aligned(ids, ib))
        return ZERO_EINVAL;
    if (vocab > 0 && !matrix_ok(table, vocab, width, width, b)) return ZERO_EINVAL;
    const View o[1] = {mat(out, tokens, width, ldo, b)};
    const View in[2] = {vec(table, vocab * width, b), vec(ids, tokens, ib)};
    if (!apart(o, 1, in, 2)) return ZERO_EINVAL;
    return done(zs::launch_embed_lookup(out, ldo, table, static_cast<int>(dt), ids,
                                        it == ZERO_I64, tokens, vocab, width, scale,
                                        static_cast<hipStream_t>(stream)),
                "zero_embed_lookup launch");
}

extern "C" int zero_embed_grad_workspace(uint64_t tokens, uint64_t vocab, uint64_t width,
                                         uint64_t *bytes) {
    if (bytes == nullptr || !extent(tokens) || !extent(vocab) || !extent(width))
        return ZERO_EINVAL;
    *bytes = tokens == 0 || vocab == 0 || width == 0 ? 0
                                                     : zs::embed_grad_workspace(tokens, vocab, width);
    return ZERO_OK;
}

extern "C" int zero_embed_grad(void *dw, zero_dtype dw_dt, int32_t first, const void *dy,
                               uint64_t lddy, zero_dtype dt, const void *ids, zero_itype it,
                               uint64_t tokens, uint64_t vocab, uint64_t width, float scale,
                               void *workspace, uint64_t workspace_bytes, void *stream) {
    if (!is_16(dt) || !is_id(it)) return ZERO_EDTYPE;
    if (!extent(tokens) || !extent(vocab) || !extent(width)) return ZERO_EINVAL;
    const int rc = grad_target(dw, dw_dt, first, dt, vocab, width);
    if (rc != ZERO_OK) return rc;
    if (vocab == 0 || width == 0) return ZERO_OK;
    if (tokens == 0)
        return zero_grad(dw, dw_dt, first, vocab * width, stream, "zero_embed_grad launch");
    const uint64_t ib = it == ZERO_I64 ? 8 : 4;
    if (!matrix_ok(dy, tokens, width, lddy, 2) || ids == nullptr || !aligned(ids, ib))
        return ZERO_EINVAL;
    const uint64_t need = zs::embed_grad_workspace(tokens, vocab, width);
    if (workspace_ok(workspace, workspace_bytes, need) != ZERO_OK) return ZERO_EINVAL;
    const View out[2] = {vec(dw, vocab * width, bytes_of(dw_dt)), vec(workspace, need, 1)};
    const View in[2] = {mat(dy, tokens, width, lddy, 2), vec(ids, tokens, ib)};
    if (!apart(out, 2, in, 2)) return ZERO_EINVAL;
    return done(zs::launch_embed_grad(dw, dw_dt == ZERO_F32, first != 0,
                                      static_cast<const uint16_t *>(dy), lddy,
                                      static_cast<int>(dt), ids, it == ZERO_I64, tokens, vocab,
                                      width, scale, workspace, static_cast<hipStream_t>(stream)),
                "zero_embed_grad launch");
}

namespace {

// Checks and launch shared by both forms of the policy loss; ctl: the control
// block of the device-resident form, or null.
int policy_loss(const zs::PolicyArgs &a, zero_dtype dt, zero_itype it, const void *ctl,
                const char *what, void *stream) {
    if (!is_any(dt) || !is_id(it)) return ZERO_EDTYPE;
    if (!extent(a.rows) || !extent(a.vocab)) return ZERO_EINVAL;
    if (!(a.clip_low >= 0.0f && a.clip_low <= 1.0f) || !(a.clip_high >= 0.0f) ||
        !std::isfinite(a.kl_coef))
        return ZERO_EINVAL;
    if (a.loss == nullptr || !aligned(a.loss, 4)) return ZERO_EINVAL;
    const uint64_t b = bytes_of(dt), ib = it == ZERO_I64 ? 8 : 4, n = a.rows;
    View out[5] = {vec(a.loss, 1, 4), vec(a.token_loss, n, 4), vec(a.logp, n, 4),
                   View{nullptr, 0, 0, 0}, View{nullptr, 0, 0, 0}};
    if (n > 0) {
        if (a.vocab == 0 || !matrix_ok(a.logits, n, a.vocab, a.ld, b)) return ZERO_EINVAL;
        if (a.dlogits != nullptr && !matrix_ok(a.dlogits, n, a.vocab, a.ldd, b))
            return ZERO_EINVAL;
        const void *need[4] = {a.token_loss, a.logp, a.advantage, a.weight};
        for (const void *p : need)
            if (p == nullptr || !aligned(p, 4)) return ZERO_EINVAL;
        if (a.targets == nullptr || !aligned(a.targets, ib)) return ZERO_EINVAL;
        if (!aligned(a.old_logp, 4) || !aligned(a.ref_logp, 4)) return ZERO_EINVAL;
        if (a.ref_logp == nullptr && a.kl_coef != 0.0f) return ZERO_EINVAL;
    }
    const View logits = n > 0 ? mat(a.logits, n, a.vocab, a.ld, b) : View{nullptr, 0, 0, 0};
    if (n > 0 && a.dlogits != nullptr) out[3] = mat(a.dlogits, n, a.vocab, a.ldd, b);
    const View in[6] = {vec(a.targets, n, ib),
                        vec(a.old_logp, a.old_logp != nullptr ? n : 0, 4),
                        vec(a.ref_logp, a.ref_logp != nullptr ? n : 0, 4),
                        vec(a.advantage, n, 4),
                        vec(a.weight, n, 4),
                        vec(ctl, ctl != nullptr ? sizeof(zero_device_ctl) : 0, 1)};
    if (!apart(out, 4, in, 6)) return ZERO_EINVAL;
    for (int i = 0; i < 3; ++i)
        if (meet(out[i], logits)) return ZERO_EINVAL;
    if (meet(out[3], logits) && !same(a.dlogits, a.ldd, a.logits, a.ld)) return ZERO_EINVAL;
    return done(zs::launch_policy_loss(a, static_cast<int>(dt), static_cast<hipStream_t>(stream)),
                what);
}

}  // namespace

extern "C" int zero_policy_loss(float *loss, float *token_loss, float *logp, void *dlogits,
                                uint64_t ldd, const void *logits, uint64_t ld, zero_dtype dt,
                                const void *targets, zero_itype it, const float *old_logp,
                                const float *ref_logp, const float *advantage,
                                const float *weight, uint64_t rows, uint64_t vocab,
                                float clip_low, float clip_high, float kl_coef, float loss_scale,
                                void *stream) {
    if (!(loss_scale > 0.0f) || !std::isfinite(loss_scale)) return ZERO_EINVAL;
    const zs::PolicyArgs a{loss, token_loss, logp, dlogits, logits, ldd, ld, targets,
                           it == ZERO_I64, old_logp, ref_logp, advantage, weight, rows, vocab,
                           clip_low, clip_high, kl_coef, loss_scale, nullptr};
    return policy_loss(a, dt, it, nullptr, "zero_policy_loss launch", stream);
}

extern "C" int zero_policy_loss_dev(float *loss, float *token_loss, float *logp, void *dlogits,
                                    uint64_t ldd, const void *logits, uint64_t ld, zero_dtype dt,
                                    const void *targets, zero_itype it, const float *old_logp,
                                    const float *ref_logp, const float *advantage,
                                    const float *weight, uint64_t rows, uint64_t vocab,
                                    float clip_low, float clip_high, float kl_coef,
                                    const zero_device_ctl *d_ctl, void *stream) {
    if (d_ctl == nullptr || !aligned(d_ctl, alignof(zero_device_ctl))) return ZERO_EINVAL;
    const zs::PolicyArgs a{loss, token_loss, logp, dlogits, logits, ldd, ld, targets,
                           it == ZERO_I64, old_logp, ref_logp, advantage, weight, rows, vocab,
                           clip_low, clip_high, kl_coef, 1.0f, &d_ctl->scaler.loss_scale};
    return policy_loss(a, dt, it, d_ctl, "zero_policy_loss_dev launch", stream);
}
