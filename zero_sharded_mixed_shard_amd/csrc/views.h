// Argument checks that the C-ABI layers of zero_shard_grad.h and
// zero_shard_block.h share: formats, matrix views and their overlaps.
#pragma once

#include <hip/hip_runtime_api.h>

#include "grad_launch.h"

namespace zs {

inline bool aligned(const void *p, uint64_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

inline uint64_t bytes_of(zero_dtype dt) { return dt == ZERO_F32 ? 4 : 2; }
inline bool is_16(zero_dtype dt) { return dt == ZERO_F16 || dt == ZERO_BF16; }
inline bool is_any(zero_dtype dt) { return is_16(dt) || dt == ZERO_F32; }
inline bool is_id(zero_itype it) { return it == ZERO_I32 || it == ZERO_I64; }

constexpr uint64_t kMaxBytes = 1ull << 56;

// A matrix view in bytes: rows of `width` bytes, `stride` bytes apart.
struct View {
    const void *p;
    uint64_t rows, width, stride;
    // bytes from the first element to the end of the last row
    uint64_t span() const { return rows == 0 || width == 0 ? 0 : (rows - 1) * stride + width; }
};

inline View vec(const void *p, uint64_t n, uint64_t elem) { return View{p, 1, n * elem, n * elem}; }

// Extents at most ZERO_MAX_EXTENT, ld at least cols, and a span below 2^56 bytes.
inline bool matrix_ok(const void *p, uint64_t rows, uint64_t cols, uint64_t ld, uint64_t elem) {
    if (p == nullptr || !aligned(p, elem)) return false;
    if (ld < cols || ld >= kMaxBytes / 8) return false;
    const unsigned __int128 span =
        (static_cast<unsigned __int128>(rows - 1) * ld + cols) * elem;
    return span < kMaxBytes;
}

inline View mat(const void *p, uint64_t rows, uint64_t cols, uint64_t ld, uint64_t elem) {
    return View{p, rows, cols * elem, ld * elem};
}

// Some byte belongs to both.  Two matrices of one stride whose columns do not
// meet are apart although their spans cross.
inline bool meet(const View &a, const View &b) {
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
inline bool apart(const View *out, int n_out, const View *in, int n_in) {
    for (int i = 0; i < n_out; ++i) {
        for (int j = i + 1; j < n_out; ++j)
            if (meet(out[i], out[j])) return false;
        for (int j = 0; j < n_in; ++j)
            if (meet(out[i], in[j])) return false;
    }
    return true;
}

inline bool extent(uint64_t n) { return n <= ZERO_MAX_EXTENT; }

// The same matrix: same pointer, same row stride.
inline bool same(const void *a, uint64_t lda, const void *b, uint64_t ldb) {
    return a == b && lda == ldb;
}

inline int done(hipError_t e, const char *what) {
    return e == hipSuccess ? ZERO_OK : fail_hip(e, what);
}

// The gradient's place in the flat buffer, and its format against dt.
inline bool grad_format_ok(zero_dtype dw_dt, zero_dtype dt) { return dw_dt == dt || dw_dt == ZERO_F32; }

inline int workspace_ok(const void *workspace, uint64_t have, uint64_t need) {
    if (need == 0) return ZERO_OK;
    return workspace != nullptr && aligned(workspace, 16) && have >= need ? ZERO_OK : ZERO_EINVAL;
}

}  // namespace zs
