// gfx950 kernels of the embedding lookup and its gradient.
//
// The lookup copies rows: one 16-B group (eight 16-bit elements, two groups of
// FP32) a lane, groups numbered over the whole output so that short and odd
// widths fill the lanes too.
//
// The gradient sums the rows of dy that share an id.  Without floating-point
// atomics and in an order that the ids alone fix:
//   1. the tokens are sorted by (id, position); ids outside the vocabulary sort
//      last (key = vocab) and are never read again.
//   2. the sorted positions are cut into chunks of C.  A chunk that lies inside
//      one id's run is summed into a partial row (FP32 workspace), so that long
//      runs (padding, frequent tokens) are spread over the whole chip.
//   3. every vocabulary row finds its run by binary search, adds the positions
//      before the first whole chunk, the whole chunks' partial rows and the
//      positions after the last one, and writes the row (zeros for an empty run).
// A run of R costs its wave at most 2C + R/C row loads; C is near the root of
// T/4, where the worst case (one id everywhere) is least.
//
// Sorting: up to kRankTokens tokens, a token's place is the number of keys that
// precede it, counted directly, in one launch (T^2 compares: 2 VALU operations
// each, measured cheaper than three dependent launches at these sizes).  More
// tokens take a stable radix sort, kDigitBits a pass, of at most kSortBlocks
// blocks.
#include "grad_device.h"

#pragma clang fp contract(off)

namespace zs {
namespace {

constexpr int kThreads = 256;

// ---- lookup -----------------------------------------------------------------

// Key of position t: its id, or vocab for an id outside [0, vocab).
__device__ __forceinline__ uint32_t key_at(const void *ids, int ids64, uint64_t t,
                                           uint32_t vocab) {
    if (ids64) {
        const int64_t v = static_cast<const int64_t *>(ids)[t];
        return v >= 0 && v < static_cast<int64_t>(vocab) ? static_cast<uint32_t>(v) : vocab;
    }
    const int32_t v = static_cast<const int32_t *>(ids)[t];
    return v >= 0 && static_cast<uint32_t>(v) < vocab ? static_cast<uint32_t>(v) : vocab;
}

constexpr int kLookUnroll = 2;

template <int F>
__global__ __launch_bounds__(kThreads) void embed_lookup_kernel(
    elem_t<F> *__restrict__ out, uint64_t ldo, const elem_t<F> *__restrict__ table,
    const void *__restrict__ ids, int ids64, uint32_t vocab, uint32_t width, FastDiv per_row,
    uint64_t n_groups, float scale) {
    constexpr uint64_t kTile = kThreads * kLookUnroll;
    for (uint64_t t0 = blockIdx.x * kTile; t0 < n_groups; t0 += gridDim.x * kTile) {
        float v[kLookUnroll][8];
#pragma unroll
        for (int u = 0; u < kLookUnroll; ++u) {
            const uint64_t g = t0 + u * kThreads + threadIdx.x;
            if (g < n_groups) {
                const uint64_t t = div_by(g, per_row);
                const uint32_t c = static_cast<uint32_t>(g - t * per_row.d) * 8;
                const uint32_t key = key_at(ids, ids64, t, vocab);
                const uint32_t n = width - c < 8 ? width - c : 8;
                const elem_t<F> *s = table + static_cast<uint64_t>(key) * width + c;
                if (key == vocab) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[u][j] = 0.0f;
                } else if (n == 8) {
                    widen8<F>(load8_cached<F>(s), v[u]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[u][j] = product32(v[u][j], scale);
                } else {
                    load_some<F>(s, n, v[u]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[u][j] = product32(v[u][j], scale);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kLookUnroll; ++u) {
            const uint64_t g = t0 + u * kThreads + threadIdx.x;
            if (g < n_groups) {
                const uint64_t t = div_by(g, per_row);
                const uint32_t c = static_cast<uint32_t>(g - t * per_row.d) * 8;
                elem_t<F> *d = out + t * ldo + c;
                if (width - c >= 8)
                    store8<F>(d, v[u]);
                else
                    store_some<F>(d, width - c, v[u]);
            }
        }
    }
}

// ---- sorting the tokens -----------------------------------------------------------

constexpr uint32_t kRankTokens = 8192;
constexpr int kRankThreads = 1024;             // 16 waves count for the same 64 tokens
constexpr int kRankWaves = kRankThreads / 64;

// keys[r], order[r]: the r-th token by (key, position).  Block b ranks tokens
// 64 b .. 64 b + 63; wave w counts over its 64-token slices of the keys.
__global__ __launch_bounds__(kRankThreads) void rank_sort_kernel(
    uint32_t *__restrict__ keys, uint32_t *__restrict__ order, const void *__restrict__ ids,
    int ids64, uint32_t tokens, uint32_t vocab) {
    __shared__ uint32_t part[kRankWaves][64];
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    const uint32_t mine = blockIdx.x * 64 + lane;
    const uint32_t key = mine < tokens ? key_at(ids, ids64, mine, vocab) : 0xffffffffu;
    uint32_t below = 0;
    const uint32_t slices = (tokens + 63) / 64;
    for (uint32_t s = wave; s < slices; s += kRankWaves) {
        const uint32_t t = s * 64 + lane;
        // past the end: a key that precedes nothing
        const uint32_t k = t < tokens ? key_at(ids, ids64, t, vocab) : 0xffffffffu;
        if (s < blockIdx.x) {          // earlier positions: equal keys precede
#pragma unroll
            for (int j = 0; j < 64; ++j)
                below += static_cast<uint32_t>(__builtin_amdgcn_readlane(k, j)) <= key ? 1u : 0u;
        } else if (s > blockIdx.x) {   // later positions: only smaller keys precede
#pragma unroll
            for (int j = 0; j < 64; ++j)
                below += static_cast<uint32_t>(__builtin_amdgcn_readlane(k, j)) < key ? 1u : 0u;
        } else {
#pragma unroll
            for (int j = 0; j < 64; ++j) {
                const uint32_t o = static_cast<uint32_t>(__builtin_amdgcn_readlane(k, j));
                below += o < key || (o == key && j < static_cast<int>(lane)) ? 1u : 0u;
            }
        }
    }
    part[wave][lane] = below;
    __syncthreads();
    if (wave == 0 && mine < tokens) {
        uint32_t r = 0;
#pragma unroll
        for (int w = 0; w < kRankWaves; ++w) r += part[w][lane];
        keys[r] = key;
        order[r] = mine;
    }
}

constexpr int kDigitBits = 9;
constexpr uint32_t kDigits = 1u << kDigitBits;
constexpr uint32_t kSortBlocks = 64;
constexpr int kSortThreads = 256;
constexpr int kSortWaves = kSortThreads / 64;
constexpr uint32_t kSortMin = 4096;           // tokens a sort block takes at least

// Lanes of the wave whose digit equals this lane's, among the active ones.
__device__ __forceinline__ uint64_t peers_of(uint32_t digit, bool on) {
    uint64_t m = __ballot(on);
#pragma unroll
    for (int b = 0; b < kDigitBits; ++b) {
        const uint64_t set = __ballot(on && ((digit >> b) & 1u));
        m &= ((digit >> b) & 1u) ? set : ~set;
    }
    return m;
}

// LDS written by some lanes of a wave, read by others of the same wave.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Digit counts of each wave's share of a block's tokens, in LDS; the shares are
// consecutive, so (wave, step, lane) is the token order.  per_wave is a multiple of 64.
template <typename Load>
__device__ __forceinline__ void wave_histogram(uint32_t (*cnt)[kDigits], uint32_t first,
                                               uint32_t last, int shift, Load key_of) {
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    for (uint32_t d = lane; d < kDigits; d += 64) cnt[wave][d] = 0;
    wave_sync();
    for (uint32_t t0 = first; t0 < last; t0 += 64) {
        const uint32_t t = t0 + lane;
        const bool on = t < last;
        const uint32_t digit = on ? (key_of(t) >> shift) & (kDigits - 1) : 0u;
        const uint64_t m = peers_of(digit, on);
        if (on && (m & ((1ull << lane) - 1)) == 0)
            cnt[wave][digit] += static_cast<uint32_t>(__popcll(m));
        wave_sync();
    }
}

struct SortShape {
    uint32_t blocks, per_block;   // per_block: a multiple of 256
};

// The first pass reads ids (keys_in null); later passes read keys and order.
__global__ __launch_bounds__(kSortThreads) void radix_count_kernel(
    uint32_t *__restrict__ hist, const uint32_t *__restrict__ keys_in,
    const void *__restrict__ ids, int ids64, uint32_t tokens, uint32_t vocab, uint32_t per_block,
    int shift) {
    __shared__ uint32_t cnt[kSortWaves][kDigits];
    const uint32_t wave = threadIdx.x >> 6, per_wave = per_block / kSortWaves;
    const uint64_t f = static_cast<uint64_t>(blockIdx.x) * per_block +
                       static_cast<uint64_t>(wave) * per_wave;
    const uint32_t first = static_cast<uint32_t>(f < tokens ? f : tokens);
    const uint32_t last = static_cast<uint32_t>(f + per_wave < tokens ? f + per_wave : tokens);
    wave_histogram(cnt, first, last, shift, [&](uint32_t t) {
        return keys_in != nullptr ? keys_in[t] : key_at(ids, ids64, t, vocab);
    });
    __syncthreads();
    for (uint32_t d = threadIdx.x; d < kDigits; d += kSortThreads) {
        uint32_t s = 0;
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) s += cnt[w][d];
        hist[d * kSortBlocks + blockIdx.x] = s;
    }
}

__global__ __launch_bounds__(kSortThreads) void radix_scatter_kernel(
    uint32_t *__restrict__ keys_out, uint32_t *__restrict__ order_out,
    const uint32_t *__restrict__ hist, const uint32_t *__restrict__ keys_in,
    const uint32_t *__restrict__ order_in, const void *__restrict__ ids, int ids64,
    uint32_t tokens, uint32_t vocab, uint32_t per_block, int shift) {
    __shared__ uint32_t cnt[kSortWaves][kDigits];
    __shared__ uint32_t total[kDigits];
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    const uint32_t per_wave = per_block / kSortWaves;
    const uint64_t f = static_cast<uint64_t>(blockIdx.x) * per_block +
                       static_cast<uint64_t>(wave) * per_wave;
    const uint32_t first = static_cast<uint32_t>(f < tokens ? f : tokens);
    const uint32_t last = static_cast<uint32_t>(f + per_wave < tokens ? f + per_wave : tokens);
    auto key_of = [&](uint32_t t) {
        return keys_in != nullptr ? keys_in[t] : key_at(ids, ids64, t, vocab);
    };
    wave_histogram(cnt, first, last, shift, key_of);
    // a digit's tokens over all blocks, and over the blocks before this one
    uint32_t before[kDigits / kSortThreads];
#pragma unroll
    for (uint32_t i = 0; i < kDigits / kSortThreads; ++i) {
        const uint32_t d = threadIdx.x + i * kSortThreads;
        uint32_t all = 0, bef = 0;
        for (uint32_t b = 0; b < gridDim.x; ++b) {
            const uint32_t h = hist[d * kSortBlocks + b];
            all += h;
            bef += b < blockIdx.x ? h : 0u;
        }
        total[d] = all;
        before[i] = bef;
    }
    __syncthreads();
    // exclusive scan of total over the digits, by wave 0: eight digits a lane
    if (wave == 0) {
        constexpr uint32_t K = kDigits / 64;
        uint32_t v[K], s = 0;
#pragma unroll
        for (uint32_t j = 0; j < K; ++j) {
            v[j] = total[lane * K + j];
            s += v[j];
        }
        uint32_t inc = s;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const uint32_t up = __shfl_up(inc, o);
            inc += static_cast<int>(lane) >= o ? up : 0u;
        }
        uint32_t ex = inc - s;
#pragma unroll
        for (uint32_t j = 0; j < K; ++j) {
            total[lane * K + j] = ex;
            ex += v[j];
        }
    }
    __syncthreads();
    // first place of each (digit, wave) of this block
#pragma unroll
    for (uint32_t i = 0; i < kDigits / kSortThreads; ++i) {
        const uint32_t d = threadIdx.x + i * kSortThreads;
        uint32_t place = total[d] + before[i];
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {
            const uint32_t c = cnt[w][d];
            cnt[w][d] = place;
            place += c;
        }
    }
    __syncthreads();
    for (uint32_t t0 = first; t0 < last; t0 += 64) {
        const uint32_t t = t0 + lane;
        const bool on = t < last;
        const uint32_t key = on ? key_of(t) : 0u;
        const uint32_t digit = (key >> shift) & (kDigits - 1);
        const uint64_t m = peers_of(digit, on);
        const uint64_t lower = m & ((1ull << lane) - 1);
        uint32_t place = 0;
        if (on) place = cnt[wave][digit] + static_cast<uint32_t>(__popcll(lower));
        wave_sync();
        if (on && lower == 0) cnt[wave][digit] += static_cast<uint32_t>(__popcll(m));
        wave_sync();
        if (on) {
            keys_out[place] = key;
            order_out[place] = order_in != nullptr ? order_in[t] : t;
        }
    }
}

// ---- summing the rows --------------------------------------------------------------

constexpr int kRowThreads = 256;
constexpr int kRowWaves = kRowThreads / 64;
constexpr uint32_t kRowsPerBlock = 16;    // vocabulary rows a block searches for at once
constexpr uint32_t kSlice = 512;          // columns a wave covers (8 a lane)

// acc[0..8) += the eight columns at col of dy's rows order[lo .. hi), in that
// order; four rows' loads in flight.
template <int F>
__device__ __forceinline__ void add_rows(float acc[8], const uint16_t *__restrict__ dy,
                                         uint64_t lddy, const uint32_t *__restrict__ order,
                                         uint32_t lo, uint32_t hi, uint32_t col, uint32_t n) {
    constexpr uint32_t U = 4;
    if (n == 8) {
        uint32_t p = lo;
        for (; p + U <= hi; p += U) {
            Raw8<F> r[U];
#pragma unroll
            for (uint32_t u = 0; u < U; ++u)
                r[u] = load8<F>(dy + static_cast<uint64_t>(order[p + u]) * lddy + col);
#pragma unroll
            for (uint32_t u = 0; u < U; ++u) {
                float x[8];
                widen8<F>(r[u], x);
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[j] += x[j];
            }
        }
        for (; p < hi; ++p) {
            float x[8];
            widen8<F>(load8<F>(dy + static_cast<uint64_t>(order[p]) * lddy + col), x);
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] += x[j];
        }
    } else {
        for (uint32_t p = lo; p < hi; ++p) {
            float x[8];
            load_some<F>(dy + static_cast<uint64_t>(order[p]) * lddy + col, n, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] += x[j];
        }
    }
}

// Partial rows of the chunks that lie inside one run.  blockIdx.x: chunk;
// blockIdx.y and the wave: slice of columns.  part holds ld_part (a multiple of
// 8) FP32 columns a chunk.
template <int F>
__global__ __launch_bounds__(kRowThreads) void chunk_sum_kernel(
    float *__restrict__ part, uint32_t ld_part, const uint16_t *__restrict__ dy, uint64_t lddy,
    const uint32_t *__restrict__ keys, const uint32_t *__restrict__ order, uint32_t vocab,
    uint32_t width, uint32_t chunk) {
    const uint32_t lo = blockIdx.x * chunk, hi = lo + chunk;   // whole chunks only
    const uint32_t key = keys[lo];
    if (key >= vocab || keys[hi - 1] != key) return;
    const uint32_t slices = (width + kSlice - 1) / kSlice;
    for (uint32_t s = blockIdx.y * kRowWaves + (threadIdx.x >> 6); s < slices;
         s += gridDim.y * kRowWaves) {
        const uint32_t col = s * kSlice + (threadIdx.x & 63u) * 8;
        if (col >= width) return;
        const uint32_t n = width - col < 8 ? width - col : 8;
        float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        add_rows<F>(acc, dy, lddy, order, lo, hi, col, n);
        f32x4 *d =
            reinterpret_cast<f32x4 *>(part + static_cast<uint64_t>(blockIdx.x) * ld_part + col);
        d[0] = f32x4{acc[0], acc[1], acc[2], acc[3]};
        d[1] = f32x4{acc[4], acc[5], acc[6], acc[7]};
    }
}

// The vocabulary rows.  O: dw's format.  FIRST false (FP32 only): rows whose id
// occurs get dw + G, the others are left alone.
template <int F, int O, bool FIRST>
__global__ __launch_bounds__(kRowThreads) void row_sum_kernel(
    elem_t<O> *__restrict__ dw, const uint16_t *__restrict__ dy, uint64_t lddy,
    const uint32_t *__restrict__ keys, const uint32_t *__restrict__ order,
    const float *__restrict__ part, uint32_t ld_part, uint32_t tokens, uint32_t vocab,
    uint32_t width, uint32_t chunk, int chunk_shift, float scale) {
    __shared__ uint32_t start[kRowsPerBlock + 1];
    for (uint32_t v0 = blockIdx.x * kRowsPerBlock; v0 < vocab; v0 += gridDim.x * kRowsPerBlock) {
    const uint32_t rows = vocab - v0 < kRowsPerBlock ? vocab - v0 : kRowsPerBlock;
    if (threadIdx.x <= rows) {      // first sorted position whose key is >= v0 + lane
        const uint32_t want = v0 + threadIdx.x;
        uint32_t lo = 0, hi = tokens;
        while (lo < hi) {
            const uint32_t mid = lo + (hi - lo) / 2;
            if (keys[mid] < want)
                lo = mid + 1;
            else
                hi = mid;
        }
        start[threadIdx.x] = lo;
    }
    __syncthreads();
    const uint32_t slices = (width + kSlice - 1) / kSlice;
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63u;
    for (uint32_t w = wave; w < rows * slices; w += kRowWaves) {
        const uint32_t r = w / slices, col = (w - r * slices) * kSlice + lane * 8;
        if (col >= width) continue;
        const uint32_t n = width - col < 8 ? width - col : 8;
        const uint32_t lo = start[r], hi = start[r + 1];
        if (!FIRST && lo == hi) continue;
        float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        const uint32_t c0 = (lo + chunk - 1) >> chunk_shift, c1 = hi >> chunk_shift;
        if (c0 < c1) {
            add_rows<F>(acc, dy, lddy, order, lo, c0 << chunk_shift, col, n);
            for (uint32_t c = c0; c < c1; ++c) {
                const f32x4 *s = reinterpret_cast<const f32x4 *>(
                    part + static_cast<uint64_t>(c) * ld_part + col);
                const f32x4 a = s[0], b = s[1];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    acc[j] += a[j];
                    acc[4 + j] += b[j];
                }
            }
            add_rows<F>(acc, dy, lddy, order, c1 << chunk_shift, hi, col, n);
        } else {
            add_rows<F>(acc, dy, lddy, order, lo, hi, col, n);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = product32(acc[j], scale);
        elem_t<O> *d = dw + static_cast<uint64_t>(v0 + r) * width + col;
        if constexpr (!FIRST) {
            float old[8];
            if (n == 8)
                widen8<O>(load8<O>(d), old);
            else
                load_some<O>(d, n, old);
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] = old[j] + acc[j];
        }
        if (n == 8)
            store8<O>(d, acc);
        else
            store_some<O>(d, n, acc);
    }
    __syncthreads();   // start is rewritten
    }
}

// Sorted positions a chunk holds: the power of two near sqrt(T) / 2, at least 32.
int chunk_shift_of(uint64_t tokens) {
    int s = 5;
    while ((1ull << (2 * s)) < tokens / 4) ++s;
    return s;
}

SortShape sort_shape(uint64_t tokens) {
    uint64_t per = (tokens + kSortBlocks - 1) / kSortBlocks;
    if (per < kSortMin) per = kSortMin;
    per = (per + kSortThreads - 1) / kSortThreads * kSortThreads;
    return SortShape{static_cast<uint32_t>((tokens + per - 1) / per), static_cast<uint32_t>(per)};
}

uint64_t round256(uint64_t b) { return (b + 255) / 256 * 256; }

// Workspace: sorted keys and order; for the radix sort a second pair and the
// digit counts; the chunks' partial rows.
struct GradSpace {
    uint64_t keys, order, keys2, order2, hist, part, total, ld_part;
    bool rank;
};

GradSpace grad_space(uint64_t tokens, uint64_t width) {
    GradSpace s{};
    s.rank = tokens <= kRankTokens;
    const uint64_t list = round256(4 * tokens);
    uint64_t at = 0;
    s.keys = at, at += list;
    s.order = at, at += list;
    if (!s.rank) {
        s.keys2 = at, at += list;
        s.order2 = at, at += list;
        s.hist = at, at += 4ull * kDigits * kSortBlocks;
    }
    s.ld_part = (width + 7) / 8 * 8;
    s.part = at;
    s.total = at + 4 * s.ld_part * (tokens >> chunk_shift_of(tokens));
    return s;
}

template <int F, int O, bool FIRST>
hipError_t sum_rows(void *dw, const uint16_t *dy, uint64_t lddy, const uint32_t *keys,
                    const uint32_t *order, float *part, uint32_t ld_part, uint64_t tokens,
                    uint64_t vocab, uint64_t width, float scale, hipStream_t stream) {
    const int shift = chunk_shift_of(tokens);
    const uint32_t chunks = static_cast<uint32_t>(tokens >> shift);
    if (chunks > 0) {
        const uint32_t per = kSlice * kRowWaves;
        const uint64_t slices = (width + per - 1) / per;
        const dim3 grid(chunks, static_cast<uint32_t>(slices < 65535 ? slices : 65535));
        chunk_sum_kernel<F><<<grid, kRowThreads, 0, stream>>>(
            part, ld_part, dy, lddy, keys, order, static_cast<uint32_t>(vocab),
            static_cast<uint32_t>(width), 1u << shift);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const uint64_t groups = (vocab + kRowsPerBlock - 1) / kRowsPerBlock, cap = max_blocks();
    const uint32_t blocks = static_cast<uint32_t>(groups < cap ? groups : cap);
    row_sum_kernel<F, O, FIRST><<<blocks, kRowThreads, 0, stream>>>(
        static_cast<elem_t<O> *>(dw), dy, lddy, keys, order, part, ld_part,
        static_cast<uint32_t>(tokens), static_cast<uint32_t>(vocab),
        static_cast<uint32_t>(width), 1u << shift, shift, scale);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_embed_lookup(void *out, uint64_t ldo, const void *table, int fmt,
                               const void *ids, bool ids64, uint64_t tokens, uint64_t vocab,
                               uint64_t width, float scale, hipStream_t stream) {
    const uint64_t per_row = (width + 7) / 8, groups = tokens * per_row;
    const FastDiv f = fast_div(static_cast<uint32_t>(per_row));
    const uint64_t tile = static_cast<uint64_t>(kThreads) * kLookUnroll;
    const uint64_t blocks = (groups + tile - 1) / tile, cap = max_blocks();
    const uint32_t grid = static_cast<uint32_t>(blocks < cap ? blocks : cap);
#define ZS_LOOK(F)                                                                              \
    if (fmt == F)                                                                               \
        embed_lookup_kernel<F><<<grid, kThreads, 0, stream>>>(                                  \
            static_cast<elem_t<F> *>(out), ldo, static_cast<const elem_t<F> *>(table), ids,     \
            ids64 ? 1 : 0, static_cast<uint32_t>(vocab), static_cast<uint32_t>(width), f,       \
            groups, scale);
    ZS_LOOK(0) ZS_LOOK(1) ZS_LOOK(2)
#undef ZS_LOOK
    return hipGetLastError();
}

uint64_t embed_grad_workspace(uint64_t tokens, uint64_t vocab, uint64_t width) {
    (void)vocab;
    return tokens == 0 ? 0 : grad_space(tokens, width).total;
}

hipError_t launch_embed_grad(void *dw, bool dw32, bool first, const uint16_t *dy, uint64_t lddy,
                             int fmt, const void *ids, bool ids64, uint64_t tokens,
                             uint64_t vocab, uint64_t width, float scale, void *workspace,
                             hipStream_t stream) {
    const GradSpace s = grad_space(tokens, width);
    auto *base = static_cast<uint8_t *>(workspace);
    auto list = [&](uint64_t at) { return reinterpret_cast<uint32_t *>(base + at); };
    uint32_t *keys = list(s.keys), *order = list(s.order);
    const uint32_t T = static_cast<uint32_t>(tokens), V = static_cast<uint32_t>(vocab);
    const int i64 = ids64 ? 1 : 0;
    if (s.rank) {
        rank_sort_kernel<<<(T + 63) / 64, kRankThreads, 0, stream>>>(keys, order, ids, i64, T, V);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    } else {
        int key_bits = 1;                        // keys are 0 .. vocab
        while ((vocab >> key_bits) != 0) ++key_bits;
        const int passes = (key_bits + kDigitBits - 1) / kDigitBits;
        const SortShape sh = sort_shape(tokens);
        uint32_t *hist = list(s.hist);
        // the last pass writes the pair (keys, order)
        uint32_t *k_out = passes % 2 ? keys : list(s.keys2);
        uint32_t *o_out = passes % 2 ? order : list(s.order2);
        const uint32_t *k_in = nullptr, *o_in = nullptr;
        for (int p = 0; p < passes; ++p) {
            radix_count_kernel<<<sh.blocks, kSortThreads, 0, stream>>>(
                hist, k_in, ids, i64, T, V, sh.per_block, p * kDigitBits);
            radix_scatter_kernel<<<sh.blocks, kSortThreads, 0, stream>>>(
                k_out, o_out, hist, k_in, o_in, ids, i64, T, V, sh.per_block, p * kDigitBits);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
            k_in = k_out;
            o_in = o_out;
            k_out = k_out == keys ? list(s.keys2) : keys;
            o_out = o_out == order ? list(s.order2) : order;
        }
    }
    auto *part = reinterpret_cast<float *>(base + s.part);
    const uint32_t ldp = static_cast<uint32_t>(s.ld_part);
#define ZS_ROWS(F, O, FIRST) \
    return sum_rows<F, O, FIRST>(dw, dy, lddy, keys, order, part, ldp, tokens, vocab, width, scale, stream)
    if (fmt == 0) {
        if (!dw32) ZS_ROWS(0, 0, true);
        if (first) ZS_ROWS(0, 2, true);
        ZS_ROWS(0, 2, false);
    }
    if (!dw32) ZS_ROWS(1, 1, true);
    if (first) ZS_ROWS(1, 2, true);
    ZS_ROWS(1, 2, false);
#undef ZS_ROWS
}

}  // namespace zs
