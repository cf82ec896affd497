// gfx950 kernels of the embedding lookup and its gradient.
//
// The lookup copies rows: long rows a wave a piece, short ones in groups of eight
// elements a lane, numbered over the whole output so that odd widths fill the lanes.
//
// The gradient sums the rows of dy that share an id, without floating-point
// atomics and in an order that the ids alone fix:
//   1. the tokens are sorted by (id, position); ids outside the vocabulary sort
//      last (key = vocab) and are never read again.
//   2. a wave walks 64 sorted positions over 512 columns, eight rows of dy in
//      flight.  A run of equal ids that lies inside its 64 positions is scaled,
//      rounded and written; what reaches over an end becomes a partial row (FP32
//      workspace).  So the work is cut evenly whatever the ids are: frequent tokens
//      and padding spread over the whole chip.  In the same launch other blocks
//      write the zero rows of ids that do not occur.
//   3. the partial rows of each run that crosses chunks are added.
// What has to move is dy once and dw once; partial rows add at most
// 2 * 2 * 4 / (64 * 2) = 1/8 of dy (1/2 where few tokens are walked 16 at a time).
// 65536 x 4096 BF16 into FP32, vocabulary 50257, 28% of the positions one id: sums and zero
// rows 240 us (5.7 TB/s of dy and dw), sorting 28, joining 20.
//
// Sorting: up to kRankTokens tokens, a token's place is the number of keys that
// precede it, counted directly in one launch (T^2 compares of two VALU operations
// each).  More tokens take a stable radix sort, kDigitBits a pass, two launches a
// pass.  Gradients of 64 columns, counted against radix: 1024 tokens 17.5 and 29.3 us,
// 8192 tokens 31.1 and 33.5, 16384 tokens 45.6 and 35.3.
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

// Rows of at least 64 vectors of 16 B: a wave takes a piece of kPiece vectors of one
// token's row, four in flight a lane, the id and the row's address in scalar registers.
// 65536 tokens x 4096 BF16 columns from a cold table: 131 us, against 149 us with the
// groups numbered over the whole output (which fill the lanes where rows are short).
constexpr uint32_t kPiece = 64 * 4;

template <int F>
__global__ __launch_bounds__(kThreads) void embed_lookup_rows_kernel(
    elem_t<F> *__restrict__ out, uint64_t ldo, const elem_t<F> *__restrict__ table,
    const void *__restrict__ ids, int ids64, uint32_t vocab, uint32_t width, FastDiv pieces,
    uint64_t n_waves, float scale) {
    constexpr uint32_t K = F == 2 ? 4 : 8;
    constexpr int U = kPiece / 64;
    const uint32_t lane = threadIdx.x & 63u;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (uint64_t w = static_cast<uint64_t>(blockIdx.x) * (kThreads / 64) + wave; w < n_waves;
         w += static_cast<uint64_t>(gridDim.x) * (kThreads / 64)) {
        const uint64_t t = div_by(w, pieces);
        const uint32_t c0 = static_cast<uint32_t>(w - t * pieces.d) * kPiece * K;
        const uint32_t key = __builtin_amdgcn_readfirstlane(key_at(ids, ids64, t, vocab));
        const elem_t<F> *src = table + static_cast<uint64_t>(key) * width + c0;
        elem_t<F> *dst = out + t * ldo + c0;
        const uint32_t left = width - c0;      // columns from the piece's first
        u32x4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t c = (u * 64 + lane) * K;
            v[u] = u32x4{0u, 0u, 0u, 0u};
            if (key != vocab && c + K <= left)
                v[u] = *reinterpret_cast<const u32x4_any *>(src + c);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t c = (u * 64 + lane) * K;
            if (c + K <= left) {
                u32x4 r;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (F == 2) {
                        r[i] = bits(product32(from_bits(v[u][i]), scale));
                    } else {
                        float x[2];
                        unpack2<F>(v[u][i], x);
                        r[i] = pack2<F>(product32(x[0], scale), product32(x[1], scale));
                    }
                }
                if (key == vocab) r = u32x4{0u, 0u, 0u, 0u};
                __builtin_nontemporal_store(r, reinterpret_cast<u32x4_any *>(dst + c));
            } else if (c < left) {             // the row's last, partial vector
                for (uint32_t j = 0; j < left - c; ++j)
                    dst[c + j] = key == vocab
                                     ? from_f32<F>(0.0f)
                                     : from_f32<F>(product32(to_f32<F>(src[c + j]), scale));
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
constexpr uint32_t kSortBlocks = 128;
constexpr int kSortThreads = 256;
constexpr int kSortWaves = kSortThreads / 64;
constexpr uint32_t kSortMin = 1024;           // tokens a sort block takes at least

constexpr uint32_t kBatch = 4;                // 64-token steps whose keys are in flight

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
// consecutive, so (wave, step, lane) is the token order.
template <typename Load>
__device__ __forceinline__ void wave_histogram(uint32_t (*cnt)[kDigits], uint32_t first,
                                               uint32_t last, int shift, Load key_of) {
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    for (uint32_t d = lane; d < kDigits; d += 64) cnt[wave][d] = 0;
    wave_sync();
    for (uint32_t t0 = first; t0 < last; t0 += 64 * kBatch) {
        uint32_t k[kBatch];
#pragma unroll
        for (uint32_t i = 0; i < kBatch; ++i) {
            const uint32_t t = t0 + i * 64 + lane;
            k[i] = t < last ? key_of(t) : 0u;
        }
#pragma unroll
        for (uint32_t i = 0; i < kBatch; ++i)
            if (t0 + i * 64 + lane < last)
                atomicAdd(&cnt[wave][(k[i] >> shift) & (kDigits - 1)], 1u);
    }
}

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
        hist[blockIdx.x * kDigits + d] = s;
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
    constexpr uint32_t kMine = kDigits / kSortThreads;
    uint32_t before[kMine] = {}, all[kMine] = {};
    constexpr uint32_t kFlight = 32;   // blocks whose counts are in flight
    for (uint32_t b0 = 0; b0 < gridDim.x; b0 += kFlight) {
        uint32_t h[kFlight][kMine];
#pragma unroll
        for (uint32_t b = 0; b < kFlight; ++b)
#pragma unroll
            for (uint32_t i = 0; i < kMine; ++i)
                h[b][i] = b0 + b < gridDim.x
                              ? hist[(b0 + b) * kDigits + threadIdx.x + i * kSortThreads]
                              : 0u;
#pragma unroll
        for (uint32_t b = 0; b < kFlight; ++b)
#pragma unroll
            for (uint32_t i = 0; i < kMine; ++i) {
                all[i] += h[b][i];
                before[i] += b0 + b < blockIdx.x ? h[b][i] : 0u;
            }
    }
#pragma unroll
    for (uint32_t i = 0; i < kMine; ++i) total[threadIdx.x + i * kSortThreads] = all[i];
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
    for (uint32_t b0 = first; b0 < last; b0 += 64 * kBatch) {
        uint32_t keys[kBatch], orders[kBatch];
#pragma unroll
        for (uint32_t i = 0; i < kBatch; ++i) {
            const uint32_t t = b0 + i * 64 + lane;
            keys[i] = t < last ? key_of(t) : 0u;
            orders[i] = t < last && order_in != nullptr ? order_in[t] : t;
        }
#pragma unroll
        for (uint32_t i = 0; i < kBatch; ++i) {
            if (b0 + i * 64 >= last) break;
            const bool on = b0 + i * 64 + lane < last;
            const uint32_t digit = (keys[i] >> shift) & (kDigits - 1);
            const uint64_t m = peers_of(digit, on);
            const uint64_t lower = m & ((1ull << lane) - 1);
            uint32_t place = 0;
            if (on) place = cnt[wave][digit] + static_cast<uint32_t>(__popcll(lower));
            wave_sync();
            if (on && lower == 0) cnt[wave][digit] += static_cast<uint32_t>(__popcll(m));
            wave_sync();
            if (on) {
                keys_out[place] = keys[i];
                order_out[place] = orders[i];
            }
        }
    }
}

// ---- summing the rows --------------------------------------------------------------

constexpr int kSumThreads = 256;
constexpr int kSumWaves = kSumThreads / 64;
constexpr uint32_t kSlice = 512;          // columns a wave covers (8 a lane)
// Sorted positions a wave walks, held one a lane: 64, or 16 where 64 would leave most
// of the chip idle (the walk is then latency: 1024 x 768 took 16.5 us with 64).
constexpr uint32_t kLongChunk = 64, kShortChunk = 16;
constexpr uint64_t kFullWaves = 2048;     // two waves on each SIMD of the chip
constexpr uint32_t kZeroRows = 64;        // vocabulary rows a zeroing block looks at: one a lane
constexpr int kJoinThreads = 512;
constexpr int kJoinWaves = kJoinThreads / 64;
constexpr uint32_t kJoinChunks = 16, kJoinColumns = 256, kShortRun = 16;

// What the summing kernels share.
struct RowSums {
    const uint16_t *dy;
    uint64_t lddy;
    const uint32_t *keys, *order;   // sorted tokens
    float *part;                    // partial rows: two a chunk, ld_part columns each
    uint32_t ld_part, tokens, vocab, width;
    uint32_t chunks, slices;
    float scale;
};

// Eight columns of a finished row: scaled, added to the old row (not FIRST), rounded.
template <int O, bool FIRST>
__device__ __forceinline__ void finish_row(elem_t<O> *dw, const RowSums &a, uint32_t key,
                                           uint32_t col, uint32_t n, const float acc[8]) {
    elem_t<O> *d = dw + static_cast<uint64_t>(key) * a.width + col;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = product32(acc[j], a.scale);
    if constexpr (!FIRST) {
        float old[8];
        if (n == 8)
            widen8<O>(load8<O>(d), old);
        else
            load_some<O>(d, n, old);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = old[j] + v[j];
    }
    if (n == 8)
        store8<O>(d, v);
    else
        store_some<O>(d, n, v);
}

__device__ __forceinline__ float *part_row(const RowSums &a, uint64_t chunk, uint32_t slot,
                                           uint32_t col) {
    return a.part + (chunk * 2 + slot) * a.ld_part + col;
}

__device__ __forceinline__ void store_part(float *p, const float v[8]) {
    f32x4 *d = reinterpret_cast<f32x4 *>(p);
    d[0] = f32x4{v[0], v[1], v[2], v[3]};
    d[1] = f32x4{v[4], v[5], v[6], v[7]};
}

// One wave: the columns [col, col + n) a lane of chunk c's positions.  A run inside
// the chunk is finished here; a run that came from the chunk before (or fills the
// whole chunk) goes to slot 0, one that starts here and goes on to slot 1.
template <int F, int O, bool FIRST, uint32_t kChunk>
__device__ __forceinline__ void sum_chunk(elem_t<O> *dw, const RowSums &a, uint32_t c,
                                          uint32_t col, uint32_t n) {
    constexpr int U = 8;              // rows in flight
    const uint32_t lane = threadIdx.x & 63u;
    const uint32_t lo = c * kChunk, p = lo + lane;
    const bool mine = lane < kChunk && p < a.tokens;
    const uint32_t key = mine ? a.keys[p] : a.vocab;
    const uint32_t row = mine ? a.order[p] : 0u;
    const uint32_t count = static_cast<uint32_t>(__popcll(__ballot(key < a.vocab)));
    if (count == 0) return;           // ids outside the vocabulary sort last
    const uint32_t next = lo + kChunk < a.tokens ? a.keys[lo + kChunk] : a.vocab;
    const uint32_t prev = lo > 0 ? a.keys[lo - 1] : a.vocab;
    uint32_t after = __shfl_down(key, 1);
    if (lane == kChunk - 1) after = next;
    const uint64_t ends = __ballot(after != key);   // last positions of their runs
    bool from_before = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(key)) == prev;
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (uint32_t i0 = 0; i0 < count; i0 += U) {
        Raw8<F> r[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t i = i0 + u < count ? i0 + u : count - 1;
            const uint64_t t = static_cast<uint32_t>(__builtin_amdgcn_readlane(row, i));
            const uint16_t *s = a.dy + t * a.lddy + col;
            if (n == 8) {
                r[u] = load8<F>(s);
            } else if (n != 0) {
                r[u].v[0] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j)
                    if (j < n) r[u].v[0][j / 2] |= static_cast<uint32_t>(s[j]) << (16 * (j % 2));
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t i = i0 + u;
            if (i >= count) break;
            float x[8];
            widen8<F>(r[u], x);
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] += x[j];
            const bool end = (ends >> i) & 1u;
            if (end || i + 1 == kChunk) {
                if (n != 0) {
                    if (from_before)
                        store_part(part_row(a, c, 0, col), acc);
                    else if (!end)
                        store_part(part_row(a, c, 1, col), acc);
                    else
                        finish_row<O, FIRST>(
                            dw, a, static_cast<uint32_t>(__builtin_amdgcn_readlane(key, i)), col,
                            n, acc);
                }
                from_before = false;
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
            }
        }
    }
}

// First sorted position whose key is at least want, by a whole wave: 64 probes a step.
__device__ __forceinline__ uint32_t wave_lower_bound(const uint32_t *keys, uint32_t tokens,
                                                     uint32_t want) {
    const uint32_t lane = threadIdx.x & 63u;
    uint32_t lo = 0, len = tokens;   // the answer is in [lo, lo + len]
    while (len > 0) {
        const uint32_t step = (len + 63) / 64;
        const uint64_t at = static_cast<uint64_t>(lane) * step + step - 1;
        const bool less = at < len && keys[lo + at] < want;
        const uint32_t n = static_cast<uint32_t>(__popcll(__ballot(less)));
        lo += n * step;
        len -= n * step;
        if (len > step - 1) len = step - 1;   // probe n is not below want
    }
    return lo;
}

// 16-B aligned zeros over [d, d + n) by the whole block, element by element at the ends.
template <typename T>
__device__ __forceinline__ void block_zero(T *d, uint64_t n) {
    constexpr uint32_t K = 16 / sizeof(T);
    const uint64_t to_line = ((16 - reinterpret_cast<uintptr_t>(d) % 16) % 16) / sizeof(T);
    const uint64_t head = to_line < n ? to_line : n;
    const uint64_t n_vec = (n - head) / K;
    if (threadIdx.x < head) d[threadIdx.x] = T(0);
    for (uint64_t i = threadIdx.x; i < n_vec; i += kSumThreads)
        __builtin_nontemporal_store(u32x4{0u, 0u, 0u, 0u},
                                    reinterpret_cast<u32x4 *>(d + head) + i);
    const uint64_t tail = head + n_vec * K + threadIdx.x;
    if (tail < n) d[tail] = T(0);
}

// Zeros in the rows of a group of kZeroRows whose id does not occur.
template <int O>
__device__ __forceinline__ void zero_rows(elem_t<O> *dw, const RowSums &a, uint32_t group) {
    __shared__ uint32_t bounds[2];
    __shared__ uint32_t seen[kZeroRows];
    const uint32_t v0 = group * kZeroRows, wave = threadIdx.x >> 6;
    const uint32_t rows = a.vocab - v0 < kZeroRows ? a.vocab - v0 : kZeroRows;
    if (threadIdx.x < kZeroRows) seen[threadIdx.x] = 0;
    if (wave < 2) {
        const uint32_t r = wave_lower_bound(a.keys, a.tokens, v0 + (wave == 0 ? 0 : rows));
        if ((threadIdx.x & 63u) == 0) bounds[wave] = r;
    }
    __syncthreads();
    for (uint32_t p = bounds[0] + threadIdx.x; p < bounds[1]; p += kSumThreads)
        seen[a.keys[p] - v0] = 1;
    __syncthreads();
    const uint32_t lane = threadIdx.x & 63u;
    uint64_t empty = __ballot(lane < rows && seen[lane] == 0);   // rows that do not occur
    while (empty != 0) {                                         // run by run
        const uint32_t r = static_cast<uint32_t>(__builtin_ctzll(empty));
        const uint64_t rest = ~(empty >> r);
        const uint32_t n = rest != 0 ? static_cast<uint32_t>(__builtin_ctzll(rest)) : 64u - r;
        block_zero(dw + static_cast<uint64_t>(v0 + r) * a.width,
                   static_cast<uint64_t>(n) * a.width);
        empty = r + n < 64 ? empty >> (r + n) << (r + n) : 0;
    }
    __syncthreads();
}

// The chunks' sums, and with FIRST the zero rows, in one launch: the sums read and
// the zeros write, so they share the memory's time.  Work items: `sum_blocks` groups
// of kSumWaves (chunk, slice) pairs, then `zero_blocks` groups of rows.
template <int F, int O, bool FIRST, uint32_t kChunk>
__global__ __launch_bounds__(kSumThreads) void chunk_sum_kernel(
    elem_t<O> *__restrict__ dw, RowSums a, FastDiv slices, uint64_t sum_blocks,
    uint64_t zero_blocks) {
    for (uint64_t b = blockIdx.x; b < sum_blocks + zero_blocks; b += gridDim.x) {
        if (b < sum_blocks) {
            const uint64_t w = b * kSumWaves + (threadIdx.x >> 6);
            const uint64_t c = div_by(w, slices);
            if (c >= a.chunks) continue;
            const uint64_t col =
                (w - c * slices.d) * kSlice + static_cast<uint64_t>(threadIdx.x & 63u) * 8;
            const uint32_t n = col >= a.width ? 0u
                               : a.width - col < 8 ? static_cast<uint32_t>(a.width - col) : 8u;
            sum_chunk<F, O, FIRST, kChunk>(
                dw, a, __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(c)),
                static_cast<uint32_t>(col), n);
        } else {
            if constexpr (FIRST)
                zero_rows<O>(dw, a, static_cast<uint32_t>(b - sum_blocks));
        }
    }
}

// acc[0..4) += parts [p0, p1) of the run that starts in chunk c: slot 1 of that chunk,
// slot 0 of the following ones, in order, U in flight.
template <uint32_t U>
__device__ __forceinline__ void add_parts(float acc[4], const RowSums &a, uint32_t c, uint32_t p0,
                                          uint32_t p1, uint32_t col) {
    for (uint32_t p = p0; p < p1; p += U) {
        f32x4 x[U];
#pragma unroll
        for (uint32_t u = 0; u < U; ++u) {
            const uint32_t i = p + u < p1 ? p + u : p1 - 1;
            x[u] = *reinterpret_cast<const f32x4 *>(
                part_row(a, static_cast<uint64_t>(c) + i, i == 0 ? 1 : 0, col));
        }
#pragma unroll
        for (uint32_t u = 0; u < U; ++u) {
            const bool on = p + u < p1;
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[j] = on ? acc[j] + x[u][j] : acc[j];
        }
    }
}

// Runs that cross chunks.  A block looks at kJoinChunks chunks and 256 columns (four
// a lane); a chunk owns the run that starts in it and goes on.  A run of at most
// kShortRun parts is added by one wave, the waves taking the chunks in turn; a longer
// one by all waves, each a consecutive share, and then the waves' sums in order.
template <int O, bool FIRST>
__global__ __launch_bounds__(kJoinThreads) void join_runs_kernel(elem_t<O> *__restrict__ dw,
                                                                 RowSums a, uint32_t chunk) {
    __shared__ float sums[kJoinWaves][kJoinColumns];
    __shared__ uint32_t reach[kJoinChunks];
    const uint32_t lane = threadIdx.x & 63u;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t c0 = blockIdx.x * kJoinChunks;
    // lane l: the key of the run that chunk c0 + l owns, or vocab
    uint32_t own = a.vocab;
    const uint64_t hi = (static_cast<uint64_t>(c0) + lane + 1) * chunk;
    if (lane < kJoinChunks && hi < a.tokens) {
        const uint64_t lo = hi - chunk;
        const uint32_t key = a.keys[hi - 1], next = a.keys[hi], first = a.keys[lo];
        const uint32_t prev = lo > 0 ? a.keys[lo - 1] : a.vocab;
        if (next == key && !(first == key && prev == key)) own = key;
    }
    const uint64_t owners = __ballot(own < a.vocab);
    if (owners == 0) return;
    // of the first kShortRun chunks after each owner's, how many the run reaches into: the
    // waves look at one owner each
    for (uint32_t l = wave; l < kJoinChunks; l += kJoinWaves) {
        const uint32_t key = static_cast<uint32_t>(__builtin_amdgcn_readlane(own, l));
        const uint64_t at = (static_cast<uint64_t>(c0) + l + 1 + lane) * chunk;
        const uint64_t in =
            __ballot(lane < kShortRun && key < a.vocab && at < a.tokens && a.keys[at] == key);
        if (lane == 0) reach[l] = static_cast<uint32_t>(__popcll(in));
    }
    __syncthreads();
    for (uint64_t col0 = static_cast<uint64_t>(blockIdx.y) * kJoinColumns; col0 < a.width;
         col0 += static_cast<uint64_t>(gridDim.y) * kJoinColumns) {
        const uint32_t col = static_cast<uint32_t>(col0) + lane * 4;
        const uint32_t n = col >= a.width ? 0u : a.width - col < 4 ? a.width - col : 4u;
        auto finish = [&](uint32_t key, const float acc[4]) {
            elem_t<O> *d = dw + static_cast<uint64_t>(key) * a.width + col;
            float v[4];
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j) {
                v[j] = product32(acc[j], a.scale);
                if (!FIRST && j < n) v[j] = to_f32<O>(d[j]) + v[j];
            }
            if (n == 4) {
                if constexpr (O == 2)
                    *reinterpret_cast<u32x4_any *>(d) =
                        u32x4{bits(v[0]), bits(v[1]), bits(v[2]), bits(v[3])};
                else
                    *reinterpret_cast<u32x2_any *>(d) =
                        u32x2{pack2<O>(v[0], v[1]), pack2<O>(v[2], v[3])};
            } else {
#pragma unroll
                for (uint32_t j = 0; j < 4; ++j)
                    if (j < n) d[j] = from_f32<O>(v[j]);
            }
        };
        uint64_t longer = 0;
        uint32_t turn = 0;
        for (uint64_t m = owners; m != 0; m &= m - 1) {
            const uint32_t l = static_cast<uint32_t>(__builtin_ctzll(m)), c = c0 + l;
            const uint32_t key = static_cast<uint32_t>(__builtin_amdgcn_readlane(own, l));
            const uint32_t n_part = 1 + reach[l];
            if (n_part > kShortRun) {
                longer |= 1ull << l;
                continue;
            }
            if (turn++ % kJoinWaves != wave) continue;
            float acc[4] = {0, 0, 0, 0};
            if (n != 0) add_parts<4>(acc, a, c, 0, n_part, col);
            finish(key, acc);
        }
        for (uint64_t m = longer; m != 0; m &= m - 1) {
            const uint32_t l = static_cast<uint32_t>(__builtin_ctzll(m)), c = c0 + l;
            const uint32_t key = static_cast<uint32_t>(__builtin_amdgcn_readlane(own, l));
            const uint32_t n_part =
                (wave_lower_bound(a.keys, a.tokens, key + 1) - 1) / chunk - c + 1;
            auto share = [&](uint32_t w) {
                return static_cast<uint32_t>(static_cast<uint64_t>(n_part) * w / kJoinWaves);
            };
            float acc[4] = {0, 0, 0, 0};
            if (n != 0) add_parts<16>(acc, a, c, share(wave), share(wave + 1), col);
            *reinterpret_cast<f32x4 *>(&sums[wave][lane * 4]) =
                f32x4{acc[0], acc[1], acc[2], acc[3]};
            __syncthreads();
            if (wave == 0) {
                for (int w = 1; w < kJoinWaves; ++w)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[j] += sums[w][lane * 4 + j];
                finish(key, acc);
            }
            __syncthreads();
        }
    }
}

uint64_t round256(uint64_t b) { return (b + 255) / 256 * 256; }

uint32_t sort_per_block(uint64_t tokens) {
    uint64_t per = (tokens + kSortBlocks - 1) / kSortBlocks;
    if (per < kSortMin) per = kSortMin;
    return static_cast<uint32_t>((per + kSortThreads - 1) / kSortThreads * kSortThreads);
}

// Workspace: sorted keys and order; for the radix sort a second pair and the
// digit counts; the chunks' partial rows (when there are two chunks).
struct GradSpace {
    uint64_t keys, order, keys2, order2, hist, part, total, ld_part;
    bool rank;
    uint32_t chunk;
};

uint32_t chunk_of(uint64_t tokens, uint64_t width) {
    const uint64_t waves = (tokens + kLongChunk - 1) / kLongChunk * ((width + kSlice - 1) / kSlice);
    return waves < kFullWaves ? kShortChunk : kLongChunk;
}

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
    s.chunk = chunk_of(tokens, width);
    const uint64_t chunks = (tokens + s.chunk - 1) / s.chunk;
    s.total = at + (chunks > 1 ? 8 * s.ld_part * chunks : 0);
    return s;
}

template <int F, int O, bool FIRST>
hipError_t sum_rows(void *dw, const RowSums &a, uint32_t chunk, hipStream_t stream) {
    auto *d = static_cast<elem_t<O> *>(dw);
    const uint64_t cap = max_blocks();
    const uint64_t sums =
        (static_cast<uint64_t>(a.chunks) * a.slices + kSumWaves - 1) / kSumWaves;
    const uint64_t zeros = FIRST ? (static_cast<uint64_t>(a.vocab) + kZeroRows - 1) / kZeroRows : 0;
    const uint64_t blocks = sums + zeros < cap ? sums + zeros : cap;
    const uint32_t grid = static_cast<uint32_t>(blocks);
    if (chunk == kLongChunk)
        chunk_sum_kernel<F, O, FIRST, kLongChunk>
            <<<grid, kSumThreads, 0, stream>>>(d, a, fast_div(a.slices), sums, zeros);
    else
        chunk_sum_kernel<F, O, FIRST, kShortChunk>
            <<<grid, kSumThreads, 0, stream>>>(d, a, fast_div(a.slices), sums, zeros);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.chunks < 2) return e;
    const uint32_t cols = (a.width + kJoinColumns - 1) / kJoinColumns;
    const dim3 joins((a.chunks + kJoinChunks - 1) / kJoinChunks, cols < 65535 ? cols : 65535);
    join_runs_kernel<O, FIRST><<<joins, kJoinThreads, 0, stream>>>(d, a, chunk);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_embed_lookup(void *out, uint64_t ldo, const void *table, int fmt,
                               const void *ids, bool ids64, uint64_t tokens, uint64_t vocab,
                               uint64_t width, float scale, hipStream_t stream) {
    const uint64_t per_vec = fmt == 2 ? 4 : 8;
    if (width >= 64 * per_vec) {
        const uint64_t pieces = (width + kPiece * per_vec - 1) / (kPiece * per_vec);
        const uint64_t waves = tokens * pieces, blocks = (waves + 3) / 4, cap = max_blocks();
        const uint32_t grid = static_cast<uint32_t>(blocks < cap ? blocks : cap);
#define ZS_LOOK(F)                                                                              \
    if (fmt == F)                                                                               \
        embed_lookup_rows_kernel<F><<<grid, kThreads, 0, stream>>>(                             \
            static_cast<elem_t<F> *>(out), ldo, static_cast<const elem_t<F> *>(table), ids,     \
            ids64 ? 1 : 0, static_cast<uint32_t>(vocab), static_cast<uint32_t>(width),          \
            fast_div(static_cast<uint32_t>(pieces)), waves, scale);
        ZS_LOOK(0) ZS_LOOK(1) ZS_LOOK(2)
#undef ZS_LOOK
        return hipGetLastError();
    }
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
        const uint32_t per = sort_per_block(tokens);
        const uint32_t blocks = static_cast<uint32_t>((tokens + per - 1) / per);
        uint32_t *hist = list(s.hist);
        // the last pass writes the pair (keys, order)
        uint32_t *k_out = passes % 2 ? keys : list(s.keys2);
        uint32_t *o_out = passes % 2 ? order : list(s.order2);
        const uint32_t *k_in = nullptr, *o_in = nullptr;
        for (int p = 0; p < passes; ++p) {
            radix_count_kernel<<<blocks, kSortThreads, 0, stream>>>(
                hist, k_in, ids, i64, T, V, per, p * kDigitBits);
            radix_scatter_kernel<<<blocks, kSortThreads, 0, stream>>>(
                k_out, o_out, hist, k_in, o_in, ids, i64, T, V, per, p * kDigitBits);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
            k_in = k_out;
            o_in = o_out;
            k_out = k_out == keys ? list(s.keys2) : keys;
            o_out = o_out == order ? list(s.order2) : order;
        }
    }
    const RowSums a{dy, lddy, keys, order, reinterpret_cast<float *>(base + s.part),
                    static_cast<uint32_t>(s.ld_part), T, V, static_cast<uint32_t>(width),
                    static_cast<uint32_t>((tokens + s.chunk - 1) / s.chunk),
                    static_cast<uint32_t>((width + kSlice - 1) / kSlice), scale};
#define ZS_ROWS(F, O, FIRST) return sum_rows<F, O, FIRST>(dw, a, s.chunk, stream)
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
