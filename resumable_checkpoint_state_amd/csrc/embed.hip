// embed.hip -- the gradient of an embedding lookup, added into the gradient of
// the embedding matrix in an order that depends on the arguments alone. gfx950
// kernels and their C ABI.
//
// Mathematics. grad[v] += scale * sum over the rows t with token[t] = v, in
// float32, rounded once to the gradient's type.
//
// Mapping. The rows' numbers are sorted by token, stably (so that equal tokens
// keep the order of their rows), by a radix sort of at most 9 bits a pass: up to
// 8,192 rows by one block in one launch, above that by two launches a pass. A wave
// then takes kSeg consecutive places of the sorted order and some columns, and walks
// its rows: a token whose rows all lie inside is added to the matrix at once, and the
// sums of one that goes over the segment's ends are left in a workspace, at most two
// a segment, which a second kernel adds up in their order. However often a token
// comes, no wave walks more than kSeg rows. Bound by HBM where it is large: each row
// is read once, each gradient row that is met read and written once.

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "rcs.h"
#include "rcs_internal.h"
#include "vocab.h"

#pragma clang fp contract(off)

namespace {

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / kWave;
constexpr int kKeys = 8;  // of a thread
constexpr int kTile = kSortThreads * kKeys;  // keys of one block of the sort
constexpr int kMaxBits = 9, kBins = 1 << kMaxBits;  // of one pass
constexpr int kSeg = 32;          // sorted places of one wave of the sums
constexpr uint32_t kNone = 0xFFFFFFFFu;  // no key

// Keys of a pass: the tokens themselves (first pass), or what the last pass
// left. Rows whose token is outside [0, vocab) get the key `vocab`.
struct SortArgs {
    const void *tokens;
    int index_type;
    int64_t rows, vocab;
    const uint32_t *keys, *ids;  // null in the first pass
    uint32_t *keys_out, *ids_out;
    uint32_t *hist;  // [tile][1 << bits]
    int shift, bits;
    int passes;  // of a block that does them all
    int tiles;
};

__device__ __forceinline__ uint32_t key_at(const SortArgs &a, int64_t t) {
    if (a.keys != nullptr) return a.keys[t];
    const int64_t v = index_at(a.tokens, t, a.index_type);
    return v < 0 || v >= a.vocab ? (uint32_t)a.vocab : (uint32_t)v;
}

__global__ __launch_bounds__(kSortThreads) void embed_count(SortArgs a) {
    __shared__ uint32_t bins[kBins];
    const int n = 1 << a.bits;
    for (int k = threadIdx.x; k < n; k += kSortThreads) bins[k] = 0;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kKeys; ++k) {
        const int64_t t = (int64_t)blockIdx.x * kTile + k * kSortThreads + threadIdx.x;
        if (t < a.rows) atomicAdd(&bins[key_at(a, t) >> a.shift & (n - 1)], 1u);
    }
    __syncthreads();
    for (int k = threadIdx.x; k < n; k += kSortThreads)
        a.hist[(int64_t)blockIdx.x * n + k] = bins[k];
}

// Each key to its place: those of lower digits first, then equal digits of earlier
// tiles, waves, turns of a wave and lanes. ALONE: the one block there is does all
// passes, in LDS; otherwise one pass, with the tiles' counts from embed_count.
template <bool ALONE>
__global__ __launch_bounds__(kSortThreads) void embed_sort(SortArgs a) {
    __shared__ uint32_t next[kSortWaves][kBins];  // of the wave: where its next key goes
    __shared__ uint32_t sums[kSortWaves];
    __shared__ uint32_t keys_at[ALONE ? kTile : 1], ids_at[ALONE ? kTile : 1];
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const int n = 1 << a.bits;
    const int first = wave * (kTile / kSortWaves) + lane;  // then every kWave-th
    const int64_t tile0 = (int64_t)blockIdx.x * kTile;
    uint32_t keys[kKeys], ids[kKeys];
#pragma unroll
    for (int k = 0; k < kKeys; ++k) {
        const int64_t t = tile0 + first + k * kWave;
        keys[k] = t < a.rows ? key_at(a, t) : kNone;
        ids[k] = t < a.rows && a.ids != nullptr ? a.ids[t] : (uint32_t)t;
    }
    for (int pass = 0; pass < (ALONE ? a.passes : 1); ++pass) {
        const int shift = ALONE ? pass * a.bits : a.shift;
        for (int k = tid; k < n; k += kSortThreads)
#pragma unroll
            for (int w = 0; w < kSortWaves; ++w) next[w][k] = 0;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kKeys; ++k)
            if (keys[k] != kNone) atomicAdd(&next[wave][keys[k] >> shift & (n - 1)], 1u);
        __syncthreads();
        // of each digit (a thread's): all keys, those of earlier tiles, and those before it
        uint32_t mine = 0, before = 0;
        if (tid < n) {
            if (ALONE) {
#pragma unroll
                for (int w = 0; w < kSortWaves; ++w) mine += next[w][tid];
            } else {
#pragma unroll 8
                for (int i = 0; i < a.tiles; ++i) {
                    const uint32_t c = a.hist[(int64_t)i * n + tid];
                    mine += c;
                    before += i < (int)blockIdx.x ? c : 0;
                }
            }
        }
        uint32_t run = mine;  // inclusive over the wave
#pragma unroll
        for (int d = 1; d < kWave; d *= 2) {
            const uint32_t up = (uint32_t)__shfl_up((int)run, d);
            if (lane >= d) run += up;
        }
        if (lane == kWave - 1) sums[wave] = run;
        __syncthreads();
        if (tid < n) {
            uint32_t at = run - mine + before;
#pragma unroll
            for (int w = 0; w < kBins / kWave; ++w)
                if (w < wave) at += sums[w];
#pragma unroll
            for (int w = 0; w < kSortWaves; ++w) {
                const uint32_t c = next[w][tid];
                next[w][tid] = at;
                at += c;
            }
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kKeys; ++k) {
            const bool in = keys[k] != kNone;
            const uint32_t digit = keys[k] >> shift & (n - 1);
            uint64_t same = __ballot(in);
            for (int b = 0; b < a.bits; ++b) {
                const uint64_t set = __ballot(digit >> b & 1);
                same &= digit >> b & 1 ? set : ~set;
            }
            const int rank = __popcll(same & ((1ull << lane) - 1));
            uint32_t to = 0;
            if (in) to = next[wave][digit] + rank;
            __builtin_amdgcn_wave_barrier();
            if (in && rank == 0) next[wave][digit] = to + __popcll(same);
            __builtin_amdgcn_wave_barrier();
            if (!in) continue;
            if (ALONE) keys_at[to] = keys[k], ids_at[to] = ids[k];
            else a.keys_out[to] = keys[k], a.ids_out[to] = ids[k];
        }
        if (!ALONE) return;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kKeys; ++k) {
            const int t = first + k * kWave;
            if (t < a.rows) keys[k] = keys_at[t], ids[k] = ids_at[t];
        }
    }
#pragma unroll
    for (int k = 0; k < kKeys; ++k) {
        const int t = first + k * kWave;
        if (t < a.rows) a.keys_out[t] = keys[k], a.ids_out[t] = ids[k];
    }
}

struct SumArgs {
    const uint32_t *keys, *ids;  // sorted
    int64_t count, vocab, dim;
    const void *rows;
    int64_t rows_ld;
    void *grad;
    int64_t grad_ld;
    float scale;
    float *open;  // [segment][2][dim]: sums of the first and of the last token of a segment
    int64_t segments;
    int parts;  // of the columns
};

constexpr int kSumThreads = 256;
constexpr int kCols = 4;    // of a lane
constexpr int kBatch = 8;   // rows that are under way at a time

// A wave does a segment of the sorted order and kCols columns a lane.
template <class R, class G>
__global__ __launch_bounds__(kSumThreads) void embed_sum(SumArgs a) {
    const int64_t item = blockIdx.x * (int64_t)(kSumThreads / kWave) +
                         __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t seg = item / a.parts;
    if (seg >= a.segments) return;
    const int lane = threadIdx.x % kWave;
    const int64_t first = seg * kSeg;
    // lane i has place first + i - 1
    uint32_t key = kNone, id = 0;
    {
        const int64_t s = first + lane - 1;
        if (lane < kSeg + 2 && s >= 0 && s < a.count) key = a.keys[s], id = a.ids[s];
    }
    const int64_t n = (item % a.parts * kWave + lane) * kCols;
    const int cols = (int)max((int64_t)0, min((int64_t)kCols, a.dim - n));
    const uint32_t vocab = (uint32_t)a.vocab;
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    bool begins = __builtin_amdgcn_readlane(key, 0) != __builtin_amdgcn_readlane(key, 1);
    for (int k0 = 0; k0 < kSeg; k0 += kBatch) {
        uint32_t v[kBatch + 1];
        f32x4 x[kBatch], y[kBatch];
#pragma unroll
        for (int k = 0; k <= kBatch; ++k) v[k] = __builtin_amdgcn_readlane(key, k0 + k + 1);
        if (v[0] >= vocab) break;  // no more tokens
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            x[k] = y[k] = f32x4{0.f, 0.f, 0.f, 0.f};
            if (v[k] >= vocab || cols == 0) continue;
            const uint32_t t = __builtin_amdgcn_readlane(id, k0 + k + 1);
            x[k] = load_some(a.rows, (int64_t)t * a.rows_ld + n, cols, R{});
            if (v[k + 1] != v[k])  // the gradient, where a token may end
                y[k] = load_some(a.grad, (int64_t)v[k] * a.grad_ld + n, cols, G{});
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (v[k] >= vocab) break;
            sum += x[k];
            const bool ends = v[k + 1] != v[k];
            if (!ends && k0 + k + 1 < kSeg) continue;
            if (cols > 0) {
                if (begins && ends) {
                    store_some(a.grad, (int64_t)v[k] * a.grad_ld + n, cols, y[k] + sum * a.scale,
                               G{});
                } else {
                    // 0: a token that came from the segment before, 1: one that begins here
                    store_some(a.open, (seg * 2 + (begins ? 1 : 0)) * a.dim + n, cols, sum, F32{});
                }
            }
            sum = f32x4{0.f, 0.f, 0.f, 0.f};
            begins = true;
        }
    }
}

// A wave does a segment and kCols columns a lane: if a token begins in the segment and
// goes on behind its end, the token's sums in the order of the segments.
template <class G>
__global__ __launch_bounds__(kSumThreads) void embed_join(SumArgs a) {
    const int64_t item = blockIdx.x * (int64_t)(kSumThreads / kWave) +
                         __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t seg = item / a.parts, last = (seg + 1) * kSeg - 1;
    if (seg >= a.segments || last + 1 >= a.count) return;
    const uint32_t v = a.keys[last];
    if (v >= (uint32_t)a.vocab || a.keys[last + 1] != v) return;
    if (seg > 0 && a.keys[seg * kSeg] == v && a.keys[seg * kSeg - 1] == v) return;
    const int64_t n = (item % a.parts * kWave + threadIdx.x % kWave) * kCols;
    // the segments that it reaches
    int64_t lo = seg + 1, hi = a.segments - 1;  // the last whose first key is v
    while (lo < hi) {
        const int64_t mid = (lo + hi + 1) / 2;
        if (a.keys[mid * kSeg] == v) lo = mid;
        else hi = mid - 1;
    }
    const int cols = (int)max((int64_t)0, min((int64_t)kCols, a.dim - n));
    if (cols == 0) return;
    f32x4 sum = load_some(a.open, (seg * 2 + 1) * a.dim + n, cols, F32{});
    for (int64_t s0 = seg + 1; s0 <= lo; s0 += kBatch) {
        f32x4 x[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            x[k] = s0 + k <= lo ? load_some(a.open, (s0 + k) * 2 * a.dim + n, cols, F32{})
                                : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < kBatch; ++k) sum += x[k];
    }
    const int64_t at = (int64_t)v * a.grad_ld + n;
    store_some(a.grad, at, cols, load_some(a.grad, at, cols, G{}) + sum * a.scale, G{});
}

// ----------------------------------------------------------------- host side

struct Plan {
    int passes, bits;
    int tiles;
    int64_t segments;
    int64_t keys[2], ids[2], hist, open, bytes;
};

Plan plan_of(int64_t rows, int64_t vocab, int64_t dim) {
    Plan p = {};
    int bits = 1;
    while ((vocab >> bits) != 0) ++bits;  // the keys are 0 to vocab
    p.passes = (bits + kMaxBits - 1) / kMaxBits;
    p.bits = (bits + p.passes - 1) / p.passes;
    p.tiles = (int)((rows + kTile - 1) / kTile);
    p.segments = (rows + kSeg - 1) / kSeg;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t was = at;
        at = round_up(at + bytes, 256);
        return was;
    };
    for (int k = 0; k < 2; ++k) p.keys[k] = take(4 * rows), p.ids[k] = take(4 * rows);
    p.hist = take(4LL * p.tiles << p.bits);
    p.open = take(8 * p.segments * dim);
    p.bytes = at;
    return p;
}

int check_sizes(int64_t rows, int64_t vocab, int64_t dim) {
    return rows < 0 || rows > kMaxRows || vocab < 1 || vocab > kMaxRows || dim < 1 ||
                   dim > kMaxWidth
               ? RCS_EINVAL
               : RCS_OK;
}

}  // namespace

extern "C" {

int64_t rcs_embed_workspace(int64_t rows, int64_t vocab, int64_t dim) {
    const int rc = check_sizes(rows, vocab, dim);
    return rc != RCS_OK ? rc : plan_of(rows, vocab, dim).bytes;
}

int embed_grad(const void *rows, int64_t rows_stride, int rows_type, int64_t count,
               const void *tokens, int index_type, void *grad, int64_t grad_stride, int grad_type,
               int64_t vocab, int64_t dim, float scale, void *workspace, int64_t workspace_bytes,
               hipStream_t stream) {
    int rc = check_sizes(count, vocab, dim);
    if (rc != RCS_OK) return rc;
    if (!is_type(rows_type) || !is_type(grad_type) || !is_index_type(index_type) ||
        !std::isfinite(scale))
        return RCS_EINVAL;
    const int isize = index_size(index_type);
    Extents reads, writes;
    if ((rc = reads.matrix(rows, count, dim, rows_stride, rows_type)) != RCS_OK ||
        (rc = reads.array(tokens, count * isize, isize)) != RCS_OK ||
        (rc = writes.matrix(grad, vocab, dim, grad_stride, grad_type)) != RCS_OK)
        return rc;
    if (count == 0) return RCS_OK;
    const Plan p = plan_of(count, vocab, dim);
    if (workspace_bytes < p.bytes) return RCS_ESIZE;
    if ((rc = writes.array(workspace, p.bytes, 256)) != RCS_OK) return rc;
    if (writes.overlap(reads)) return RCS_EINVAL;

    char *ws = static_cast<char *>(workspace);
    SortArgs s = {};
    s.tokens = tokens, s.index_type = index_type, s.rows = count, s.vocab = vocab;
    s.hist = reinterpret_cast<uint32_t *>(ws + p.hist), s.bits = p.bits;
    s.passes = p.passes, s.tiles = p.tiles;
    const auto to = [&](int k) {
        s.keys_out = reinterpret_cast<uint32_t *>(ws + p.keys[k]);
        s.ids_out = reinterpret_cast<uint32_t *>(ws + p.ids[k]);
    };
    if (p.tiles == 1) {
        to(0);
        embed_sort<true><<<1, kSortThreads, 0, stream>>>(s);
    }
    for (int k = 0; k < p.passes && p.tiles > 1; ++k) {
        to(k & 1);
        s.shift = k * p.bits;
        embed_count<<<dim3((unsigned)p.tiles), kSortThreads, 0, stream>>>(s);
        embed_sort<false><<<dim3((unsigned)p.tiles), kSortThreads, 0, stream>>>(s);
        s.keys = s.keys_out, s.ids = s.ids_out;
    }
    SumArgs a = {};
    a.keys = s.keys_out, a.ids = s.ids_out, a.count = count, a.vocab = vocab, a.dim = dim;
    a.rows = rows, a.rows_ld = rows_stride;
    a.grad = grad, a.grad_ld = grad_stride, a.scale = scale;
    a.open = reinterpret_cast<float *>(ws + p.open), a.segments = p.segments;
    a.parts = (int)((dim + kCols * kWave - 1) / (kCols * kWave));
    const dim3 grid((unsigned)((p.segments * a.parts + 3) / 4));
    by_type(grad_type, [&](auto g) {
        using G = decltype(g);
        by_type(rows_type, [&](auto r) {
            embed_sum<decltype(r), G><<<grid, kSumThreads, 0, stream>>>(a);
        });
        embed_join<G><<<grid, kSumThreads, 0, stream>>>(a);
    });
    return hipGetLastError() == hipSuccess ? RCS_OK : RCS_EHIP;
}

}  // extern "C"
