// embed.hip -- the gradient of an embedding lookup, added into the gradient of
// the embedding matrix in an order that depends on the arguments alone. gfx950
// kernels and their C ABI.
//
// Mathematics. grad[v] += scale * sum over the rows t with token[t] = v, in
// float32, rounded once to the gradient's type.
//
// Mapping. The rows' numbers are sorted by token, stably (so that equal tokens
// keep the order of their rows), by one or two passes of a radix sort; a block
// then takes kSeg consecutive places of the sorted order and some columns, and
// walks its rows: a token whose rows all lie inside is added to the matrix at
// once, and the sums of one that goes over the block's ends are left in a
// workspace, at most two a block, which a second kernel adds up in their order.
// However often a token comes, no wave walks more than kSeg rows. Bound by HBM:
// each row is read once, each gradient row that is met read and written once.

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "rcs.h"
#include "rcs_internal.h"
#include "vocab.h"

#pragma clang fp contract(off)

namespace {

constexpr int kSortThreads = 256;
constexpr int kSortWaves = kSortThreads / kWave;
constexpr int kTile = 1024;       // keys of one block of the sort
constexpr int kPerWave = kTile / kSortWaves;
constexpr int kMaxBits = 9;       // of one pass
constexpr int kSeg = 32;          // sorted places of one block of the sums
constexpr uint32_t kNone = 0xFFFFFFFFu;  // a row that adds nothing: sorted to the end

// Keys of a pass: the tokens themselves (first pass), or what the last pass
// left. Rows whose token is outside [0, vocab) get the key `vocab`.
struct SortArgs {
    const void *tokens;
    int index_type;
    int64_t rows, vocab;
    const uint32_t *keys, *ids;  // null in the first pass
    uint32_t *keys_out, *ids_out;
    uint32_t *hist;  // [tile][bins]
    int shift, bits;
};

__device__ __forceinline__ uint32_t key_at(const SortArgs &a, int64_t t) {
    if (a.keys != nullptr) return a.keys[t];
    const int64_t v = index_at(a.tokens, t, a.index_type);
    return v < 0 || v >= a.vocab ? (uint32_t)a.vocab : (uint32_t)v;
}

__global__ __launch_bounds__(kSortThreads) void embed_count(SortArgs a) {
    __shared__ uint32_t bins[1 << kMaxBits];
    const int n = 1 << a.bits;
    for (int k = threadIdx.x; k < n; k += kSortThreads) bins[k] = 0;
    __syncthreads();
    for (int k = threadIdx.x; k < kTile; k += kSortThreads) {
        const int64_t t = (int64_t)blockIdx.x * kTile + k;
        if (t < a.rows) atomicAdd(&bins[key_at(a, t) >> a.shift & (n - 1)], 1u);
    }
    __syncthreads();
    for (int k = threadIdx.x; k < n; k += kSortThreads)
        a.hist[(int64_t)blockIdx.x * n + k] = bins[k];
}

// Each key to its place: those of lower digits first, then equal digits of
// earlier tiles, waves and lanes.
__global__ __launch_bounds__(kSortThreads) void embed_place(SortArgs a, int tiles) {
    __shared__ uint32_t base[1 << kMaxBits];              // of the tile, for each digit
    __shared__ uint32_t next[kSortWaves][1 << kMaxBits];  // of the wave
    __shared__ uint32_t sums[kSortWaves];
    const int n = 1 << a.bits, tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    for (int k = tid; k < n; k += kSortThreads)
        for (int w = 0; w < kSortWaves; ++w) next[w][k] = 0;
    // totals of each digit, and of the tiles before
    uint32_t total[(1 << kMaxBits) / kSortThreads], before[(1 << kMaxBits) / kSortThreads];
    const int each = (n + kSortThreads - 1) / kSortThreads;  // consecutive digits of a thread
    uint32_t mine = 0;
#pragma unroll
    for (int d = 0; d < (1 << kMaxBits) / kSortThreads; ++d) {
        total[d] = before[d] = 0;
        const int k = tid * each + d;
        if (d >= each || k >= n) continue;
        for (int i = 0; i < tiles; ++i) {
            const uint32_t c = a.hist[(int64_t)i * n + k];
            total[d] += c;
            if (i < (int)blockIdx.x) before[d] += c;
        }
        mine += total[d];
    }
    uint32_t run = mine;  // inclusive over the wave
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
        const uint32_t up = (uint32_t)__shfl_up((int)run, d);
        if (lane >= d) run += up;
    }
    if (lane == kWave - 1) sums[wave] = run;
    __syncthreads();
    uint32_t at = run - mine;
    for (int w = 0; w < wave; ++w) at += sums[w];
#pragma unroll
    for (int d = 0; d < (1 << kMaxBits) / kSortThreads; ++d) {
        const int k = tid * each + d;
        if (d >= each || k >= n) continue;
        base[k] = at + before[d];
        at += total[d];
    }
    // digits of each wave's keys
    uint32_t keys[kPerWave / kWave];
    const int64_t first = (int64_t)blockIdx.x * kTile + wave * kPerWave + lane;
#pragma unroll
    for (int k = 0; k < kPerWave / kWave; ++k) {
        const int64_t t = first + k * kWave;
        keys[k] = t < a.rows ? key_at(a, t) : 0;
        if (t < a.rows) atomicAdd(&next[wave][keys[k] >> a.shift & (n - 1)], 1u);
    }
    __syncthreads();
    for (int k = tid; k < n; k += kSortThreads) {
        uint32_t b = base[k];
        for (int w = 0; w < kSortWaves; ++w) {
            const uint32_t c = next[w][k];
            next[w][k] = b;
            b += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kPerWave / kWave; ++k) {
        const int64_t t = first + k * kWave;
        const bool in = t < a.rows;
        const uint32_t digit = keys[k] >> a.shift & (n - 1);
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
        if (in) {
            a.keys_out[to] = keys[k];
            a.ids_out[to] = a.ids != nullptr ? a.ids[t] : (uint32_t)t;
        }
    }
}

struct SumArgs {
    const uint32_t *keys, *ids;  // sorted
    int64_t count, vocab, dim;
    const void *rows;
    int64_t rows_ld;
    int rows_type;
    void *grad;
    int64_t grad_ld;
    int grad_type;
    float scale;
    float *open;  // [segment][2][dim]: sums of the first and of the last token of a segment
    int64_t segments;
};

__device__ __forceinline__ void add4(const SumArgs &a, uint32_t v, int64_t n, int cols, f32x4 x) {
    const int64_t at = (int64_t)v * a.grad_ld + n;
    if (cols == 4) {
        store4(a.grad, at, a.grad_type, load4(a.grad, at, a.grad_type) + x * a.scale);
    } else {
        for (int r = 0; r < cols; ++r)
            put(a.grad, at + r, a.grad_type,
                element(a.grad, at + r, a.grad_type) + pick(x, r) * a.scale);
    }
}

constexpr int kSumThreads = 256;

// blockIdx.x: segment of the sorted order, blockIdx.y: columns, four a lane.
__global__ __launch_bounds__(kSumThreads) void embed_sum(SumArgs a) {
    __shared__ uint32_t key[kSeg + 2], id[kSeg];
    const int64_t first = (int64_t)blockIdx.x * kSeg;
    const int tid = threadIdx.x;
    if (tid < kSeg + 2) {
        const int64_t s = first + tid - 1;
        key[tid] = s >= 0 && s < a.count ? a.keys[s] : kNone;
    }
    if (tid < kSeg) id[tid] = first + tid < a.count ? a.ids[first + tid] : 0;
    __syncthreads();
    const int64_t n = ((int64_t)blockIdx.y * kSumThreads + tid) * 4;
    if (n >= a.dim) return;
    const int cols = (int)min((int64_t)4, a.dim - n);
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    bool begins = key[0] != key[1];  // whether the token's first row is in this segment
    int slot = 0;
    for (int k0 = 0; k0 < kSeg; k0 += 8) {
        f32x4 x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            x[k] = f32x4{0.f, 0.f, 0.f, 0.f};
            if (key[k0 + k + 1] >= (uint32_t)a.vocab) continue;
            const int64_t at = (int64_t)id[k0 + k] * a.rows_ld + n;
            if (cols == 4) {
                x[k] = load4(a.rows, at, a.rows_type);
            } else {
                for (int r = 0; r < 3; ++r)
                    if (r < cols) x[k][r] = element(a.rows, at + r, a.rows_type);
            }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int i = k0 + k + 1;
            const uint32_t v = key[i];
            if (v >= (uint32_t)a.vocab) break;  // none follow
            sum += x[k];
            const bool ends = key[i + 1] != v;
            if (!ends && i < kSeg) continue;
            if (begins && ends) {
                add4(a, v, n, cols, sum);
            } else {
                // 0: a token that came from the segment before, 1: one that begins here
                float *to = a.open + ((int64_t)blockIdx.x * 2 + (begins ? 1 : 0)) * a.dim + n;
                for (int r = 0; r < cols; ++r) to[r] = pick(sum, r);
            }
            sum = f32x4{0.f, 0.f, 0.f, 0.f};
            begins = true;
            slot = 1;
        }
    }
    (void)slot;
}

// blockIdx.x: segment; if a token begins in it and goes on behind its end, the
// token's sums in the order of the segments.
__global__ __launch_bounds__(kSumThreads) void embed_join(SumArgs a) {
    const int64_t seg = blockIdx.x, last = (seg + 1) * kSeg - 1;
    if (last + 1 >= a.count) return;
    const uint32_t v = a.keys[last];
    if (v >= (uint32_t)a.vocab || a.keys[last + 1] != v) return;
    if (seg > 0 && a.keys[seg * kSeg] == v && a.keys[seg * kSeg - 1] == v) return;
    const int64_t n = ((int64_t)blockIdx.y * kSumThreads + threadIdx.x) * 4;
    // the segments that it reaches
    int64_t lo = seg + 1, hi = a.segments - 1;  // the last whose first key is v
    while (lo < hi) {
        const int64_t mid = (lo + hi + 1) / 2;
        if (a.keys[mid * kSeg] == v) lo = mid;
        else hi = mid - 1;
    }
    if (n >= a.dim) return;
    const int cols = (int)min((int64_t)4, a.dim - n);
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    for (int64_t s = seg; s <= lo; ++s) {
        const float *from = a.open + (s * 2 + (s == seg ? 1 : 0)) * a.dim + n;
        f32x4 x = {0.f, 0.f, 0.f, 0.f};
        for (int r = 0; r < 4; ++r)
            if (r < cols) x[r] = from[r];
        sum += x;
    }
    add4(a, v, n, cols, sum);
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
    for (int k = 0; k < p.passes; ++k) {
        s.shift = k * p.bits;
        s.keys_out = reinterpret_cast<uint32_t *>(ws + p.keys[k & 1]);
        s.ids_out = reinterpret_cast<uint32_t *>(ws + p.ids[k & 1]);
        embed_count<<<dim3((unsigned)p.tiles), kSortThreads, 0, stream>>>(s);
        embed_place<<<dim3((unsigned)p.tiles), kSortThreads, 0, stream>>>(s, p.tiles);
        s.keys = s.keys_out, s.ids = s.ids_out;
    }
    SumArgs a = {};
    a.keys = s.keys, a.ids = s.ids, a.count = count, a.vocab = vocab, a.dim = dim;
    a.rows = rows, a.rows_ld = rows_stride, a.rows_type = rows_type;
    a.grad = grad, a.grad_ld = grad_stride, a.grad_type = grad_type, a.scale = scale;
    a.open = reinterpret_cast<float *>(ws + p.open), a.segments = p.segments;
    const dim3 grid((unsigned)p.segments, (unsigned)((dim + 4 * kSumThreads - 1) / (4 * kSumThreads)));
    embed_sum<<<grid, kSumThreads, 0, stream>>>(a);
    embed_join<<<grid, kSumThreads, 0, stream>>>(a);
    return hipGetLastError() == hipSuccess ? RCS_OK : RCS_EHIP;
}

}  // extern "C"
