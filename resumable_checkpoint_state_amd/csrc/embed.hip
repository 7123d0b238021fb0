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
// comes, no wave walks more than kSeg rows.
//
// Bounds. Each row is read once, and each gradient row that is met is read and written
// once: for 65,536 rows of 4,096 in bfloat16, 20,097 different tokens, one of them
// 3,787 times, 866 MB, which take 181 us at the 4.79 TB/s of a large copy. Measured: 246
// us, of which the sort is 24 (four launches), the sums 189 and the join 36. 8,192 float32
// rows of 768: the sort 20 us (one block's arithmetic), the sums 10, the join 6. 1,023
// rows: 5, 5 and 4, which launches alone take.

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "rcs.h"
#include "rcs_internal.h"
#include "vocab.h"

#pragma clang fp contract(off)

namespace {

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / kWave;
// Keys of a thread: at most, of the one block that sorts alone, and of one of several.
constexpr int kAloneKeys = 8, kTileKeys = 2;
constexpr int kAlone = kSortThreads * kAloneKeys, kTile = kSortThreads * kTileKeys;
constexpr int kMinBits = 6, kMaxBits = 9;  // of one pass
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
    __shared__ uint32_t bins[1 << kMaxBits];
    const int n = 1 << a.bits;
    for (int k = threadIdx.x; k < n; k += kSortThreads) bins[k] = 0;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kTileKeys; ++k) {
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
template <bool ALONE, int BITS, int KEYS>
__global__ __launch_bounds__(kSortThreads) void embed_sort(SortArgs a) {
    constexpr int kKeys = KEYS, kPlaces = kSortThreads * kKeys;
    constexpr int kBins = 1 << BITS;
    __shared__ uint32_t next[kSortWaves][kBins];  // of the wave: its keys so far, then where they begin
    __shared__ uint32_t sums[kSortWaves];
    __shared__ uint32_t keys_at[ALONE ? kPlaces : 1], ids_at[ALONE ? kPlaces : 1];
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const int first = wave * (kPlaces / kSortWaves) + lane;  // then every kWave-th
    const int64_t tile0 = (int64_t)blockIdx.x * kPlaces;
    uint32_t keys[kKeys], ids[kKeys];
#pragma unroll
    for (int k = 0; k < kKeys; ++k) {
        const int64_t t = tile0 + first + k * kWave;
        keys[k] = t < a.rows ? key_at(a, t) : kNone;
        ids[k] = t < a.rows && a.ids != nullptr ? a.ids[t] : (uint32_t)t;
    }
    for (int pass = 0; pass < (ALONE ? a.passes : 1); ++pass) {
        const int shift = ALONE ? pass * BITS : a.shift;
        // of each digit: all keys, and those of earlier tiles
        uint32_t mine = 0, before = 0;
        if (!ALONE && tid < kBins) {
#pragma unroll 8
            for (int i = 0; i < a.tiles; ++i) {
                const uint32_t c = a.hist[(int64_t)i * kBins + tid];
                mine += c;
                before += i < (int)blockIdx.x ? c : 0;
            }
        }
        for (int k = lane; k < kBins; k += kWave) next[wave][k] = 0;
        // each key's place among the wave's keys of its digit
        uint32_t place[kKeys];
#pragma unroll
        for (int k = 0; k < kKeys; ++k) {
            const bool in = keys[k] != kNone;
            const uint32_t digit = keys[k] >> shift & (kBins - 1);
            uint64_t same = __ballot(in);
#pragma unroll
            for (int b = 0; b < BITS; ++b) {
                const bool bit = digit >> b & 1;
                const uint64_t set = __ballot(bit);
                same &= bit ? set : ~set;
            }
            const int rank = __popcll(same & ((1ull << lane) - 1));
            place[k] = (in ? next[wave][digit] : 0) + rank;
            __builtin_amdgcn_wave_barrier();
            if (in && rank == 0) next[wave][digit] = place[k] + __popcll(same);
            __builtin_amdgcn_wave_barrier();
        }
        __syncthreads();
        if (ALONE && tid < kBins) {
#pragma unroll
            for (int w = 0; w < kSortWaves; ++w) mine += next[w][tid];
        }
        uint32_t run = mine;  // inclusive over the wave
#pragma unroll
        for (int d = 1; d < kWave; d *= 2) {
            const uint32_t up = (uint32_t)__shfl_up((int)run, d);
            if (lane >= d) run += up;
        }
        if (lane == kWave - 1) sums[wave] = run;
        __syncthreads();
        if (tid < kBins) {
            uint32_t at = run - mine + before;
#pragma unroll
            for (int w = 0; w < (kBins + kWave - 1) / kWave; ++w)
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
            if (keys[k] == kNone) continue;
            const uint32_t to = next[wave][keys[k] >> shift & (kBins - 1)] + place[k];
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
// Sorted places of one wave of the sums: few of them where there are few rows, so that
// more waves share them (1,023 rows of 321: 25 us with 32 places).
constexpr int kManySeg = 32, kFewSeg = 8;
constexpr int64_t kFewRows = 16384;

// A lane's columns n to n + cols - 1 of a row. A row's last few are read as the last of
// its last four: all loads are then alike, with no branch between them, and are under
// way together (values are made of them afterwards). NARROW: rows of fewer columns.
template <class T>
using Four = typename std::conditional<T::kBytes == 4, u32x4, u32x2>::type;
template <bool NARROW>
struct Cols {
    int64_t n, from;
    int cols;
    __device__ __forceinline__ Cols(int64_t at, int64_t dim) {
        n = at;
        cols = (int)max((int64_t)0, min((int64_t)kCols, dim - n));
        from = NARROW ? 0 : min(n, dim - kCols);
    }
    template <class T>
    __device__ __forceinline__ Four<T> load(const void *p, int64_t row, T) const {
        if constexpr (NARROW) {
            const f32x4 x = load_some(p, row, cols, T{});
            if constexpr (T::kBytes == 4) return __builtin_bit_cast(u32x4, x);
            else return u32x2{two(x[0], x[1], T{}), two(x[2], x[3], T{})};
        } else if constexpr (T::kBytes == 4) {
            return *reinterpret_cast<const u32x4_any *>(static_cast<const float *>(p) + row + from);
        } else {
            return *reinterpret_cast<const u32x2_any *>(static_cast<const uint16_t *>(p) + row +
                                                        from);
        }
    }
    template <class T>
    __device__ __forceinline__ f32x4 values(Four<T> raw, T) const {
        f32x4 x;
        if constexpr (T::kBytes == 4) x = __builtin_bit_cast(f32x4, raw);
        else x = four(raw, T{});
        if (NARROW || cols == 4) return x;
        return cols == 3   ? f32x4{x[1], x[2], x[3], 0.f}
               : cols == 2 ? f32x4{x[2], x[3], 0.f, 0.f}
                           : f32x4{x[3], 0.f, 0.f, 0.f};
    }
    template <class T>
    __device__ __forceinline__ void store(void *p, int64_t row, f32x4 x, T) const {
        store_some(p, row + n, cols, x, T{});
    }
};

// A wave does a segment of the sorted order and kCols columns a lane.
template <class R, class G, int kSeg, bool NARROW>
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
    const Cols<NARROW> c((item % a.parts * kWave + lane) * kCols, a.dim);
    const uint32_t vocab = (uint32_t)a.vocab;
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    bool begins = __builtin_amdgcn_readlane(key, 0) != __builtin_amdgcn_readlane(key, 1);
    for (int k0 = 0; k0 < kSeg; k0 += kBatch) {
        uint32_t v[kBatch + 1];
        Four<R> x[kBatch];
        Four<G> y[kBatch];  // the gradient: where a token goes on, it is not used
#pragma unroll
        for (int k = 0; k <= kBatch; ++k) v[k] = __builtin_amdgcn_readlane(key, k0 + k + 1);
        if (v[0] >= vocab) break;  // no more tokens
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const uint32_t t = __builtin_amdgcn_readlane(id, k0 + k + 1);
            const uint32_t row = v[k] < vocab ? v[k] : v[0];
            x[k] = c.load(a.rows, (int64_t)(v[k] < vocab ? t : 0) * a.rows_ld, R{});
            y[k] = c.load(a.grad, (int64_t)row * a.grad_ld, G{});
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (v[k] >= vocab) break;
            sum += c.values(x[k], R{});
            const bool ends = v[k + 1] != v[k];
            if (!ends && k0 + k + 1 < kSeg) continue;
            if (c.cols > 0) {
                if (begins && ends) {
                    c.store(a.grad, (int64_t)v[k] * a.grad_ld, c.values(y[k], G{}) + sum * a.scale,
                            G{});
                } else {
                    // 0: a token that came from the segment before, 1: one that begins here
                    c.store(a.open, (seg * 2 + (begins ? 1 : 0)) * a.dim, sum, F32{});
                }
            }
            sum = f32x4{0.f, 0.f, 0.f, 0.f};
            begins = true;
        }
    }
}

// blockIdx.x: segment; if a token begins in it and goes on behind its end, the token's
// sums in the order of the segments, kCols columns a lane, the block's four waves a
// quarter of the segments each. The blocks of a segment share its columns.
constexpr int kJoinParts = 8;
template <class G, int kSeg, bool NARROW>
__global__ __launch_bounds__(kSumThreads) void embed_join(SumArgs a) {
    __shared__ f32x4 shared[kSumThreads];
    const int64_t seg = blockIdx.x, last = (seg + 1) * kSeg - 1;
    if (last + 1 >= a.count) return;
    const uint32_t v = a.keys[last], after = a.keys[last + 1], begin = a.keys[seg * kSeg];
    const uint32_t before = seg > 0 ? a.keys[seg * kSeg - 1] : kNone;
    if (v >= (uint32_t)a.vocab || after != v || (begin == v && before == v)) return;
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    // the last segment that it reaches: the last whose first key it is
    int64_t lo = seg;
    for (bool all = true; all;) {
        const int64_t s = lo + 1 + lane;
        const uint64_t here = __ballot(s < a.segments && a.keys[min(s, a.segments - 1) * kSeg] == v);
        all = here == ~0ull;
        lo += all ? kWave : __builtin_ctzll(~here);
    }
    constexpr int kWaves = kSumThreads / kWave;
    const int64_t each = (lo - seg + kWaves) / kWaves;  // of lo - seg + 1 segments
    const int64_t first = seg + wave * each, behind = min(first + each, lo + 1);
    for (int part = blockIdx.y; part < a.parts; part += gridDim.y) {
        const Cols<NARROW> c(((int64_t)part * kWave + lane) * kCols, a.dim);
        const int64_t row = (int64_t)v * a.grad_ld;
        const Four<G> old = c.load(a.grad, row, G{});
        f32x4 sum = {0.f, 0.f, 0.f, 0.f};
        for (int64_t s0 = first; s0 < behind; s0 += kBatch) {
            u32x4 x[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int64_t s = min(s0 + k, behind - 1);
                x[k] = c.load(a.open, (s * 2 + (s == seg ? 1 : 0)) * a.dim, F32{});
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (s0 + k < behind) sum += c.values(x[k], F32{});
        }
        shared[threadIdx.x] = sum;
        __syncthreads();
        if (wave == 0 && c.cols > 0) {
#pragma unroll
            for (int w = 1; w < kWaves; ++w) sum += shared[w * kWave + lane];
            c.store(a.grad, row, c.values(old, G{}) + sum * a.scale, G{});
        }
        __syncthreads();
    }
}

// ----------------------------------------------------------------- host side

constexpr int64_t kMaxTokens = 1 << 30;

struct Plan {
    int passes, bits;
    int tiles, seg;
    int64_t segments;
    int64_t keys[2], ids[2], hist, open, bytes;
};

Plan plan_of(int64_t rows, int64_t vocab, int64_t dim) {
    Plan p = {};
    int bits = 1;
    while ((vocab >> bits) != 0) ++bits;  // the keys are 0 to vocab
    p.passes = (bits + kMaxBits - 1) / kMaxBits;
    p.bits = kMinBits;
    while (p.bits * p.passes < bits) ++p.bits;
    p.tiles = (int)((rows + kTile - 1) / kTile);
    if (rows <= kAlone) p.tiles = 1;
    p.seg = rows <= kFewRows || dim < kCols ? kFewSeg : kManySeg;
    p.segments = (rows + p.seg - 1) / p.seg;
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

template <class F>
void by_bits(int bits, F f) {
    if (bits == 6) f(std::integral_constant<int, 6>{});
    else if (bits == 7) f(std::integral_constant<int, 7>{});
    else if (bits == 8) f(std::integral_constant<int, 8>{});
    else f(std::integral_constant<int, 9>{});
}

int check_sizes(int64_t rows, int64_t vocab, int64_t dim) {
    return rows < 0 || rows > kMaxRows || vocab < 1 || vocab > kMaxTokens || dim < 1 ||
                   dim > kMaxDim
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
    Allocations seen;
    Extents reads(seen), writes(seen);
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
        by_bits(p.bits, [&](auto bits) {
            constexpr int kBits = decltype(bits)::value;
            if (count <= kSortThreads)
                embed_sort<true, kBits, 1><<<1, kSortThreads, 0, stream>>>(s);
            else if (count <= 3 * kSortThreads)
                embed_sort<true, kBits, 3><<<1, kSortThreads, 0, stream>>>(s);
            else embed_sort<true, kBits, kAloneKeys><<<1, kSortThreads, 0, stream>>>(s);
        });
    }
    for (int k = 0; k < p.passes && p.tiles > 1; ++k) {
        to(k & 1);
        s.shift = k * p.bits;
        embed_count<<<dim3((unsigned)p.tiles), kSortThreads, 0, stream>>>(s);
        by_bits(p.bits, [&](auto bits) {
            embed_sort<false, decltype(bits)::value, kTileKeys>
                <<<dim3((unsigned)p.tiles), kSortThreads, 0, stream>>>(s);
        });
        s.keys = s.keys_out, s.ids = s.ids_out;
    }
    SumArgs a = {};
    a.keys = s.keys_out, a.ids = s.ids_out, a.count = count, a.vocab = vocab, a.dim = dim;
    a.rows = rows, a.rows_ld = rows_stride;
    a.grad = grad, a.grad_ld = grad_stride, a.scale = scale;
    a.open = reinterpret_cast<float *>(ws + p.open), a.segments = p.segments;
    a.parts = (int)((dim + kCols * kWave - 1) / (kCols * kWave));
    const dim3 grid((unsigned)((p.segments * a.parts + 3) / 4));
    const dim3 joins((unsigned)p.segments, (unsigned)(a.parts < kJoinParts ? a.parts : kJoinParts));
    by_type(grad_type, [&](auto g) {
        using G = decltype(g);
        const auto run = [&](auto seg, auto narrow) {
            constexpr int kSeg = decltype(seg)::value;
            constexpr bool kNarrow = decltype(narrow)::value;
            by_type(rows_type, [&](auto r) {
                embed_sum<decltype(r), G, kSeg, kNarrow><<<grid, kSumThreads, 0, stream>>>(a);
            });
            embed_join<G, kSeg, kNarrow><<<joins, kSumThreads, 0, stream>>>(a);
        };
        const std::integral_constant<int, kFewSeg> few{};
        if (dim < kCols) run(few, std::true_type{});
        else if (p.seg == kFewSeg) run(few, std::false_type{});
        else run(std::integral_constant<int, kManySeg>{}, std::false_type{});
    });
    return hipGetLastError() == hipSuccess ? RCS_OK : RCS_EHIP;
}

}  // extern "C"
