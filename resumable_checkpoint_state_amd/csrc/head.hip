// head.hip -- losses of a language model's output head and their gradients,
// without the matrix of logits: softmax cross entropy, and the divergence from
// a teacher's top logits. gfx950 kernels and their C ABI.
//
// Mathematics. z = h w^T / tau, one row of `vocab` logits for each row of `dim` of h
// that has a loss, l = log sum_v exp z[v].
//   cross entropy (tau = 1, q the target's one place): loss = l - z[target]
//   a teacher's entries, q their softmax at tau:
//     loss = tau^2 sum_k q[k] (log q[k] - (z[index[k]] - l))
//   either way, with p = exp(z - l):
//     d loss / dh = tau (p - q) w,  d loss / dw = tau (p - q)^T h
// Exponentials are powers of two and logits in units of log 2 throughout.
//
// Mapping. The rows that have a loss are counted and placed one after another
// (head_count, head_prep), so that the rest costs nothing. Three matrix products with
// one body (`product`): the logits' tiles end as exponentials of 16 bits with a sum of
// each row's, the only thing of the size of the logits that is kept, and not without
// gradients; head_rows makes losses of the sums, and of the exponentials what the
// other two products read; head_finish adds up what was split. Rows are done in groups
// where their exponentials would exceed the caller's limit. Each sum has one order, and
// no float is added atomically.
//
// Float32 matrices are two half-precision planes, x 2^lift = high + low (22 bits; the
// low by low products, below 2^-22, are left out): three products of 16 bits are three
// times as fast as one of float32 on the matrix units, of which 153 TFLOP/s were
// measured, against 1,400 in half precision.
//
// Bounds. The three products of 8,192 x 50,257 x 768 in bfloat16 are 1,897 GFLOP: 1.26
// ms at the 1,504 TFLOP/s that a product of 16,384^3 reaches on this card. The whole
// call takes 1.70 to 1.74 ms; in a trace, where kernels are some 10% longer, the products take
// 618 us (logits, with their exponentials), 612 (hidden) and 595 (weight). At 131,072 x
// 4,096 with a tenth of the rows masked 18.6 to 19.0 ms, 6.16, 6.38 and 5.91 of it the
// products, 1,240 to 1,340 TFLOP/s. There, loads with a quarter of the
// matrix instructions took 5.54, 5.46 and 4.78 ms, and those instructions without loads
// 5.32, 5.52 and 5.47, at a clock that such work lowers to 2.0 GHz: what is lost is
// that the two do not overlap wholly.

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "rcs.h"
#include "rcs_internal.h"
#include "vocab.h"

#pragma clang fp contract(off)

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

#ifdef __HIP_DEVICE_COMPILE__
__device__ __forceinline__ f32x4 mfma(s16x8 a, s16x8 b, f32x4 c, BF16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma(s16x8 a, s16x8 b, f32x4 c, F16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
#endif
__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

template <int N>
struct Int {
    static constexpr int value = N;
};

// Tiles of a product: kX by kY outputs by a block of 2 by kY / 64 waves, each kX / 2
// by 64 of them, kK at a time, from two places in LDS in turn. The large ones (one
// block a CU) read least: 64 KB for 256 x 256 x 64 products. Products that have fewer
// of them than there are CUs are done in small ones (two blocks a CU). Four places of
// 32 columns each instead of two of 64 were slower.
constexpr int kK = 64;
template <bool SMALL>
struct Shape {
    static constexpr int kX = SMALL ? 128 : 256, kY = kX;
    static constexpr int kThreads = 2 * kY, kWaves = kThreads / kWave;
    static constexpr int kFx = kX / 32, kFy = 4;  // fragments of a wave
    static constexpr int kGroup = kX / 2;  // columns of the logits with a reference of their own
    static constexpr int kXBytes = kX * kK * 2, kStageBytes = 2 * kXBytes;
};

// What the kernels of one call tell each other, in device memory.
struct Scalars {
    int32_t count;        // rows that have a loss
    uint32_t retry;       // not 0: a row's largest logit was beyond its reference's reach
    uint32_t top_h, top_w;  // float32 only: bits of the largest finite magnitudes
};

// The power of two that brings a largest magnitude of these bits to [2^14, 2^15).
__device__ __forceinline__ int lift_of(uint32_t top) {
    const int e = (int)(top >> 23);
    return e == 0 ? 126 : min(141 - e, 126);
}
__device__ __forceinline__ float pow2(int e) { return ldexpf(1.f, e); }

// --------------------------------------------------------------- preparation

// Over the wave, by permutes within rows of 16 lanes and broadcasts between them.
template <class F>
__device__ __forceinline__ float wave_all(float x, float none, F f) {
    const auto step = [&](auto control, auto rows) {
        const int y = __builtin_amdgcn_update_dpp(
            __builtin_bit_cast(int, none), __builtin_bit_cast(int, x), decltype(control)::value,
            decltype(rows)::value, 0xF, false);
        x = f(x, __builtin_bit_cast(float, y));
    };
    step(Int<0x111>{}, Int<0xF>{});  // from 1, 2, 4 and 8 lanes before in the row
    step(Int<0x112>{}, Int<0xF>{});
    step(Int<0x114>{}, Int<0xF>{});
    step(Int<0x118>{}, Int<0xF>{});
    step(Int<0x142>{}, Int<0xA>{});  // the row before's last lane, to the second and fourth
    step(Int<0x143>{}, Int<0xC>{});  // the second row's last lane, to the third and fourth
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 63));
}
__device__ __forceinline__ float wave_sum(float x) {
    return wave_all(x, 0.f, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ float wave_max(float x) {
    return wave_all(x, -INFINITY, [](float a, float b) { return fmaxf(a, b); });
}

// What the rows' kernels read: the rows, their targets and where their results go.
struct RowArgs {
    Scalars *scalars;
    int32_t *rowmap;  // [i]: the i-th row that has a loss
    int64_t row0;
    const f32x2 *parts;
    int64_t groups, parts_ld, vocab;
    int group;  // columns
    void *g[2];
    int64_t gld;
    bool store;
    int gshift;
    const void *hidden, *weight;
    int64_t hld, wld, dim;
    int type;
    const void *index, *logits;
    int index_type, logits_type;
    int64_t entries, ignore;
    bool distill;
    float tau;
    float *losses, *compact;  // of the rows, and of those that have one
    float *targets;  // [i][entry]: logits of the targets, in units of log 2
    // DIRECT only, of each row: its reference, 2^(reference - lse) and the row times that
    float *ref, *factor;
    const uint16_t *h;
    uint16_t *scaled;
    int64_t pad;
    float *only_loss;  // where there is one row, the result too
};

// Column of entry k of the row, -1 where there is none; bad is set if it is not one
// of the vocabulary.
__device__ __forceinline__ int64_t target_at(const RowArgs &a, int64_t t, int k, bool &bad) {
    const int64_t at = a.distill ? t * a.entries + k : t;
    const int64_t v = index_at(a.index, at, a.index_type);
    if (a.distill && (v < 0 || element(a.logits, at, a.logits_type) == -INFINITY)) return -1;
    if (v >= 0 && v < a.vocab) return v;
    bad = true;
    return -1;
}

// flags[t]: whether row t has a loss; counts[b]: how many of the b-th `chunk` rows.
struct CountArgs {
    uint8_t *flags;
    int32_t *counts;
    int64_t rows, chunk;
    int chunks;
};
__global__ __launch_bounds__(256) void head_count(RowArgs a, CountArgs c) {
    __shared__ int32_t shared[256 / kWave];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int64_t first = blockIdx.x * c.chunk, behind = min(first + c.chunk, c.rows);
    int32_t n = 0;
    if (a.distill) {
        for (int64_t t = first + wave; t < behind; t += 256 / kWave) {
            bool any = false;
            for (int64_t k = lane; k < a.entries; k += kWave)
                any |= index_at(a.index, t * a.entries + k, a.index_type) >= 0 &&
                       element(a.logits, t * a.entries + k, a.logits_type) != -INFINITY;
            const bool flag = __any(any);
            if (lane == 0) c.flags[t] = flag;
            n += flag;
        }
    } else {
        for (int64_t t0 = first + wave * kWave; t0 < behind; t0 += 256) {
            const int64_t t = t0 + lane;
            const bool flag = t < behind && index_at(a.index, t, a.index_type) != a.ignore;
            if (t < behind) c.flags[t] = flag;
            n += __popcll(__ballot(flag));
        }
    }
    if (lane == 0) shared[wave] = n;
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int w = 1; w < 256 / kWave; ++w) n += shared[w];
    c.counts[blockIdx.x] = n;
    if (blockIdx.x == 0) *a.scalars = Scalars{};
}

// Rows of a matrix as the products read them: padded with zeros to `pad` columns,
// float32 as two half-precision planes (x * 2^lift = high + low).
struct Rows {
    const void *src;
    uint16_t *hi, *lo;
    int64_t ld, rows;
};
struct PrepArgs {
    Rows hidden, weight;  // weight.rows: 0 if the products read it where it is
    int64_t dim, pad;
    int type;
    void *grad;  // gradient of the hidden rows, or null
    int64_t grad_ld;
};

// float32 only: the largest finite magnitudes of the hidden rows that have a loss (the
// first kTopHidden blocks) and of the weight. One atomic a block: more would queue.
// Reads both once: 47 us for 4,096 rows and 50,257, of 768.
constexpr int kTopHidden = 64, kTopWeight = 192;
__global__ __launch_bounds__(1024) void head_top(PrepArgs a, const uint8_t *flags,
                                                 Scalars *scalars) {
    __shared__ uint32_t shared[1024 / kWave];
    const bool hidden = blockIdx.x < kTopHidden;
    const Rows &m = hidden ? a.hidden : a.weight;
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int64_t waves = (hidden ? kTopHidden : kTopWeight) * (1024 / kWave);
    uint32_t best = 0;
    auto take = [&](float x) {
        const uint32_t b = __float_as_uint(x) & 0x7FFFFFFFu;
        if (b < 0x7F800000u && b > best) best = b;
    };
    for (int64_t r = (blockIdx.x - (hidden ? 0 : kTopHidden)) * (int64_t)(1024 / kWave) + wave;
         r < m.rows; r += waves) {
        if (hidden && flags[r] == 0) continue;
        for (int64_t k = 4 * lane; k < a.dim; k += 4 * kWave) {
            if (k + 4 <= a.dim) {
                const f32x4 x = load4(m.src, r * m.ld + k, RCS_F32);
#pragma unroll
                for (int j = 0; j < 4; ++j) take(x[j]);
            } else {
                for (int64_t j = k; j < a.dim; ++j)
                    take(static_cast<const float *>(m.src)[r * m.ld + j]);
            }
        }
    }
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) best = max(best, (uint32_t)__shfl_xor((int)best, d));
    if (lane == 0) shared[wave] = best;
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int w = 1; w < 1024 / kWave; ++w) best = max(best, shared[w]);
    atomicMax(hidden ? &scalars->top_h : &scalars->top_w, best);
}

// Over a block of 256, every thread gets it.
__device__ __forceinline__ int32_t block_count(int32_t x, int32_t *shared) {
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) x += __shfl_xor(x, d);
    __syncthreads();
    if (threadIdx.x % kWave == 0) shared[threadIdx.x / kWave] = x;
    __syncthreads();
    return (shared[0] + shared[1]) + (shared[2] + shared[3]);
}

// Eight consecutive elements as they lie in memory.
template <class T>
struct Eight {
    static constexpr int kParts = T::kBytes / 2;
    u32x4 raw[kParts];
    __device__ __forceinline__ void load(const void *p, int64_t i) {
        const u32x4_half *q = reinterpret_cast<const u32x4_half *>(static_cast<const char *>(p) +
                                                                   i * T::kBytes);
#pragma unroll
        for (int k = 0; k < kParts; ++k) raw[k] = q[k];
    }
    __device__ __forceinline__ float at(int r) const {
        if constexpr (T::kBytes == 4) return __uint_as_float(raw[r / 4][r % 4]);
        else return value((uint16_t)(raw[0][r / 2] >> (16 * (r & 1))), T{});
    }
};

// A row's logits of kFew of its targets, each lane 8 columns at a time, two times 512
// columns of all of them under way together: the loads have no branch between them. A
// lane at the row's end reads the last eight columns, and leaves out those that are
// another's. (In head_targets 73 us for 8,192 rows of 32 entries and 768 columns, a
// gather of 403 MB at 5.5 TB/s; with each load waited for before the next, 132.)
template <class T, int kFew>
__device__ __forceinline__ void target_logits(const RowArgs &a, int64_t t, int k0, bool &bad,
                                              float &top, float *to) {
    const int lane = threadIdx.x % kWave;
    const int few = (int)min((int64_t)kFew, a.entries - k0);
    int column = -1;
    if (lane < few) column = (int)target_at(a, t, k0 + lane, bad);
    bad = __any(bad);
    int v[kFew];
    float dot[kFew] = {};
#pragma unroll
    for (int k = 0; k < kFew; ++k) v[k] = __builtin_amdgcn_readlane(column, k);
    if (a.dim < 8) {
        for (int k = 0; k < kFew; ++k)
            if (lane < a.dim)
                dot[k] = element(a.hidden, t * a.hld + lane, T::kType) *
                         element(a.weight, max(v[k], 0) * a.wld + lane, T::kType);
    } else {
        constexpr int kTimes = 2;
        for (int64_t n0 = 0; n0 < a.dim; n0 += kTimes * 8 * kWave) {
            Eight<T> x[kTimes], y[kTimes][kFew];
            int64_t skip[kTimes];
#pragma unroll
            for (int i = 0; i < kTimes; ++i) {
                const int64_t n = n0 + (i * kWave + lane) * 8, from = min(n, a.dim - 8);
                skip[i] = n - from;
                x[i].load(a.hidden, t * a.hld + from);
#pragma unroll
                for (int k = 0; k < kFew; ++k)  // (of a column that there is, in any case)
                    y[i][k].load(a.weight, max(v[k], 0) * a.wld + from);
            }
#pragma unroll
            for (int i = 0; i < kTimes; ++i)
#pragma unroll
                for (int k = 0; k < kFew; ++k)
#pragma unroll
                    for (int r = 0; r < 8; ++r)
                        if (r >= skip[i]) dot[k] = fmaf(x[i].at(r), y[i][k].at(r), dot[k]);
        }
    }
#pragma unroll
    for (int k = 0; k < kFew; ++k) {
        if (k >= few) continue;
        dot[k] = v[k] < 0 ? 0.f : wave_sum(dot[k]) * (kLog2e / a.tau);
        if (v[k] >= 0) top = fmaxf(top, dot[k]);
        if (lane == 0) to[k0 + k] = dot[k];
    }
}
// As a row's reference, the largest of its targets' logits: no larger than the row's
// largest. A target that is not a column leaves NaN in the first place.
__device__ __forceinline__ void target_row(const RowArgs &a, int64_t i, bool bad, float top) {
    if (bad) a.targets[i * a.entries] = __uint_as_float(0x7FC00000u);
    if (a.ref != nullptr) a.ref[i] = fabsf(top) < INFINITY ? top : 0.f;
}

// A wave does a row. A hidden row goes to the place that it has among those with a
// loss, and with one entry its target's logit is worked out; a row without a loss is
// left out, and its gradient and loss are cleared; kK rows more are zeros behind the
// last one, up to a whole step of the products. SOLO: there are no flags and counts of
// the rows yet: each block looks at all targets before its own, which saves a launch
// (5 us) where there are few. Bound by HBM: 42 us for 8,192 rows of 4,096, a tenth
// masked, which with their copies and their targets' rows are 181 MB.
template <class T, bool SOLO>
__global__ __launch_bounds__(256) void head_prep(PrepArgs a, RowArgs rows, CountArgs c) {
    __shared__ int32_t shared[256 / kWave];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int64_t blocks = (a.hidden.rows + 3) / 4, padding = blocks + kK / 4;
    const int64_t block = blockIdx.x;
    const bool hidden = block < padding;
    const Rows &m = hidden ? a.hidden : a.weight;
    int64_t r = 4 * (hidden ? block : block - padding) + wave, to = r;
    bool zero = false;
    if (hidden) {
        // rows with a loss before the block's first one; before the padding, all
        const int64_t first = min(4 * block, a.hidden.rows);
        const auto has = [&](int64_t t) {
            return SOLO ? index_at(rows.index, t, rows.index_type) != rows.ignore
                        : c.flags[t] != 0;
        };
        const bool all = block >= blocks;
        const int64_t chunk = SOLO || all ? 0 : first / c.chunk;
        int32_t n = 0;
        if (!SOLO)
            for (int k = threadIdx.x; k < (all ? c.chunks : chunk); k += 256) n += c.counts[k];
        if (SOLO || !all)
            for (int64_t t = (SOLO ? 0 : chunk * c.chunk) + threadIdx.x; t < first; t += 256)
                n += has(t);
        const int32_t before = block_count(n, shared);
        if (all) {
            if (block == blocks && threadIdx.x == 0) {
                rows.scalars->count = before;
                rows.scalars->retry = 0;
            }
            to = before + (4 * (block - blocks) + wave);
            if (to >= (before + kK - 1) / kK * kK) return;
            zero = true;
        } else {
            if (r >= a.hidden.rows) return;
            if (!has(r)) {
                if (lane == 0) rows.losses[r] = 0.f;
                if (a.grad != nullptr)
                    for (int64_t k = 4 * lane; k < a.dim; k += 4 * kWave)
                        put4(a.grad, r * a.grad_ld + k, a.type, f32x4{0.f, 0.f, 0.f, 0.f},
                             a.dim - k, false);
                return;
            }
            to = before;
            for (int64_t t = first; t < r; ++t) to += has(t);
            if (lane == 0) rows.rowmap[to] = (int32_t)r;
            if (rows.entries == 1) {
                bool bad = false;
                float top = -INFINITY;
                target_logits<T, 1>(rows, r, 0, bad, top, rows.targets + to);
                if (lane == 0) target_row(rows, to, bad, top);
            }
        }
    }
    if (r >= m.rows && !zero) return;
    uint16_t *hi = m.hi + to * a.pad;
    if (a.type == RCS_F32) {
        uint16_t *lo = m.lo + to * a.pad;
        const float up = pow2(lift_of(hidden ? rows.scalars->top_h : rows.scalars->top_w));
        for (int64_t k = 4 * lane; k < a.pad; k += 4 * kWave) {
            f32x4 x = {0.f, 0.f, 0.f, 0.f};
            if (!zero && k + 4 <= a.dim) {
                x = load4(m.src, r * m.ld + k, RCS_F32);
            } else if (!zero) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (k + j < a.dim) x[j] = static_cast<const float *>(m.src)[r * m.ld + k + j];
            }
            x *= up;
            const u32x2 h = {two(x[0], x[1], F16{}), two(x[2], x[3], F16{})};
            const f32x4 rest = x - four(h, F16{});
            *reinterpret_cast<u32x2 *>(hi + k) = h;
            *reinterpret_cast<u32x2 *>(lo + k) =
                u32x2{two(rest[0], rest[1], F16{}), two(rest[2], rest[3], F16{})};
        }
        return;
    }
    const uint16_t *from = static_cast<const uint16_t *>(m.src) + r * m.ld;
    for (int64_t k = 8 * lane; k < a.pad; k += 8 * kWave) {
        u32x4 x = {0, 0, 0, 0};
        if (!zero && k + 8 <= a.dim) {
            x = *reinterpret_cast<const u32x4_half *>(from + k);
        } else if (!zero) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (k + j < a.dim) x[j / 2] |= (uint32_t)from[k + j] << (16 * (j & 1));
        }
        *reinterpret_cast<u32x4 *>(hi + k) = x;
    }
}

// ------------------------------------------------------------------ products

enum Op { kLogits, kHidden, kWeight };

// How far, in units of log 2, a logit may be above its row's reference: the
// exponentials and the products with them then stay within float32's range.
constexpr float kReach = 64.f;

struct GemmArgs {
    const void *x[2], *y[2];  // planes; the second of each only with float32
    int64_t xld, yld;         // elements
    int64_t xsize, ysize;     // elements from the first to the last one in memory
    int64_t nx, ny, nk;       // extent of the product (ny, or nk of kWeight, at most: see count)
    int64_t kper;             // of nk, for one split of kHidden
    int xtiles, ytiles, splits;
    int whole, parts_of_rest;  // kWeight: tiles done whole, and splits of each of the rest
    int64_t row0;             // first row of this group of rows
    Scalars *scalars;
    // kLogits
    void *e[2];
    int64_t eld;
    f32x2 *parts;
    int64_t groups;
    float zscale;
    bool store, retry;
    const float *ref;
    // kHidden, and the rest of kWeight's tiles
    float *partial;
    int64_t pld;
    // kWeight
    void *out;
    int64_t old;
    int out_type;
    bool add;
    float scale;
    bool mean;
    int gshift;
};

typedef __attribute__((address_space(3))) char lds_char;

constexpr int kRefPlaces = 4;  // items whose rows' references are in LDS, at most
[[maybe_unused]] constexpr int kCalls = 4;  // loads of a wave for one operand

// How an operand's tile of R by kK lies in LDS: in `kCalls` loads a wave, each of
// 1,024 consecutive bytes (source: where a lane's 16 come from), and how a wave
// reads its fragments of 16 by 32 (base: of the first one; read: fragment i of the
// tile's half `half` of the sum).
template <bool KCONTIG, int R, bool PERM>
struct Side;

// The sum runs along memory's rows: R rows of kK consecutive values, eight
// 16-byte chunks (a line of 128 bytes) each, chunk c of row r at slot c ^ turn(r).
// A read of 16 rows is served 16 lanes at a time, the lanes of rows 0-3 and 12-15
// with those of rows 4-11 of the next chunk: turned so, each such group meets all
// 64 banks once. With PERM, fragments 2i and 2i + 1 take their 32 rows in turns of
// four, so that a lane's results from both are of eight consecutive rows.
template <int R, bool PERM>
struct Side<true, R, PERM> {
    static __device__ __forceinline__ int turn(int r) {
        return PERM ? (r >> 2 & 6) | (r >> 1 & 1) : r >> 1 & 7;
    }
    static __device__ __forceinline__ uint32_t source(int call, int lane, int64_t ld) {
        const int r = call * 8 + lane / 8, c = (lane % 8) ^ turn(r);
        return (uint32_t)(r * ld * 2 + c * 16);
    }
    static __device__ __forceinline__ uint32_t base(int at, int lane) {
        const int m = lane % 16, g = lane / 16;
        const int r = PERM ? 8 * (m >> 2) + (m & 3) : m;
        return (uint32_t)((at + r) * 128 + ((g ^ turn(r)) * 16));
    }
    static __device__ __forceinline__ s16x8 read(const lds_char *p, uint32_t base, int i,
                                                 int half) {
        const uint32_t at = (base ^ (uint32_t)(half * 64)) +
                            (PERM ? (i / 2) * 4096 + (i & 1) * 512 : i * 2048);
        return *(const __attribute__((address_space(3))) s16x8 *)(p + at);
    }
};

// The sum runs across memory's rows: kK rows of R consecutive values, read back
// transposed. The R / 16 pairs of chunks of row k are turned by a number that differs
// between the rows that one read takes.
template <int R, bool PERM>
struct Side<false, R, PERM> {
    static __device__ __forceinline__ int turn(int k) {
        return ((k & 3) | (k >> 3 & 3) << 2) & (R / 16 - 1);
    }
    static __device__ __forceinline__ uint32_t source(int call, int lane, int64_t ld) {
        constexpr int kSlots = R / 8;
        const int k = call * (kWave / kSlots) + lane / kSlots, slot = lane % kSlots;
        const int c = (((slot >> 1) ^ turn(k)) << 1) | (slot & 1);
        return (uint32_t)(k * ld * 2 + c * 16);
    }
    static __device__ __forceinline__ uint32_t base(int at, int lane) {
        const int s = lane % 16, k = 8 * (lane / 16) + s / 4;
        return (uint32_t)(k * R * 2 + (((at / 16) ^ turn(k)) * 32) + (s % 4) * 8);
    }
    static __device__ __forceinline__ s16x8 read(const lds_char *p, uint32_t base, int i,
                                                 int half) {
        typedef __attribute__((address_space(3))) s16x4 v;
        const lds_char *q = p + (base ^ (uint32_t)(i * 32)) + half * 32 * R * 2;
        const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((v *)q);
        const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((v *)(q + 4 * R * 2));
        return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    }
};

// The b-th of n items in an order that suits the chip's caches. A block does b, b +
// gridDim.x, ...; blocks are dispatched round-robin over the 8 XCDs, each with an L2
// of its own: an XCD takes a stretch of its own, so that what its 32 CUs do at once
// shares operand tiles.
[[maybe_unused]] __device__ __forceinline__ int near_item(int b, int n) {
    const int per = n / 8, more = n % 8, xcd = b % 8;
    return xcd * per + min(xcd, more) + b / 8;
}
// The tiles in bands of BAND y tiles, and along a band all y of an x, then the next. Of
// 4, 8 and 16, 8 is best for the logits, and 4 for the others (weight at 131,072 x
// 4,096: 5,901 us, with 8 6,142; at 50,257 x 768 they are the same).
template <int BAND>
__device__ __forceinline__ void tile_of(int at, int xtiles, int ytiles, int &tx, int &ty) {
    const int band = at / (BAND * xtiles), rest = at % (BAND * xtiles);
    const int high = min(BAND, ytiles - band * BAND);
    tx = rest / high;
    ty = band * BAND + rest % high;
}

// 16 bytes a lane from `at` bytes into the buffer on, to 1,024 consecutive bytes of
// LDS. (Written out, because the compiler would let each transposing read of LDS
// wait for all such loads, the ones for later steps too. It has no result
// register, and `arrive` below waits for it. The wait states: between a vector
// instruction that wrote one of the scalars and the load.)
[[maybe_unused]] __device__ __forceinline__ void load_lds(u32x4 buffer, uint32_t at, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(to),
                 "v"(at), "s"(buffer)
                 : "memory");
}

[[maybe_unused]] __device__ __forceinline__ void load_lds_dword(u32x4 buffer, uint32_t at, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(to),
                 "v"(at), "s"(buffer)
                 : "memory");
}

// The buffer of what an array of `size` bytes has from `at` on: loads behind its end
// give zeros.
[[maybe_unused]] __device__ __forceinline__ u32x4 buffer_of(const void *p, int64_t at, int64_t size) {
    const uint64_t from = reinterpret_cast<uint64_t>(p) + (uint64_t)at;
    const int64_t left = max((int64_t)0, min(size - at, (int64_t)0xFFFFFFFFLL));
    return u32x4{(uint32_t)from, (uint32_t)(from >> 32) & 0xFFFFu, (uint32_t)left, 0x00020000u};
}

// Part of a product: an output tile, or a split of its sum.
struct Item {
    int64_t x0, y0, k0;
    int per;  // steps of one pair of planes
    bool empty;  // a sum over nothing: one step, of zeros
    int split;  // kHidden: the split; kWeight: place among the partial tiles, or -1
};

// a and b of an even lane and of the odd one after it, as the even lane's a and b in
// the two lanes' a, and the odd one's in their b.
[[maybe_unused]] __device__ __forceinline__ void swap_rows(u32x4 &a, u32x4 &b, bool odd) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const uint32_t give = odd ? a[r] : b[r];
        const uint32_t got = (uint32_t)__builtin_amdgcn_mov_dpp((int)give, 0xB1, 0xF, 0xF, true);
        a[r] = odd ? got : a[r];
        b[r] = odd ? b[r] : got;
    }
}

// A store's cache policy: the exponentials are not kept in L2, where the product's tiles
// are (then 736 -> 700 us for 8,192 x 50,257 x 768).
[[maybe_unused]] constexpr int kStreamed = 2;

// LDS of a product's block.
template <bool DIRECT, bool SMALL>
constexpr int kSharedBytes =
    2 * Shape<SMALL>::kStageBytes + (DIRECT ? kRefPlaces * Shape<SMALL>::kY * 4 : 0);

// What the block-th of `blocks` blocks does of a product: items one after another, the
// loads running two steps ahead of the matrix instructions across their bounds, and an
// item's results stored while the next one's first step is multiplied.
template <class T, int OP, int PLANES, bool DIRECT, bool SMALL>
__device__ __forceinline__ void product(const GemmArgs &a, char *shared, int block, int blocks) {
#ifdef __HIP_DEVICE_COMPILE__  // the host needs the kernels' launch stubs alone
    using S = Shape<SMALL>;
    constexpr int kX = S::kX, kY = S::kY, kXBytes = S::kXBytes, kStageBytes = S::kStageBytes;
    constexpr int kFx = S::kFx, kFy = S::kFy;
    using X = Side<OP == kLogits, kX, OP == kLogits>;
    using Y = Side<OP != kWeight, kY, false>;
    static_assert(kX / 8 == kCalls * S::kWaves && kY / 8 == kCalls * S::kWaves, "whole tiles");
    static_assert(!DIRECT || OP == kLogits, "a form of the logits");
    lds_char *lds = (lds_char *)shared;
    const uint32_t lds_at = (uint32_t)(uintptr_t)lds;
    const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int wx = wave & 1, wy = wave >> 1;

    // the items of this launch, and this block's first one
    const int64_t count = a.scalars->count - a.row0;
    const int64_t ny = OP == kWeight ? a.ny : min(a.ny, count);
    const int64_t nk = OP == kWeight ? max((int64_t)0, min(a.nk, count)) : a.nk;
    if (ny <= 0 || (OP == kWeight && a.add && nk == 0)) return;
    if (OP == kLogits && a.retry && a.scalars->retry == 0) return;
    const int ytiles = (int)((ny + kY - 1) / kY), tiles = a.xtiles * ytiles;
    const int items = OP == kHidden   ? tiles * a.splits
                      : OP == kWeight ? a.whole + (tiles - a.whole) * a.parts_of_rest
                                      : tiles;
    int at = block;
    if (at >= items) return;
    auto item_of = [&](int index) {
        Item m;
        int tx, ty;
        int64_t kper = nk;
        m.k0 = 0;
        m.split = OP == kWeight ? -1 : 0;
        if (OP == kHidden) {
            index = near_item(index, items);
            m.split = index / tiles;
            index %= tiles;
            kper = a.kper;
            m.k0 = m.split * kper;
        } else if (OP == kLogits || index < a.whole) {
            index = near_item(index, OP == kLogits ? tiles : a.whole);
        } else {
            if (a.parts_of_rest > 1) {
                m.split = index - a.whole;
                const int64_t steps = (nk + kK - 1) / kK;
                kper = (steps + a.parts_of_rest - 1) / a.parts_of_rest * kK;
                m.k0 = m.split % a.parts_of_rest * kper;
            }
            index = a.whole + (index - a.whole) / a.parts_of_rest;
        }
        tile_of<OP == kLogits ? 8 : 4>(index, a.xtiles, ytiles, tx, ty);
        m.x0 = (int64_t)tx * kX;
        m.y0 = (int64_t)ty * kY;
        const int64_t n = max((int64_t)0, min(kper, nk - m.k0));
        m.per = (int)((n + kK - 1) / kK);
        m.empty = m.per == 0;
        if (m.empty) m.per = 1;
        return m;
    };
    constexpr int kPairsOfPlanes = PLANES == 1 ? 1 : 3;

    // loads, step after step and item after item
    uint32_t xsrc[kCalls], ysrc[kCalls];
#pragma unroll
    for (int c = 0; c < kCalls; ++c) {
        xsrc[c] = X::source(wave * kCalls + c, lane, a.xld);
        ysrc[c] = Y::source(wave * kCalls + c, lane, a.yld);
    }
    Item load = item_of(at);
    int load_at = at, load_pair = 0, load_step = 0;
    u32x4 bx, by;
    auto place_loads = [&] {
        const int64_t k = load.k0 + (int64_t)load_step * kK;
        const int64_t x = OP == kLogits ? load.x0 * a.xld + k : k * a.xld + load.x0;
        const int64_t y = OP != kWeight ? load.y0 * a.yld + k : k * a.yld + load.y0;
        const void *px = a.x[0], *py = a.y[0];
        if (PLANES > 1) {  // low by high, high by low, high by high: the large sums last,
            px = load_pair == 0 ? a.x[1] : px;  // which the small ones would add roundings to
            py = load_pair == 1 ? a.y[1] : py;
        }
        bx = buffer_of(px, x * 2, load.empty ? 0 : a.xsize * 2);
        by = buffer_of(py, y * 2, load.empty ? 0 : a.ysize * 2);
    };
    place_loads();
    // the c-th of the loads of a step's tiles (behind the last step: of zeros)
    auto load_one = [&](int stage, int c) {
        const uint32_t to = lds_at + (uint32_t)(stage * kStageBytes);
        if (c < kCalls) load_lds(bx, xsrc[c], to + (wave * kCalls + c) * 1024);
        else load_lds(by, ysrc[c - kCalls], to + kXBytes + (wave * kCalls + c - kCalls) * 1024);
    };
    // the references of the rows of an item
    int load_place = 0;
    auto load_refs = [&] {
        if constexpr (DIRECT) {
            const int r = wave % (kY / kWave) * kWave;
            const u32x4 rows = buffer_of(a.ref, (load.y0 + r) * 4, load.empty ? 0 : ny * 4);
            load_lds_dword(rows, (uint32_t)(lane * 4),
                           lds_at + 2 * kStageBytes + (load_place * kY + r) * 4);
            load_place = (load_place + 1) % kRefPlaces;
        }
    };
    auto next_loads = [&] {
        ++load_step;
        if (load_step == load.per) {
            load_step = 0;
            ++load_pair;
            if (load_pair == kPairsOfPlanes) {
                load_pair = 0;
                load_at += blocks;
                if (load_at < items) load = item_of(load_at);
                else load.empty = true;
                load_refs();
            }
        }
        place_loads();
    };

    f32x4 acc[kFx][kFy];
    auto clear = [&] {
#pragma unroll
        for (int i = 0; i < kFx; ++i)
#pragma unroll
            for (int j = 0; j < kFy; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    };
    // Float32 in small tiles, which leave the registers for it: every two steps' sums are
    // added up apart, a quarter of the roundings at the whole sum's size (half of the
    // gradients' error; 3 us of 33 for the products of 65 rows by 8,191 x 321).
    constexpr bool kPairwise = PLANES > 1 && SMALL;
    f32x4 whole[kPairwise ? kFx : 1][kPairwise ? kFy : 1];
    [[maybe_unused]] auto move = [&](auto how) {  // 0: none yet, 1: these too, 2: that is all
#pragma unroll
        for (int i = 0; i < kFx; ++i)
#pragma unroll
            for (int j = 0; j < kFy; ++j) {
                if constexpr (!kPairwise) continue;
                else if constexpr (decltype(how)::value == 0) whole[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
                else if constexpr (decltype(how)::value == 1) whole[i][j] += acc[i][j];
                else acc[i][j] = whole[i][j];
            }
    };
    const uint32_t xbase = X::base(wx * (kX / 2), lane);
    const uint32_t ybase = Y::base(wy * 64, lane);

    // While one half of a step is multiplied out of registers, the next half is read
    // into others. Between a step's halves, when every wave has read the whole of its
    // tile and the next one has arrived, the one after that is loaded in its place.
    // Each four products come with a read and, in a step's second half, a load: as a
    // stretch of loads, these would keep the products waiting while they queue (the
    // order is held by barriers to the compiler's scheduling).
    s16x8 fx[2][kFx], fy[2][kFy];
    auto read_one = [&](int stage, int i, auto half) {
        constexpr int h = decltype(half)::value;
        const lds_char *px = lds + stage * kStageBytes, *py = px + kXBytes;
        if (i < kFy) fy[h][i] = Y::read(py, ybase, i, h);
        fx[h][i] = X::read(px, xbase, i, h);
    };
    auto multiply = [&](auto half, auto between) {
        constexpr int h = decltype(half)::value;
#pragma unroll
        for (int i = 0; i < kFx; ++i) {
            between(i);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < kFy; ++j) acc[i][j] = mfma(fx[h][i], fy[h][j], acc[i][j], T{});
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // this wave's reads of LDS are done, and all but the last n of its accesses to
    // memory (which end in their order); then every wave's
    auto arrive = [&](auto behind) {
        constexpr int n = decltype(behind)::value;
        static_assert(n < 64, "of the counter");
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt((n & 15) | (n >> 4) << 14 | 7 << 4);  // vmcnt n, lgkmcnt 0
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };

    // The results of an item. kLogits: kStores stores, always, so that the next step's
    // tile, which was loaded before them, can be waited for without them.
    constexpr int kStores = OP == kLogits ? kFy * (1 + kFx / 2 * PLANES) : 0;
    float c1 = 1.f;
    if constexpr (OP == kLogits) {
        c1 = a.zscale;
        if (PLANES > 1) c1 = c1 * pow2(-lift_of(a.scalars->top_h)) * pow2(-lift_of(a.scalars->top_w));
    } else if constexpr (OP == kWeight) {
        c1 = a.scale * pow2(-a.gshift);
        if (a.mean) c1 /= (float)max(a.scalars->count, 1);
        if (PLANES > 1) c1 *= pow2(-lift_of(a.scalars->top_h));
    }
    auto finish = [&](const Item &m, int place) {
        int at_lane = lane;
        asm volatile("" : "+v"(at_lane));  // addresses are worked out here, not kept through the loop
        const int g = at_lane / 16, l16 = at_lane % 16;
        if constexpr (OP == kLogits) {
            const int64_t v0 = m.x0 + wx * (kX / 2);
            constexpr float kHead = __is_same(T, F16) ? 15.f : 0.f;
            if (m.x0 + kX > a.nx) {  // the last tile's columns behind the vocabulary
#pragma unroll
                for (int f = 0; f < kFx; ++f)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (v0 + 32 * (f / 2) + 8 * g + 4 * (f & 1) + r >= a.nx)
#pragma unroll
                            for (int j = 0; j < kFy; ++j) acc[f][j][r] = -INFINITY;
            }
            // rows behind the last one lie behind the buffers' ends, and are not stored
            const int64_t rows = min((int64_t)kY, ny - m.y0);
            const auto ebuf = [&](int k) {
                return __builtin_amdgcn_make_buffer_rsrc(
                    static_cast<uint16_t *>(a.e[k]) + m.y0 * a.eld, 0,
                    a.store ? (int)(uint32_t)(rows * a.eld * 2) : 0, 0x00020000);
            };
            const __amdgpu_buffer_rsrc_t eh = ebuf(0), el = ebuf(PLANES - 1);
            const __amdgpu_buffer_rsrc_t pb = __builtin_amdgcn_make_buffer_rsrc(
                a.parts + m.y0 * a.groups, 0, (int)(uint32_t)(rows * a.groups * 8), 0x00020000);
            const uint32_t part = g == 0 && v0 < a.nx ? (uint32_t)(v0 / S::kGroup * 8) : 0xFFFFFF00u;
#pragma unroll
            for (int j = 0; j < kFy; ++j) {
                const int i = wy * 64 + 16 * j + l16;
                float top = -INFINITY, sum = 0.f;
                const float less =
                    DIRECT ? -*(const __attribute__((address_space(3))) float *)(
                                  lds + 2 * kStageBytes + (place * kY + i) * 4)
                            : 0.f;
#pragma unroll
                for (int f = 0; f < kFx; ++f)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        acc[f][j][r] = fmaf(acc[f][j][r], c1, less);
                        top = fmaxf(top, acc[f][j][r]);
                    }
                top = fmaxf(top, __shfl_xor(top, 16));
                top = fmaxf(top, __shfl_xor(top, 32));
                if (DIRECT && top > kReach && i < rows) atomicOr(&a.scalars->retry, 1u);
                const float ref = DIRECT ? top : top == -INFINITY ? 0.f : top - kHead;
#pragma unroll
                for (int f = 0; f < kFx; ++f)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float e = exp2_(DIRECT ? acc[f][j][r] : acc[f][j][r] - ref);
                        acc[f][j][r] = e;
                        sum += e;
                    }
                sum += __shfl_xor(sum, 16);
                sum += __shfl_xor(sum, 32);
                __builtin_amdgcn_raw_buffer_store_b64(
                    u32x2{__float_as_uint(ref), __float_as_uint(sum)}, pb,
                    part == 0xFFFFFF00u ? part : part + (uint32_t)(i * a.groups * 8), 0, 0);
                u32x4 h[kFx / 2], l[kFx / 2];
#pragma unroll
                for (int p = 0; p < kFx / 2; ++p)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float x = acc[2 * p + r / 2][j][2 * r % 4];
                        const float y = acc[2 * p + r / 2][j][2 * r % 4 + 1];
                        h[p][r] = two(x, y, T{});
                        if (PLANES > 1)
                            l[p][r] = two(x - value((uint16_t)h[p][r], T{}),
                                          y - value((uint16_t)(h[p][r] >> 16), T{}), T{});
                    }
                // whole lines: first the even row of a pair of lanes, then the odd one
#pragma unroll
                for (int p = 0; p < kFx / 2; p += 2) {
                    const uint32_t to =
                        (uint32_t)(((i & ~1) * a.eld + v0 + 32 * (p + (l16 & 1)) + 8 * g) * 2);
                    const uint32_t row = (uint32_t)(a.eld * 2);
                    swap_rows(h[p], h[p + 1], l16 & 1);
                    __builtin_amdgcn_raw_buffer_store_b128(h[p], eh, to, 0, kStreamed);
                    __builtin_amdgcn_raw_buffer_store_b128(h[p + 1], eh, to + row, 0, kStreamed);
                    if (PLANES > 1) {
                        swap_rows(l[p], l[p + 1], l16 & 1);
                        __builtin_amdgcn_raw_buffer_store_b128(l[p], el, to, 0, kStreamed);
                        __builtin_amdgcn_raw_buffer_store_b128(l[p + 1], el, to + row, 0, kStreamed);
                    }
                }
            }
        } else if constexpr (OP == kHidden) {
#pragma unroll
            for (int j = 0; j < kFy; ++j) {
                const int64_t i = m.y0 + wy * 64 + 16 * j + l16;
                if (i >= ny) continue;
#pragma unroll
                for (int f = 0; f < kFx; ++f) {
                    const int64_t n = m.x0 + wx * (kX / 2) + 16 * f + 4 * g;
                    if (n >= a.pld) continue;
                    *reinterpret_cast<f32x4 *>(a.partial + (m.split * a.ny + i) * a.pld + n) =
                        acc[f][j];
                }
            }
        } else if (m.split >= 0) {
            float *to = a.partial + (int64_t)m.split * kX * kY;
#pragma unroll
            for (int j = 0; j < kFy; ++j)
#pragma unroll
                for (int f = 0; f < kFx; ++f)
                    *reinterpret_cast<f32x4 *>(to + (wy * 64 + 16 * j + l16) * kX + wx * (kX / 2) +
                                               16 * f + 4 * g) = acc[f][j] * c1;
        } else {
#pragma unroll
            for (int j = 0; j < kFy; ++j) {
                const int64_t v = m.y0 + wy * 64 + 16 * j + l16;
                if (v >= a.ny) continue;
#pragma unroll
                for (int f = 0; f < kFx; ++f) {
                    const int64_t n = m.x0 + wx * (kX / 2) + 16 * f + 4 * g;
                    put4(a.out, v * a.old + n, a.out_type, acc[f][j] * c1, a.nx - n, a.add);
                }
            }
        }
    };

    load_refs();
    constexpr int kEach = 2 * kCalls / kFx;  // loads with each read
    for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int c = 0; c < 8; ++c) load_one(k, c);
        next_loads();
    }
    arrive(Int<0>{});
#pragma unroll
    for (int i = 0; i < kFx; ++i) read_one(0, i, Int<0>{});
    int stage = 0, place = 0;
    bool stored = false;
    for (; at < items; at += blocks) {
        const Item m = item_of(at);
        clear();
        if constexpr (kPairwise) move(Int<0>{});
        for (int left = m.per * kPairsOfPlanes; left > 0; --left) {
            multiply(Int<0>{}, [&](int i) { read_one(stage, i, Int<1>{}); });
            if (kStores > 0 && stored) arrive(Int<kStores>{});
            else arrive(Int<0>{});
            stored = false;
            multiply(Int<1>{}, [&](int i) {
                read_one(stage ^ 1, i, Int<0>{});  // of nothing, behind the last step
#pragma unroll
                for (int c = 0; c < kEach; ++c) load_one(stage, i * kEach + c);
            });
            next_loads();
            stage ^= 1;
            if constexpr (kPairwise) {
                if (left & 1) move(Int<1>{}), clear();  // every other step, and the last one
            }
        }
        if constexpr (kPairwise) move(Int<2>{});
        finish(m, place);
        place = (place + 1) % kRefPlaces;
        stored = true;
    }
    arrive(Int<0>{});  // the loads of nothing have ended, too
#endif
}

template <class T, int OP, int PLANES, bool DIRECT, bool SMALL>
__global__ __launch_bounds__(Shape<SMALL>::kThreads, 2) void head_gemm(GemmArgs a) {
    __shared__ __attribute__((aligned(1024))) char shared[kSharedBytes<DIRECT, SMALL>];
    product<T, OP, PLANES, DIRECT, SMALL>(a, shared, (int)blockIdx.x, (int)gridDim.x);
}
// Both gradients' products, where neither fills the chip: 20 us for 512 rows by 8,191
// by 321 in half precision.
template <class T, int PLANES>
__global__ __launch_bounds__(Shape<true>::kThreads, 2) void head_gemms(GemmArgs hidden,
                                                                       GemmArgs weight,
                                                                       int hidden_blocks) {
    __shared__ __attribute__((aligned(1024))) char shared[kSharedBytes<false, true>];
    const int block = (int)blockIdx.x;
    if (block < hidden_blocks)
        product<T, kHidden, PLANES, false, true>(hidden, shared, block, hidden_blocks);
    else
        product<T, kWeight, PLANES, false, true>(weight, shared, block - hidden_blocks,
                                                 (int)gridDim.x - hidden_blocks);
}

// Four values of each of n splits, `apart` floats apart, added up in their order, the
// loads of up to eight splits under way together (16 need more registers and are slower
// where there are few: 44 us instead of 40 for head_finish with 5).
template <int N>
__device__ __forceinline__ void add_some(const float *from, int64_t apart, int n, int &k0,
                                         f32x4 &sum) {
    f32x4 x[N];
#pragma unroll
    for (int k = 0; k < N; ++k)
        x[k] = *reinterpret_cast<const f32x4 *>(from + min(k0 + k, n - 1) * apart);
#pragma unroll
    for (int k = 0; k < N; ++k)
        if (k0 + k < n) sum += x[k];
    k0 += N;
}
__device__ __forceinline__ f32x4 add_up(const float *from, int64_t apart, int n) {
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    int k = 0;
    while (n - k > 4) add_some<8>(from, apart, n, k, sum);
    if (n - k > 0) add_some<4>(from, apart, n, k, sum);
    return sum;
}

// The tiles of kWeight that were split: sums in the order of the splits, a wave a row.
template <bool SMALL>
__device__ __forceinline__ void weight_join(const GemmArgs &a, int block) {
    constexpr int kX = Shape<SMALL>::kX, kY = Shape<SMALL>::kY;
    const int64_t count = a.scalars->count - a.row0;
    if (a.add && count <= 0) return;
    const int rows = block * (256 / kWave) + threadIdx.x / kWave;
    const int lane = threadIdx.x % kWave, tile = a.whole + rows / kY, row = rows % kY;
    int tx, ty;
    tile_of<4>(tile, a.xtiles, a.ytiles, tx, ty);
    const int64_t v = (int64_t)ty * kY + row, n = (int64_t)tx * kX + 4 * lane;
    if (4 * lane >= kX || v >= a.ny || n >= a.nx) return;
    const float *from = a.partial + (int64_t)(tile - a.whole) * a.parts_of_rest * kX * kY +
                        row * kX + 4 * lane;
    const f32x4 x = add_up(from, kX * kY, a.parts_of_rest);
    put4(a.out, v * a.old + n, a.out_type, x, a.nx - n, a.add);
}

// ------------------------------------------------------------- rows of logits

constexpr int kRowThreads = 256;
constexpr int kMaxEntries = RCS_HEAD_MAX_ENTRIES;

struct Sum {
    static __device__ __forceinline__ float of(float a, float b) { return a + b; }
    static __device__ __forceinline__ float wave(float a) { return wave_sum(a); }
};
struct Max {
    static __device__ __forceinline__ float of(float a, float b) { return fmaxf(a, b); }
    static __device__ __forceinline__ float wave(float a) { return wave_max(a); }
};
// Over the block, in a fixed order; every lane gets it.
template <class F>
__device__ __forceinline__ float block_all(float x, float *shared) {
    x = F::wave(x);
    __syncthreads();
    if (threadIdx.x % kWave == 0) shared[threadIdx.x / kWave] = x;
    __syncthreads();
    float y = shared[0];
#pragma unroll
    for (int w = 1; w < kRowThreads / kWave; ++w) y = F::of(y, shared[w]);
    return y;
}

// The targets' logits where a row has several; a block does a row.
template <class T>
__global__ __launch_bounds__(kRowThreads) void head_targets(RowArgs a) {
    __shared__ float shared[kRowThreads / kWave];
    const int64_t i = a.row0 + blockIdx.x;
    if (i >= a.scalars->count) return;
    const int64_t t = a.rowmap[i];
    float top = -INFINITY;
    bool bad = false;
    constexpr int kFew = 4;
    for (int k0 = threadIdx.x / kWave * kFew; k0 < a.entries; k0 += kRowThreads / kWave * kFew)
        target_logits<T, kFew>(a, t, k0, bad, top, a.targets + i * a.entries);
    top = block_all<Max>(top, shared);
    bad = block_all<Max>(bad ? 1.f : 0.f, shared) > 0.f;  // (the first place has been written)
    if (threadIdx.x == 0) target_row(a, i, bad, top);
}

// Rows whose largest logit is beyond the reach of their reference get that logit as
// their reference. (Does nothing if there are none, like the product after it.)
__global__ __launch_bounds__(kRowThreads) void head_reach(RowArgs a) {
    const int lane = threadIdx.x % kWave;
    const int64_t local = blockIdx.x * (int64_t)(kRowThreads / kWave) + threadIdx.x / kWave;
    if (a.scalars->retry == 0 || a.row0 + local >= a.scalars->count) return;
    const f32x2 *parts = a.parts + local * a.parts_ld;
    float top = -INFINITY;
    for (int64_t k = lane; k < a.groups; k += kWave) top = fmaxf(top, parts[k][0]);
    top = wave_max(top);
    if (lane == 0 && top > kReach) a.ref[a.row0 + local] += top;
}

// Row i of the logits: the sum of its exponentials, the loss, and the exponentials
// made into what the gradients' products take. In general that is (softmax - target)
// * 2^gshift, from exponentials relative to a reference of each group of columns.
// DIRECT (bfloat16, whose range is float32's, and one target): they are relative to
// the row's reference, and so the row's factor is left to the other sides: the hidden
// gradient's rows are multiplied by it in the end, and the hidden rows for the
// weight's gradient here. This saves a pass over all exponentials (20 us instead of
// 330, which are 5 TB/s, with 8,192 rows of 50,257), and is one more rounding of what
// the weight's gradient is made of: with a teacher's many targets, too much of one.
template <class T, int PLANES, bool DIRECT>
__global__ __launch_bounds__(kRowThreads) void head_rows(RowArgs a) {
    __shared__ float shared[kRowThreads / kWave];
    __shared__ float sp[kMaxEntries], sz[kMaxEntries];
    __shared__ int64_t sv[kMaxEntries];
    const int tid = threadIdx.x;
    const int64_t local = blockIdx.x, i = a.row0 + local;
    const int64_t count = a.scalars->count;
    if (i >= count) {
        if (a.only_loss != nullptr && tid == 0) *a.only_loss = 0.f;
        // zeros up to a whole step of the products' sums over the rows
        if (!a.store || i >= a.row0 + (max((int64_t)0, count - a.row0) + kK - 1) / kK * kK) return;
        const u32x4 zero = {0, 0, 0, 0};
        for (int p = 0; p < PLANES; ++p) {
            u32x4 *g = reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(a.g[p]) + local * a.gld);
            for (int64_t k = tid; k < a.gld / 8; k += kRowThreads) g[k] = zero;
        }
        if (DIRECT) {
            u32x4 *h = reinterpret_cast<u32x4 *>(a.scaled + local * a.pad);
            for (int64_t k = tid; k < a.pad / 8; k += kRowThreads) h[k] = zero;
        }
        return;
    }
    const int64_t t = a.rowmap[i];
    const f32x2 *parts = a.parts + local * a.parts_ld;
    const float ref = DIRECT ? a.ref[i] : 0.f;
    float top = 0.f;
    if (!DIRECT) {
        top = -INFINITY;
        for (int64_t k = tid; k < a.groups; k += kRowThreads) top = fmaxf(top, parts[k][0]);
        top = block_all<Max>(top, shared);
    }
    float sum = 0.f;
    for (int64_t k = tid; k < a.groups; k += kRowThreads)
        sum += DIRECT ? parts[k][1] : parts[k][1] * exp2_(parts[k][0] - top);
    sum = block_all<Sum>(sum, shared);
    float lse2 = (DIRECT ? ref : top) + __log2f(sum);

    // the targets: their columns, probabilities and logits
    const int entries = (int)a.entries;
    for (int k = tid; k < entries; k += kRowThreads) {
        bool bad = false;
        sv[k] = target_at(a, t, k, bad);
        sz[k] = a.targets[i * a.entries + k];
        sp[k] = !a.distill ? 0.f
                : sv[k] < 0
                    ? -INFINITY
                    : element(a.logits, t * a.entries + k, a.logits_type) * (kLog2e / a.tau);
    }
    __syncthreads();
    if (sz[0] != sz[0]) lse2 = sz[0];
    float loss;
    if (!a.distill) {
        loss = (lse2 - sz[0]) * kLn2;
        if (loss < 0.f) loss = 0.f;
        if (tid == 0) sp[0] = 1.f;
    } else {
        float m = -INFINITY;
        for (int k = tid; k < entries; k += kRowThreads) m = fmaxf(m, sp[k]);
        m = block_all<Max>(m, shared);
        float s = 0.f;
        for (int k = tid; k < entries; k += kRowThreads)
            if (sv[k] >= 0) s += exp2_(sp[k] - m);
        s = block_all<Sum>(s, shared);
        const float l2 = m + __log2f(s);
        float x = 0.f;
        for (int k = tid; k < entries; k += kRowThreads) {
            const float y = sp[k] - l2, p = sv[k] >= 0 ? exp2_(y) : 0.f;
            if (sv[k] >= 0) x += p * (y - (sz[k] - lse2));
            sp[k] = p;
        }
        x = block_all<Sum>(x, shared);
        loss = x * kLn2 * a.tau * a.tau;
    }
    if (lse2 != lse2) loss = lse2;
    if (tid == 0) a.losses[t] = a.compact[i] = loss;
    if (tid == 0 && a.only_loss != nullptr) *a.only_loss = loss;
    if (!a.store) return;

    if constexpr (DIRECT) {
        // the factor is moved, by less than half a step of bfloat16, to where the target's
        // place, which most of the gradients comes from, rounds to no error
        float f = exp2_(ref - lse2);
        const float own = exp2_(sz[0] - lse2) - 1.f;
        const uint16_t held = (uint16_t)two(own / f, 0.f, T{});
        if (fabsf(own) > 0x1p-10f) f = own / value(held, T{});
        if (tid == 0) {
            a.factor[local] = f;
            if (sv[0] >= 0) static_cast<uint16_t *>(a.g[0])[local * a.gld + sv[0]] = held;
        }
        const u32x4 *from = reinterpret_cast<const u32x4 *>(a.h + i * a.pad);
        u32x4 *to = reinterpret_cast<u32x4 *>(a.scaled + local * a.pad);
        for (int64_t k = tid; k < a.pad / 8; k += kRowThreads) {
            u32x4 x = from[k];
#pragma unroll
            for (int r = 0; r < 4; ++r)
                x[r] = two(value((uint16_t)x[r], T{}) * f, value((uint16_t)(x[r] >> 16), T{}) * f,
                           T{});
            to[k] = x;
        }
        return;
    } else {
        // the row: exponentials times 2^(reference - lse + gshift)
        for (int64_t k = tid; k < a.gld / 8; k += kRowThreads) {
            const int64_t v = 8 * k;
            u32x4 *gh =
                reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(a.g[0]) + local * a.gld) + k;
            u32x4 *gl = reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(a.g[PLANES - 1]) +
                                                  local * a.gld) + k;
            u32x4 h = {0, 0, 0, 0}, l = {0, 0, 0, 0};
            if (v < a.vocab) {
                const float f = exp2_(parts[v / a.group][0] - lse2 + (float)a.gshift);
                h = *gh;
                if (PLANES > 1) l = *gl;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float x = value((uint16_t)h[r], T{}), y = value((uint16_t)(h[r] >> 16), T{});
                    if (PLANES > 1) {
                        x += value((uint16_t)l[r], T{});
                        y += value((uint16_t)(l[r] >> 16), T{});
                    }
                    x = v + 2 * r < a.vocab ? x * f : 0.f;
                    y = v + 2 * r + 1 < a.vocab ? y * f : 0.f;
                    h[r] = two(x, y, T{});
                    if (PLANES > 1)
                        l[r] = two(x - value((uint16_t)h[r], T{}),
                                   y - value((uint16_t)(h[r] >> 16), T{}), T{});
                }
            }
            *gh = h;
            if (PLANES > 1) *gl = l;
        }
    }
    __syncthreads();
    // less the targets: an index that comes several times once, with their sum
    for (int k = tid; k < entries; k += kRowThreads) {
        const int64_t v = sv[k];
        if (v < 0) continue;
        float p = 0.f;
        bool seen = false;
        for (int j = 0; j < entries; ++j)
            if (sv[j] == v) {
                p += sp[j];
                seen |= j < k;
            }
        if (seen) continue;
        // float32: of the softmax value that the others of the row were summed with, so
        // that one near 1 is off by its own roundings only, not by the logits'
        float own = exp2_(sz[k] - lse2);
        if (PLANES > 1)
            own = (value(static_cast<const uint16_t *>(a.g[0])[local * a.gld + v], T{}) +
                   value(static_cast<const uint16_t *>(a.g[1])[local * a.gld + v], T{})) *
                  pow2(-a.gshift);
        const float x = (own - p) * pow2(a.gshift);
        const uint32_t h = two(x, 0.f, T{});
        static_cast<uint16_t *>(a.g[0])[local * a.gld + v] = (uint16_t)h;
        if (PLANES > 1)
            static_cast<uint16_t *>(a.g[1])[local * a.gld + v] =
                (uint16_t)two(x - value((uint16_t)h, T{}), 0.f, T{});
    }
}

// ------------------------------------------------------------------- results

struct TotalArgs {
    const Scalars *scalars;
    const float *losses;  // of the rows that have one
    bool mean;
    float *loss;
};

// The sum or mean of the losses, in an order of its own: each of a block's 256 threads
// takes every 256th, in eight sums (whose loads are under way together).
__device__ __forceinline__ void total(const TotalArgs &a) {
    __shared__ double shared[256 / kWave];
    const int64_t count = a.scalars->count;
    constexpr int kSums = 8;
    double x[kSums] = {};
    for (int64_t i = threadIdx.x; i < count; i += 256 * kSums) {
        float loss[kSums];
#pragma unroll
        for (int k = 0; k < kSums; ++k) loss[k] = a.losses[min(i + 256 * k, count - 1)];
#pragma unroll
        for (int k = 0; k < kSums; ++k) x[k] += i + 256 * k < count ? (double)loss[k] : 0.0;
    }
    double y = ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) y += __shfl_xor(y, d);
    if (threadIdx.x % kWave == 0) shared[threadIdx.x / kWave] = y;
    __syncthreads();
    if (threadIdx.x == 0) {
        y = (shared[0] + shared[1]) + (shared[2] + shared[3]);
        *a.loss = (float)(a.mean ? y / (double)max(count, (int64_t)1) : y);
    }
}
__global__ __launch_bounds__(256) void head_total(TotalArgs a) { total(a); }

struct ReduceArgs {
    const Scalars *scalars;
    const int32_t *rowmap;
    int64_t row0, rows, dim, pld;
    const float *partial;
    int splits;
    void *out;
    int64_t old;
    int type;
    float scale;
    bool mean;
    int gshift;
    const float *factor;  // of each row, or null
    TotalArgs total;
};

// What follows the gradients' products: the gradients of the hidden rows, a wave a row,
// the sum of its splits in their order; behind them the weight's tiles that were split;
// and with the last group of rows the loss, by the first block. 40 us for 8,192 rows of
// 768 in 5 splits with 50,257 of the weight, and 42 for 4,096 columns in one.
struct FinishArgs {
    ReduceArgs hidden;
    GemmArgs weight;
    int first, hidden_blocks;
    bool small_weight;
};
__global__ __launch_bounds__(256) void head_finish(FinishArgs f) {
    const ReduceArgs &a = f.hidden;
    int block = (int)blockIdx.x;
    if (block < f.first) {
        total(a.total);
        return;
    }
    block -= f.first;
    if (block >= f.hidden_blocks) {
        block -= f.hidden_blocks;
        if (f.small_weight) weight_join<true>(f.weight, block);
        else weight_join<false>(f.weight, block);
        return;
    }
    const int64_t i = block * (int64_t)(256 / kWave) + threadIdx.x / kWave;
    const int64_t count = a.scalars->count;
    if (i >= a.rows || a.row0 + i >= count) return;
    float s = a.scale * pow2(-a.gshift);
    if (a.mean) s /= (float)count;
    if (a.type == RCS_F32) s *= pow2(-lift_of(a.scalars->top_w));
    if (a.factor != nullptr) s *= a.factor[i];
    const int64_t t = a.rowmap[a.row0 + i];
    for (int64_t n = 4 * (threadIdx.x % kWave); n < a.dim; n += 4 * kWave) {
        const float *from = a.partial + i * a.pld + n;
        const f32x4 x = add_up(from, a.rows * a.pld, a.splits);
        put4(a.out, t * a.old + n, a.type, x * s, a.dim - n, false);
    }
}

__global__ __launch_bounds__(256) void head_weight_out(const float *from, int64_t rows,
                                                       int64_t dim, void *out, int64_t ld,
                                                       int type, bool add) {
    const int64_t v = blockIdx.x * (int64_t)(256 / kWave) + threadIdx.x / kWave;
    if (v >= rows) return;
    for (int64_t n = 4 * (threadIdx.x % kWave); n < dim; n += 4 * kWave) {
        f32x4 x = {0.f, 0.f, 0.f, 0.f};
        for (int r = 0; r < 4; ++r)
            if (n + r < dim) x[r] = from[v * dim + n + r];
        put4(out, v * ld + n, type, x, dim - n, add);
    }
}

// ----------------------------------------------------------------- host side

constexpr int64_t kCus = 256;
constexpr int64_t kItemSteps = 24;   // what an item costs beside its steps, in steps
constexpr int64_t kSoloRows = 1024;  // of which each block counts those before its own
constexpr int64_t kChunks = 256;     // that the rows are counted in, at most
constexpr int64_t kMaxVocab = 1 << 22;  // a tile's rows of exponentials fit a buffer of 4 GB
constexpr int64_t kMinChunk = 128;  // rows done at a time at least

struct Plan {
    int planes;
    int64_t rows, vocab, dim, pad;   // pad: columns of the prepared rows
    int64_t chunk;                   // rows of a group
    int64_t eld, groups;
    int splits, whole, parts_of_rest;
    int64_t kper;
    bool copy_w, wide_out, direct, solo, small_logits, small_hidden, small_weight;
    // offsets in the workspace
    int64_t scalars, flags, counts, rowmap, losses, compact, h[2], w[2], e[2], parts, targets, ref, factor, scaled, partial, rest, acc, bytes;
};

bool direct_weight(const rcs_head *a) {
    return a->type != RCS_F32 && a->dim % kK == 0 && a->weight_stride % 8 == 0 &&
           (reinterpret_cast<uintptr_t>(a->weight) & 15u) == 0;
}

Plan plan_of(const rcs_head *a, int64_t entries, bool distill) {
    Plan p = {};
    const bool grads = a->grad_hidden != nullptr || a->grad_weight != nullptr;
    p.planes = a->type == RCS_F32 ? 2 : 1;
    p.rows = a->rows, p.vocab = a->vocab, p.dim = a->dim;
    p.pad = round_up(a->dim, kK);
    constexpr int kX = Shape<false>::kX;
    p.groups = round_up(a->vocab, kX) / Shape<true>::kGroup;  // or half as many
    p.eld = round_up(a->vocab, kX);
    p.copy_w = !direct_weight(a);
    // rows of a group: as many as fit the limit, in whole tiles
    const int64_t row_bytes = (grads ? p.eld * 2 * p.planes : 0) + p.groups * 8 +
                              (a->grad_hidden != nullptr ? 4 * p.pad : 0);
    p.chunk = round_up(a->rows > 0 ? a->rows : 1, kMinChunk);
    const int64_t fit = a->limit / row_bytes / kMinChunk * kMinChunk;
    if (p.chunk > fit) p.chunk = fit < kMinChunk ? kMinChunk : fit;
    // rows done at a time, and the logits' tiles
    const int64_t rows = p.chunk < a->rows ? p.chunk : a->rows;
    const auto tiles_of = [](int64_t x, int64_t y, int64_t tile) {
        return (x + tile - 1) / tile * ((y + tile - 1) / tile);
    };
    p.small_logits = tiles_of(a->vocab, rows, kX) < kCus;
    p.direct = a->type == RCS_BF16 && !distill && grads && !p.small_logits;
    p.solo = a->type != RCS_F32 && !distill && a->rows <= kSoloRows;
    // the weight's tiles in whole rounds, and the rest split to fill one more
    p.small_weight = tiles_of(a->dim, a->vocab, kX) < kCus;
    const int64_t weight_tile = p.small_weight ? Shape<true>::kX : kX;
    const int64_t weight_slots = p.small_weight ? 2 * kCus : kCus;
    const int64_t wtiles = tiles_of(a->dim, a->vocab, weight_tile);
    const int64_t rest = wtiles % weight_slots, wsteps = round_up(p.chunk, kK) / kK;
    p.parts_of_rest = 1;
    if (rest > 0) {
        int64_t n = weight_slots / rest;
        if (n > wsteps / kItemSteps) n = wsteps / kItemSteps;
        if (n > 1) p.parts_of_rest = (int)n;
    }
    p.whole = (int)(p.parts_of_rest > 1 ? wtiles - rest : wtiles);
    // splits of the hidden gradient's sum over the vocabulary: the number that fills
    // the chip's rounds best, each item costing about as much as kItemSteps steps more;
    // in large tiles unless even small ones have no 64 steps each
    const int64_t steps = round_up(a->vocab, kK) / kK;
    p.small_hidden = tiles_of(a->dim, rows, kX) * steps < 64 * kCus;
    const int64_t hidden_tile = p.small_hidden ? Shape<true>::kX : kX;
    int64_t slots = p.small_hidden ? 2 * kCus : kCus;
    if (a->grad_weight != nullptr && p.small_hidden && p.small_weight) {
        // both in one launch: what the weight's items leave of one round, if half of it
        const int64_t others = p.whole + (wtiles - p.whole) * p.parts_of_rest;
        if (others <= slots / 2) slots -= others;
    }
    const int64_t tiles = tiles_of(a->dim, rows, hidden_tile);
    int64_t best = 0;
    for (int64_t n = 1; n <= 64 && n <= steps; ++n) {
        const int64_t rounds = (tiles * n + slots - 1) / slots;
        const int64_t cost = rounds * ((steps + n - 1) / n + kItemSteps);
        if (n == 1 || cost < best) best = cost, p.splits = (int)n;
    }
    p.kper = (steps + p.splits - 1) / p.splits * kK;
    p.splits = (int)((steps * kK + p.kper - 1) / p.kper);
    p.wide_out = a->grad_weight != nullptr && a->grad_weight_type != RCS_F32 && p.chunk < a->rows;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t was = at;
        at = round_up(at + bytes, 256);
        return was;
    };
    p.scalars = take(sizeof(Scalars));
    p.flags = take(a->rows);
    p.counts = take(4 * kChunks);
    p.rowmap = take(4 * a->rows);
    p.losses = take(4 * a->rows);
    p.compact = take(4 * a->rows);
    for (int k = 0; k < p.planes; ++k) p.h[k] = take(2 * (a->rows + kK) * p.pad);
    if (p.copy_w)
        for (int k = 0; k < p.planes; ++k) p.w[k] = take(2 * a->vocab * p.pad);
    p.parts = take(8 * p.chunk * p.groups);
    p.targets = take(4 * a->rows * entries);
    if (p.direct) {
        p.ref = take(4 * a->rows);
        p.factor = take(4 * p.chunk);
        if (grads) p.scaled = take(2 * p.chunk * p.pad);
    }
    if (grads)
        for (int k = 0; k < p.planes; ++k) p.e[k] = take(2 * p.chunk * p.eld);
    if (a->grad_hidden != nullptr) p.partial = take(4 * p.splits * p.chunk * p.pad);
    if (a->grad_weight != nullptr && p.parts_of_rest > 1)
        p.rest = take(4 * weight_tile * weight_tile * (wtiles - p.whole) * p.parts_of_rest);
    if (p.wide_out) p.acc = take(4 * a->vocab * a->dim);
    p.bytes = at;
    return p;
}

struct Targets {
    const void *index;
    int index_type;
    int64_t entries;
    const void *logits;
    int logits_type;
    int64_t ignore;
    float tau;
    bool distill;
};

int check_head(const rcs_head *a) {
    if (a == nullptr) return RCS_EINVAL;
    if (a->rows < 0 || a->rows > kMaxRows || a->vocab < 1 || a->vocab > kMaxVocab || a->dim < 1 ||
        a->dim > kMaxDim || !is_type(a->type))
        return RCS_EINVAL;
    if (a->grad_weight != nullptr && !is_type(a->grad_weight_type)) return RCS_EINVAL;
    return RCS_OK;
}

// Tiles of a product, and the blocks that do it.
template <int OP, bool SMALL>
int64_t blocks_of(GemmArgs &g) {
    constexpr int kX = Shape<SMALL>::kX, kY = Shape<SMALL>::kY;
    g.xtiles = (int)(round_up(g.nx, kX) / kX);
    g.ytiles = (int)(round_up(g.ny, kY) / kY);
    const int64_t tiles = (int64_t)g.xtiles * g.ytiles;
    int64_t items = tiles;
    if (OP == kHidden) items *= g.splits;
    if (OP == kWeight) items = g.whole + (tiles - g.whole) * g.parts_of_rest;
    const int64_t slots = SMALL ? 2 * kCus : kCus;
    return items < slots ? items : slots;
}

template <class T, int OP, int PLANES, bool DIRECT, bool SMALL>
void launch_shape(GemmArgs &g, hipStream_t stream) {
    const unsigned blocks = (unsigned)blocks_of<OP, SMALL>(g);
    head_gemm<T, OP, PLANES, DIRECT, SMALL>
        <<<dim3(blocks), Shape<SMALL>::kThreads, 0, stream>>>(g);
}

template <class T, int OP, int PLANES, bool DIRECT>
void launch_gemm(GemmArgs &g, bool small, hipStream_t stream) {
    if constexpr (!DIRECT) {
        if (small) {
            launch_shape<T, OP, PLANES, DIRECT, true>(g, stream);
            return;
        }
    }
    launch_shape<T, OP, PLANES, DIRECT, false>(g, stream);
}

TotalArgs total_of(const rcs_head *a, const Plan &p, char *ws) {
    return TotalArgs{reinterpret_cast<Scalars *>(ws + p.scalars),
                     reinterpret_cast<float *>(ws + p.compact), a->mean != 0, a->loss};
}

template <class T, int PLANES, bool DIRECT>
void launch_products(const rcs_head *a, const Targets &tg, const Plan &p, const RowArgs &all,
                     char *ws, hipStream_t stream) {
    const bool grads = a->grad_hidden != nullptr || a->grad_weight != nullptr;
    Scalars *scalars = reinterpret_cast<Scalars *>(ws + p.scalars);
    const int gshift = __is_same(T, F16) ? 14 : 0;
    const float scale = a->scale * tg.tau;
    for (int64_t row0 = 0; row0 == 0 || row0 < a->rows; row0 += p.chunk) {
        const int64_t rows = a->rows - row0 < p.chunk ? a->rows - row0 : p.chunk;
        GemmArgs g = {};
        g.scalars = scalars;
        g.row0 = row0;
        g.scale = scale;
        g.mean = a->mean != 0;
        g.gshift = gshift;
        for (int k = 0; k < PLANES; ++k) {
            g.x[k] = p.copy_w ? ws + p.w[k] : a->weight;
            g.y[k] = ws + p.h[k] + 2 * row0 * p.pad;
            g.e[k] = ws + p.e[k];
        }
        const int64_t wld = p.copy_w ? p.pad : a->weight_stride;
        g.xld = wld, g.xsize = (a->vocab - 1) * wld + (p.copy_w ? p.pad : a->dim);
        g.yld = p.pad, g.ysize = (a->rows + kK - row0) * p.pad;
        g.nx = a->vocab, g.ny = rows, g.nk = p.pad, g.kper = p.pad;
        g.eld = p.eld, g.parts = reinterpret_cast<f32x2 *>(ws + p.parts), g.groups = p.groups;
        g.zscale = kLog2e / tg.tau;
        g.store = grads;
        RowArgs r = all;
        r.row0 = row0;
        r.parts = g.parts;
        r.group = p.small_logits ? Shape<true>::kGroup : Shape<false>::kGroup;
        r.groups = (a->vocab + r.group - 1) / r.group;
        for (int k = 0; k < PLANES; ++k) r.g[k] = g.e[k];
        r.gshift = gshift;
        if (DIRECT) g.ref = r.ref + row0;
        if (rows > 0) {
            if (tg.entries > 1) {
                const dim3 grid((unsigned)rows);
                if (PLANES > 1) head_targets<F32><<<grid, kRowThreads, 0, stream>>>(r);
                else head_targets<T><<<grid, kRowThreads, 0, stream>>>(r);
            }
            launch_gemm<T, kLogits, PLANES, DIRECT>(g, p.small_logits, stream);
            if (DIRECT) {
                head_reach<<<dim3((unsigned)((rows + 3) / 4)), kRowThreads, 0, stream>>>(r);
                g.retry = true;
                launch_gemm<T, kLogits, PLANES, DIRECT>(g, p.small_logits, stream);
            }
            const int64_t row_blocks = grads ? round_up(rows, kK) : rows;
            head_rows<T, PLANES, DIRECT><<<dim3((unsigned)row_blocks), kRowThreads, 0, stream>>>(r);
        }

        const bool hidden = a->grad_hidden != nullptr && rows > 0;
        const bool weight = a->grad_weight != nullptr;
        FinishArgs f = {};
        GemmArgs q = g;
        if (hidden) {
            for (int k = 0; k < PLANES; ++k) q.y[k] = g.e[k];
            q.yld = p.eld, q.ysize = p.chunk * p.eld;
            q.nx = a->dim, q.ny = rows, q.nk = round_up(a->vocab, kK), q.kper = p.kper;
            q.partial = reinterpret_cast<float *>(ws + p.partial), q.pld = p.pad;
            q.splits = p.splits;
            ReduceArgs &d = f.hidden;
            d.scalars = scalars, d.rowmap = r.rowmap, d.row0 = row0, d.rows = rows;
            d.dim = a->dim, d.pld = p.pad, d.partial = q.partial, d.splits = p.splits;
            d.out = a->grad_hidden, d.old = a->grad_hidden_stride, d.type = a->type;
            d.scale = scale, d.mean = g.mean, d.gshift = gshift;
            d.factor = r.factor;
            f.hidden_blocks = (int)((rows + 3) / 4);
            if (row0 + p.chunk >= a->rows) {
                d.total = total_of(a, p, ws);
                f.first = 1;
            }
        }
        GemmArgs &w = f.weight;
        int64_t joins = 0;
        if (weight) {
            w = g;
            for (int k = 0; k < PLANES; ++k)
                w.x[k] = DIRECT ? ws + p.scaled : static_cast<const char *>(g.y[k]),
                w.y[k] = g.e[k];
            w.xld = p.pad, w.xsize = DIRECT ? p.chunk * p.pad : g.ysize;
            w.yld = p.eld, w.ysize = p.chunk * p.eld;
            w.nx = a->dim, w.ny = a->vocab, w.nk = rows;
            w.out = p.wide_out ? ws + p.acc : a->grad_weight;
            w.old = p.wide_out ? a->dim : a->grad_weight_stride;
            w.out_type = p.wide_out ? RCS_F32 : a->grad_weight_type;
            w.add = row0 > 0 || (a->accumulate != 0 && !p.wide_out);
            w.partial = reinterpret_cast<float *>(ws + p.rest);
            w.whole = p.whole, w.parts_of_rest = p.parts_of_rest;
            f.small_weight = p.small_weight;
        }
        if (hidden && weight && p.small_hidden && p.small_weight) {
            const int64_t first = blocks_of<kHidden, true>(q), more = blocks_of<kWeight, true>(w);
            head_gemms<T, PLANES><<<dim3((unsigned)(first + more)), Shape<true>::kThreads, 0,
                                    stream>>>(q, w, (int)first);
        } else {
            if (hidden) launch_gemm<T, kHidden, PLANES, false>(q, p.small_hidden, stream);
            if (weight) launch_gemm<T, kWeight, PLANES, false>(w, p.small_weight, stream);
        }
        if (weight && p.parts_of_rest > 1) {
            const int tile = p.small_weight ? Shape<true>::kY : Shape<false>::kY;
            joins = ((int64_t)w.xtiles * w.ytiles - w.whole) * (tile / 4);
        }
        const int64_t blocks = f.first + f.hidden_blocks + joins;
        if (blocks > 0) head_finish<<<dim3((unsigned)blocks), 256, 0, stream>>>(f);
    }
    if (p.wide_out)
        head_weight_out<<<dim3((unsigned)((a->vocab + 3) / 4)), 256, 0, stream>>>(
            reinterpret_cast<float *>(ws + p.acc), a->vocab, a->dim, a->grad_weight,
            a->grad_weight_stride, a->grad_weight_type, a->accumulate != 0);
}

int head_call(const rcs_head *a, const Targets &tg, hipStream_t stream) {
    int rc = check_head(a);
    if (rc != RCS_OK) return rc;
    if (!is_index_type(tg.index_type)) return RCS_EINVAL;
    // (what is made of the temperature, too)
    if (!(tg.tau > 0.f && std::isfinite(kLog2e / tg.tau) && std::isfinite(tg.tau * tg.tau) &&
          std::isfinite(a->scale) && std::isfinite(a->scale * tg.tau)))
        return RCS_EINVAL;
    const int isize = index_size(tg.index_type);
    const int64_t entries = a->rows * tg.entries;
    Allocations seen;
    Extents reads(seen), writes(seen);
    if ((rc = reads.matrix(a->hidden, a->rows, a->dim, a->hidden_stride, a->type)) != RCS_OK ||
        (rc = reads.matrix(a->weight, a->vocab, a->dim, a->weight_stride, a->type)) != RCS_OK ||
        (rc = reads.array(tg.index, entries * isize, isize)) != RCS_OK)
        return rc;
    if (tg.distill) {
        if (!is_type(tg.logits_type)) return RCS_EINVAL;
        const int size = type_size(tg.logits_type);
        if ((rc = reads.array(tg.logits, entries * size, size)) != RCS_OK) return rc;
    }
    if (a->grad_hidden != nullptr &&
        (rc = writes.matrix(a->grad_hidden, a->rows, a->dim, a->grad_hidden_stride, a->type)) !=
            RCS_OK)
        return rc;
    if (a->grad_weight != nullptr &&
        (rc = writes.matrix(a->grad_weight, a->vocab, a->dim, a->grad_weight_stride,
                            a->grad_weight_type)) != RCS_OK)
        return rc;
    if (a->losses != nullptr && (rc = writes.array(a->losses, 4 * a->rows, 4)) != RCS_OK)
        return rc;
    if ((rc = writes.array(a->loss, 4, 4)) != RCS_OK) return rc;
    const Plan p = plan_of(a, tg.entries, tg.distill);
    if (a->workspace_bytes < p.bytes) return RCS_ESIZE;
    if ((rc = writes.array(a->workspace, p.bytes, 256)) != RCS_OK) return rc;
    if (writes.overlap(reads)) return RCS_EINVAL;

    char *ws = static_cast<char *>(a->workspace);
    Scalars *scalars = reinterpret_cast<Scalars *>(ws + p.scalars);
    RowArgs r = {};
    r.scalars = scalars;
    r.rowmap = reinterpret_cast<int32_t *>(ws + p.rowmap);
    r.parts_ld = p.groups, r.vocab = a->vocab;
    r.gld = p.eld, r.store = a->grad_hidden != nullptr || a->grad_weight != nullptr;
    r.hidden = a->hidden, r.weight = a->weight, r.hld = a->hidden_stride;
    r.wld = a->weight_stride, r.dim = a->dim, r.type = a->type;
    r.index = tg.index, r.logits = tg.logits, r.index_type = tg.index_type;
    r.logits_type = tg.logits_type, r.entries = tg.entries, r.ignore = tg.ignore;
    r.distill = tg.distill, r.tau = tg.tau;
    r.losses = a->losses != nullptr ? a->losses : reinterpret_cast<float *>(ws + p.losses);
    r.compact = reinterpret_cast<float *>(ws + p.compact);
    r.targets = reinterpret_cast<float *>(ws + p.targets);
    r.h = reinterpret_cast<const uint16_t *>(ws + p.h[0]), r.pad = p.pad;
    if (p.direct) {
        r.ref = reinterpret_cast<float *>(ws + p.ref);
        r.factor = reinterpret_cast<float *>(ws + p.factor);
        r.scaled = reinterpret_cast<uint16_t *>(ws + p.scaled);
    }
    const bool only = a->rows == 1 && !r.store;
    if (only) r.only_loss = a->loss;
    CountArgs c = {};
    c.flags = reinterpret_cast<uint8_t *>(ws + p.flags);
    c.counts = reinterpret_cast<int32_t *>(ws + p.counts);
    c.rows = a->rows;
    c.chunk = round_up((a->rows + kChunks - 1) / kChunks, 32);
    if (c.chunk == 0) c.chunk = 32;
    c.chunks = (int)((a->rows + c.chunk - 1) / c.chunk);
    PrepArgs h = {};
    const auto plane = [&](int64_t at) { return reinterpret_cast<uint16_t *>(ws + at); };
    h.hidden = Rows{a->hidden, plane(p.h[0]), plane(p.h[1]), a->hidden_stride, a->rows};
    h.weight = Rows{a->weight, plane(p.w[0]), plane(p.w[1]), a->weight_stride,
                    p.copy_w ? a->vocab : 0};
    h.dim = a->dim, h.pad = p.pad, h.type = a->type;
    h.grad = a->grad_hidden, h.grad_ld = a->grad_hidden_stride;
    if (!p.solo)
        head_count<<<dim3((unsigned)(c.chunks > 0 ? c.chunks : 1)), 256, 0, stream>>>(r, c);
    if (a->type == RCS_F32)
        head_top<<<kTopHidden + kTopWeight, 1024, 0, stream>>>(h, c.flags, scalars);
    const dim3 blocks((unsigned)((a->rows + 3) / 4 + kK / 4 + (h.weight.rows + 3) / 4));
    by_type(a->type, [&](auto type) {
        using T = decltype(type);
        if (p.solo) head_prep<T, true><<<blocks, 256, 0, stream>>>(h, r, c);
        else head_prep<T, false><<<blocks, 256, 0, stream>>>(h, r, c);
    });
    if (a->type == RCS_F32) launch_products<F16, 2, false>(a, tg, p, r, ws, stream);
    else if (a->type == RCS_F16) launch_products<F16, 1, false>(a, tg, p, r, ws, stream);
    else if (p.direct) launch_products<BF16, 1, true>(a, tg, p, r, ws, stream);
    else launch_products<BF16, 1, false>(a, tg, p, r, ws, stream);
    if ((a->grad_hidden == nullptr || a->rows == 0) && !only)
        head_total<<<1, 256, 0, stream>>>(total_of(a, p, ws));
    return hipGetLastError() == hipSuccess ? RCS_OK : RCS_EHIP;
}

}  // namespace

extern "C" {

int64_t rcs_head_workspace(const rcs_head *a, int64_t entries) {
    const int rc = check_head(a);
    if (rc != RCS_OK) return rc;
    if (entries < 0 || entries > kMaxEntries) return RCS_EINVAL;
    return plan_of(a, entries > 0 ? entries : 1, entries > 0).bytes;
}

int head_loss(const rcs_head *a, const void *targets, int index_type, int64_t ignore_index,
              hipStream_t stream) {
    Targets tg = {targets, index_type, 1, nullptr, 0, ignore_index, 1.f, false};
    return head_call(a, tg, stream);
}

int head_distill(const rcs_head *a, const void *indices, int index_type, const void *logits,
                 int logits_type, int64_t entries, float temperature, hipStream_t stream) {
    if (entries < 1 || entries > kMaxEntries) return RCS_EINVAL;
    Targets tg = {indices, index_type, entries, logits, logits_type, 0, temperature, true};
    return head_call(a, tg, stream);
}

}  // extern "C"
