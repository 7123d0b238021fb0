// list.inl -- the clipped AdamW update over a list of tensors: weights and
// gradients of 32 or 16 bits, moments in 32 or in 8 bits, and the list's state
// as the flat arrays of a step file. gfx950 kernels and their C ABI; the last
// part of rcs.hip, whose final reduction, workspaces and checks it uses.
//
// Mathematics. For tensor k of the list, element i, with every float32
// operation rounded on its own:
//   norm = sqrt(sum_k sum_i (double)(g_k[i] * gscale)^2), in float64
//   s    = (float)(clip / norm) if norm > clip else 1
//   gp   = (g * gscale) * s
//   m    = b1 m + (1 - b1) gp           v = b2 v + (1 - b2) (gp gp)
//   w    = w (1 - lr wd_k) - (lr (m / bc1)) / (sqrt(v / bc2) + eps)
// with bc = 1 - b^t; nothing changes if norm is not finite. With float32
// weights, gradients and moments and the default betas and eps this is
// adamw_clip_step's sequence, bit for bit for equal s.
//
// Moments in 8 bits. Each tensor is cut into blocks of 128 elements; a block
// has one exponent byte for m and one for v. A value is a float of 3 mantissa
// bits, held as its distance, in units of the last of these bits, from the
// bottom of the block's range: with B = 8 e - 127 (m) or 8 e - 255 (v), e the
// biased exponent of the smallest power of two not below the block's largest
// magnitude, code k > 0 stands for the float whose bits are (k + B) << 20 and
// k = 0 for zero. The range is 15.75 octaves for m and 31.75 for v (as many
// for sqrt(v)). Decoding is an add and a shift, encoding an add, a shift and a
// subtraction, all on the float's bits: no table, no division, no product with
// a scale, and decode(encode(decode(x))) is decode(x) exactly, so a state
// that went through a step file continues bit-identically.
//   Rounding: an update adds 20 random bits below the third mantissa bit and
// cuts (stochastic rounding, which keeps the mean). v changes by at most one
// part in a thousand per update while its grid's steps are 1/16 to 1/8, so with
// nearest rounding it would never move again once it is near its scale. The
// random bits are a hash of (seed, t, element), so an update is a function of
// its inputs and a resumed run repeats it. Below the smallest value, m goes to
// the nearer of it and zero (rounding up at random there would now and then
// make a step of the whole range), and v > 0 goes to the smallest value: v is
// zero only if it is exactly zero, so that no m is divided by eps alone.
//
// Mapping. A table row per tensor (pointers, length, decay, types) and one
// entry per chunk of 512 elements (tensor, chunk within it) live in device
// memory and are made once, when the list is. One wave takes one chunk: it
// reads its entry and row through scalar loads and then streams its elements in
// two rounds of 4 consecutive ones per lane, so that each access of a wave
// covers whole lines (8 a lane put the halves of a float32 line into two
// accesses: 802 against 683 us); the accesses need only the element's own
// alignment, so tensors may be views at any offset. Chunks
// are sorted by the types of weights and gradients; each pair of them has a
// kernel and a launch of its own. Bound by HBM, beside 8-bit moments of 16-bit
// weights nearly as much by the vector instructions.

#include <algorithm>
#include <cfloat>
#include <new>
#include <type_traits>

namespace {

constexpr int kBlock = RCS_LIST_BLOCK;  // elements that share a block exponent
// Elements of one wave. The update of the 124,356,864-element float32 list in
// one process, same buffers: 607 us a step with 512 elements, 615 with 256,
// 624 with 1,024 (the flat update: 604).
constexpr int kChunk = 512;
static_assert(kChunk % kBlock == 0 && kChunk % (8 * kWave) == 0, "whole blocks and vectors");
// Norm pass: a block of 16 waves per CU, each with 4 loads of 16 bytes a lane in
// flight, in runs of 4 chunks (of float32 or bfloat16 gradients of the same
// list: 86 and 51 us; 8 waves with 8 loads and runs of 8: 89 and 52; runs of
// one stretch per wave: 97 and 57).
constexpr int kListNormThreads = 1024;
constexpr int kRun = 4;
constexpr int kDeep = 4;
// The norm's buffers: partial sums, record, the count of blocks that have left
// theirs, and, in a stream's workspace, which has the same layout, the norm of
// its last update over a list (whose record is the list's own).
constexpr size_t kNormRecordAt = (size_t)kNormMaxBlocks * sizeof(double);
constexpr size_t kNormArrivedAt = kNormRecordAt + 128;
constexpr size_t kNormLastAt = kNormRecordAt + 192;
constexpr size_t kNormBytes = kNormRecordAt + 256;
static_assert(sizeof(ClipScalars) <= 128, "the record ends before the count");
// Lowest block exponents (biased): the smallest value and, for m, half of it
// are then normal floats.
constexpr int kLowM = 18, kLowV = 33;
constexpr uint32_t kHashA = 0x9E3779B1u, kHashB = 0xC2A3F1D7u, kHashC = 0x5BD9E4B5u,
                   kHashK = 0x7F4A7C15u;

// One tensor of the list, in device memory. All but c is one scalar load of 64
// bytes.
struct Row {
    void *w;
    const void *g;  // null: the tensor has no gradient and is left alone
    void *m, *v;
    union {
        uint16_t *e;    // block exponents of the 8-bit moments: m's low, v's high byte
        int64_t shift;  // 32-bit moments: chunks begin this many elements early
    };
    int64_t n;
    int64_t off;  // elements of the list before this tensor
    float wd;
    uint32_t types;  // RCS_F32, RCS_BF16, RCS_F16 of w, of g and of c, a byte each
    void *c;         // low-precision copy of w, or null
    __host__ __device__ int wt() const { return (int)(types & 0xFFu); }
    __host__ __device__ int gt() const { return (int)((types >> 8) & 0xFFu); }
    __host__ __device__ int ct() const { return (int)((types >> 16) & 0xFFu); }
};

// A chunk: the row of its tensor in the lower half, its number there in the
// upper one. With 8-bit moments chunk k begins at element k * kChunk. With
// 32-bit ones the boundaries lie where m's address is a multiple of 256 bytes
// (as far as arrays share their phase, whole lines then belong to one wave:
// 65 -> 58 us a step of a 12.7M-element bfloat16 list of odd sizes), so the
// first chunk may be short: chunk k begins `shift` elements before that.
typedef uint64_t Chunk;
__device__ __forceinline__ uint32_t row_of(Chunk c) { return (uint32_t)c; }

// The chunk of block blockIdx.x: a permutation of [0, gridDim.x). Blocks are
// dispatched round-robin over the 8 XCDs, so taken in order, neighbouring
// chunks run on different ones, and each fetches the lines they share on its
// own (of arrays off a line boundary, of the block exponents, of the table).
// Within each window of 8 * kNear chunks an XCD here gets kNear neighbours.
// us with chunks in order and so: 8-bit moments, float32 weights with bfloat16
// gradients and copies, 348 and 338 at 124,356,864 elements, 47.7 and 45.0 at
// 12.7M of odd sizes; export 328 and 319, import 432 and 426; 32-bit moments
// 60.6 and 57.5 (12.7M bfloat16, odd sizes), 187 and 185 (37M float32), 247
// and 245 (50M). Beside 32-bit moments above 2^26 elements they stay in order:
// at 124,356,864 elements, on the same arrays, 602 and 612 (float32), 443 and 450
// (bfloat16), 445 and 449 (float16), 576 and 580 (float32 weights, bfloat16
// gradients and copies); at 537.6M 2,860 and 2,904, 2,139 and 2,152, 2,111 and
// 2,177, 2,750 and 2,756. (Odd sizes there: 172.5M float32 878 and 894, but
// bfloat16 660 and 657, with float32 weights and copies 854 and 838. Why the order
// that saves lines costs aligned streams of this length is not known. 16
// neighbours: 343 for export; 128 or 256: as 64. Each XCD on an eighth of the
// list, as in the flat update: 651 for 607.)
constexpr uint32_t kNear = 64;
constexpr int64_t kNearMaxN = 1LL << 26;  // beside 32-bit moments
constexpr uint32_t kWindow = 8 * kNear;
// in_windows: the blocks of whole windows, 0 to take all chunks in order (a
// kernel argument: the grid's size would be a load of its own).
__device__ __forceinline__ uint32_t near_chunk(uint32_t in_windows) {
    const uint32_t b = blockIdx.x, i = b % kWindow;
    const uint32_t near = b - i + (i % 8) * kNear + i / 8;
    return b < in_windows ? near : b;
}

// Elements first .. end - 1 of a tensor; a chunk's are whole if it lies inside.
struct Range {
    int64_t first, end;
    bool whole;
};
template <bool Q8>
__device__ __forceinline__ Range range_of(Chunk c, const Row &t) {
    const int64_t a = (int64_t)(c >> 32) * kChunk - (Q8 ? 0 : t.shift), b = a + kChunk;
    return Range{Q8 || a >= 0 ? a : 0, b <= t.n ? b : t.n, (Q8 || a >= 0) && b <= t.n};
}

struct ListScalars {
    float lr, bc1, bc2, b1, c1, b2, c2, eps, gscale;
    float da, db, sc;  // for the free evaluation of the weight: weight_free, weight_wide
    uint32_t key;   // of the update's random bits
    // of decode_moments; 0 for a beta of 0, which forgets the 8-bit moment, an
    // infinite one too (0 times that would be a NaN; so no moment is ever one)
    uint32_t mask_m, mask_v;
    int32_t fits;  // the update's arrays fit the last-level cache
};

// ------------------------------------------------------------- element types

// Bytes of an element type; 0 if there is no such type.
__host__ __device__ constexpr int type_bytes(int t) {
    return t == RCS_F32 ? 4 : t == RCS_BF16 || t == RCS_F16 ? 2 : 0;
}

struct F32 {
    static constexpr int kBytes = 4;
};
struct BF16 {
    static constexpr int kBytes = 2;
};
struct F16 {
    static constexpr int kBytes = 2;
};

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// 16 bytes at the alignment of an element: the hardware's vector accesses need
// no more.
template <int DWORDS, int ALIGN>
struct Vector;
template <>
struct Vector<4, 4> {
    typedef u32x4 type __attribute__((aligned(4)));
};
template <>
struct Vector<4, 2> {
    typedef u32x4 type __attribute__((aligned(2)));
};
template <>
struct Vector<2, 4> {
    typedef u32x2 type __attribute__((aligned(4)));
};
template <>
struct Vector<2, 2> {
    typedef u32x2 type __attribute__((aligned(2)));
};

// A pointer that came out of a table is one to device memory: said so, its
// accesses are global ones rather than flat ones, which would wait for LDS too.
template <class V>
using Global = __attribute__((address_space(1))) V *;
template <class V>
__device__ __forceinline__ Global<V> global(const void *p) {
    return (Global<V>)reinterpret_cast<uintptr_t>(p);
}

template <class T, int V>
struct Raw {  // V elements as they lie in memory
    uint32_t d[V * T::kBytes / 4];
};

__device__ __forceinline__ float elem_f32(uint32_t bits, F32) { return __uint_as_float(bits); }
__device__ __forceinline__ float elem_f32(uint32_t bits, BF16) {
    return __uint_as_float(bits << 16);
}
__device__ __forceinline__ float elem_f32(uint32_t bits, F16) {
    return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
}

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// One rounding each to nearest even; a NaN stays one.
__device__ __forceinline__ uint32_t two_bits(float x, float y, BF16) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{x, y}, bf16x2));
}
__device__ __forceinline__ uint32_t two_bits(float x, float y, F16) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{x, y}, f16x2));
}

template <class T, int V>
__device__ __forceinline__ void unpack(const Raw<T, V> &r, float (&x)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if constexpr (T::kBytes == 4) x[i] = elem_f32(r.d[i], T{});
        else x[i] = elem_f32((r.d[i / 2] >> (16 * (i & 1))) & 0xFFFFu, T{});
    }
}

template <class T, int V>
__device__ __forceinline__ Raw<T, V> pack(const float (&x)[V]) {
    Raw<T, V> r;
#pragma unroll
    for (int i = 0; i < V; i += 2) {
        if constexpr (T::kBytes == 4) {
            r.d[i] = __float_as_uint(x[i]);
            r.d[i + 1] = __float_as_uint(x[i + 1]);
        } else {
            r.d[i / 2] = two_bits(x[i], x[i + 1], T{});
        }
    }
    return r;
}

// The V elements from element first + at of p on, `first` uniform in the wave;
// cnt of them exist (the others come as zero), all of them with FULL. Streaming
// loads unless KEEP.
template <class T, int V, bool FULL, bool KEEP = false>
__device__ __forceinline__ Raw<T, V> load(const void *p, int64_t first, uint32_t at, int cnt) {
    Raw<T, V> r;
    constexpr int kDwords = (int)sizeof(r) / 4, kWide = kDwords < 4 ? kDwords : 4;
    const Global<char> a =
        global<char>(static_cast<const char *>(p) + first * T::kBytes) + at * T::kBytes;
    if (FULL || cnt == V) {
        using X = typename Vector<kWide, T::kBytes>::type;
        const Global<X> q = (Global<X>)a;
#pragma unroll
        for (int k = 0; k < kDwords / kWide; ++k) {
            const X x = KEEP ? q[k] : __builtin_nontemporal_load(q + k);
#pragma unroll
            for (int j = 0; j < kWide; ++j) r.d[kWide * k + j] = x[j];
        }
    } else {
#pragma unroll
        for (int k = 0; k < kDwords; ++k) r.d[k] = 0;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            if (k >= cnt) continue;
            if constexpr (T::kBytes == 4)
                r.d[k] = ((Global<uint32_t>)a)[k];
            else
                r.d[k / 2] |= (uint32_t)((Global<uint16_t>)a)[k] << (16 * (k & 1));
        }
    }
    return r;
}

template <bool FULL, class T, int V>
__device__ __forceinline__ void store(void *p, int64_t first, uint32_t at, int cnt,
                                      const Raw<T, V> &r) {
    constexpr int kDwords = (int)sizeof(r) / 4, kWide = kDwords < 4 ? kDwords : 4;
    const Global<char> a =
        global<char>(static_cast<char *>(p) + first * T::kBytes) + at * T::kBytes;
    if (FULL || cnt == V) {
        using X = typename Vector<kWide, T::kBytes>::type;
        const Global<X> q = (Global<X>)a;
#pragma unroll
        for (int k = 0; k < kDwords / kWide; ++k) {
            X x;
#pragma unroll
            for (int j = 0; j < kWide; ++j) x[j] = r.d[kWide * k + j];
            __builtin_nontemporal_store(x, q + k);
        }
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            if (k >= cnt) continue;
            if constexpr (T::kBytes == 4)
                ((Global<uint32_t>)a)[k] = r.d[k];
            else
                ((Global<uint16_t>)a)[k] = (uint16_t)(r.d[k / 2] >> (16 * (k & 1)));
        }
    }
}

// Whether an array's chunks begin off a line boundary, and its waves so share
// lines with their neighbours: its loads are then left in the cache for them
// (KEEP) rather than streamed, which would fetch those lines twice. The two
// cases are told apart by f(true) or f(false), each behind a barrier of its own:
// the compiler would merge loads that only differ in this.
template <class F>
__device__ __forceinline__ void by_lines(bool shared, F f) {
    if (shared) {
        asm volatile("; shared lines" ::: "memory");
        f(std::true_type{});
    } else {
        asm volatile("; whole lines" ::: "memory");
        f(std::false_type{});
    }
}
__device__ __forceinline__ bool off_line(const void *p, int64_t bytes) {
    return ((reinterpret_cast<uintptr_t>(p) + (uintptr_t)bytes) & 127u) != 0;
}

// (Update beside 8-bit moments, float32 weights at odd offsets, bfloat16
// gradients and copies, streamed against kept: 51.6 and 48.1 us at 12.7M
// elements, 89.5 and 87.1 at 24.7M, 129 and 130 at 36.7M, 164 and 171 at 50M:
// kept while all its arrays fit the cache. Export 49.7 and 44.6 us at 12.7M,
// 488 and 476 at 124.6M, import 421 and 395: kept always.)

// f(T) for the element type t (uniform in the wave).
template <class F>
__device__ __forceinline__ void by_type(int t, F f) {
    if (t == RCS_F32) f(F32{});
    else if (t == RCS_BF16) f(BF16{});
    else f(F16{});
}

// How many of the V elements that begin `at` elements after a point lie in the
// tensor, which has `left` from that point on.
template <int V>
__device__ __forceinline__ int count_of(int64_t left, int at) {
    const int64_t r = left - at;
    return r >= V ? V : r > 0 ? (int)r : 0;
}

// ----------------------------------------------------------- 8-bit moments

// Hash of an element's index and the update: the mixing step of x = index *
// kHashA + (index >> 32) * kHashB + key.
__host__ __device__ __forceinline__ uint32_t mixed(uint32_t x) {
    x = (x ^ (x >> 16)) * kHashC;
    return x ^ (x >> 15);
}

// The random bits of elements first + at .. first + at + V - 1 of the list,
// `first` uniform; carry: the upper half of an index may change among the
// wave's.
template <int V>
__device__ __forceinline__ void random_bits(int64_t first, uint32_t at, uint32_t key, bool carry,
                                            uint32_t (&r)[V]) {
    const uint32_t x =
        (uint32_t)first * kHashA + (uint32_t)(first >> 32) * kHashB + key + at * kHashA;
    if (!carry) {
#pragma unroll
        for (int k = 0; k < V; ++k) r[k] = mixed(x + (uint32_t)k * kHashA);
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const uint32_t up = (uint32_t)((first + at + k) >> 32) - (uint32_t)(first >> 32);
            r[k] = mixed(x + (uint32_t)k * kHashA + up * kHashB);
        }
    }
}

// The larger of each pair of 16-lane rows' values, in every lane of the pair.
__device__ __forceinline__ uint32_t row_pair_max(uint32_t x) {
    const auto y = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    return y[0] > y[1] ? y[0] : y[1];
}

// The largest of the values of the lanes that share a block of V elements
// each, in every one of them.
template <int V>
__device__ __forceinline__ uint32_t block_max(uint32_t x) {
    auto with = [&](uint32_t y) { x = x > y ? x : y; };
    with((uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0xB1, 0xF, 0xF, true));   // pairs
    with((uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x4E, 0xF, 0xF, true));   // quads
    with((uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x141, 0xF, 0xF, true));  // 8 lanes
    with((uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x140, 0xF, 0xF, true));  // 16 lanes
    return V == 8 ? x : row_pair_max(x);
}

// The codes' arithmetic runs on two elements at once, in the upper 16 bits of
// their floats: sign, exponent and 7 mantissa bits, of which the format keeps 3.
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ u16x2 both(uint32_t x) { return u16x2{(uint16_t)x, (uint16_t)x}; }
__device__ __forceinline__ u16x2 halves(uint32_t x) { return __builtin_bit_cast(u16x2, x); }
// A 1 that the compiler does not see through: it would turn min(k, 1) * x, one
// instruction each for two elements, into a comparison and a selection for each.
__device__ __forceinline__ uint32_t hidden_one(uint32_t x) {
    asm("" : "+v"(x));
    return x;
}
__device__ __forceinline__ uint32_t word(u16x2 x) { return __builtin_bit_cast(uint32_t, x); }

// Upper halves of two words.
__device__ __forceinline__ u16x2 upper(uint32_t x0, uint32_t x1) {
    return halves(__builtin_amdgcn_perm(x1, x0, 0x07060302u));
}

__device__ __forceinline__ int base_m(int e) { return 8 * e - 127; }
__device__ __forceinline__ int base_v(int e) { return 8 * e - 255; }

// Biased exponent of the smallest power of two not below a block's largest
// magnitude, given the upper half of that magnitude's bits plus 0x7FFFFF; at
// least low, and 255 for what is not finite.
__device__ __forceinline__ int block_exponent(uint32_t half, int low) {
    const int e = (int)(half >> 7);
    return e < low ? low : e > 255 ? 255 : e;
}

// V codes of one byte. The arithmetic takes codes j and j + 2 of a word
// together, j = 0 or 1: a mask puts them into 16 bits each.
template <int V>
struct Codes {
    uint32_t d[V / 4];
};
template <int V>
__device__ __forceinline__ constexpr int first_of_pair(int p) {  // of the V / 2 pairs
    return 4 * (p / 2) + (p & 1);
}

template <int V>
__device__ __forceinline__ Codes<V> load_codes(const void *p, int64_t first, uint32_t at) {
    Codes<V> c;
    const Global<char> a = global<char>(static_cast<const char *>(p) + first) + at;
    if constexpr (V == 8) {
        const u32x2 x = __builtin_nontemporal_load((Global<u32x2>)a);
        c.d[0] = x.x;
        c.d[1] = x.y;
    } else {
        c.d[0] = __builtin_nontemporal_load((Global<uint32_t>)a);
    }
    return c;
}

template <int V>
__device__ __forceinline__ void store_codes(void *p, int64_t first, uint32_t at,
                                            const Codes<V> &c) {
    const Global<char> a = global<char>(static_cast<char *>(p) + first) + at;
    if constexpr (V == 8)
        __builtin_nontemporal_store(u32x2{c.d[0], c.d[1]}, (Global<u32x2>)a);
    else
        __builtin_nontemporal_store(c.d[0], (Global<uint32_t>)a);
}

// The exponents of the block that holds element first + at (first begins one).
__device__ __forceinline__ Global<uint16_t> exponents_at(const Row &t, int64_t first,
                                                         uint32_t at) {
    return global<uint16_t>(t.e + first / kBlock) + at / kBlock;
}

// A float's upper half is 16 (k + B), plus the sign for m, and 0 for k = 0; its
// lower half is zero. mask_m, mask_v: kMaskM and kMaskV, or 0 to take all codes
// as 0.
constexpr uint32_t kMaskM = 0x07F007F0u, kMaskV = 0x0FF00FF0u;  // 16 k of two codes
template <int V>
__device__ __forceinline__ void decode_moments(const Codes<V> &cm, const Codes<V> &cv, uint32_t e,
                                               uint32_t mask_m, uint32_t mask_v, float (&m)[V],
                                               float (&v)[V]) {
    const uint32_t bm = 16u * (uint32_t)base_m((int)(e & 0xFFu));
    const u16x2 bv = both(16u * (uint32_t)base_v((int)(e >> 8)));
    const uint32_t bm2 = (bm | (bm << 16)) & 0x7FFF7FFFu;
    const u16x2 one = halves(hidden_one(0x00010001u));
#pragma unroll
    for (int p = 0; p < V / 2; ++p) {
        const int i = first_of_pair<V>(p);
        const uint32_t c = cm.d[p / 2], l = cv.d[p / 2];
        const u16x2 k = halves((p & 1 ? c >> 4 : c << 4) & mask_m);
        const u16x2 signed_base = halves(((p & 1 ? c : c << 8) & 0x80008000u) | bm2);
        const uint32_t x = word(k + __builtin_elementwise_min(k, one) * signed_base);
        m[i] = __uint_as_float(x << 16);
        m[i + 2] = __uint_as_float(x & 0xFFFF0000u);
        const u16x2 n = halves((p & 1 ? l >> 4 : l << 4) & mask_v);
        const uint32_t y = word(n + __builtin_elementwise_min(n, one) * bv);
        v[i] = __uint_as_float(y << 16);
        v[i + 2] = __uint_as_float(y & 0xFFFF0000u);
    }
}

// What is added below the third mantissa bit before the rest is cut off, for
// the nearest value (ties to even).
__device__ __forceinline__ uint32_t half_unit(uint32_t bits) { return 0x7FFFFu + ((bits >> 20) & 1u); }

// Block exponents and codes of the lane's m and v (those past the tensor's end
// are zero), written to their block; every lane of the block calls this.
// add_m, add_v: below 2^20, what is added to the bits of element k before they
// are cut (random bits, or half a unit). v is not below zero, and neither is a
// NaN.
template <int V, class AddM, class AddV>
__device__ __forceinline__ void store_moments(const Row &t, int64_t first, uint32_t at,
                                              const float (&m)[V], const float (&v)[V],
                                              bool active, AddM add_m, AddV add_v) {
    // ym: upper halves of |m|'s bits plus 0x7FFFFF. Their largest gives the
    // block's exponent; and as the smallest value L and half of it are a power
    // of two apart and end in 20 zero bits, ym >= L exactly where |m| > L / 2.
    u16x2 ym[V / 2], big = both(0);
    uint32_t av = 0;
#pragma unroll
    for (int p = 0; p < V / 2; ++p) {
        const int i = first_of_pair<V>(p);
        const uint32_t y0 = __float_as_uint(m[i]) + 0x7FFFFFu;
        const uint32_t y1 = __float_as_uint(m[i + 2]) + 0x7FFFFFu;
        ym[p] = halves(word(upper(y0, y1)) & 0x7FFF7FFFu);
        big = __builtin_elementwise_max(big, ym[p]);
        const uint32_t u0 = __float_as_uint(v[i]), u1 = __float_as_uint(v[i + 2]);
        av = av > u0 ? av : u0;
        av = av > u1 ? av : u1;
    }
    const uint32_t one = hidden_one(1u);
    const uint32_t am = big.x > big.y ? big.x : big.y;
    const int em = block_exponent(block_max<V>(am), kLowM);
    const int ev = block_exponent((block_max<V>(av) + 0x7FFFFFu) >> 16, kLowV);
    const u16x2 bm = both((uint32_t)base_m(em)), bv = both((uint32_t)base_v(ev));
    const u16x2 least = both(16u * (uint32_t)(base_m(em) + 1));
    Codes<V> cm, cv;
#pragma unroll
    for (int p = 0; p < V / 2; ++p) {
        const int i = first_of_pair<V>(p);
        const uint32_t u0 = __float_as_uint(m[i]), u1 = __float_as_uint(m[i + 2]);
        const u16x2 x = upper(u0 + add_m(i), u1 + add_m(i + 2));
        u16x2 y = __builtin_elementwise_max(halves(word(x) & 0x7FFF7FFFu),
                                            __builtin_elementwise_min(ym[p], least));
        y = __builtin_elementwise_sub_sat(y >> both(4), bm);  // (infinity comes to the top code)
        const uint32_t s0 = __float_as_uint(v[i]), s1 = __float_as_uint(v[i + 2]);
        const u16x2 z = upper(s0 + add_v(i), s1 + add_v(i + 2));
        const u16x2 some = halves((s0 < one ? s0 : one) | ((s1 < one ? s1 : one) << 16));
        const u16x2 k =
            __builtin_elementwise_max(__builtin_elementwise_sub_sat(z >> both(4), bv), some);
        if (p & 1) {
            cm.d[p / 2] |= (word(y) << 8) | (word(x) & 0x80008000u);
            cv.d[p / 2] |= word(k) << 8;
        } else {
            cm.d[p / 2] = ((word(x) >> 8) & 0x00800080u) | word(y);
            cv.d[p / 2] = word(k);
        }
    }
    if (!active) return;
    store_codes(t.m, first, at, cm);
    store_codes(t.v, first, at, cv);
    if ((threadIdx.x & (kBlock / V - 1)) == 0)
        *exponents_at(t, first, at) = (uint16_t)(em | (ev << 8));
}

// ------------------------------------------------------------------- kernels

template <class G, int V>
__device__ __forceinline__ void add_squares(const Raw<G, V> &r, float gscale, double &acc) {
    float x[V];
    unpack(r, x);
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const double d = (double)(x[k] * gscale);
        acc = __builtin_fma(d, d, acc);  // the square of a float is exact in float64
    }
}

// Sum of squares of elements first .. stop - 1 of a gradient, this lane's part.
template <class G, bool KEEP>
__device__ __forceinline__ double squares_of(const void *g, int64_t first, int64_t stop,
                                             float gscale) {
    constexpr int V = 16 / G::kBytes;  // one 16-byte vector
    constexpr int kStep = kWave * V;
    const int lane = ((int)threadIdx.x & (kWave - 1)) * V;
    double acc[kDeep] = {};
    int64_t i = first;
    for (; i + kDeep * kStep <= stop; i += kDeep * kStep) {
        Raw<G, V> r[kDeep];
#pragma unroll
        for (int q = 0; q < kDeep; ++q) r[q] = load<G, V, true, KEEP>(g, i, lane + q * kStep, V);
#pragma unroll
        for (int q = 0; q < kDeep; ++q) add_squares(r[q], gscale, acc[q]);
    }
    if (i < stop) {  // the rest, also in flight at once: whole steps, then lane by lane
        const int steps = (int)((stop - i) / kStep);
        const int64_t last = i + steps * kStep;
        Raw<G, V> r[kDeep - 1], z = {};
#pragma unroll
        for (int q = 0; q < kDeep - 1; ++q)
            if (q < steps) r[q] = load<G, V, true, KEEP>(g, i, lane + q * kStep, V);
        if (last < stop)
            z = load<G, V, false, KEEP>(g, last, lane, count_of<V>(stop - last, lane));
#pragma unroll
        for (int q = 0; q < kDeep - 1; ++q)
            if (q < steps) add_squares(r[q], gscale, acc[q]);
        if (last < stop) add_squares(z, gscale, acc[kDeep - 1]);
    }
    return (acc[0] + acc[1]) + (acc[2] + acc[3]);
}

// Per-block float64 partial sums of squares of the list's gradients. The waves
// of the grid take runs of kRun consecutive chunks in turn, and go through a run
// one stretch of a tensor at a time; the order depends on the list's chunks
// alone. The table entries of a run are fetched while the one before it is
// summed. Bound by HBM; of 16-bit gradients, by the start and end of so short a
// pass too: 124,356,864 float32 gradients 79 us = 6.3 TB/s, bfloat16 ones 39 us =
// 6.4 TB/s where the last-level cache holds them, 48 us = 5.2 TB/s behind an
// update that left other things there (right behind kernels that left it full
// of written lines, which have to go out first, 140 and 103 us). A run is kRun
// chunks whatever the list's length: up to 16,384 chunks some blocks have no run,
// at 8 blocks of 32 with 262,144 elements, and above the last turn of runs is
// not full (12.7M elements: 1.52 turns' work in 2).
//   The end (unless arrived is null: the update then reduces the partials): the
// block that finds itself the last to leave its partial reduces them all, in
// their order, whichever it is. A partial goes out as an exchange whose answer
// is waited for: it then has been performed where the atomics of all XCDs meet,
// before the block counts itself; the last block's loads, issued after its own
// count came back, are device-scope ones that no cache answers. (With a plain
// store and fences, which write back and drop whole caches, 54.5 us for 48.5 at
// 124,356,864 bfloat16 gradients; a kernel of its own 50.1, and 6.5 for 4.8 at
// 262,144.) The count wraps to zero by itself.
template <bool Q8>
__global__ __launch_bounds__(kListNormThreads) void list_norm(
    const Row *__restrict__ rows, const Chunk *__restrict__ chunks, int64_t nchunks,
    int64_t keep_from, float gscale, double *partials, uint32_t *arrived, float clip,
    ClipScalars *__restrict__ record, double *__restrict__ norm_out, double *__restrict__ last) {
    __shared__ double lds[kListNormThreads / kWave];
    constexpr int kWaves = kListNormThreads / kWave;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
    const int64_t step = (int64_t)gridDim.x * kWaves * kRun;
    int64_t run = ((int64_t)blockIdx.x * kWaves + wave) * kRun;
    double sum = 0.0;
    if (run < nchunks) {
        Chunk c = chunks[run];
        Chunk next = chunks[run + step < nchunks ? run + step : run];
        Row t = rows[row_of(c)];
        for (; run < nchunks; run += step) {
            const Chunk after = chunks[run + 2 * step < nchunks ? run + 2 * step : run];
            const Row next_row = rows[row_of(next)];
            const int64_t end = run + kRun < nchunks ? run + kRun : nchunks;
            for (int64_t j = run;;) {
                const int64_t shift = Q8 ? 0 : t.shift, k = (int64_t)(c >> 32);
                const int64_t rest = (t.n + shift + kChunk - 1) / kChunk - k;
                const int64_t mine = rest < end - j ? rest : end - j;
                int64_t first = k * kChunk - shift, stop = first + mine * kChunk;
                if (first < 0) first = 0;
                if (stop > t.n) stop = t.n;
                if (t.g != nullptr)
                    by_type(t.gt(), [&](auto G) {
                        using T = decltype(G);
                        sum += run < keep_from ? squares_of<T, false>(t.g, first, stop, gscale)
                                               : squares_of<T, true>(t.g, first, stop, gscale);
                    });
                j += mine;
                if (j >= end) break;
                c = chunks[j];
                t = rows[row_of(c)];
            }
            c = next;
            t = next_row;
            next = after;
        }
    }
    sum = block_sum<kListNormThreads>(sum, lds);
    if (arrived == nullptr) {
        if (threadIdx.x == 0) partials[blockIdx.x] = sum;
        return;
    }
    if (threadIdx.x >= kWave) return;
    uint32_t before = 0;
    if (threadIdx.x == 0) {
        const unsigned long long old = __hip_atomic_exchange(
            reinterpret_cast<unsigned long long *>(partials + blockIdx.x),
            (unsigned long long)__double_as_longlong(sum), __ATOMIC_RELAXED,
            __HIP_MEMORY_SCOPE_AGENT);
        asm volatile("; the partial has arrived" ::"v"(old) : "memory");
        before = atomicInc(arrived, gridDim.x - 1);
    }
    if ((uint32_t)__builtin_amdgcn_readfirstlane((int)before) != gridDim.x - 1) return;
    double x[kPartsPerLane];
#pragma unroll
    for (int k = 0; k < kPartsPerLane; ++k) {
        const int j = (int)threadIdx.x + k * kUpdThreads, end = (int)gridDim.x - 1;
        x[k] = __hip_atomic_load(partials + (j < end ? j : end), __ATOMIC_RELAXED,
                                 __HIP_MEMORY_SCOPE_AGENT);
    }
    const ClipScalars r = final_reduce(x, (int)gridDim.x, clip, nullptr);
    if (threadIdx.x == 0) {
        *record = r;
        if (norm_out != nullptr) *norm_out = r.norm;
        if (last != nullptr) *last = r.norm;
    }
}

// Sets a workspace's count of arrived blocks to zero, once.
__global__ void list_norm_init(uint32_t *arrived) { *arrived = 0; }

// New moments of one element from its scaled gradient; the operations and their
// roundings are part of the definition (8-bit moments are rounded from exactly
// these).
__device__ __forceinline__ void moments(float ga, float &m, float &v, float s,
                                        const ListScalars &h) {
    const float gp = ga * s;
    m = h.b1 * m + h.c1 * gp;
    v = h.b2 * v + h.c2 * (gp * gp);
}

// g * gscale, which a uniform branch leaves out where it changes nothing.
template <int V>
__device__ __forceinline__ void scale(float (&g)[V], const ListScalars &h) {
    if (h.gscale == 1.0f) return;
#pragma unroll
    for (int k = 0; k < V; ++k) g[k] = g[k] * h.gscale;
}

// The weight in the flat update's operation sequence: divisions and root
// correctly rounded (beside 32-bit moments, where memory hides them).
__device__ __forceinline__ float weight(float w, float m, float v, float decay,
                                        const ListScalars &h) {
    const float mh = m / h.bc1;
    const float vh = v / h.bc2;
    const float den = __builtin_sqrtf(vh) + h.eps;
    return w * decay - (h.lr * mh) / den;
}

// The weight beside 8-bit moments, where the arithmetic is what counts:
//   w decay - lr (m / bc1) / (sqrt(v / bc2) + eps) = w decay - m / (da sqrt(v) + db)
// with da = bc1 / (lr sqrt(bc2)), db = bc1 eps / lr; root and reciprocal are the
// hardware's, 1 ulp each over the normal floats. The root of a subnormal v comes
// out as zero: da sqrt(v) then lacks up to 2^-63 da of a denominator of at least
// db = sqrt(bc2) eps da, which is for the caller to weigh (kWideEps), and so is
// a denominator whose reciprocal is no normal float (kWideDen).
__device__ __forceinline__ float weight_free(float w, float m, float v, float decay,
                                             const ListScalars &h) {
    const float den = __builtin_fmaf(__builtin_amdgcn_sqrtf(v), h.da, h.db);
    return __builtin_fmaf(-m, __builtin_amdgcn_rcpf(den), w * decay);
}

// Below this sqrt(bc2) eps, weight_wide takes the place of weight_free: from it
// on what the root of a subnormal v lacks is at most 2^-27 of the denominator, an
// eighth of a rounding. (us a step in either form: 218 and 223 at 124,356,864
// bfloat16 elements, 19.5 and 20.6 at 8.0M; float32 weights 372 and 373, 25.8
// and 26.0.)
constexpr double kWideEps = 0x1p-36;

// And where the largest denominator, da sqrt(2^128) + db, passes this one (an lr
// below about 1e-18, or eps / lr beyond 1e37): da and db are then scaled down to
// it by a power of two, sc, and so is the quotient.
constexpr double kWideDen = 0x1p125;

// weight_free with the root right for every v (a small one is scaled by 2^64 and
// its root by 2^-32, both exactly) and the quotient scaled by sc (one rounding
// more, so not for an sc of 1).
__device__ __forceinline__ float weight_wide(float w, float m, float v, float decay,
                                             const ListScalars &h) {
    const bool small = v < 0x1p-64f;
    const float root = __builtin_amdgcn_sqrtf(small ? v * 0x1p64f : v);
    const float den = __builtin_fmaf(small ? root * 0x1p-32f : root, h.da, h.db);
    const float over = __builtin_amdgcn_rcpf(den);
    return h.sc == 1.0f ? __builtin_fmaf(-m, over, w * decay)
                        : __builtin_fmaf(-(m * over), h.sc, w * decay);
}

// R groups of 32-bit moments from element `first` on: W, G the types of weights
// and gradients; FULL: all of them lie in the tensor.
template <class W, class G, int V, int R, bool FULL, class Factor>
__device__ __forceinline__ void update32(const Row &t, int64_t first, int64_t end,
                                         Factor clip_factor, const ListScalars &h) {
    const int64_t left = end - first;
    int at[R], cnt[R];
    Raw<W, V> w[R];
    Raw<G, V> g[R];
    Raw<F32, V> m[R], v[R];
#pragma unroll
    for (int q = 0; q < R; ++q) {
        at[q] = (q * kWave + (int)threadIdx.x) * V;
        cnt[q] = FULL ? V : count_of<V>(left, at[q]);
        g[q] = load<G, V, FULL>(t.g, first, at[q], cnt[q]);
        w[q] = load<W, V, FULL>(t.w, first, at[q], cnt[q]);
        m[q] = load<F32, V, FULL>(t.m, first, at[q], cnt[q]);
        v[q] = load<F32, V, FULL>(t.v, first, at[q], cnt[q]);
    }
    float s;
    if (!clip_factor(s)) return;
    const float decay = (float)(1.0 - (double)h.lr * (double)t.wd);
#pragma unroll
    for (int q = 0; q < R; ++q) {
        float ww[V], gg[V], mm[V], vv[V];
        unpack(w[q], ww);
        unpack(g[q], gg);
        unpack(m[q], mm);
        unpack(v[q], vv);
        scale(gg, h);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            moments(gg[k], mm[k], vv[k], s, h);
            ww[k] = weight(ww[k], mm[k], vv[k], decay, h);
        }
        store<FULL>(t.w, first, at[q], cnt[q], pack<W>(ww));
        store<FULL>(t.m, first, at[q], cnt[q], pack<F32>(mm));
        store<FULL>(t.v, first, at[q], cnt[q], pack<F32>(vv));
        if constexpr (W::kBytes == 4) {
            if (t.c != nullptr) {
                if (t.ct() == RCS_BF16) store<FULL>(t.c, first, at[q], cnt[q], pack<BF16>(ww));
                else store<FULL>(t.c, first, at[q], cnt[q], pack<F16>(ww));
            }
        }
    }
}

// The same with 8-bit moments. The code arrays are filled up to whole blocks,
// so a code access is always a whole vector; a block past the tensor's end is
// not touched. WIDE: the weight's form.
template <class W, class G, int V, int R, bool FULL, bool KEEP, bool WIDE, class Factor>
__device__ __forceinline__ void update8(const Row &t, int64_t first, int64_t end,
                                        Factor clip_factor, const ListScalars &h) {
    const int64_t left = end - first;
    // (uniform: the group's first and last element of the list)
    const bool carry = ((t.off + first) >> 32) != ((t.off + first + R * kWave * V - 1) >> 32);
    int at[R], cnt[R];
    bool active[R];
    Raw<W, V> w[R];
    Raw<G, V> g[R];
    Codes<V> cm[R], cv[R];
    uint32_t e[R];
#pragma unroll
    for (int q = 0; q < R; ++q) {
        at[q] = (q * kWave + (int)threadIdx.x) * V;
        cnt[q] = FULL ? V : count_of<V>(left, at[q]);
        active[q] = FULL || (at[q] & ~(kBlock - 1)) < left;
        g[q] = load<G, V, FULL, KEEP>(t.g, first, at[q], cnt[q]);
        w[q] = load<W, V, FULL, KEEP>(t.w, first, at[q], cnt[q]);
        const int there = active[q] ? at[q] : 0;
        cm[q] = load_codes<V>(t.m, first, there);
        cv[q] = load_codes<V>(t.v, first, there);
        e[q] = *exponents_at(t, first, there);
    }
    float s;
    if (!clip_factor(s)) return;
    const float decay = (float)(1.0 - (double)h.lr * (double)t.wd);
#pragma unroll
    for (int q = 0; q < R; ++q) {
        float ww[V], gg[V], mm[V], vv[V];
        unpack(w[q], ww);
        unpack(g[q], gg);
        decode_moments(cm[q], cv[q], e[q], h.mask_m, h.mask_v, mm, vv);
        scale(gg, h);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            moments(gg[k], mm[k], vv[k], s, h);
            ww[k] = WIDE ? weight_wide(ww[k], mm[k], vv[k], decay, h)
                         : weight_free(ww[k], mm[k], vv[k], decay, h);
            if (!FULL && k >= cnt[q]) mm[k] = vv[k] = 0.0f;
        }
        store<FULL>(t.w, first, at[q], cnt[q], pack<W>(ww));
        if constexpr (W::kBytes == 4) {
            if (t.c != nullptr) {
                if (t.ct() == RCS_BF16) store<FULL>(t.c, first, at[q], cnt[q], pack<BF16>(ww));
                else store<FULL>(t.c, first, at[q], cnt[q], pack<F16>(ww));
            }
        }
        uint32_t r[V];
        random_bits(t.off + first, at[q], h.key, carry, r);
        store_moments(t, first, at[q], mm, vv, active[q], [&](int k) { return r[k] & 0xFFFFFu; },
                      [&](int k) { return r[k] >> 12; });
    }
}

// The update, one wave per chunk. The clip record was written by list_norm; it
// is read beside the table. FOLD: every wave does the final reduction of the
// norm itself (as the flat update does at small n), behind its loads, and the
// first one writes the record. W, G: the types of weights and gradients; a list
// with several pairs of types has a launch for each (one kernel that branched on
// them held 92 vector registers for every pair and spilled scalar ones). WIDE:
// the weight beside 8-bit moments in weight_wide's form, kernels of their own
// too (a branch in update8 that left the compiler one order of instructions for
// both forms: 24.8 and 25.3 us at 8.0M float32 elements).
//   At 124,356,864 elements, each pass once over its bytes: float32 weights and
// gradients with 32-bit moments 524 us = 6.6 TB/s, bfloat16 ones 411 us =
// 6.7 TB/s; with 8-bit moments, float32 weights, bfloat16 gradients and copies
// 291 us = 6.9 TB/s, bfloat16 weights and gradients 202 us = 6.2 TB/s. Bound by
// HBM; the last one, at 397 vector instructions a chunk (49.6 an element), by
// them as well: 230 us in a run at a lower clock.
template <class W, class G, bool Q8, bool FOLD, bool WIDE = false>
__global__ __launch_bounds__(kUpdThreads) void list_update(
    const Row *__restrict__ rows, const Chunk *__restrict__ chunks, uint32_t in_windows,
    int nparts, const double *__restrict__ partials, float clip, ClipScalars *__restrict__ record,
    double *__restrict__ norm_out, double *__restrict__ last, ListScalars h) {
    const Chunk c = chunks[near_chunk(in_windows)];
    double x[kPartsPerLane];
    ClipScalars cs = {};
    if constexpr (FOLD) load_partials(partials, nparts, x);
    else cs = *record;
    const Row t = rows[row_of(c)];
    auto factor = [&](float &s) -> bool {
        if constexpr (FOLD) {
            asm volatile("" ::: "memory");  // the loads before this stay before it
            cs = final_reduce(x, nparts, clip, nullptr);
            if (blockIdx.x == 0 && threadIdx.x == 0) {
                *record = cs;
                if (norm_out != nullptr) *norm_out = cs.norm;
                if (last != nullptr) *last = cs.norm;
            }
        }
        s = cs.scale;
        return cs.apply != 0;
    };
    // all of the row before the branch, in one trip
    asm volatile("" ::"s"(t.n), "s"(t.off), "s"(t.types), "s"(h.lr), "s"(h.eps), "s"(h.key));
    if (t.g == nullptr || (!FOLD && !cs.apply)) {
        float s;
        if constexpr (FOLD) (void)factor(s);
        return;
    }
    const Range r = range_of<Q8>(c, t);
    // 16-bit weights and gradients beside 8-bit moments: 8 elements a lane still
    // cover whole lines and halve the work per block exponent
    constexpr int V = Q8 && W::kBytes == 2 && G::kBytes == 2 ? 8 : 4;
    constexpr int R = kChunk / (kWave * V);
    if (r.whole) {
        if constexpr (Q8)
            by_lines(h.fits != 0 && off_line(t.w, 0), [&](auto K) {
                update8<W, G, V, R, true, K.value, WIDE>(t, r.first, r.end, factor, h);
            });
        else
            update32<W, G, V, R, true>(t, r.first, r.end, factor, h);
        return;
    }
    float s;  // a tensor's first or last chunk: one group at a time
    if (!factor(s)) return;
    auto same = [s](float &y) {
        y = s;
        return true;
    };
#pragma unroll 1
    for (int64_t at = r.first; at < r.end; at += kWave * V) {
        if constexpr (Q8) update8<W, G, V, 1, false, true, WIDE>(t, at, r.end, same, h);
        else update32<W, G, V, 1, false>(t, at, r.end, same, h);
    }
}

// Flat arrays of the list's elements, in list order: w, m and v, each float32
// or bfloat16, or null for one that is left out. Bound by HBM: at 124,356,864
// elements with bfloat16 weights and 8-bit moments, export to float32 takes
// 329 us = 6.1 TB/s (three quarters of it written), of the moments alone to
// bfloat16 119 us = 6.3 TB/s (8 elements a lane there, whole lines of it), import
// from float32 313 us = 6.4 TB/s.
struct Flat {
    void *w, *m, *v;
    int wt, mt, vt;
};

template <bool FULL, int V>
__device__ __forceinline__ void store_as(int type, void *p, int64_t first, uint32_t at, int cnt,
                                         const float (&x)[V]) {
    if (type == RCS_F32) store<FULL>(p, first, at, cnt, pack<F32>(x));
    else store<FULL>(p, first, at, cnt, pack<BF16>(x));
}

template <bool FULL, bool KEEP, int V>
__device__ __forceinline__ void load_as(int type, const void *p, int64_t first, uint32_t at,
                                        int cnt, float (&x)[V]) {
    if (type == RCS_F32) unpack(load<F32, V, FULL, KEEP>(p, first, at, cnt), x);
    else unpack(load<BF16, V, FULL, KEEP>(p, first, at, cnt), x);
}

// One group of V elements a lane from element `first` of t on.
template <bool Q8, int V, bool FULL, bool KEEP>
__device__ __forceinline__ void export_group(const Row &t, int64_t first, int64_t end,
                                             const Flat &f) {
    const int at = (int)threadIdx.x * V;
    const int cnt = FULL ? V : count_of<V>(end - first, at);
    if (cnt == 0) return;
    float m[V], v[V];
    if (f.m != nullptr || f.v != nullptr) {
        if constexpr (Q8) {
            decode_moments(load_codes<V>(t.m, first, at), load_codes<V>(t.v, first, at),
                           *exponents_at(t, first, at), kMaskM, kMaskV, m, v);
        } else {
            if (f.m != nullptr) unpack(load<F32, V, FULL>(t.m, first, at, cnt), m);
            if (f.v != nullptr) unpack(load<F32, V, FULL>(t.v, first, at, cnt), v);
        }
    }
    if (f.w != nullptr)
        by_type(t.wt(), [&](auto W) {
            float x[V];
            unpack(load<decltype(W), V, FULL, KEEP>(t.w, first, at, cnt), x);
            store_as<FULL>(f.wt, f.w, t.off + first, at, cnt, x);
        });
    if (f.m != nullptr) store_as<FULL>(f.mt, f.m, t.off + first, at, cnt, m);
    if (f.v != nullptr) store_as<FULL>(f.vt, f.v, t.off + first, at, cnt, v);
}

template <bool Q8, int V>
__global__ __launch_bounds__(kUpdThreads) void list_export(const Row *__restrict__ rows,
                                                           const Chunk *__restrict__ chunks,
                                                           uint32_t in_windows, Flat f) {
    const Chunk c = chunks[near_chunk(in_windows)];
    const Row t = rows[row_of(c)];
    const Range r = range_of<Q8>(c, t);
    if (r.whole) {
        by_lines(off_line(t.w, r.first * type_bytes(t.wt())), [&](auto K) {
#pragma unroll
            for (int q = 0; q < kChunk / (kWave * V); ++q)
                export_group<Q8, V, true, K.value>(t, r.first + q * kWave * V, r.end, f);
        });
        return;
    }
#pragma unroll 1
    for (int64_t at = r.first; at < r.end; at += kWave * V)
        export_group<Q8, V, false, true>(t, at, r.end, f);
}

// With 8-bit moments, m and v come together (the host sees to it): a block's
// two exponents are one store.
template <bool Q8, int V, bool FULL, bool KEEP>
__device__ __forceinline__ void import_group(const Row &t, int64_t first, int64_t end,
                                             const Flat &f) {
    const int at = (int)threadIdx.x * V;
    const int64_t left = end - first;
    const int cnt = FULL ? V : count_of<V>(left, at);
    float m[V], v[V];
    if (f.m != nullptr) load_as<FULL, KEEP>(f.mt, f.m, t.off + first, at, cnt, m);
    if (f.v != nullptr) load_as<FULL, KEEP>(f.vt, f.v, t.off + first, at, cnt, v);
    if (f.w != nullptr && cnt > 0) {
        float x[V];
        load_as<FULL, KEEP>(f.wt, f.w, t.off + first, at, cnt, x);
        by_type(t.wt(), [&](auto W) { store<FULL>(t.w, first, at, cnt, pack<decltype(W)>(x)); });
        if (t.c != nullptr) {
            if (t.ct() == RCS_BF16) store<FULL>(t.c, first, at, cnt, pack<BF16>(x));
            else store<FULL>(t.c, first, at, cnt, pack<F16>(x));
        }
    }
    if constexpr (Q8) {
        if (f.m == nullptr) return;
#pragma unroll
        for (int k = 0; k < V; ++k) {  // a NaN becomes an infinity, v below zero zero
            const uint32_t a = __float_as_uint(m[k]), u = __float_as_uint(v[k]);
            const uint32_t a1 = a & 0x7FFFFFFFu, u1 = u & 0x7FFFFFFFu;
            m[k] = __uint_as_float((a1 < 0x7F800000u ? a1 : 0x7F800000u) | (a & 0x80000000u));
            v[k] = __uint_as_float(u1 > 0x7F800000u ? 0x7F800000u : u == u1 ? u : 0u);
        }
        store_moments(t, first, at, m, v, FULL || (at & ~(kBlock - 1)) < left,
                      [&](int k) { return half_unit(__float_as_uint(m[k])); },
                      [&](int k) { return half_unit(__float_as_uint(v[k])); });
    } else {
        if (f.m != nullptr && cnt > 0) store<FULL>(t.m, first, at, cnt, pack<F32>(m));
        if (f.v != nullptr && cnt > 0) store<FULL>(t.v, first, at, cnt, pack<F32>(v));
    }
}

template <bool Q8, int V>
__global__ __launch_bounds__(kUpdThreads) void list_import(const Row *__restrict__ rows,
                                                           const Chunk *__restrict__ chunks,
                                                           uint32_t in_windows, Flat f) {
    const Chunk c = chunks[near_chunk(in_windows)];
    const Row t = rows[row_of(c)];
    const Range r = range_of<Q8>(c, t);
    if (r.whole) {
        by_lines(off_line(f.m, (t.off + r.first) * type_bytes(f.mt)), [&](auto K) {
#pragma unroll
            for (int q = 0; q < kChunk / (kWave * V); ++q)
                import_group<Q8, V, true, K.value>(t, r.first + q * kWave * V, r.end, f);
        });
        return;
    }
#pragma unroll 1
    for (int64_t at = r.first; at < r.end; at += kWave * V)
        import_group<Q8, V, false, true>(t, at, r.end, f);
}

// Other gradients for rows first .. first + count - 1. The pointers travel in
// the kernel's arguments, so the call is in stream order and needs no staging.
constexpr int kBind = 256;
struct Pointers {
    const void *p[kBind];
};
__global__ __launch_bounds__(kBind) void list_bind(Row *__restrict__ rows, int count,
                                                   Pointers g) {
    if ((int)threadIdx.x < count) rows[threadIdx.x].g = g.p[threadIdx.x];
}

// ----------------------------------------------------------------- host side

// The shift of a tensor whose m begins at p (32-bit moments).
int64_t shift_of(const void *p, int64_t n) {
    const int64_t head = (int64_t)((256u - (reinterpret_cast<uintptr_t>(p) & 255u)) & 255u) / 4;
    return head == 0 || n <= kChunk ? 0 : kChunk - head;
}

int64_t chunks_of(const rcs_list_tensor &t, int bits) {
    return (t.n + (bits == 8 ? 0 : shift_of(t.m, t.n)) + kChunk - 1) / kChunk;
}

struct Span {
    const char *lo, *hi;
};

// The chunks whose weights and gradients are of one pair of types.
struct Group {
    int wt, gt;
    int64_t first, count;
};

bool by_start(const Span &a, const Span &b) { return a.lo < b.lo; }

}  // namespace

struct rcs_list {
    int dev = 0;
    int bits = 32;
    int64_t n = 0;        // elements of all tensors
    int64_t nchunks = 0;
    int64_t bytes = 0;     // of weights, gradients, copies and 8-bit moments
    int64_t keep_from = 0;  // first chunk whose gradient the norm pass leaves in the cache
    std::vector<Row> rows;
    std::vector<Group> groups;
    std::vector<Span> written;  // what an update writes, sorted
    // gradients of captured bindings, which a replay may put in the place of the
    // rows', up to the next eager binding
    std::vector<Span> captured;
    char *mem = nullptr;        // everything below, one allocation
    Row *d_rows = nullptr;
    Chunk *d_chunks = nullptr;
    // norm buffers of the update, and of a norm call that is being captured
    // (an eager one uses its stream's)
    NormBuffers norm[2];

    // Whether [p, p + bytes) shares a byte with what an update writes.
    bool touches(const void *p, int64_t bytes) const {
        const Span s{static_cast<const char *>(p), static_cast<const char *>(p) + bytes};
        auto it = std::upper_bound(written.begin(), written.end(), s, by_start);
        if (it != written.end() && it->lo < s.hi) return true;
        return it != written.begin() && (it - 1)->hi > s.lo;
    }

    int norm_blocks() const {
        const int64_t b = (nchunks + kListNormThreads / kWave - 1) / (kListNormThreads / kWave);
        return (int)(b < kNormMaxBlocks ? b : kNormMaxBlocks);
    }
};

namespace {

// The largest list whose update folds the final reduction of the norm; above it
// the norm pass ends with it. us a step with and without: 7.4 and 8.4 at 262,144
// float32 elements, 10.6 and 12.0 at 1M, 25.2 and 26.8 at 4M, 44.1 and 47.2 at
// 8.4M; 8-bit moments at 8.0M 33.0 and 32.6.
constexpr int64_t kListFoldMaxN = 8388608;
// Bytes at the end of the gradients that the norm pass reads with cache-
// allocating loads, so that the update finds them in the last-level cache.
constexpr int64_t kCachedTailBytes = 320LL << 20;
constexpr int64_t kCacheBytes = 256LL << 20;  // the last-level cache
// Waves of a launch: the grid's work-items have to fit 32 bits.
constexpr int64_t kMaxChunks = 0xFFFFFFFFLL / kUpdThreads;

bool aligned(const void *p, int align) {
    return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(align - 1)) == 0;
}

// Checks pointers of one call: aligned to their element and, as for the other
// entry points, inside one allocation of the current device. The allocations
// seen are remembered for the call: a list's arrays mostly lie in few of them,
// and each question to the runtime costs more than the rest of the check.
class Arrays {
public:
    int check(const void *p, int64_t bytes, int align) {
        if (!aligned(p, align)) return RCS_EINVAL;
        const char *q = static_cast<const char *>(p);
        for (const Span &s : seen_)
            if (s.lo <= q && q < s.hi) return bytes <= s.hi - q ? RCS_OK : RCS_ESIZE;
        const int rc = check_device_range(p, bytes);
        if (rc != RCS_OK) return rc;
        hipDeviceptr_t base = nullptr;
        size_t size = 0;
        if (hipMemGetAddressRange(&base, &size, const_cast<void *>(p)) == hipSuccess && base) {
            const char *lo = static_cast<const char *>(base);
            seen_[next_++ % kSeen] = Span{lo, lo + size};
        } else {
            (void)hipGetLastError();
        }
        return RCS_OK;
    }

private:
    static constexpr unsigned kSeen = 16;
    Span seen_[kSeen] = {};
    unsigned next_ = 0;
};

int check_list(const rcs_list *list) {
    if (list == nullptr) return RCS_EINVAL;
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess) return RCS_EHIP;
    return dev == list->dev ? RCS_OK : RCS_EINVAL;
}

// norm_out on the device, where the kernels can write it; null if it is host
// memory (copied there afterwards) or not wanted.
bool on_device(const double *p) {
    hipPointerAttribute_t pa;
    if (p == nullptr || hipPointerGetAttributes(&pa, p) != hipSuccess) {
        (void)hipGetLastError();
        return false;
    }
    return pa.type != hipMemoryTypeHost;
}

bool capturing(hipStream_t stream) {
    hipStreamCaptureStatus st = hipStreamCaptureStatusNone;
    if (hipStreamIsCapturing(stream, &st) != hipSuccess) {
        (void)hipGetLastError();
        return false;
    }
    return st != hipStreamCaptureStatusNone;
}

// The workspace of a stream that is not being captured. It may be made while
// another stream is: an allocation of this thread is no part of that capture.
int list_workspace(int dev, hipStream_t stream, Workspace **out) {
    if (t_ws.ws != nullptr && t_ws.dev == dev && t_ws.stream == stream) {
        *out = t_ws.ws;
        return RCS_OK;
    }
    hipStreamCaptureMode mode = hipStreamCaptureModeRelaxed;
    const bool swapped = hipThreadExchangeStreamCaptureMode(&mode) == hipSuccess;
    const int rc = get_workspace(stream, out);
    if (swapped) (void)hipThreadExchangeStreamCaptureMode(&mode);
    return rc;
}

double *last_norm(const NormBuffers &nb) {
    return reinterpret_cast<double *>(reinterpret_cast<char *>(nb.partials) + kNormLastAt);
}

uint32_t *arrived(const NormBuffers &nb) {
    return reinterpret_cast<uint32_t *>(reinterpret_cast<char *>(nb.partials) + kNormArrivedAt);
}

// fold: the update will reduce the partials itself. dev_out, last: further places
// for the norm, or null.
void launch_norm(const rcs_list *l, float gscale, const NormBuffers &nb, bool fold, float clip,
                 double *dev_out, double *last, hipStream_t stream) {
    auto *kernel = l->bits == 8 ? list_norm<true> : list_norm<false>;
    hipLaunchKernelGGL(kernel, dim3(l->norm_blocks()), dim3(kListNormThreads), 0,
                       stream, (const Row *)l->d_rows, (const Chunk *)l->d_chunks, l->nchunks,
                       l->keep_from, gscale, nb.partials, fold ? nullptr : arrived(nb), clip,
                       nb.scalars, dev_out, last);
}

uint32_t in_windows(int64_t blocks) { return (uint32_t)(blocks - blocks % kWindow); }

template <bool Q8, bool FOLD, bool WIDE>
auto *update_kernel(const Group &g) {
    auto *kernel = list_update<F32, F32, Q8, FOLD, WIDE>;
    auto with = [&](auto W) {
        using WT = decltype(W);
        kernel = g.gt == RCS_F32    ? list_update<WT, F32, Q8, FOLD, WIDE>
                 : g.gt == RCS_BF16 ? list_update<WT, BF16, Q8, FOLD, WIDE>
                                    : list_update<WT, F16, Q8, FOLD, WIDE>;
    };
    if (g.wt == RCS_F32) with(F32{});
    else if (g.wt == RCS_BF16) with(BF16{});
    else with(F16{});
    return kernel;
}

int check_flat(Arrays &arrays, const rcs_list *l, const void *p, int type, bool writes) {
    if (p == nullptr) return RCS_OK;
    if (type != RCS_F32 && type != RCS_BF16) return RCS_EINVAL;
    const int64_t bytes = l->n * type_bytes(type);
    const int rc = arrays.check(p, bytes, type_bytes(type));
    if (rc != RCS_OK) return rc;
    if (l->touches(p, bytes)) return RCS_EINVAL;
    if (writes)  // an exported array is not a gradient either
        for (const Row &r : l->rows) {
            const char *g = static_cast<const char *>(r.g), *q = static_cast<const char *>(p);
            if (g != nullptr && g < q + bytes && q < g + r.n * type_bytes(r.gt())) return RCS_EINVAL;
        }
    if (writes)
        for (const Span &g : l->captured) {
            const char *q = static_cast<const char *>(p);
            if (g.lo < q + bytes && q < g.hi) return RCS_EINVAL;
        }
    return RCS_OK;
}

bool apart(const void *a, int ta, const void *b, int tb, int64_t n) {
    const char *x = static_cast<const char *>(a), *y = static_cast<const char *>(b);
    return a == nullptr || b == nullptr || x + n * type_bytes(ta) <= y ||
           y + n * type_bytes(tb) <= x;
}

}  // namespace

extern "C" {

int rcs_list_create(const rcs_list_tensor *tensors, int64_t count, int state_bits,
                    rcs_list **out) {
    if (out == nullptr) return RCS_EINVAL;
    *out = nullptr;
    if (tensors == nullptr || count < 1 || count > 0x7FFFFFFF ||
        (state_bits != 32 && state_bits != 8))
        return RCS_EINVAL;
    int64_t total = 0, nchunks = 0, bytes = 0;
    for (int64_t k = 0; k < count; ++k) {
        const rcs_list_tensor &t = tensors[k];
        if (t.n < 0 || t.n > (1LL << 40)) return RCS_EINVAL;
        if (type_bytes(t.w_type) == 0 || type_bytes(t.g_type) == 0 || !std::isfinite(t.wd))
            return RCS_EINVAL;
        if (t.copy != nullptr &&
            (t.w_type != RCS_F32 || (t.copy_type != RCS_BF16 && t.copy_type != RCS_F16)))
            return RCS_EINVAL;
        const int sa = state_bits == 32 ? 4 : 16;
        if (t.n > 0 && (!aligned(t.w, type_bytes(t.w_type)) || !aligned(t.m, sa) ||
                        !aligned(t.v, sa) || (state_bits == 8 && !aligned(t.exps, 2)) ||
                        (t.g != nullptr && !aligned(t.g, type_bytes(t.g_type))) ||
                        (t.copy != nullptr && !aligned(t.copy, 2))))
            return RCS_EINVAL;
        total += t.n;
        nchunks += chunks_of(t, state_bits);
        bytes += t.n * (type_bytes(t.w_type) + type_bytes(t.g_type) +
                        (t.copy != nullptr ? 2 : 0) + 2);
        if (nchunks > kMaxChunks) return RCS_EINVAL;
    }
    if (total < 1) return RCS_EINVAL;
    int rc;
    try {
        rcs_list *l = new rcs_list;
        struct Drop {
            rcs_list *l;
            ~Drop() { delete l; }
        } drop{l};
        Arrays arrays;
        l->bits = state_bits;
        l->n = total;
        l->nchunks = nchunks;
        l->bytes = bytes;
        if (hipGetDevice(&l->dev) != hipSuccess) return RCS_EHIP;
        std::vector<Chunk> chunks;
        chunks.reserve((size_t)nchunks);
        int64_t off = 0;
        for (int64_t k = 0; k < count; ++k) {
            const rcs_list_tensor &t = tensors[k];
            const uint32_t types = (uint32_t)t.w_type | (uint32_t)t.g_type << 8 |
                                   (t.copy != nullptr ? (uint32_t)t.copy_type << 16 : 0u);
            Row r{t.w, t.g, t.m, t.v, {}, t.n, off, t.wd, types, t.copy};
            if (state_bits == 8) r.e = static_cast<uint16_t *>(t.exps);
            else r.shift = shift_of(t.m, t.n);
            if (t.n == 0) {
                l->rows.push_back(r);
                continue;
            }
            const int wb = type_bytes(t.w_type), gb = type_bytes(t.g_type);
            const int64_t blocks = (t.n + kBlock - 1) / kBlock;
            const int64_t sb = state_bits == 32 ? 4 * t.n : blocks * kBlock;
            const int sa = state_bits == 32 ? 4 : 16;
            if ((rc = arrays.check(t.w, wb * t.n, wb)) != RCS_OK) return rc;
            if ((rc = arrays.check(t.m, sb, sa)) != RCS_OK) return rc;
            if ((rc = arrays.check(t.v, sb, sa)) != RCS_OK) return rc;
            if (t.g != nullptr && (rc = arrays.check(t.g, gb * t.n, gb)) != RCS_OK) return rc;
            if (t.copy != nullptr && (rc = arrays.check(t.copy, 2 * t.n, 2)) != RCS_OK) return rc;
            if (state_bits == 8 && (rc = arrays.check(t.exps, 2 * blocks, 2)) != RCS_OK) return rc;
            auto add = [&](const void *p, int64_t bytes) {
                const char *c = static_cast<const char *>(p);
                l->written.push_back(Span{c, c + bytes});
            };
            add(t.w, wb * t.n);
            add(t.m, sb);
            add(t.v, sb);
            if (t.copy != nullptr) add(t.copy, 2 * t.n);
            if (state_bits == 8) add(t.exps, 2 * blocks);
            l->rows.push_back(r);
            off += t.n;
        }
        for (int pair = 0; pair < 9; ++pair) {
            const Group g{pair / 3, pair % 3, (int64_t)chunks.size(), 0};
            for (int64_t k = 0; k < count; ++k)
                if (tensors[k].w_type == g.wt && tensors[k].g_type == g.gt)
                    for (int64_t c = 0; c < chunks_of(tensors[k], state_bits); ++c)
                        chunks.push_back((Chunk)c << 32 | (Chunk)k);
            if ((int64_t)chunks.size() > g.first)
                l->groups.push_back(
                    Group{g.wt, g.gt, g.first, (int64_t)chunks.size() - g.first});
        }
        // the last chunks, as many as hold kCachedTailBytes of gradients
        l->keep_from = nchunks;
        int64_t tail = 0;
        for (size_t k = l->groups.size(); k-- > 0 && tail < kCachedTailBytes;) {
            const Group &g = l->groups[k];
            const int64_t per = (int64_t)kChunk * type_bytes(g.gt);
            const int64_t want = (kCachedTailBytes - tail + per - 1) / per;
            const int64_t take = g.count < want ? g.count : want;
            l->keep_from -= take;
            tail += take * per;
        }
        std::sort(l->written.begin(), l->written.end(), by_start);
        for (size_t k = 1; k < l->written.size(); ++k)
            if (l->written[k].lo < l->written[k - 1].hi) return RCS_EINVAL;
        for (const Row &r : l->rows)
            if (r.n > 0 && r.g != nullptr && l->touches(r.g, r.n * type_bytes(r.gt())))
                return RCS_EINVAL;

        const size_t rows_b = (l->rows.size() * sizeof(Row) + 255) / 256 * 256;
        const size_t chunks_b = (chunks.size() * sizeof(Chunk) + 255) / 256 * 256;
        std::vector<char> tables(rows_b + chunks_b + 2 * kNormBytes);
        std::memcpy(tables.data(), l->rows.data(), l->rows.size() * sizeof(Row));
        std::memcpy(tables.data() + rows_b, chunks.data(), chunks.size() * sizeof(Chunk));
        void *p = nullptr;
        if (hipMalloc(&p, tables.size()) != hipSuccess) {
            (void)hipGetLastError();
            return RCS_ENOMEM;
        }
        l->mem = static_cast<char *>(p);
        l->d_rows = reinterpret_cast<Row *>(l->mem);
        l->d_chunks = reinterpret_cast<Chunk *>(l->mem + rows_b);
        for (int k = 0; k < 2; ++k) {
            char *q = l->mem + rows_b + chunks_b + (size_t)k * kNormBytes;
            l->norm[k].partials = reinterpret_cast<double *>(q);
            l->norm[k].scalars = reinterpret_cast<ClipScalars *>(q + kNormRecordAt);
        }
        if (hipMemcpy(l->mem, tables.data(), tables.size(), hipMemcpyHostToDevice) !=
                hipSuccess ||
            hipStreamSynchronize(nullptr) != hipSuccess) {
            (void)hipGetLastError();
            (void)hipFree(p);
            return RCS_EHIP;
        }
        drop.l = nullptr;
        *out = l;
        return RCS_OK;
    } catch (const std::bad_alloc &) {
        return RCS_ENOMEM;
    }
}

int rcs_list_destroy(rcs_list *list) {
    if (list == nullptr) return RCS_OK;
    // hipFree is not among the calls that a capture under way elsewhere
    // tolerates by default; this thread's calls are no part of one
    hipStreamCaptureMode mode = hipStreamCaptureModeRelaxed;
    const bool swapped = hipThreadExchangeStreamCaptureMode(&mode) == hipSuccess;
    const hipError_t e = hipFree(list->mem);  // waits for the work that uses it
    if (swapped) (void)hipThreadExchangeStreamCaptureMode(&mode);
    delete list;
    if (e == hipSuccess) return RCS_OK;
    (void)hipGetLastError();
    return RCS_EHIP;
}

int64_t rcs_list_elements(const rcs_list *list) { return list == nullptr ? -1 : list->n; }

int rcs_list_bind_grads(rcs_list *list, const void *const *g, int64_t count, hipStream_t stream) {
    int rc;
    Arrays arrays;
    if (list == nullptr || g == nullptr || count != (int64_t)list->rows.size()) return RCS_EINVAL;
    if ((rc = check_list(list)) != RCS_OK) return rc;
    for (int64_t k = 0; k < count; ++k) {
        const Row &r = list->rows[(size_t)k];
        if (r.n == 0 || g[k] == nullptr) continue;
        const int b = type_bytes(r.gt());
        if ((rc = arrays.check(g[k], b * r.n, b)) != RCS_OK) return rc;
        if (list->touches(g[k], b * r.n)) return RCS_EINVAL;
    }
    const bool later = capturing(stream);
    if (later) {
        const size_t before = list->captured.size();
        try {
            for (int64_t k = 0; k < count; ++k) {
                const Row &r = list->rows[(size_t)k];
                const char *p = static_cast<const char *>(g[k]);
                if (r.n > 0 && p != nullptr)
                    list->captured.push_back(Span{p, p + r.n * type_bytes(r.gt())});
            }
        } catch (const std::bad_alloc &) {
            list->captured.resize(before);
            return RCS_ENOMEM;
        }
    } else {
        list->captured.clear();
    }
    for (int64_t k = 0; k < count; k += kBind) {
        const int some = (int)(count - k < kBind ? count - k : kBind);
        Pointers p;
        for (int j = 0; j < kBind; ++j) p.p[j] = j < some ? g[k + j] : nullptr;
        hipLaunchKernelGGL(list_bind, dim3(1), dim3(kBind), 0, stream, list->d_rows + k, some, p);
        for (int j = 0; !later && j < some; ++j) list->rows[(size_t)(k + j)].g = g[k + j];
    }
    return hipGetLastError() == hipSuccess ? RCS_OK : RCS_EHIP;
}

int rcs_stream_capturing(hipStream_t stream) { return capturing(stream) ? 1 : 0; }

int grad_global_norm_list(const rcs_list *list, float grad_scale, double *norm_out,
                          hipStream_t stream) {
    int rc;
    if (list == nullptr || norm_out == nullptr) return RCS_EINVAL;
    if (!std::isfinite(grad_scale) || !(grad_scale > 0.0f)) return RCS_EINVAL;
    if ((rc = check_list(list)) != RCS_OK) return rc;
    if ((rc = check_norm_out(norm_out, list->dev)) != RCS_OK) return rc;
    NormBuffers nb = list->norm[1];
    Workspace *ws = nullptr;
    if (!capturing(stream)) {
        if ((rc = list_workspace(list->dev, stream, &ws)) != RCS_OK) return rc;
        nb = *ws;
        std::lock_guard<std::mutex> lk(g_mu);
        if (!ws->counts) {  // in stream order before the first pass that counts there
            hipLaunchKernelGGL(list_norm_init, dim3(1), dim3(1), 0, stream, arrived(nb));
            if (hipGetLastError() != hipSuccess) return RCS_EHIP;
            ws->counts = true;
        }
    }
    const bool direct = on_device(norm_out);
    launch_norm(list, grad_scale, nb, false, INFINITY, direct ? norm_out : nullptr, nullptr,
                stream);
    if (hipGetLastError() != hipSuccess) return RCS_EHIP;
    if (ws != nullptr) ws->last = &ws->scalars->norm;
    if (!direct && hipMemcpyAsync(norm_out, &nb.scalars->norm, sizeof(double), hipMemcpyDefault,
                                  stream) != hipSuccess)
        return RCS_EHIP;
    return RCS_OK;
}

int adamw_clip_step_list(rcs_list *list, int32_t t, float lr, float clip, float grad_scale,
                         double beta1, double beta2, float eps, uint32_t seed, double *norm_out,
                         hipStream_t stream) {
    int rc;
    if (list == nullptr || t < 1) return RCS_EINVAL;
    if (!std::isfinite(lr) || std::isnan(clip) || !(clip > 0.0f)) return RCS_EINVAL;
    if (!std::isfinite(grad_scale) || !(grad_scale > 0.0f)) return RCS_EINVAL;
    if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0)) return RCS_EINVAL;
    if (!std::isnormal(eps) || !(eps > 0.0f)) return RCS_EINVAL;
    if ((rc = check_list(list)) != RCS_OK) return rc;
    if (norm_out != nullptr && (rc = check_norm_out(norm_out, list->dev)) != RCS_OK) return rc;
    ListScalars h;
    h.lr = lr;
    h.bc1 = (float)(1.0 - std::pow(beta1, (double)t));
    h.bc2 = (float)(1.0 - std::pow(beta2, (double)t));
    h.b1 = (float)beta1;
    h.c1 = (float)(1.0 - beta1);
    h.b2 = (float)beta2;
    h.c2 = (float)(1.0 - beta2);
    h.eps = eps;
    h.gscale = grad_scale;
    h.fits = list->bytes <= kCacheBytes;
    h.mask_m = h.b1 == 0.0f ? 0u : kMaskM;
    h.mask_v = h.b2 == 0.0f ? 0u : kMaskV;
    // weight_free's constants; a learning rate of zero divides by infinity
    const double over = (1.0 - std::pow(beta1, (double)t)) / (double)lr;
    const double root2 = std::sqrt(1.0 - std::pow(beta2, (double)t));
    const double da = over / root2, db = over * (double)eps;
    const double most = std::fabs(da) * 0x1p64 + std::fabs(db);
    bool wide = root2 * (double)eps < kWideEps;
    h.da = (float)da;
    h.db = (float)db;
    h.sc = 1.0f;
    if (lr == 0.0f) {
        h.da = 1.0f;
        h.db = INFINITY;
    } else if (list->bits == 8 && std::fabs(db) < (double)FLT_MIN) {
        return RCS_EINVAL;  // lr so large that v = 0 would divide by nothing
    } else if (most > kWideDen) {
        const int k = std::ilogb(most / kWideDen) + 1;
        h.da = (float)std::ldexp(da, -k);
        h.db = (float)std::ldexp(db, -k);
        h.sc = (float)std::ldexp(1.0, -k);
        wide = true;
    }
    h.key = mixed(mixed(seed * kHashA + (uint32_t)t * kHashB) + kHashK);
    const bool fold = list->n <= kListFoldMaxN, q8 = list->bits == 8;
    const bool direct = norm_out != nullptr && on_device(norm_out);
    double *dev_out = direct ? norm_out : nullptr;
    const NormBuffers &nb = list->norm[0];
    // for last_grad_norm; a replay reports only where norm_out says
    Workspace *ws = nullptr;
    if (!capturing(stream) && (rc = list_workspace(list->dev, stream, &ws)) != RCS_OK) return rc;
    double *last = ws != nullptr ? last_norm(*ws) : nullptr;
    launch_norm(list, grad_scale, nb, fold, clip, dev_out, last, stream);
    const bool near = q8 || list->n <= kNearMaxN;
    for (const Group &g : list->groups) {
        auto *kernel = fold ? update_kernel<false, true, false>(g)
                            : update_kernel<false, false, false>(g);
        if (q8 && wide)
            kernel = fold ? update_kernel<true, true, true>(g) : update_kernel<true, false, true>(g);
        else if (q8)
            kernel = fold ? update_kernel<true, true, false>(g)
                          : update_kernel<true, false, false>(g);
        hipLaunchKernelGGL(kernel, dim3((unsigned)g.count), dim3(kUpdThreads), 0, stream,
                           (const Row *)list->d_rows, (const Chunk *)list->d_chunks + g.first,
                           near ? in_windows(g.count) : 0u, list->norm_blocks(),
                           (const double *)nb.partials, clip, nb.scalars, dev_out, last, h);
    }
    if (hipGetLastError() != hipSuccess) return RCS_EHIP;
    if (ws != nullptr) ws->last = last;
    if (norm_out != nullptr && !direct &&
        hipMemcpyAsync(norm_out, &nb.scalars->norm, sizeof(double), hipMemcpyDefault, stream) !=
            hipSuccess)
        return RCS_EHIP;
    return RCS_OK;
}

int rcs_list_export(const rcs_list *list, void *w, int w_type, void *m, int m_type, void *v,
                    int v_type, hipStream_t stream) {
    int rc;
    if (list == nullptr || (w == nullptr && m == nullptr && v == nullptr)) return RCS_EINVAL;
    if ((rc = check_list(list)) != RCS_OK) return rc;
    Arrays arrays;
    if ((rc = check_flat(arrays, list, w, w_type, true)) != RCS_OK) return rc;
    if ((rc = check_flat(arrays, list, m, m_type, true)) != RCS_OK) return rc;
    if ((rc = check_flat(arrays, list, v, v_type, true)) != RCS_OK) return rc;
    if (!apart(w, w_type, m, m_type, list->n) || !apart(w, w_type, v, v_type, list->n) ||
        !apart(m, m_type, v, v_type, list->n))
        return RCS_EINVAL;
    const Flat f{w, m, v, w_type, m_type, v_type};
    const bool wide = (w == nullptr || w_type == RCS_BF16) && (m == nullptr || m_type == RCS_BF16) &&
                      (v == nullptr || v_type == RCS_BF16);
    auto *kernel = list->bits == 8 ? (wide ? list_export<true, 8> : list_export<true, 4>)
                                   : list_export<false, 4>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)list->nchunks), dim3(kUpdThreads), 0, stream,
                       (const Row *)list->d_rows, (const Chunk *)list->d_chunks,
                       in_windows(list->nchunks), f);
    return hipGetLastError() == hipSuccess ? RCS_OK : RCS_EHIP;
}

int rcs_list_import(rcs_list *list, const void *w, int w_type, const void *m, int m_type,
                    const void *v, int v_type, hipStream_t stream) {
    int rc;
    if (list == nullptr || (w == nullptr && m == nullptr && v == nullptr)) return RCS_EINVAL;
    if (list->bits == 8 && (m == nullptr) != (v == nullptr)) return RCS_EINVAL;
    if ((rc = check_list(list)) != RCS_OK) return rc;
    Arrays arrays;
    if ((rc = check_flat(arrays, list, w, w_type, false)) != RCS_OK) return rc;
    if ((rc = check_flat(arrays, list, m, m_type, false)) != RCS_OK) return rc;
    if ((rc = check_flat(arrays, list, v, v_type, false)) != RCS_OK) return rc;
    const Flat f{const_cast<void *>(w), const_cast<void *>(m), const_cast<void *>(v), w_type,
                 m_type, v_type};
    const bool wide = (w == nullptr || w_type == RCS_BF16) && (m == nullptr || m_type == RCS_BF16);
    auto *kernel = list->bits == 8 ? (wide ? list_import<true, 8> : list_import<true, 4>)
                                   : list_import<false, 4>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)list->nchunks), dim3(kUpdThreads), 0, stream,
                       (const Row *)list->d_rows, (const Chunk *)list->d_chunks,
                       in_windows(list->nchunks), f);
    return hipGetLastError() == hipSuccess ? RCS_OK : RCS_EHIP;
}

}  // extern "C"
