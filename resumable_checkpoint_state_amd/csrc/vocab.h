// vocab.h -- what the output head's and the embedding's kernels share: elements
// of three types, and the checks of their calls' arguments.
#ifndef RCS_VOCAB_H
#define RCS_VOCAB_H

#include <hip/hip_runtime.h>

#include <cstdint>

#include "rcs.h"
#include "rcs_internal.h"

#pragma clang fp contract(off)

namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

struct F32 {
    static constexpr int kType = RCS_F32, kBytes = 4;
};
struct BF16 {
    static constexpr int kType = RCS_BF16, kBytes = 2;
};
struct F16 {
    static constexpr int kType = RCS_F16, kBytes = 2;
};

__device__ __forceinline__ uint32_t two(float a, float b, BF16) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}
__device__ __forceinline__ uint32_t two(float a, float b, F16) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, f16x2));
}
__device__ __forceinline__ float value(uint16_t b, BF16) {
    return __uint_as_float((uint32_t)b << 16);
}
__device__ __forceinline__ float value(uint16_t b, F16) {
    return (float)__builtin_bit_cast(_Float16, b);
}

// Element i of an array of type t (RCS_F32, RCS_BF16, RCS_F16).
__device__ __forceinline__ float element(const void *p, int64_t i, int t) {
    if (t == RCS_F32) return static_cast<const float *>(p)[i];
    const uint16_t b = static_cast<const uint16_t *>(p)[i];
    return t == RCS_BF16 ? value(b, BF16{}) : value(b, F16{});
}
__device__ __forceinline__ void put(void *p, int64_t i, int t, float x) {
    if (t == RCS_F32) static_cast<float *>(p)[i] = x;
    else static_cast<uint16_t *>(p)[i] =
        (uint16_t)(t == RCS_BF16 ? two(x, 0.f, BF16{}) : two(x, 0.f, F16{}));
}
// Four consecutive elements, aligned to one: the hardware's vector accesses need
// no more.
typedef u32x4 u32x4_any __attribute__((aligned(4)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));
template <class T>
__device__ __forceinline__ f32x4 four(u32x2 b, T) {
    return f32x4{value((uint16_t)b[0], T{}), value((uint16_t)(b[0] >> 16), T{}),
                 value((uint16_t)b[1], T{}), value((uint16_t)(b[1] >> 16), T{})};
}
__device__ __forceinline__ f32x4 load4(const void *p, int64_t i, int t) {
    if (t == RCS_F32)
        return __builtin_bit_cast(
            f32x4, *reinterpret_cast<const u32x4_any *>(static_cast<const float *>(p) + i));
    const u32x2 b = *reinterpret_cast<const u32x2_any *>(static_cast<const uint16_t *>(p) + i);
    return t == RCS_BF16 ? four(b, BF16{}) : four(b, F16{});
}
typedef u32x4 u32x4_half __attribute__((aligned(2)));
__device__ __forceinline__ void store4(void *p, int64_t i, int t, f32x4 x) {
    if (t == RCS_F32) {
        *reinterpret_cast<u32x4_any *>(static_cast<float *>(p) + i) = __builtin_bit_cast(u32x4, x);
        return;
    }
    const u32x2 b = t == RCS_BF16 ? u32x2{two(x[0], x[1], BF16{}), two(x[2], x[3], BF16{})}
                                  : u32x2{two(x[0], x[1], F16{}), two(x[2], x[3], F16{})};
    *reinterpret_cast<u32x2_any *>(static_cast<uint16_t *>(p) + i) = b;
}
__device__ __forceinline__ float pick(f32x4 x, int r) {
    return r == 0 ? x[0] : r == 1 ? x[1] : r == 2 ? x[2] : x[3];
}
// x to elements i to i + 3 of p, or to those of them that there are (`left`); added
// to what is there, with add.
__device__ __forceinline__ void put4(void *p, int64_t i, int t, f32x4 x, int64_t left, bool add) {
    if (left >= 4) {
        if (add) x += load4(p, i, t);
        store4(p, i, t, x);
        return;
    }
    for (int r = 0; r < 3; ++r)
        if (r < left) put(p, i + r, t, add ? pick(x, r) + element(p, i + r, t) : pick(x, r));
}
// Elements i to i + cols - 1 of p, of type T, cols at most 4 (zeros behind them).
template <class T>
__device__ __forceinline__ f32x4 load_some(const void *p, int64_t i, int cols, T) {
    if (cols >= 4) return load4(p, i, T::kType);
    f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int r = 0; r < 3; ++r)
        if (r < cols) x[r] = element(p, i + r, T::kType);
    return x;
}
template <class T>
__device__ __forceinline__ void store_some(void *p, int64_t i, int cols, f32x4 x, T) {
    if (cols >= 4) {
        store4(p, i, T::kType, x);
        return;
    }
#pragma unroll
    for (int r = 0; r < 3; ++r)
        if (r < cols) put(p, i + r, T::kType, pick(x, r));
}
__device__ __forceinline__ int64_t index_at(const void *p, int64_t i, int t) {
    return t == RCS_I32 ? (int64_t) static_cast<const int32_t *>(p)[i]
                        : static_cast<const int64_t *>(p)[i];
}

constexpr int kWave = 64;

// ----------------------------------------------------------------- host side

constexpr int64_t kMaxStride = 1 << 20;  // of a matrix: offsets within a tile fit 32 bits
constexpr int64_t kMaxRows = 1 << 23, kMaxDim = 1 << 16;  // the grids' threads do, too

inline int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }
inline int type_size(int type) { return type == RCS_F32 ? 4 : 2; }
inline bool is_type(int t) { return t == RCS_F32 || t == RCS_BF16 || t == RCS_F16; }
inline int index_size(int type) { return type == RCS_I32 ? 4 : 8; }
inline bool is_index_type(int t) { return t == RCS_I32 || t == RCS_I64; }

// f(T) for the element type t.
template <class F>
void by_type(int t, F f) {
    if (t == RCS_F32) f(F32{});
    else if (t == RCS_BF16) f(BF16{});
    else f(F16{});
}

// The allocations that a call's arrays lie in: often few, and each question to the
// runtime costs more than the rest of a check.
class Allocations {
public:
    int check(const void *p, int64_t bytes) {
        const char *q = static_cast<const char *>(p);
        for (int k = 0; k < n_; ++k)
            if (lo_[k] <= q && q < hi_[k]) return bytes <= hi_[k] - q ? RCS_OK : RCS_ESIZE;
        const char *lo, *hi;
        const int rc = rcs_device_allocation(p, &lo, &hi);
        if (rc != RCS_OK || lo == nullptr) return rc;
        if (n_ < kMost) lo_[n_] = lo, hi_[n_++] = hi;
        return bytes <= hi - q ? RCS_OK : RCS_ESIZE;
    }

private:
    static constexpr int kMost = 8;
    const char *lo_[kMost], *hi_[kMost];
    int n_ = 0;
};

// What a call reads, or what it writes: each checked as it is added.
class Extents {
public:
    explicit Extents(Allocations &seen) : seen_(seen) {}
    int array(const void *p, int64_t bytes, int align) {
        if (bytes == 0) return RCS_OK;
        if (p == nullptr || (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(align - 1)) != 0)
            return RCS_EINVAL;
        const int rc = seen_.check(p, bytes);
        if (rc == RCS_OK) all_[n_++] = Extent{p, bytes};
        return rc;
    }
    int matrix(const void *p, int64_t rows, int64_t cols, int64_t stride, int type) {
        if (stride < cols || stride > kMaxStride) return RCS_EINVAL;
        const int size = type_size(type);
        return array(p, rows == 0 ? 0 : ((rows - 1) * stride + cols) * size, size);
    }
    // Whether these (written) share a byte with those (read) or with each other.
    bool overlap(const Extents &reads) const {
        for (int k = 0; k < n_; ++k) {
            for (int j = 0; j < reads.n_; ++j)
                if (rcs_overlaps(all_[k].p, all_[k].bytes, reads.all_[j].p, reads.all_[j].bytes))
                    return true;
            for (int j = 0; j < k; ++j)
                if (rcs_overlaps(all_[k].p, all_[k].bytes, all_[j].p, all_[j].bytes)) return true;
        }
        return false;
    }

private:
    struct Extent {
        const void *p;
        int64_t bytes;
    };
    Allocations &seen_;
    Extent all_[6];
    int n_ = 0;
};

}  // namespace

#endif
