// rcs_device.h -- device code that the library's kernels share: the wave and
// block sums, the final reduction of the norm pass with the clip record and the
// streaming accesses. Everything has internal linkage (each source file
// compiles its own copy).
#ifndef RCS_DEVICE_H
#define RCS_DEVICE_H

#include <hip/hip_runtime.h>

#include <cstdint>

#pragma clang fp contract(off)

namespace {

constexpr int kWave = 64;
// The norm pass never has more blocks, and so partial sums, than this.
constexpr int kNormMaxBlocks = 256;
// At most this many partials reach the final reduction.
constexpr int kParts = kNormMaxBlocks;
// Lanes per block of the update and in-place scale kernels, one 16-byte
// vector of each array per lane; the final reduction (in those kernels and in
// grad_norm_final) runs on blocks of the same size, lane i summing partials
// i, i + L, i + 2L, ... in that order, so all three give the same bits.
// One wave per block measured fastest: the update takes 529.7 us at the
// ANDREA-120M size against 546.1 us with 256 lanes (same process).
constexpr int kUpdThreads = 64;
static_assert(kUpdThreads == 64 || kUpdThreads == 128 || kUpdThreads == 256, "lanes per block");
constexpr int kPartsPerLane = kParts / kUpdThreads;

// Native 16-byte vector (the nontemporal builtins need a clang vector type).
typedef float f32x4 __attribute__((ext_vector_type(4)));

struct ClipScalars {
    double norm;    // pre-clip global L2 norm
    float scale;    // clip factor s
    int32_t apply;  // 1 when the norm is finite, else the update is skipped
};

// ---------------------------------------------------------------- reductions

__device__ __forceinline__ double as_double(uint32_t lo, uint32_t hi) {
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

template <int CTRL>
__device__ __forceinline__ double dpp_f64(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const int lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, 0xF, 0xF, true);
    const int hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, 0xF, 0xF, true);
    return as_double((uint32_t)lo, (uint32_t)hi);
}

// Sum over the 64 lanes; every lane ends with the same value (each step adds
// a value to its mirror partner, and a + b == b + a exactly).
__device__ __forceinline__ double wave_sum(double x) {
    x += dpp_f64<0xB1>(x);   // quad_perm [1,0,3,2]: pairs
    x += dpp_f64<0x4E>(x);   // quad_perm [2,3,0,1]: quads
    x += dpp_f64<0x141>(x);  // row_half_mirror: 8 lanes
    x += dpp_f64<0x140>(x);  // row_mirror: 16-lane row
    x += __shfl_xor(x, 16, kWave);
    x += __shfl_xor(x, 32, kWave);
    return x;
}

// Block sum in wave order; the result is valid in thread 0 only.
template <int THREADS>
__device__ __forceinline__ double block_sum(double x, double *lds) {
    x = wave_sum(x);
    const int lane = threadIdx.x & (kWave - 1);
    const int wid = threadIdx.x / kWave;
    if (lane == 0) lds[wid] = x;
    __syncthreads();
    double r = 0.0;
    if (threadIdx.x == 0) {
        r = lds[0];
#pragma unroll
        for (int i = 1; i < THREADS / kWave; ++i) r += lds[i];
    }
    return r;
}

// a2, first half: lane i of a kUpdThreads-lane block loads partials i, i + L,
// i + 2L, ... (L = kUpdThreads). Every load is issued (lanes past nparts
// re-read the last partial; final_reduce drops them), so that a caller can
// issue its own loads behind these and still wait for these alone.
__device__ __forceinline__ void load_partials(const double *__restrict__ partials, int nparts,
                                              double (&x)[kPartsPerLane]) {
#pragma unroll
    for (int k = 0; k < kPartsPerLane; ++k) {
        const int j = (int)threadIdx.x + k * kUpdThreads;
        x[k] = partials[j < nparts ? j : nparts - 1];
    }
}

// a2, second half: each lane sums its partials in index order (0 beyond
// nparts), the block sums the lanes in the fixed wave/LDS tree, then the
// float64 square root and the clip factor. The result is valid in every lane.
__device__ __forceinline__ ClipScalars final_reduce(const double (&x)[kPartsPerLane], int nparts,
                                                    float clip, double *lds) {
    double acc = 0.0;
#pragma unroll
    for (int k = 0; k < kPartsPerLane; ++k)
        acc += ((int)threadIdx.x + k * kUpdThreads < nparts) ? x[k] : 0.0;
    double S;
    if constexpr (kUpdThreads == kWave) {
        S = wave_sum(acc);  // the same bits in every lane
    } else {
        const double b = block_sum<kUpdThreads>(acc, lds);
        if (threadIdx.x == 0) lds[0] = b;  // block_sum's reads of lds are done by now
        __syncthreads();
        S = lds[0];
    }
    ClipScalars r;
    r.norm = sqrt(S);
    r.apply = isfinite(r.norm) ? 1 : 0;
    r.scale = (r.norm > (double)clip) ? (float)((double)clip / r.norm) : 1.0f;
    return r;
}

template <typename T>
__device__ __forceinline__ T ld_stream(const T *p) {
    return __builtin_nontemporal_load(p);
}

template <typename T>
__device__ __forceinline__ void st_stream(T *p, T x) {
    __builtin_nontemporal_store(x, p);
}

}  // namespace

#endif
