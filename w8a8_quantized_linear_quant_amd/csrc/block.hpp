// block.hpp -- helpers of the kernels beside the 8-bit linear: element types,
// wave and workgroup reductions.
#pragma once

#include "../../include/w8a8_block.h"
#include "common.hpp"

namespace w8a8 {

inline bool valid_dtype(w8a8_dtype t) { return t == W8A8_BF16 || t == W8A8_F32; }

struct Bf16 {
    typedef uint16_t type;
    static __device__ __forceinline__ float load(const uint16_t *p) { return bf16_bits_to_f32(*p); }
    // the hardware conversion: nearest even, infinities and NaN kept
    static __device__ __forceinline__ void store(uint16_t *p, float v) { *p = __builtin_bit_cast(uint16_t, (__bf16)v); }
};
struct F32 {
    typedef float type;
    static __device__ __forceinline__ float load(const float *p) { return *p; }
    static __device__ __forceinline__ void store(float *p, float v) { *p = v; }
};

// Element k of a weight vector of type wt; `none` where there is no vector.
__device__ __forceinline__ float load_param(const void *p, int wt, int64_t k, float none) {
    if (!p) return none;
    return wt == W8A8_BF16 ? bf16_bits_to_f32(static_cast<const uint16_t *>(p)[k]) : static_cast<const float *>(p)[k];
}

// Sum over the 64 lanes, the same value in every lane.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
    return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) v = fmaxf(v, __shfl_xor(v, d));
    return v;
}

// Sum over a workgroup of WAVES waves, the same value in every thread; `part`
// holds WAVES floats and may be used again after the next barrier.
template <int WAVES>
__device__ __forceinline__ float group_sum(float v, float *part) {
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = part[0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) s += part[w];
    return s;
}
template <int WAVES>
__device__ __forceinline__ float group_max(float v, float *part) {
    v = wave_max(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = part[0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) s = fmaxf(s, part[w]);
    return s;
}

}  // namespace w8a8
