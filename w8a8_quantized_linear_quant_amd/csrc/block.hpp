// block.hpp -- helpers of the kernels beside the 8-bit linear: element types,
// wave and workgroup reductions.
#pragma once

#include "../../include/w8a8_block.h"
#include "common.hpp"

namespace w8a8 {

inline bool valid_dtype(w8a8_dtype t) { return t == W8A8_BF16 || t == W8A8_F32; }

// 16-byte accesses at the alignment of one element: rows of any stride take
// the same full-width instructions (global memory allows unaligned ones).
typedef v4u v4u_at2 __attribute__((aligned(2)));
typedef v4u v4u_at4 __attribute__((aligned(4)));

// An element type and its 16-byte chunks of kVec elements.
struct Bf16 {
    typedef uint16_t type;
    static constexpr int kVec = 8;
    static __device__ __forceinline__ float load(const uint16_t *p) { return bf16_bits_to_f32(*p); }
    // the hardware conversion: nearest even, infinities and NaN kept
    static __device__ __forceinline__ void store(uint16_t *p, float v) { *p = __builtin_bit_cast(uint16_t, (__bf16)v); }
    static __device__ __forceinline__ v4u load_chunk(const uint16_t *p) { return *reinterpret_cast<const v4u_at2 *>(p); }
    static __device__ __forceinline__ void store_chunk(uint16_t *p, v4u d) { *reinterpret_cast<v4u_at2 *>(p) = d; }
    // elements 0 .. n - 1 of a chunk, the others 0
    static __device__ __forceinline__ v4u load_part(const uint16_t *p, int n) {
        v4u d = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int e = 0; e < kVec; ++e)
            if (e < n) d[e / 2] |= (uint32_t)p[e] << (16 * (e & 1));
        return d;
    }
    static __device__ __forceinline__ void unpack(v4u d, float *v) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            v[2 * w] = __uint_as_float(d[w] << 16);
            v[2 * w + 1] = __uint_as_float(d[w] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ v4u pack(const float *v) {
        return v4u{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
    }
};
struct F32 {
    typedef float type;
    static constexpr int kVec = 4;
    static __device__ __forceinline__ float load(const float *p) { return *p; }
    static __device__ __forceinline__ void store(float *p, float v) { *p = v; }
    static __device__ __forceinline__ v4u load_chunk(const float *p) { return *reinterpret_cast<const v4u_at4 *>(p); }
    static __device__ __forceinline__ void store_chunk(float *p, v4u d) { *reinterpret_cast<v4u_at4 *>(p) = d; }
    static __device__ __forceinline__ v4u load_part(const float *p, int n) {
        v4u d = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int e = 0; e < kVec; ++e)
            if (e < n) d[e] = __float_as_uint(p[e]);
        return d;
    }
    static __device__ __forceinline__ void unpack(v4u d, float *v) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(d[e]);
    }
    static __device__ __forceinline__ v4u pack(const float *v) {
        return v4u{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
    }
};

// The chunk of X::kVec elements at column `col` of a row of K, as floats;
// elements past K are 0.
template <class X>
__device__ __forceinline__ v4u load_row_chunk(const typename X::type *row, int col, int K) {
    if (col + X::kVec <= K) return X::load_chunk(row + col);
    return X::load_part(row + col, K - col);
}
template <class X>
__device__ __forceinline__ void store_row_chunk(typename X::type *row, int col, int K, const float *v) {
    if (col + X::kVec <= K) {
        X::store_chunk(row + col, X::pack(v));
    } else {
#pragma unroll
        for (int e = 0; e < X::kVec; ++e)
            if (col + e < K) X::store(row + col + e, v[e]);
    }
}

// Element k of a weight vector of type wt; `none` where there is no vector.
__device__ __forceinline__ float load_param(const void *p, int wt, int64_t k, float none) {
    if (!p) return none;
    return wt == W8A8_BF16 ? bf16_bits_to_f32(static_cast<const uint16_t *>(p)[k]) : static_cast<const float *>(p)[k];
}

// Sum and maximum over the 64 lanes, the same value in every lane: DPP row
// shifts gather each 16-lane row in its lane 15, four lane reads join the rows.
__device__ __forceinline__ float dpp_shr(float v, float none, int by) {
    const int o = __float_as_int(none), s = __float_as_int(v);
    switch (by) {  // row_shr:by (dpp ctrl 0x110 + by); lanes shifted in from outside the row read `none`
    case 1: return __int_as_float(__builtin_amdgcn_update_dpp(o, s, 0x111, 0xF, 0xF, false));
    case 2: return __int_as_float(__builtin_amdgcn_update_dpp(o, s, 0x112, 0xF, 0xF, false));
    case 4: return __int_as_float(__builtin_amdgcn_update_dpp(o, s, 0x114, 0xF, 0xF, false));
    default: return __int_as_float(__builtin_amdgcn_update_dpp(o, s, 0x118, 0xF, 0xF, false));
    }
}
__device__ __forceinline__ float lane_value(float v, int lane) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 1; d < 16; d *= 2) v += dpp_shr(v, 0.f, d);
    return (lane_value(v, 15) + lane_value(v, 31)) + (lane_value(v, 47) + lane_value(v, 63));
}
// The greater of two values, NaN if either is (fmaxf would drop it): one
// instruction, as fmaxf is.
__device__ __forceinline__ float max_or_nan(float a, float b) { return __builtin_elementwise_maximum(a, b); }
__device__ __forceinline__ float wave_max(float v) {  // of values >= 0 or NaN
#pragma unroll
    for (int d = 1; d < 16; d *= 2) v = max_or_nan(v, dpp_shr(v, 0.f, d));
    return max_or_nan(max_or_nan(lane_value(v, 15), lane_value(v, 31)), max_or_nan(lane_value(v, 47), lane_value(v, 63)));
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
    for (int w = 1; w < WAVES; ++w) s = max_or_nan(s, part[w]);
    return s;
}

}  // namespace w8a8
