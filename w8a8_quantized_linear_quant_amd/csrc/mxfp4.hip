// mxfp4.hip -- quantizers and dequantizer of the microscaled 4-bit format.
//
// A block of 32 values along a row shares the scale 2^e, one byte e + 127; a
// value is an E2M1 code, two a byte (OCP Microscaling Formats v1.0, MXFP4).
// The scale needs no floating-point logarithm: with the absmax's bits b,
// floor(log2) + 127 is its exponent field b >> 23, so the byte is
// max((b >> 23) - 2, 0), and 255 exactly where the block holds an infinity or
// a NaN (their bits are the largest as integers too).  x / 2^e is exact in f32
// (v_ldexp_f32) and the hardware conversion rounds it to nearest even.
//
// All three are bound by memory (and below ~1 MB by the launch).  5120 x 4096 in
// bf16 and f32, twelve sets of operands in turn, that is from HBM: quantizer
// 12.1 and 19.9 us (4.4 and 4.8 TB/s), transposed 14.2 and 22.3, dequantizer
// 11.8 and 22.8; three sets, partly from the Infinity Cache: 10.4 and 16.7,
// 11.5 and 19.2, 10.3 and 21.8.  One pass, 16-byte loads, a unit of 512 columns
// a wave, so that a row's scales leave as 16 bytes a unit.
#include "../../include/w8a8_experts.h"
#include "block.hpp"
#include "internal.hpp"

namespace w8a8 {
namespace {

constexpr int kThreads = 256;
constexpr int kUnit = 512;      // columns of a row that a wave takes at a time: 16 scale bytes
// units in flight a wave (5120 x 4096 from HBM, bf16: quantizer 12.7 us with 1, 12.3 with 2, 12.1 with 4, 13.8 with 8;
// dequantizer 14.0, 13.3, 13.1, 11.8; f32: 18.2, 18.5, 19.9, 21.3; 23.9, 26.0, 25.5, 22.8)
constexpr int kQuantizeUnits = 4, kDequantizeUnits = 8;
constexpr int kPadByte = 127;   // padding of a row's scales: the scale 1

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// The scale byte of a block from its absmax's bits.
__device__ __forceinline__ int scale_byte(uint32_t amax) {
    const int exponent = (int)(amax >> 23);
    return exponent == 255 ? 255 : max(exponent - 2, 0);
}

// 8 values as 8 codes with the block's scale byte; codes 0 beside a NaN scale.
__device__ __forceinline__ uint32_t codes_of(const float *v, int byte) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __builtin_amdgcn_fmed3f(__builtin_ldexpf(v[i], 127 - byte), -6.0f, 6.0f);
    uint32_t r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, y[0], y[1], 1.0f, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, y[2], y[3], 1.0f, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, y[4], y[5], 1.0f, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, y[6], y[7], 1.0f, 3);
    return byte == 255 ? 0u : r;
}

// 8 consecutive elements of a row as floats, those past K as 0.
template <class X>
struct Eight {
    v4u d[8 / X::kVec];
    __device__ __forceinline__ void load(const typename X::type *row, int col, int K) {
#pragma unroll
        for (int i = 0; i < 8 / X::kVec; ++i) {
            if (col + i * X::kVec < K) d[i] = load_row_chunk<X>(row, col + i * X::kVec, K);
            else d[i] = v4u{0u, 0u, 0u, 0u};
        }
    }
    __device__ __forceinline__ void unpack(float *v) const {
#pragma unroll
        for (int i = 0; i < 8 / X::kVec; ++i) X::unpack(d[i], v + i * X::kVec);
    }
};

// Units of a row: whole ones cover the padded scales too.
__host__ __device__ inline int64_t units_of(int64_t ldq) { return (ldq + kUnit - 1) / kUnit; }

// A wave takes kQuantizeUnits consecutive units, their loads all in flight
// before the first is converted.  Lane l holds columns 8 l .. 8 l + 7 of a
// unit; the four lanes of a block share its absmax.
template <class X>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const typename X::type *x, int64_t units, int per_row, int K,
                                                            int64_t ldx, uint8_t *xq, int ldq, uint8_t *xs) {
    const int lane = threadIdx.x & 63;
    const int64_t wave = (int64_t)blockIdx.x * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t first = wave * kQuantizeUnits;
    if (first >= units) return;
    int64_t row = first / per_row;
    int unit = (int)(first - row * per_row);
    Eight<X> in[kQuantizeUnits];
    {
        int64_t r = row;
        int u = unit;
#pragma unroll
        for (int i = 0; i < kQuantizeUnits; ++i) {
            if (first + i < units) in[i].load(x + r * ldx, u * kUnit + lane * 8, K);
            if (++u == per_row) {
                u = 0;
                ++r;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kQuantizeUnits; ++i) {
        if (first + i >= units) return;
        float v[8];
        in[i].unpack(v);
        uint32_t amax = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = max(amax, abs_bits(v[e]));
        // quad_perm [1,0,3,2], then [2,3,0,1]: the greatest of the block's four lanes
        amax = max(amax, (uint32_t)__builtin_amdgcn_mov_dpp((int)amax, 0xB1, 0xF, 0xF, true));
        amax = max(amax, (uint32_t)__builtin_amdgcn_mov_dpp((int)amax, 0x4E, 0xF, 0xF, true));
        const int col = unit * kUnit + lane * 8;
        const int byte = scale_byte(amax);
        if (col < ldq) *reinterpret_cast<uint32_t *>(xq + row * (ldq / 2) + col / 2) = codes_of(v, byte);
        if ((lane & 3) == 0) xs[(row * per_row + unit) * 16 + lane / 4] = (uint8_t)(col < ldq ? byte : kPadByte);
        if (++unit == per_row) {
            unit = 0;
            ++row;
        }
    }
}

// Transposed: a workgroup takes kTileN rows of w (columns of the result: 8
// blocks) by kTileK columns (rows of the result), loads them row by row, turns
// them in LDS, converts, and writes the results' rows 128 bytes at a time.
constexpr int kTileN = 256, kTileK = 64;

template <class X>
__global__ __launch_bounds__(kThreads) void quantize_transposed_kernel(const typename X::type *w, int N, int K,
                                                                       int64_t ldx, uint8_t *wq, int ldq, uint8_t *ws,
                                                                       int tiles_n, int tiles_k) {
    typedef typename X::type T;
    // words XOR-swizzled by row, so that a write to several rows meets every bank, as a read of 64 columns of one row
    // does by itself; no padding: bf16 takes 32 KB, five
    // workgroups a CU (5120 x 4096, three sets of operands: 11.5 us; three with padding and the results beside the tile,
    // 12.4)
    constexpr int kWord = 4 / sizeof(T);             // elements of a word
    constexpr int kPitch = kTileK / kWord;           // words of a row
    auto turn = [](int row) { return (row / kWord) & 3; };
    __shared__ __attribute__((aligned(16))) uint32_t tile[kTileN * kPitch];
    const int64_t b = blockIdx.y;
    const int tk = blockIdx.x % tiles_k, tn = blockIdx.x / tiles_k;
    const int n0 = tn * kTileN, k0 = tk * kTileK;
    const T *src = w + b * (int64_t)N * ldx;
    constexpr int kLanes = kTileK / X::kVec;         // lanes along a row
    constexpr int kRows = kThreads / kLanes;         // rows a step
    const int c = threadIdx.x % kLanes * X::kVec, r0 = threadIdx.x / kLanes;
    v4u d[kTileN / kRows];
#pragma unroll
    for (int i = 0; i < kTileN / kRows; ++i) {
        const int n = n0 + i * kRows + r0;
        d[i] = v4u{0u, 0u, 0u, 0u};
        if (n < N && k0 + c < K) d[i] = load_row_chunk<X>(src + n * ldx, k0 + c, K);
    }
#pragma unroll
    for (int i = 0; i < kTileN / kRows; ++i) {
        const int row = i * kRows + r0;
#pragma unroll
        for (int e = 0; e < 4; ++e) tile[row * kPitch + c / kWord + (e ^ turn(row))] = d[i][e];
    }
    __syncthreads();
    // One block of one result row a thread and step; its codes and scale back to LDS, so that they leave along rows:
    // in the tile's place.
    v4u *codes = reinterpret_cast<v4u *>(tile);  // [row][chunk, XOR-swizzled by row]
    uint8_t *scales = reinterpret_cast<uint8_t *>(codes + kTileK * 8);
    static_assert(sizeof(tile) >= kTileK * 8 * 17, "results in the tile's place");
    const int k = threadIdx.x % kTileK;
    v4u out[2];
    int byte[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int nb = threadIdx.x / kTileK + 4 * i;  // block of the tile
        float v[32];
        uint32_t amax = 0;
#pragma unroll
        for (int e = 0; e < 32; ++e) {
            v[e] = X::load(reinterpret_cast<const T *>(tile + (nb * 32 + e) * kPitch) + (k ^ (turn(e) * kWord)));
            amax = max(amax, abs_bits(v[e]));
        }
        byte[i] = scale_byte(amax);
#pragma unroll
        for (int e = 0; e < 4; ++e) out[i][e] = codes_of(v + 8 * e, byte[i]);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int nb = threadIdx.x / kTileK + 4 * i;
        codes[k * 8 + (nb ^ (k & 7))] = out[i];
        scales[k * 8 + nb] = (uint8_t)(n0 + nb * 32 < ldq ? byte[i] : kPadByte);
    }
    __syncthreads();
    const int stride = (int)units_of(ldq) * 16;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = threadIdx.x / 8 + 32 * i, nb = threadIdx.x & 7;
        if (k0 + r < K && n0 + nb * 32 < ldq)
            *reinterpret_cast<v4u *>(wq + (b * K + k0 + r) * (int64_t)(ldq / 2) + n0 / 2 + nb * 16) = codes[r * 8 + (nb ^ (r & 7))];
    }
    if (threadIdx.x < kTileK && k0 + (int)threadIdx.x < K)
        *reinterpret_cast<uint2 *>(ws + (b * K + k0 + threadIdx.x) * (int64_t)stride + n0 / 32) =
            *reinterpret_cast<const uint2 *>(scales + threadIdx.x * 8);
}

// 8 codes a lane and step, as quantize_kernel.
template <class Y>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(const uint8_t *xq, const uint8_t *xs, int64_t units,
                                                              int per_row, int K, int ldq, typename Y::type *y,
                                                              int64_t ldy) {
    const int lane = threadIdx.x & 63;
    const int64_t wave = (int64_t)blockIdx.x * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t first = wave * kDequantizeUnits;
    if (first >= units) return;
    int64_t row = first / per_row;
    int unit = (int)(first - row * per_row);
    uint32_t codes[kDequantizeUnits];
    int bytes[kDequantizeUnits];
    {
        int64_t r = row;
        int u = unit;
#pragma unroll
        for (int i = 0; i < kDequantizeUnits; ++i) {
            const int col = u * kUnit + lane * 8;
            codes[i] = 0;
            bytes[i] = 0;
            if (first + i < units && col < K) {
                codes[i] = *reinterpret_cast<const uint32_t *>(xq + r * (ldq / 2) + col / 2);
                bytes[i] = xs[(r * per_row + u) * 16 + lane / 4];
            }
            if (++u == per_row) {
                u = 0;
                ++r;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kDequantizeUnits; ++i) {
        if (first + i >= units) return;
        const int col = unit * kUnit + lane * 8;
        if (col < K) {
            typedef float v2f __attribute__((ext_vector_type(2)));
            const v2f p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes[i], 1.0f, 0),
                              __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes[i], 1.0f, 1),
                              __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes[i], 1.0f, 2),
                              __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes[i], 1.0f, 3)};
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = bytes[i] == 255 ? __builtin_nanf("") : __builtin_ldexpf(p[e / 2][e & 1], bytes[i] - 127);
#pragma unroll
            for (int e = 0; e < 8; e += Y::kVec)
                if (col + e < K) store_row_chunk<Y>(y + row * ldy, col + e, K, v + e);
        }
        if (++unit == per_row) {
            unit = 0;
            ++row;
        }
    }
}

w8a8_status check_rows(int64_t M, int64_t K, int64_t ldx, int64_t ldq) {
    if (M < 0) return W8A8_ERR_INVALID_ARG;
    if (M > (1 << 30) || K < 1 || K > (1 << 22) || ldx < K || ldx > (1 << 24)) return W8A8_ERR_SHAPE;
    if (ldq < K || ldq > (1 << 22) || ldq % 32 != 0) return W8A8_ERR_SHAPE;
    // one launch: units / 16 workgroups of 256 threads, below 2^32 threads
    if (M * units_of(ldq) > ((int64_t)1 << 27)) return W8A8_ERR_SHAPE;
    return W8A8_OK;
}

unsigned unit_blocks(int64_t units, int a_wave) {
    const int a_block = kThreads / 64 * a_wave;
    return (unsigned)((units + a_block - 1) / a_block);
}

}  // namespace
}  // namespace w8a8

extern "C" int64_t mxfp4_scale_stride(int64_t ldq) { return ldq <= 0 ? 0 : w8a8::units_of(ldq) * 16; }

extern "C" w8a8_status mxfp4_quantize(w8a8_dtype xt, const void *x, int64_t M, int64_t K, int64_t ldx, uint8_t *xq,
                                      int64_t ldq, uint8_t *xs, hipStream_t stream) {
    using namespace w8a8;
    if (!valid_dtype(xt)) return W8A8_ERR_INVALID_ARG;
    const w8a8_status st = check_rows(M, K, ldx, ldq);
    if (st != W8A8_OK) return st;
    if (M == 0) return W8A8_OK;
    if (!x || !xq || !xs) return W8A8_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(xq) || !aligned16(xs)) return W8A8_ERR_ALIGN;
    const int per_row = (int)units_of(ldq);
    const int64_t units = M * per_row;
    if (xt == W8A8_BF16)
        quantize_kernel<Bf16><<<unit_blocks(units, kQuantizeUnits), kThreads, 0, stream>>>(static_cast<const uint16_t *>(x), units,
                                                                           per_row, (int)K, ldx, xq, (int)ldq, xs);
    else
        quantize_kernel<F32><<<unit_blocks(units, kQuantizeUnits), kThreads, 0, stream>>>(static_cast<const float *>(x), units, per_row,
                                                                          (int)K, ldx, xq, (int)ldq, xs);
    return launch_status();
}

extern "C" w8a8_status mxfp4_quantize_transposed(w8a8_dtype xt, const void *w, int64_t B, int64_t N, int64_t K,
                                                 int64_t ldx, uint8_t *wq, int64_t ldq, uint8_t *ws,
                                                 hipStream_t stream) {
    using namespace w8a8;
    if (!valid_dtype(xt) || B < 0) return W8A8_ERR_INVALID_ARG;
    if (B > 65535 || N < 1 || N > (1 << 22) || K < 1 || K > (1 << 22) || ldx < K || ldx > (1 << 24))
        return W8A8_ERR_SHAPE;
    if (ldq < N || ldq > (1 << 22) || ldq % 32 != 0) return W8A8_ERR_SHAPE;
    if (B == 0) return W8A8_OK;
    if (N * ldx > ((int64_t)1 << 40) / B) return W8A8_ERR_SHAPE;
    // the tiles that hold the padding of the scales too
    const int64_t tiles_n = units_of(ldq) * (kUnit / kTileN), tiles_k = (K + kTileK - 1) / kTileK;
    if (tiles_n * tiles_k * B >= ((int64_t)1 << 24)) return W8A8_ERR_SHAPE;  // 2^32 threads
    if (!w || !wq || !ws) return W8A8_ERR_INVALID_ARG;
    if (!aligned16(w) || !aligned16(wq) || !aligned16(ws)) return W8A8_ERR_ALIGN;
    const dim3 grid((unsigned)(tiles_n * tiles_k), (unsigned)B);
    if (xt == W8A8_BF16)
        quantize_transposed_kernel<Bf16><<<grid, kThreads, 0, stream>>>(static_cast<const uint16_t *>(w), (int)N,
                                                                        (int)K, ldx, wq, (int)ldq, ws, (int)tiles_n,
                                                                        (int)tiles_k);
    else
        quantize_transposed_kernel<F32><<<grid, kThreads, 0, stream>>>(static_cast<const float *>(w), (int)N, (int)K,
                                                                       ldx, wq, (int)ldq, ws, (int)tiles_n,
                                                                       (int)tiles_k);
    return launch_status();
}

extern "C" w8a8_status mxfp4_dequantize(const uint8_t *xq, const uint8_t *xs, int64_t M, int64_t K, int64_t ldq,
                                        w8a8_dtype yt, void *y, int64_t ldy, hipStream_t stream) {
    using namespace w8a8;
    if (!valid_dtype(yt)) return W8A8_ERR_INVALID_ARG;
    const w8a8_status st = check_rows(M, K, ldy, ldq);
    if (st != W8A8_OK) return st;
    if (M == 0) return W8A8_OK;
    if (!xq || !xs || !y) return W8A8_ERR_INVALID_ARG;
    if (!aligned16(xq) || !aligned16(xs) || !aligned16(y)) return W8A8_ERR_ALIGN;
    const int per_row = (int)units_of(ldq);
    const int64_t units = M * per_row;
    if (yt == W8A8_BF16)
        dequantize_kernel<Bf16><<<unit_blocks(units, kDequantizeUnits), kThreads, 0, stream>>>(
            xq, xs, units, per_row, (int)K, (int)ldq, static_cast<uint16_t *>(y), ldy);
    else
        dequantize_kernel<F32><<<unit_blocks(units, kDequantizeUnits), kThreads, 0, stream>>>(xq, xs, units, per_row, (int)K, (int)ldq,
                                                                            static_cast<float *>(y), ldy);
    return launch_status();
}
