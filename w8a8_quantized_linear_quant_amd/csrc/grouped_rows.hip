// grouped_rows.hip -- products of groups with few rows each: every weight is
// read once and multiplied by 16 to 64 rows, so the weights' bytes are the
// bound.
//
// A workgroup takes 16 MB rows of one group by 16 NB columns; its four waves
// split K between them, 128 bytes of every row at a time in turn, and add
// their sums up in LDS.  Operands go from memory straight to the matrix
// instructions' registers: a weight is used once in a workgroup, staging it
// would only cost.  Lane l reads row l & 15 of a 16-row block, bytes
// 32 (l >> 4) .. + 31 of the 128: which k a lane holds is free as long as both
// operands agree, so a row's 128-byte line is read whole by four lanes.  In the
// 4-bit format those 32 bytes are blocks 2 (l >> 4) and + 1: one 16-bit load
// holds both scales, and the instruction's operand selector takes the byte.
#include <type_traits>

#include "grouped.hpp"

namespace w8a8 {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kChunk = 128;  // bytes of a row a wave multiplies at a time

__device__ __forceinline__ v4u buffer_load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
}
__device__ __forceinline__ int buffer_load2(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, (int)off, 0, 0);
}

template <int QT, int MB, int NB, int DEPTH>
__global__ __launch_bounds__(kThreads) void grouped_rows_kernel(GroupedArgs p, int tiles_n, int columns) {
    constexpr bool kMx = QT == kTypeMx4;
    typedef typename std::conditional<QT == kTypeInt8, v4i, v4f>::type acc_t;
    __shared__ acc_t part[kWaves][MB * NB][64];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // `columns` is tiles_n rounded up to a multiple of 8: the row tiles of one
    // column tile, which read the same weights, run on the same XCD
    const int tm = blockIdx.x / columns, tn = blockIdx.x - tm * columns;
    if (tn >= tiles_n) return;
    GroupWindow w = {};
    load_window<16 * MB>(w, p.offsets, p.E, p.M, lane);
    const GroupTile t = find_tile<16 * MB>(w, tm, p.offsets, p.E, p.M, lane);
    if (t.group < 0) return;
    const int n0 = tn * 16 * NB;
    const int rows_w = min(p.N - n0, 16 * NB);
    const size_t w0 = (size_t)t.group * p.N + n0;
    const int kb = p.kb;

    // Operand descriptors: rows past the end and row indices outside x lie past num_records and read as 0.
    const __amdgpu_buffer_rsrc_t rw =
        __builtin_amdgcn_make_buffer_rsrc((void *)(p.wq + w0 * kb), (short)0, rows_w * kb, kBufferRsrcWord3);
    const bool gather = p.rows != nullptr;
    const int rows_x = gather ? (int)p.X : min(t.end - t.m0, 16 * MB);
    const size_t x0 = gather ? 0 : t.m0;
    const __amdgpu_buffer_rsrc_t rx =
        __builtin_amdgcn_make_buffer_rsrc((void *)(p.xq + x0 * kb), (short)0, (int)(rows_x * (int64_t)kb), kBufferRsrcWord3);
    __amdgpu_buffer_rsrc_t rws, rxs;
    if constexpr (kMx) {
        rws = __builtin_amdgcn_make_buffer_rsrc((void *)(p.ws + w0 * p.stride), (short)0, rows_w * p.stride,
                                                kBufferRsrcWord3);
        rxs = __builtin_amdgcn_make_buffer_rsrc((void *)(p.xs + x0 * p.stride), (short)0,
                                                (int)(rows_x * (int64_t)p.stride), kBufferRsrcWord3);
    }
    const int r = lane & 15, q = lane >> 4;
    int xrow[MB];  // the lane's rows of x, relative to the descriptor; -1: none
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
        const int m = t.m0 + mb * 16 + r;
        xrow[mb] = -1;
        if (m < t.end) {
            const int s = gather ? p.rows[m] : m - t.m0;
            if (s >= 0 && s < rows_x) xrow[mb] = s;
        }
    }
    uint32_t woff[NB], xoff[MB], wsoff[kMx ? NB : 1], xsoff[kMx ? MB : 1];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        woff[nb] = (uint32_t)(nb * 16 + r) * kb + q * 32;
        if constexpr (kMx) wsoff[nb] = (uint32_t)(nb * 16 + r) * p.stride + q * 2;
    }
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
        xoff[mb] = (uint32_t)xrow[mb] * kb + q * 32;
        if constexpr (kMx) xsoff[mb] = (uint32_t)xrow[mb] * p.stride + q * 2;
    }

    struct Chunk {
        v4u w[NB][2], x[MB][2];
        int ws[kMx ? NB : 1], xs[kMx ? MB : 1];
    } ring[DEPTH];
    const int chunks = (kb + kChunk - 1) / kChunk;
    // (K travels in the lane's offset: a scalar offset past num_records would
    // wrap the range check)
    auto load = [&](Chunk &c, int chunk) {
        const int k = chunk * kChunk;
        const int left = kb - k - q * 32;  // bytes of the row from the lane's first on
        constexpr uint32_t kOut = (uint32_t)kOobOffset;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const bool in = left > h * 16;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) c.w[nb][h] = buffer_load16(rw, in ? woff[nb] + k + h * 16 : kOut);
#pragma unroll
            for (int mb = 0; mb < MB; ++mb)
                c.x[mb][h] = buffer_load16(rx, in && xrow[mb] >= 0 ? xoff[mb] + k + h * 16 : kOut);
        }
        if constexpr (kMx) {
            // scale bytes past the row's blocks count as 1 (their codes are 0, but 0 times NaN is not)
            const int keep = left > 16 ? 0xFFFF : left > 0 ? 0xFF : 0;
            const int one = 0x7F7F & ~keep;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
                c.ws[nb] = (buffer_load2(rws, left > 0 ? wsoff[nb] + k / 16 : kOut) & keep) | one;
#pragma unroll
            for (int mb = 0; mb < MB; ++mb)
                c.xs[mb] = (buffer_load2(rxs, left > 0 && xrow[mb] >= 0 ? xsoff[mb] + k / 16 : kOut) & keep) | one;
        }
    };
    acc_t acc[MB][NB];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = acc_t{};
    auto multiply = [&](const Chunk &c) {
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const v4u *a = c.w[nb], *b = c.x[mb];
                if constexpr (QT == kTypeInt8) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        acc[mb][nb] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(v4i, a[h]),
                                                                            __builtin_bit_cast(v4i, b[h]), acc[mb][nb], 0, 0, 0);
                } else if constexpr (QT == kTypeE4m3) {
                    const v8i va = {(int)a[0][0], (int)a[0][1], (int)a[0][2], (int)a[0][3],
                                    (int)a[1][0], (int)a[1][1], (int)a[1][2], (int)a[1][3]};
                    const v8i vb = {(int)b[0][0], (int)b[0][1], (int)b[0][2], (int)b[0][3],
                                    (int)b[1][0], (int)b[1][1], (int)b[1][2], (int)b[1][3]};
                    acc[mb][nb] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(va, vb, acc[mb][nb], 0, 0, 0, 127, 0, 127);
                } else {
                    const v8i a0 = {(int)a[0][0], (int)a[0][1], (int)a[0][2], (int)a[0][3], 0, 0, 0, 0};
                    const v8i b0 = {(int)b[0][0], (int)b[0][1], (int)b[0][2], (int)b[0][3], 0, 0, 0, 0};
                    const v8i a1 = {(int)a[1][0], (int)a[1][1], (int)a[1][2], (int)a[1][3], 0, 0, 0, 0};
                    const v8i b1 = {(int)b[1][0], (int)b[1][1], (int)b[1][2], (int)b[1][3], 0, 0, 0, 0};
                    acc[mb][nb] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a0, b0, acc[mb][nb], 4, 4, 0, c.ws[nb], 0, c.xs[mb]);
                    acc[mb][nb] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a1, b1, acc[mb][nb], 4, 4, 1, c.ws[nb], 1, c.xs[mb]);
                }
            }
    };

    // Wave w takes chunks w, w + 4, ...; the ring holds the next DEPTH of them.
    // Past the end every offset is out of range: zeros.
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) load(ring[d], wave + d * kWaves);
    for (int c = wave; c < chunks; c += DEPTH * kWaves) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            multiply(ring[d]);
            load(ring[d], c + (d + DEPTH) * kWaves);
        }
    }

    // The waves' sums: wave w adds up blocks w, w + 4, ...
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) part[wave][mb * NB + nb][lane] = acc[mb][nb];
    __syncthreads();
#pragma unroll
    for (int b = 0; b < MB * NB; ++b) {
        if ((b & (kWaves - 1)) != wave) continue;
        const int mb = b / NB, nb = b % NB;
        acc_t s = part[0][b][lane];
#pragma unroll
        for (int i = 1; i < kWaves; ++i) s += part[i][b][lane];
        // lane l: row l & 15 of the block, columns 4 (l >> 4) .. + 3
        const int m = t.m0 + mb * 16 + r, n = n0 + nb * 16 + q * 4;
        if (m >= t.end || n >= p.N) continue;
        float tm = 1.0f;
        if constexpr (!kMx) {
            tm = xrow[mb] < 0 ? 0.0f : p.sx[x0 + xrow[mb]];
            if (!p.per_channel) tm *= p.sw[t.group];
        }
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (n + i >= p.N) {
                y[i] = 0.0f;
                continue;
            }
            const size_t at = (size_t)t.group * p.N + n + i;
            const float bias = p.bias ? bf16_bits_to_f32(p.bias[at]) : 0.0f;
            if constexpr (kMx) y[i] = s[i] + bias;
            else y[i] = __builtin_fmaf((float)s[i], p.per_channel ? tm * p.sw[at] : tm, bias);
        }
        uint16_t *dst = p.out + (size_t)m * p.N + n;
        if ((p.N & 3) == 0) {
            *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n + i < p.N) Bf16::store(dst + i, y[i]);
        }
    }
}

template <int QT, int MB, int NB, int DEPTH>
void launch(const GroupedArgs &a, hipStream_t stream) {
    const int64_t rows = 16 * MB;
    const int tiles_n = (a.N + 16 * NB - 1) / (16 * NB);
    const int columns = (tiles_n + 7) / 8 * 8;
    // every group may leave one tile partly filled
    const int64_t tiles_m = a.M / rows + (a.E < a.M ? a.E : a.M);
    grouped_rows_kernel<QT, MB, NB, DEPTH><<<(unsigned)(tiles_m * columns), kThreads, 0, stream>>>(a, tiles_n, columns);
}

}  // namespace

template <int QT>
void launch_grouped_rows(const GroupedArgs &a, hipStream_t stream) {
    const int64_t mean = (a.M + a.E - 1) / a.E;
    if (mean <= 16) launch<QT, 1, 1, 4>(a, stream);
    else if (mean <= 32) launch<QT, 2, 2, 3>(a, stream);
    else launch<QT, 4, 4, 2>(a, stream);
}
template void launch_grouped_rows<kTypeInt8>(const GroupedArgs &, hipStream_t);
template void launch_grouped_rows<kTypeE4m3>(const GroupedArgs &, hipStream_t);
template void launch_grouped_rows<kTypeMx4>(const GroupedArgs &, hipStream_t);

}  // namespace w8a8
