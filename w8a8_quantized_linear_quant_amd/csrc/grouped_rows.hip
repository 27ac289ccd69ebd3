// grouped_rows.hip -- products of groups with few rows each: every weight is
// read once and multiplied by 16 to 64 rows, so the weights' bytes are the
// bound.
//
// A workgroup takes 16 MB rows of one group by 16 NB columns; its four waves
// split K between them, a unit of every row at a time in turn, and add their
// sums up in LDS.  A wave stages its own units in LDS, by loads that go there
// without registers, and waits for its own loads alone: no barrier until the
// sums.  The detour is for the loads' sake: as the product wants its operands,
// 16 rows in 16 lanes, each lane is a request of its own (about 85 cycles of a
// CU's address unit for 1 KB), where 8 lanes along a row's 128-byte line make
// one of it (16 cycles).  32 int8 experts of 2048 x 4096, 25 rows each: 61 us
// against 73 with operands loaded straight to registers; 4-bit 12288 x 4096, 32
// rows: 9.2 against 11.7.  With 8 e4m3 experts of 4096 x 4096 and 8 rows each (24.3
// us) the weights arrive at 5.5 TB/s.
//
// A unit is 128 bytes of every row, its 16-byte chunks XOR-swizzled by row; in
// the 4-bit format that is 256 values with 8 scale bytes, loaded as two words.
// Which k goes with which lane is free as long as both operands agree: in the
// 4-bit format lane (r, q) takes chunks 2 q and 2 q + 1, whose two scales are
// one 16-bit word; the product's operand selector takes the byte.
//
// e4m3: the matrix cores line eight neighbouring products up with the greatest
// of them and cut them off 13 bits below its leading bit, in this instruction
// and in the unscaled one of half the rate alike (both probed): the sums are
// f32 but for that, and there is no other product of e4m3 codes to choose.
#include <type_traits>
#include <utility>

#include "grouped.hpp"

namespace w8a8 {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kUnit = 128;  // bytes of a row that eight lanes load

typedef __attribute__((address_space(3))) void *lds_ptr_t;

__device__ __forceinline__ v8i codes4(v4i d) {  // the operand of 4-bit codes: 16 of its 32 bytes
    return v8i{d[0], d[1], d[2], d[3], 0, 0, 0, 0};
}
__device__ __forceinline__ int swizzle(int row) { return (row & 7) ^ ((row >> 3) & 1); }

template <int QT, int MB, int NB>
__global__ __launch_bounds__(kThreads) void grouped_rows_kernel(GroupedArgs p, int tiles_n, int columns) {
    constexpr bool kMx = QT == kTypeMx4;
    typedef typename std::conditional<QT == kTypeInt8, v4i, v4f>::type acc_t;
    constexpr int kRows = 16 * (MB + NB);             // x's, then the weight's
    constexpr int kCodeBytes = kRows * kUnit;
    constexpr int kXsLoads = kMx ? (MB + 1) / 2 : 0;  // scales of 32 rows a load
    constexpr int kWsLoads = kMx ? (NB + 1) / 2 : 0;
    constexpr int kSlotBytes = kCodeBytes + (kXsLoads + kWsLoads) * 256;
    constexpr int kPartBytes = kWaves * MB * NB * 64 * 16;
    // two units a wave; one array each, so that the compiler can tell the loads into one from the reads of the other
    __shared__ __attribute__((aligned(1024))) uint8_t slot0[kWaves * kSlotBytes];
    __shared__ __attribute__((aligned(1024))) uint8_t slot1[kWaves * kSlotBytes];
    static_assert(kPartBytes <= (int)sizeof(slot0), "the sums take the first units' place");

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
    const bool gather = p.rows != nullptr;
    const int rows_x = gather ? (int)p.X : min(t.end - t.m0, 16 * MB);
    const size_t x0 = gather ? 0 : t.m0;

    // Rows past the end, row indices outside x and chunks past K lie past num_records and read as 0.  (K travels in
    // the lane's offset: a scalar offset past num_records would wrap the range check.)
    constexpr uint32_t kOut = (uint32_t)kOobOffset;
    const __amdgpu_buffer_rsrc_t rw =
        __builtin_amdgcn_make_buffer_rsrc((void *)(p.wq + w0 * kb), (short)0, rows_w * kb, kBufferRsrcWord3);
    const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc((void *)(p.xq + x0 * kb), (short)0,
                                                                        (int)((int64_t)rows_x * kb), kBufferRsrcWord3);
    auto row_of_x = [&](int i) -> int {  // row i of the tile, relative to the descriptor; -1: none
        const int m = t.m0 + i;
        if (m >= t.end) return -1;
        const int s = gather ? p.rows[m] : i;
        return s >= 0 && s < rows_x ? s : -1;
    };
    // Lane l of load j brings row 8 j + l / 8, physical chunk l % 8 of a line; the weight's first.
    const int r8 = lane >> 3;
    uint32_t woff[2 * NB], xoff[2 * MB];
#pragma unroll
    for (int j = 0; j < 2 * NB; ++j)
        woff[j] = (uint32_t)(j * 8 + r8) * kb + (((lane & 7) ^ swizzle(j * 8 + r8)) << 4);
    const int col0 = ((lane & 7) ^ swizzle(r8)) << 4, col1 = ((lane & 7) ^ swizzle(8 + r8)) << 4;
    // 4-bit format: lane l of load j brings word l % 2 of the unit's scales of row 32 j + l / 2.
    uint32_t wsoff[kMx ? kWsLoads : 1], xsoff[kMx ? kXsLoads : 1];
    __amdgpu_buffer_rsrc_t rws, rxs;
    if constexpr (kMx) {
        rws = __builtin_amdgcn_make_buffer_rsrc((void *)(p.ws + w0 * p.stride), (short)0, rows_w * p.stride,
                                                kBufferRsrcWord3);
        rxs = __builtin_amdgcn_make_buffer_rsrc((void *)(p.xs + x0 * p.stride), (short)0,
                                                (int)((int64_t)rows_x * p.stride), kBufferRsrcWord3);
#pragma unroll
        for (int j = 0; j < kWsLoads; ++j) {
            const int row = j * 32 + (lane >> 1);
            wsoff[j] = row < 16 * NB ? (uint32_t)row * p.stride + (lane & 1) * 4 : kOut;
        }
    }

    const int units = (kb + kUnit - 1) / kUnit;
    // Units are taken in an order that starts elsewhere in every column tile: all of them reading x's rows from
    // their start would queue at the same memory channels (32 int8 experts, 1 row each: 26.8 against 29.2 us).
    const int span = (units + kWaves - 1) / kWaves * kWaves, turn = tn % span;
    auto place = [&](int i) {
        if (i >= span) return i;
        i += turn;
        return i >= span ? i - span : i;
    };
    auto load_weights = [&](uint8_t *slot, int unit) __attribute__((always_inline)) {
        const uint32_t k = unit * kUnit;
#pragma unroll
        for (int j = 0; j < 2 * NB; ++j) {
            const uint32_t o = k + ((j & 1) ? col1 : col0) < (uint32_t)kb ? woff[j] + k : kOut;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_ptr_t)(slot + 16 * MB * kUnit + j * 1024), 16, o, 0, 0, 0);
        }
        if constexpr (kMx) {
#pragma unroll
            for (int j = 0; j < kWsLoads; ++j) {
                const uint32_t o = wsoff[j] != kOut && k < (uint32_t)kb ? wsoff[j] + k / 16 : kOut;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rws, (lds_ptr_t)(slot + kCodeBytes + (kXsLoads + j) * 256), 4, o, 0, 0, 0);
            }
        }
    };
    auto load_x = [&](uint8_t *slot, int unit) __attribute__((always_inline)) {
        const uint32_t k = unit * kUnit;
#pragma unroll
        for (int j = 0; j < 2 * MB; ++j) {
            const uint32_t o = xoff[j] != kOut && k + ((j & 1) ? col1 : col0) < (uint32_t)kb ? xoff[j] + k : kOut;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_ptr_t)(slot + j * 1024), 16, o, 0, 0, 0);
        }
        if constexpr (kMx) {
#pragma unroll
            for (int j = 0; j < kXsLoads; ++j) {
                const uint32_t o = xsoff[j] != kOut && k < (uint32_t)kb ? xsoff[j] + k / 16 : kOut;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rxs, (lds_ptr_t)(slot + kCodeBytes + j * 256), 4, o, 0, 0, 0);
            }
        }
    };
    constexpr int kXLoads = 2 * MB + kXsLoads, kLoads = kXLoads + 2 * NB + kWsLoads;
    uint8_t *const s0 = slot0 + wave * kSlotBytes, *const s1 = slot1 + wave * kSlotBytes;
    // the first weights before the rows' indices are known
    load_weights(s0, place(wave));
    load_weights(s1, place(wave + kWaves));
#pragma unroll
    for (int j = 0; j < 2 * MB; ++j) {
        const int s = row_of_x(j * 8 + r8);
        xoff[j] = s < 0 ? kOut : (uint32_t)s * kb + ((j & 1) ? col1 : col0);
    }
    if constexpr (kMx) {
#pragma unroll
        for (int j = 0; j < kXsLoads; ++j) {
            const int row = j * 32 + (lane >> 1), s = row < 16 * MB ? row_of_x(row) : -1;
            xsoff[j] = s < 0 ? kOut : (uint32_t)s * p.stride + (lane & 1) * 4;
        }
    }
    load_x(s0, place(wave));
    load_x(s1, place(wave + kWaves));

    const int r = lane & 15, q = lane >> 4;
    acc_t acc[MB][NB];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = acc_t{};
    auto multiply = [&](const uint8_t *slot, int unit) __attribute__((always_inline)) {
        const uint8_t *base = slot + r * kUnit;
        // the lane's two chunks: halves of one product's operand (e4m3), or one for each of two products
        const int c0 = QT == kTypeInt8 ? q : 2 * q, c1 = QT == kTypeInt8 ? 4 + q : 2 * q + 1;
        const int o0 = (c0 ^ swizzle(r)) << 4, o1 = (c1 ^ swizzle(r)) << 4;
        v4i a[NB][2], b[MB][2];
        int ws[kMx ? NB : 1], xs[kMx ? MB : 1];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            a[nb][0] = *reinterpret_cast<const v4i *>(base + (MB + nb) * 16 * kUnit + o0);
            a[nb][1] = *reinterpret_cast<const v4i *>(base + (MB + nb) * 16 * kUnit + o1);
        }
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
            b[mb][0] = *reinterpret_cast<const v4i *>(base + mb * 16 * kUnit + o0);
            b[mb][1] = *reinterpret_cast<const v4i *>(base + mb * 16 * kUnit + o1);
        }
        if constexpr (kMx) {
            // bytes past the row's blocks count as 2^-127 (their codes are 0, but 0 times NaN is not)
            const int left = kb / 16 - unit * 8 - 2 * q, keep = left >= 2 ? 0xFFFF : left == 1 ? 0xFF : 0;
            const uint8_t *sc = slot + kCodeBytes + r * 8 + q * 2;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) ws[nb] = *reinterpret_cast<const uint16_t *>(sc + kXsLoads * 256 + nb * 128) & keep;
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) xs[mb] = *reinterpret_cast<const uint16_t *>(sc + mb * 128) & keep;
        }
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                if constexpr (QT == kTypeInt8) {
                    acc[mb][nb] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[nb][0], b[mb][0], acc[mb][nb], 0, 0, 0);
                    acc[mb][nb] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[nb][1], b[mb][1], acc[mb][nb], 0, 0, 0);
                } else if constexpr (QT == kTypeE4m3) {
                    const v8i va = {a[nb][0][0], a[nb][0][1], a[nb][0][2], a[nb][0][3],
                                    a[nb][1][0], a[nb][1][1], a[nb][1][2], a[nb][1][3]};
                    const v8i vb = {b[mb][0][0], b[mb][0][1], b[mb][0][2], b[mb][0][3],
                                    b[mb][1][0], b[mb][1][1], b[mb][1][2], b[mb][1][3]};
                    acc[mb][nb] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(va, vb, acc[mb][nb], 0, 0, 0, 127, 0, 127);
                } else {
                    acc[mb][nb] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        codes4(a[nb][0]), codes4(b[mb][0]), acc[mb][nb], 4, 4, 0, ws[nb], 0, xs[mb]);
                    acc[mb][nb] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        codes4(a[nb][1]), codes4(b[mb][1]), acc[mb][nb], 4, 4, 1, ws[nb], 1, xs[mb]);
                }
            }
    };
    // Wave w takes units w, w + 4, ... of the turned order; past the end zeros.  A slot is loaded again once it has
    // been read.  `newer`: loads in flight that are not the slot's.
    static_assert(kLoads < 64, "vmcnt range");
    auto step = [&](uint8_t *slot, int i, auto newer) __attribute__((always_inline)) {
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(decltype(newer)::value) : "memory");
        multiply(slot, place(i));
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        load_weights(slot, place(i + 2 * kWaves));
        load_x(slot, place(i + 2 * kWaves));
    };
    // (the first slot's last loads were x's, before the second's x)
    step(s0, wave, std::integral_constant<int, kXLoads>{});
    step(s1, wave + kWaves, std::integral_constant<int, kLoads>{});
    for (int i = wave + 2 * kWaves; i < span; i += 2 * kWaves) {
        step(s0, i, std::integral_constant<int, kLoads>{});
        step(s1, i + kWaves, std::integral_constant<int, kLoads>{});
    }

    // The waves' sums, in the first units' place once no load is on its way there.
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    acc_t *part = reinterpret_cast<acc_t *>(slot0);
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) part[(wave * MB * NB + mb * NB + nb) * 64 + lane] = acc[mb][nb];
    __syncthreads();
    // wave w adds up blocks w, w + 4, ...
#pragma unroll
    for (int b = 0; b < MB * NB; ++b) {
        if ((b & (kWaves - 1)) != wave) continue;
        const int mb = b / NB, nb = b % NB;
        acc_t s = part[b * 64 + lane];
#pragma unroll
        for (int i = 1; i < kWaves; ++i) {
            const acc_t other = part[(i * MB * NB + b) * 64 + lane];
            if constexpr (QT == kTypeInt8) s = (acc_t)((v4u)s + (v4u)other);  // modulo 2^32, as the products add up
            else s += other;
        }
        // lane l: row l & 15 of the block, columns 4 (l >> 4) .. + 3
        const int i = mb * 16 + r, m = t.m0 + i, n = n0 + nb * 16 + q * 4;
        if (m >= t.end || n >= p.N) continue;
        float tm = 1.0f;
        if constexpr (!kMx) {
            const int row = row_of_x(i);
            tm = row < 0 ? 0.0f : p.sx[x0 + row];
            if (!p.per_channel) tm *= p.sw[t.group];
        }
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (n + e >= p.N) {
                y[e] = 0.0f;
                continue;
            }
            const size_t at = (size_t)t.group * p.N + n + e;
            const float bias = p.bias ? bf16_bits_to_f32(p.bias[at]) : 0.0f;
            if constexpr (kMx) y[e] = s[e] + bias;
            else y[e] = __builtin_fmaf((float)s[e], p.per_channel ? tm * p.sw[at] : tm, bias);
        }
        uint16_t *dst = p.out + (size_t)m * p.N + n;
        if (n + 3 < p.N) {
            // at the alignment of one value: rows of any N start anywhere
            typedef uint32_t v2u_at2 __attribute__((ext_vector_type(2), aligned(2)));
            typedef uint32_t v2u __attribute__((ext_vector_type(2)));
            *reinterpret_cast<v2u_at2 *>(dst) = v2u{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n + e < p.N) Bf16::store(dst + e, y[e]);
        }
    }
}

template <int QT, int MB, int NB>
void launch(const GroupedArgs &a, hipStream_t stream) {
    const int tiles_n = (a.N + 16 * NB - 1) / (16 * NB), columns = (tiles_n + 7) / 8 * 8;
    grouped_rows_kernel<QT, MB, NB>
        <<<(unsigned)(rows_tiles(a, 16 * MB) * columns), kThreads, 0, stream>>>(a, tiles_n, columns);
}

}  // namespace

template <int QT>
void launch_grouped_rows(const GroupedArgs &a, GroupedKind kind, hipStream_t stream) {
    if (kind == kRows16x16) launch<QT, 1, 1>(a, stream);
    else if (kind == kRows16x32) launch<QT, 1, 2>(a, stream);
    else if (kind == kRows32x32) launch<QT, 2, 2>(a, stream);
    else launch<QT, 4, 4>(a, stream);
}
template void launch_grouped_rows<kTypeInt8>(const GroupedArgs &, GroupedKind, hipStream_t);
template void launch_grouped_rows<kTypeE4m3>(const GroupedArgs &, GroupedKind, hipStream_t);
template void launch_grouped_rows<kTypeMx4>(const GroupedArgs &, GroupedKind, hipStream_t);

}  // namespace w8a8
