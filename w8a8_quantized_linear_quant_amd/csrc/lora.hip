// lora.hip -- low-rank adapters of many requests beside a shared projection.
//
// Row m of X belongs to a request that uses adapter l (or none):
//   u = s_l x A_l^T           (down, over K)       out = base + u B_l^T   (up)
//   g = s_l dy B_l            (down, over N)       dx  = base + g A_l     (up)
//   dA_l = sum_m g^T x        dB_l = sum_m dy^T u  (over the rows of l)
// The kernels, on the bf16 MFMA: a down-projection of the rows, an up-projection
// added to a base, both in one for few rows and ranks, and a sum of outer
// products over an adapter's rows.  (The splits of these sums are added up in
// the up-projection's launch, or in one of their own where there is none.)  The
// weight of the projections is A [R, K] or B [N, R]: one of the two has the
// MFMA's contraction index contiguous in memory, the other (TR) is transposed on
// its way to the registers.
//
// All are bound by streaming the wide tensors (x, dy, base, out): R is small, so
// each takes 2 R operations for the 2 bytes of an element, far below the 500 or
// so at which the matrix pipes would be the bound.  Measured (MI355X, a large
// copy moves 5.3 TB/s; medians under rocprofv3, inputs rotated over three sets):
//   M 8192, K 4096, N 12288, R 64, forward: down 28 us (67 MB of x; the rest is
//   the weight, 512 KB a workgroup from L2), up 83 us (403 MB, 4.8 TB/s)
//   M 8192, K = N 4096, R 32, backward: down 18.6 us (67 MB), outer sums 32 us
//   (134 MB, 4.2 TB/s), up with their splits 29.6 us (134 MB, 4.5 TB/s)
// The comparisons at the single choices below are of one set of inputs taken over
// and over, part of which the caches hold.
#include <algorithm>

#include "block.hpp"

namespace w8a8 {
namespace {

constexpr int kTileRows = W8A8_LORA_TILE_ROWS;
constexpr int kMaxR = 128;
constexpr int64_t kMaxL = 65535;

struct Tile {
    int64_t row0;
    int rows, adapter;
};

// Tile t of the plan; rows = 0 where the entry does not fit M and L (checked
// without branches, so that the entry is one 16-byte scalar load).
__device__ __forceinline__ Tile load_tile(const int32_t *plan, int t, int64_t M, int L) {
    const v4i e = reinterpret_cast<const v4i *>(plan)[t];
    const int row0 = e[0], rows = e[1], adapter = e[2];
    const bool ok = (row0 >= 0) & (rows >= 0) & (rows <= kTileRows) & (row0 <= M - rows) & (adapter >= -1) &
                    (adapter < L);
    return {ok ? row0 : 0, ok ? rows : 0, ok ? adapter : -1};
}

__device__ __forceinline__ int rank_of(const int32_t *ranks, int l, int R) {
    return l < 0 ? 0 : ranks ? min(max(ranks[l], 0), R) : R;
}

// A buffer of `rows` rows of `cols` bf16 elements, ld apart, from row0: reads
// past the last row's end give 0.  The base is 64-bit, the offsets inside a
// tile are below 2^31 (64 rows of at most 2^22 elements).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const uint16_t *p, int64_t row0, int rows, int64_t ld,
                                                            int cols) {
    const int bytes = rows > 0 ? (int)(((rows - 1) * ld + cols) * 2) : 0;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t *>(p) + row0 * ld, (short)0, bytes, kBufferRsrcWord3);
}
// The rows of a tile in v f32 [M, R].
__device__ __forceinline__ __amdgpu_buffer_rsrc_t v_rsrc(const float *v, int64_t row0, int rows, int R) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<float *>(v) + row0 * R, (short)0, rows * R * 4,
                                             kBufferRsrcWord3);
}
__device__ __forceinline__ v4u load16(__amdgpu_buffer_rsrc_t r, int offset) {
    return __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(r, offset, 0, 0));
}
__device__ __forceinline__ v4f mfma(v4u a, v4u b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0,
                                                   0);
}

// Lanes: MFMA 16x16x32, A row (and B column) lane % 16, contraction elements
// 8 (lane / 16) .. + 7; D row 4 (lane / 16) + e, column lane % 16.

// ---------------------------------------------------------------- down
// One workgroup takes 16 RB rows of a tile over all of C; its waves take
// 128-wide slices of the contraction in turn and their sums meet in LDS, so
// that no partial sums leave the workgroup.  JB: 16-wide blocks of the rank.
//
// A fragment wants 16 rows in 16 consecutive lanes, which from memory would be
// 64 separate 16-byte requests a load (85 cycles of a CU's address unit where
// 16 do: 38 us at M 8192, C 4096, R 64).  So x and the weight are loaded with
// 16 lanes along a row (256 bytes) and turned in a 4 KB piece of LDS of the
// wave's own: a block is written there, its registers are loaded again at once
// with the next one's data, and its fragments are read back.  LDS accesses of
// a wave stay in order, so no barrier is needed.
constexpr int kSlice = 128;
// 16 waves where 128 registers hold a wave's sums and its blocks in flight.
constexpr int down_waves(int JB, int RB) { return RB == 1 && JB <= 4 ? 16 : 8; }

// Block of 16 rows x 256 bytes: chunk c of row i in slot c ^ i, so that 16
// rows' reads of one chunk fall on distinct banks.
__device__ __forceinline__ void turn_in(char *area, const v4u (&d)[4], int lane) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = i * 4 + (lane >> 4), c = lane & 15;
        *reinterpret_cast<v4u *>(area + row * 256 + ((c ^ row) << 4)) = d[i];
    }
}
__device__ __forceinline__ v4u turn_out(const char *area, int step, int lane) {
    const int row = lane & 15, c = step * 4 + (lane >> 4);
    return *reinterpret_cast<const v4u *>(area + row * 256 + ((c ^ row) << 4));
}

// TR's weight fragments: 32 rows n of B by 16 JB ranks, written as they lie,
// read transposed (ds_read_b64_tr_b16: each 16 lanes read 4 rows of 16
// columns, lane i receives column i's 4 values).
template <int JB>
__device__ __forceinline__ v4u transposed_fragment(const char *area, int jb, int lane) {
    typedef short v4s __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) v4s lds_v4s;
    const int g = lane >> 4, q = lane & 15;
    const char *p = area + (8 * g + q / 4) * (32 * JB) + jb * 32 + (q % 4) * 8;
    const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)p);
    const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)(p + 4 * 32 * JB));
    const uint2 a = __builtin_bit_cast(uint2, lo), b = __builtin_bit_cast(uint2, hi);
    return v4u{a.x, a.y, b.x, b.y};
}

// acc += this wave's slices of rows x weight, for the 16 RB rows from `first`
// of a tile and the 16 JB ranks from j0; area: the wave's LDS; block: which
// workgroup asks (all that share a result must give the same, for the order of
// its sums).
template <int JB, int RB, bool TR, int W>
__device__ __forceinline__ void down_sums(v4f (&acc)[RB][JB], const uint16_t *x, const Tile &tile, int first, int C,
                                          int64_t ldx, const uint16_t *w, int R, int j0, char *area, unsigned block) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int slices = (C + kSlice - 1) / kSlice;
    if (wave >= slices) return;
    const auto rx = rows_rsrc(x, tile.row0 + first, tile.rows - first, ldx, C);
    const auto rw = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t *>(w) + (int64_t)tile.adapter * R * C, (short)0,
                                                      R * C * 2, kBufferRsrcWord3);
    const int li = lane >> 4, lc = (lane & 15) * 8;  // row and column of a lane in a load of 4 rows x 128
    // past C both factors read 0: neither may be whatever lies behind a row
    auto fetch_x = [&](int slice, int a, v4u (&d)[4]) {
        const int k = slice * kSlice + lc;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            d[i] = load16(rx, k < C ? (int)((a * 16 + i * 4 + li) * ldx + k) * 2 : kOobOffset);
    };
    constexpr int kUnits = TR ? 4 : JB, kUnit = TR ? JB : 4;  // weight blocks of a slice, loads of a block
    auto fetch_w = [&](int slice, int unit, v4u (&d)[kUnit]) {
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
            if constexpr (TR) {  // 32 rows n of a step, all ranks
                const int c = i * 64 + lane, row = slice * kSlice + unit * 32 + c / (2 * JB);
                const int j = j0 + c % (2 * JB) * 8;
                d[i] = load16(rw, row < C && j < R ? (row * R + j) * 2 : kOobOffset);
            } else {             // 16 ranks of a slice
                const int k = slice * kSlice + lc;
                d[i] = load16(rw, k < C ? ((j0 + unit * 16 + i * 4 + li) * C + k) * 2 : kOobOffset);
            }
        }
    };
    // Workgroups start at different slices: in step, they would all read
    // the same few kilobytes of every row (with rows a power of two apart
    // a quarter of the memory channels) and the same lines of the weight
    // (8 XCDs: blocks 8 apart share an L2).
    const int turns = (slices + W - 1) / W;
    int turn = (int)((block / 8 + block) % (unsigned)turns);
    // Weight blocks in flight: two for ranks past 64, whose 8 blocks a slice
    // are most of the loads (R 128, M 8192, C 4096: 48 us with one, 34 with
    // two; R 64: 23 and 24; a whole slice's, ahead of the next rows of x, 25).
    constexpr int DW = JB == 8 && !TR ? 2 : 1;
    v4u xd[RB][4], wd[DW][kUnit];
    int slice = turn * W + wave;
#pragma unroll
    for (int a = 0; a < RB; ++a) fetch_x(slice, a, xd[a]);
#pragma unroll
    for (int q = 0; q < DW; ++q) fetch_w(slice, q, wd[q]);
    for (int n = 0; n < turns; ++n) {  // a slice past the end reads 0 without touching memory
        turn = turn + 1 < turns ? turn + 1 : 0;
        const int next = n + 1 < turns ? turn * W + wave : slices;
        v4u xf[RB][4];
#pragma unroll
        for (int a = 0; a < RB; ++a) {
            turn_in(area, xd[a], lane);
            fetch_x(next, a, xd[a]);
#pragma unroll
            for (int t = 0; t < 4; ++t) xf[a][t] = turn_out(area, t, lane);
        }
#pragma unroll
        for (int q = 0; q < kUnits; ++q) {
            if constexpr (TR) {
#pragma unroll
                for (int i = 0; i < kUnit; ++i) *reinterpret_cast<v4u *>(area + (i * 64 + lane) * 16) = wd[q % DW][i];
            } else {
                turn_in(area, wd[q % DW], lane);
            }
            if (q + DW < kUnits) fetch_w(slice, q + DW, wd[q % DW]);
            else fetch_w(next, q + DW - kUnits, wd[q % DW]);
#pragma unroll
            for (int i = 0; i < (TR ? JB : 4); ++i) {
                const v4u f = TR ? transposed_fragment<JB>(area, i, lane) : turn_out(area, i, lane);
                const int t = TR ? q : i, b = TR ? i : q;
#pragma unroll
                for (int a = 0; a < RB; ++a) acc[a][b] = mfma(xf[a][t], f, acc[a][b]);
            }
        }
        slice = next;
    }
}

template <int JB, int RB, bool TR>
__global__ __launch_bounds__(64 * down_waves(JB, RB)) void lora_down_kernel(const uint16_t *x, int64_t M, int C,
                                                                            int64_t ldx, const uint16_t *w, int L,
                                                                            int R, const float *scale,
                                                                            const int32_t *ranks, const int32_t *plan,
                                                                            int T, int j_parts, float *v) {
    constexpr int W = down_waves(JB, RB);
    constexpr int kArea = TR && JB > 4 ? JB * 1024 : 4096;  // bytes of a wave
    constexpr int kSums = W * RB * 16 * 17 * 4;
    __shared__ __attribute__((aligned(16))) char lds[W * kArea > kSums ? W * kArea : kSums];
    // the tiles' first parts come first: short tiles have no others, and the
    // blocks that are left must not fall on the same few XCDs
    const int block = blockIdx.x / j_parts, j0 = blockIdx.x % j_parts * (16 * JB);
    const Tile tile = load_tile(plan, block % T, M, L);
    const int first = block / T * (16 * RB);
    if (first >= tile.rows) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = rank_of(ranks, tile.adapter, R);
    const float s = tile.adapter >= 0 && scale ? scale[tile.adapter] : 1.f;
    v4f acc[RB][JB];
#pragma unroll
    for (int a = 0; a < RB; ++a)
#pragma unroll
        for (int b = 0; b < JB; ++b) acc[a][b] = v4f{0.f, 0.f, 0.f, 0.f};
    // (the rank masks what is written; no load waits for it)
    if (tile.adapter >= 0)
        down_sums<JB, RB, TR, W>(acc, x, tile, first, C, ldx, w, R, j0, lds + wave * kArea, blockIdx.x);
    auto part = reinterpret_cast<float (*)[RB * 16][17]>(lds);
#pragma unroll
    for (int b = 0; b < JB; ++b) {
        __syncthreads();
#pragma unroll
        for (int a = 0; a < RB; ++a)
#pragma unroll
            for (int e = 0; e < 4; ++e) part[wave][a * 16 + 4 * (lane >> 4) + e][lane & 15] = acc[a][b][e];
        __syncthreads();
        const int row = threadIdx.x / 16, j = j0 + b * 16 + threadIdx.x % 16;
        if (row < RB * 16 && first + row < tile.rows && j < R) {
            float t = 0.f;
#pragma unroll
            for (int k = 0; k < W; ++k) t += part[k][row][threadIdx.x % 16];
            v[(tile.row0 + first + row) * R + j] = j < r ? t * s : 0.f;
        }
    }
}

// ------------------------------------------------------------------ up
// A wave takes 128 columns of all the tile's rows, its weights in registers
// and all of base in flight at once.  MFMA t of 8 has column 8 i + t as its
// column i: a lane then holds 8 consecutive columns of a row, 16 lanes 256
// bytes of it, and base (the sums' start) and out move as 16-byte accesses.
// (The transposed product, 16 rows in 16 consecutive lanes, makes 64 requests
// of each access: 99 us against 84 at M 8192, C 12288, R 64.)  The workgroup
// turns v into two bf16 halves (hi + lo, ~16 bits) in LDS; up to R = 16 both
// fit one 32-wide contraction, the weight twice.
constexpr int kUpWaves = 4;
// Waves to a SIMD that the registers allow: 32 (RB = 2) or 64 of base, 32 for
// each 32 ranks of the weight, 32 of sums.
constexpr int up_simd_waves(int JB, int RB) {
    if (JB <= 2) return RB == 2 ? 4 : 3;
    return JB == 4 ? (RB == 2 ? 3 : 2) : 1;
}

// Four f32 values as bf16 halves; lo = 0 beside an infinite hi.  A finite value
// nearest to no finite bf16 takes the largest one for its hi.
__device__ __forceinline__ float split_hi(float f) {
    constexpr float most = 0x1.FEp127f;
    return __builtin_isfinite(f) ? __builtin_amdgcn_fmed3f(f, -most, most) : f;
}
__device__ __forceinline__ void split2(v4f f, uint2 &hi, uint2 &lo) {
    uint32_t h[2], l[2];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        h[p] = pack_bf16x2(split_hi(f[2 * p]), split_hi(f[2 * p + 1]));
        const float a = __uint_as_float(h[p] << 16), b = __uint_as_float(h[p] & 0xFFFF0000u);
        l[p] = pack_bf16x2(__builtin_isfinite(a) ? f[2 * p] - a : 0.f, __builtin_isfinite(b) ? f[2 * p + 1] - b : 0.f);
    }
    hi = make_uint2(h[0], h[1]), lo = make_uint2(l[0], l[1]);
}

// The 16-bit halves of (a, b): the low ones, or the high ones.
__device__ __forceinline__ uint32_t halves(uint32_t a, uint32_t b, bool high) {
    return __builtin_amdgcn_perm(b, a, high ? 0x07060302u : 0x05040100u);
}

// The weight fragments of a wave's 128 columns, one 32-wide contraction k at a
// time: loaded with lanes along memory, then turned into wf[t][k].  Entries
// beyond the adapter's rank become 0, whatever lies there.  TR: 8 ranks of the
// lane's 8 columns, paired into the 8 fragments.  Else: 128 rows of 2 or 4
// chunks of 8 ranks through the wave's own LDS (4 KB for JB = 1, else 8),
// slots swizzled for the reads 8 rows apart.
constexpr int up_loads(int JB, bool TR) { return JB == 1 && !TR ? 4 : 8; }

template <bool TR>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t up_rsrc(const uint16_t *w, int adapter, int C, int R, int r) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t *>(w) + (int64_t)adapter * R * C, (short)0,
                                             (TR ? r : R) * C * 2, kBufferRsrcWord3);
}

template <int JB, bool TR>
__device__ __forceinline__ void up_fetch(v4u (&d)[up_loads(JB, TR)], __amdgpu_buffer_rsrc_t rw, int col0, int C, int R,
                                         int k) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < up_loads(JB, TR); ++i) {
        if constexpr (TR) {
            const int jg = JB == 1 ? lane >> 4 & 1 : lane >> 4, j = k * 32 + jg * 8 + i, c = col0 + 8 * (lane & 15);
            d[i] = load16(rw, c < C ? (j * C + c) * 2 : kOobOffset);
        } else {
            constexpr int kCh = JB == 1 ? 2 : 4;
            const int q = i * 64 + lane, n = col0 + q / kCh, j = k * 32 + q % kCh * 8;
            d[i] = load16(rw, n < C && j < R ? (n * R + j) * 2 : kOobOffset);
        }
    }
}

template <int JB, bool TR, int KB>
__device__ __forceinline__ void up_fragments(v4u (&wf)[8][KB], int k, const v4u (&d)[up_loads(JB, TR)], char *ws, int R,
                                             int r) {
    const int lane = threadIdx.x & 63, fi = lane & 15, jg = JB == 1 ? lane >> 4 & 1 : lane >> 4;
    if constexpr (TR) {
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int p = 0; p < 4; ++p) wf[t][k][p] = halves(d[2 * p][t / 2], d[2 * p + 1][t / 2], t & 1);
    } else {
        constexpr int kCh = JB == 1 ? 2 : 4;
#pragma unroll
        for (int i = 0; i < 2 * kCh; ++i) {
            const int q = i * 64 + lane;
            *reinterpret_cast<v4u *>(ws + ((q ^ (q / kCh >> 3 & 7)) << 4)) = d[i];
        }
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            const int q = (8 * fi + t) * kCh + jg;
            wf[t][k] = *reinterpret_cast<const v4u *>(ws + ((q ^ (fi & 7)) << 4));
        }
        if (r < R) {
            const int j = k * 32 + jg * 8;
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const uint32_t keep = (j + 2 * p < r ? 0xFFFFu : 0u) | (j + 2 * p + 1 < r ? 0xFFFF0000u : 0u);
#pragma unroll
                for (int t = 0; t < 8; ++t) wf[t][k][p] &= keep;
            }
        }
    }
}

// v's fragment of 16 rows for contraction k: from its hi or its lo half (JB = 1:
// both in one contraction, the lanes of fg 2 and 3 hold lo).
template <int JB, int P>
__device__ __forceinline__ v4u v_fragment(const uint16_t (*hi)[P], const uint16_t (*lo)[P], int k, int h, int lane) {
    const int fi = lane & 15, fg = lane >> 4, jg = JB == 1 ? fg & 1 : fg;
    return *reinterpret_cast<const v4u *>(&((JB == 1 ? fg >> 1 : h) ? lo : hi)[fi][k * 32 + jg * 8]);
}

// One block of 16 rows of a wave's 128 columns: base (bf) plus v (its halves in
// LDS rows hi, lo of this block) times the weight, stored, unless a lane holds a
// NaN in it: returns whether.  (Looking costs 16 instructions.  With a rank of 0
// the block is base, and there is no weight to take it again with.)
template <int JB, int KB, int P>
__device__ __forceinline__ bool up_rows(const v4u (&bf)[4], const uint16_t (*hi)[P], const uint16_t (*lo)[P],
                                        const v4u (&wf)[8][KB], int r, uint16_t *out, int64_t ldout, int rows, int col0,
                                        int C) {
    const int lane = threadIdx.x & 63, fg = lane >> 4;
    v4f acc[8];
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[t][e] = __uint_as_float(t & 1 ? bf[e][t / 2] & 0xFFFF0000u : bf[e][t / 2] << 16);
    if (r > 0) {
#pragma unroll
        for (int k = 0; k < KB; ++k) {
#pragma unroll
            for (int h = 0; h < (JB == 1 ? 1 : 2); ++h) {
                const v4u f = v_fragment<JB, P>(hi, lo, k, h, lane);
#pragma unroll
                for (int t = 0; t < 8; ++t) acc[t] = mfma(f, wf[t][k], acc[t]);
            }
        }
    }
    const int c = col0 + 8 * (lane & 15);
    float any = 0.f;
    v4u d[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            any = max_or_nan(max_or_nan(any, acc[2 * p][e]), acc[2 * p + 1][e]);
            d[e][p] = pack_bf16x2(acc[2 * p][e], acc[2 * p + 1][e]);
        }
    if (__builtin_expect(r > 0 && __any(any != any && c < C), false)) return false;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int row = 4 * fg + e;
        if (row < rows && c < C) *reinterpret_cast<v4u *>(out + row * ldout + c) = d[e];
    }
    return true;
}

// A pair of bf16 with its infinities and NaN as 0.
__device__ __forceinline__ uint32_t finite_halves(uint32_t w) {
    return ((w & 0x7F80u) != 0x7F80u ? w & 0xFFFFu : 0u) | ((w & 0x7F800000u) != 0x7F800000u ? w & 0xFFFF0000u : 0u);
}

// The blocks (bits of `again`) that up_rows did not store.  Against an infinite
// weight the two halves of v may give inf - inf or inf * 0 where v gives an
// infinity: here lo meets the weight's finite entries alone, and the infinities
// hi, which has v's sign.  base is still in place and read again.  Two columns
// at a time, their results over their base, to need no more registers than up_rows.
template <int JB, int KB, int P>
__device__ __forceinline__ void up_again(unsigned again, __amdgpu_buffer_rsrc_t rb, int64_t ldbase,
                                         const uint16_t (*hi)[P], const uint16_t (*lo)[P], const v4u (&wf)[8][KB],
                                         uint16_t *out, int64_t ldout, int rows, int col0, int C) {
    const int lane = threadIdx.x & 63, fg = lane >> 4, c = col0 + 8 * (lane & 15);
#pragma unroll 1
    for (; again != 0; again &= again - 1) {
        const int first = __builtin_ctz(again) * 16;
        v4u d[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) d[e] = load16(rb, (int)((first + 4 * fg + e) * ldbase + c) * 2);
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            v4f acc[2];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc[0][e] = __uint_as_float(d[e][p] << 16), acc[1][e] = __uint_as_float(d[e][p] & 0xFFFF0000u);
#pragma unroll
            for (int k = 0; k < KB; ++k)
#pragma unroll
                for (int h = 0; h < (JB == 1 ? 1 : 2); ++h) {
                    const v4u f = v_fragment<JB, P>(hi + first, lo + first, k, h, lane);
                    const bool is_lo = JB == 1 ? fg >> 1 : h;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        v4u w = wf[2 * p + i][k];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            asm volatile("" : "+v"(w[q]));  // or all of them are made, and held, ahead of the loop
                            w[q] = is_lo ? finite_halves(w[q]) : w[q];
                        }
                        acc[i] = mfma(f, w, acc[i]);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
#pragma unroll
            for (int e = 0; e < 4; ++e) d[e][p] = pack_bf16x2(acc[0][e], acc[1][e]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (4 * fg + e < rows - first && c < C)
                *reinterpret_cast<v4u *>(out + (first + 4 * fg + e) * ldout + c) = d[e];
    }
}

// The outer sums' splits, to be added up: da = sum of pa [splits][na], db of pb
// (na, nb multiples of 4), 1024 elements a block of 256 threads.  With an input
// gradient wanted too, these blocks go first in the up-projection's launch,
// which hides their memory's latency (4.5 us as a launch of their own).
struct SplitSums {
    const float *pa, *pb;
    float *da, *db;
    int64_t na, nb;
    int splits, blocks;
};
__device__ __forceinline__ void add_splits(const SplitSums &sums, int block) {
    int64_t i = ((int64_t)block * 256 + threadIdx.x) * 4;
    const bool is_a = i < sums.na;
    const float *p = is_a ? sums.pa : sums.pb;
    float *d = is_a ? sums.da : sums.db;
    const int64_t n = is_a ? sums.na : sums.nb;
    if (!is_a) i -= sums.na;
    if (i >= n) return;
    v4f s = {0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < sums.splits; k += 8) {
        v4f q[8];
#pragma unroll
        for (int c = 0; c < 8; ++c)
            q[c] = k + c < sums.splits ? *reinterpret_cast<const v4f *>(p + (k + c) * n + i) : v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 8; ++c) s += q[c];
    }
    *reinterpret_cast<v4f *>(d + i) = s;
}

template <int JB, bool TR, int RB>
__global__ __launch_bounds__(64 * kUpWaves, up_simd_waves(JB, RB)) void lora_up_kernel(
    const float *v, const uint16_t *w, int64_t M, int C, int L, int R, const int32_t *ranks, const int32_t *plan,
    int groups, const uint16_t *base, int64_t ldbase, uint16_t *out, int64_t ldout, SplitSums sums) {
    if ((int)blockIdx.x < sums.blocks) return add_splits(sums, blockIdx.x);
    constexpr int KB = JB == 1 ? 1 : JB / 2;  // 32-wide contractions
    constexpr int P = JB * 16 + 8;  // halves of an LDS row: 16 rows' reads fall on distinct banks
    constexpr int kRows = 16 * RB, kParts = kTileRows / kRows;
    __shared__ __attribute__((aligned(16))) uint16_t vs[2][kRows][P];
    __shared__ __attribute__((aligned(16))) char ws[TR ? 1 : kUpWaves][TR ? 16 : JB == 1 ? 4096 : 8192];
    // blocks of a tile's rows: columns, then its next 16 RB rows
    const int block = blockIdx.x - sums.blocks, part = block / groups;
    Tile tile = load_tile(plan, part / kParts, M, L);
    tile.row0 += part % kParts * kRows;
    tile.rows = min(tile.rows - part % kParts * kRows, kRows);
    if (tile.rows <= 0) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col0 = (block % groups * kUpWaves + wave) * 128;
    const auto rv = v_rsrc(v, tile.row0, tile.rows, R);
    constexpr int kChunks = (kRows * JB * 4 + 64 * kUpWaves - 1) / (64 * kUpWaves);  // 4-float chunks of v per thread
    v4u vd[kChunks];
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const int q = i * 64 * kUpWaves + threadIdx.x, row = q / (JB * 4), j = q % (JB * 4) * 4;
        vd[i] = load16(rv, j < R ? (row * R + j) * 4 : kOobOffset);
    }
    const int r = rank_of(ranks, tile.adapter, R);
    const int fi = lane & 15, fg = lane >> 4;

    v4u bf[RB][4];
    const auto rb = rows_rsrc(base, tile.row0, base ? tile.rows : 0, ldbase, C);
#pragma unroll
    for (int a = 0; a < RB; ++a) {
        if (a * 16 >= tile.rows) break;
#pragma unroll
        for (int e = 0; e < 4; ++e) bf[a][e] = load16(rb, (int)((a * 16 + 4 * fg + e) * ldbase + col0 + 8 * fi) * 2);
    }
    v4u wf[8][KB];
    if (r > 0 && col0 < C) {
        const auto rw = up_rsrc<TR>(w, tile.adapter, C, R, r);
#pragma unroll
        for (int k = 0; k < KB; ++k) {
            v4u d[up_loads(JB, TR)];
            up_fetch<JB, TR>(d, rw, col0, C, R, k);
            up_fragments<JB, TR>(wf, k, d, ws[TR ? 0 : wave], R, r);
        }
    }
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const int q = i * 64 * kUpWaves + threadIdx.x, row = q / (JB * 4), j = q % (JB * 4) * 4;
        if (row >= kRows) break;
        uint2 hi, lo;
        split2(__builtin_bit_cast(v4f, vd[i]), hi, lo);
        *reinterpret_cast<uint2 *>(&vs[0][row][j]) = hi;
        *reinterpret_cast<uint2 *>(&vs[1][row][j]) = lo;
    }
    __syncthreads();
    if (col0 >= C) return;
    unsigned again = 0;
#pragma unroll
    for (int a = 0; a < RB; ++a) {
        if (a * 16 >= tile.rows) break;
        if (!up_rows<JB, KB, P>(bf[a], &vs[0][a * 16], &vs[1][a * 16], wf, r, out + (tile.row0 + a * 16) * ldout,
                                       ldout, tile.rows - a * 16, col0, C))
            again |= 1u << a;
    }
    up_again<JB, KB, P>(again, rb, ldbase, vs[0], vs[1], wf, out + tile.row0 * ldout, ldout, tile.rows, col0, C);
}

// ---------------------------------------------------------------- both
// The down- and the up-projection of 16 rows in one workgroup of 16 waves, 128
// columns a wave: one launch, with base and the up-projection's weights loaded
// ahead of the sums, ranks up to 16.  Where 2048 columns a workgroup do not
// cover C2, each further one takes the sums again (`groups` workgroups a block
// of rows).  Bound by the latency of its chain of loads: 4.9 us for one row at
// C = C2 1024, 9.1 for 48 requests' rows at 4096 (8.6 MB of weights, which the
// caches do not hold; 7.7 where they do).
template <bool TR>
__global__ __launch_bounds__(1024) void lora_both_kernel(const uint16_t *x, int64_t M, int C, int64_t ldx,
                                                         const uint16_t *w, int L, int R, const float *scale,
                                                         const int32_t *ranks, const int32_t *plan, int T, float *v,
                                                         const uint16_t *w2, int C2, int groups, const uint16_t *base,
                                                         int64_t ldbase, uint16_t *out, int64_t ldout) {
    constexpr int W = 16, JB = 1, KB = 1, P = JB * 16 + 8, kArea = 4096;
    __shared__ __attribute__((aligned(16))) char lds[W * kArea];
    __shared__ __attribute__((aligned(16))) uint16_t vs[2][16][P];
    const unsigned block = blockIdx.x / groups;
    const Tile tile = load_tile(plan, block % T, M, L);
    const int first = block / T * 16;
    if (first >= tile.rows) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = rank_of(ranks, tile.adapter, R);
    const float s = tile.adapter >= 0 && scale ? scale[tile.adapter] : 1.f;
    const int group = blockIdx.x % groups, col0 = (group * W + wave) * 128;
    const int64_t row0 = tile.row0 + first;
    const int rows = min(tile.rows - first, 16);
    v4u bf[4], d[up_loads(JB, TR)], wf[8][KB];
    const auto rb = rows_rsrc(base, row0, base ? rows : 0, ldbase, C2);
#pragma unroll
    for (int e = 0; e < 4; ++e)
        bf[e] = load16(rb, col0 < C2 ? (int)((4 * (lane >> 4) + e) * ldbase + col0 + 8 * (lane & 15)) * 2 : kOobOffset);
    up_fetch<JB, TR>(d, up_rsrc<TR>(w2, max(tile.adapter, 0), C2, R, r), col0, C2, R, 0);
    v4f acc[1][JB];
#pragma unroll
    for (int b = 0; b < JB; ++b) acc[0][b] = v4f{0.f, 0.f, 0.f, 0.f};
    if (tile.adapter >= 0) down_sums<JB, 1, TR, W>(acc, x, tile, first, C, ldx, w, R, 0, lds + wave * kArea, block);
    auto part = reinterpret_cast<float (*)[16][17]>(lds);
#pragma unroll
    for (int b = 0; b < JB; ++b) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 4; ++e) part[wave][4 * (lane >> 4) + e][lane & 15] = acc[0][b][e];
        __syncthreads();
        if (threadIdx.x < 256) {
            const int row = threadIdx.x / 16, j = b * 16 + threadIdx.x % 16;
            float t = 0.f;
#pragma unroll
            for (int k = 0; k < W; ++k) t += part[k][row][threadIdx.x % 16];
            t = j < r ? t * s : 0.f;
            if (v && group == 0 && row < rows && j < R) v[(row0 + row) * R + j] = t;
            const float hi = __uint_as_float(pack_bf16x2(split_hi(t), 0.f) << 16);
            vs[0][row][j] = (uint16_t)(__float_as_uint(hi) >> 16);
            vs[1][row][j] = (uint16_t)pack_bf16x2(__builtin_isfinite(hi) ? t - hi : 0.f, 0.f);
        }
    }
    __syncthreads();
    if (col0 >= C2) return;
    up_fragments<JB, TR>(wf, 0, d, lds + wave * kArea, R, r);
    const bool stored = up_rows<JB, KB, P>(bf, vs[0], vs[1], wf, r, out + row0 * ldout, ldout, rows, col0, C2);
    up_again<JB, KB, P>(stored ? 0u : 1u, rb, ldbase, vs[0], vs[1], wf, out + row0 * ldout, ldout, rows, col0, C2);
}

// --------------------------------------------------------------- outer sums
// d[c][j] = sum over an adapter's rows of y[m][c] v[m][j]: a product whose
// contraction runs over rows, across memory in both factors.  A workgroup
// takes 128 columns c and all ranks j; a tile of 64 rows of y and of v is
// staged in LDS as it lies, and the fragments come back transposed
// (ds_read_b64_tr_b16).  Two tiles' loads are in flight in registers.  v is
// three bf16 parts, which hold all 24 bits of it, so the gradients are as
// exact as f32 sums are.
constexpr int kOuterWaves = 4;

struct Outer {
    const uint16_t *y;
    int64_t ldy;
    const float *v;   // f32 [M, R]
    float *d;         // split s of d starts at s * L * R * C
    int C, groups;    // columns; workgroups of 128 columns
};
struct OuterPair {
    Outer a, b;       // dA [R, C]: y = x, v = g; dB [C, R]: y = dy, v = u
};

// Four f32 values as three bf16 parts: the first two are cut (not rounded) off
// the remainder, so each remainder is exact; an infinity has none, a NaN's is NaN
// (the first part alone may be an infinity, where the payload is in the low bits).
__device__ __forceinline__ void split3(v4f f, uint2 (&s)[3]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t h[2];
#pragma unroll
        for (int p = 0; p < 2; ++p) h[p] = halves(__float_as_uint(f[2 * p]), __float_as_uint(f[2 * p + 1]), true);
        s[i] = make_uint2(h[0], h[1]);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            f[k] = i || !__builtin_isinf(f[k]) ? f[k] - __uint_as_float(__float_as_uint(f[k]) & 0xFFFF0000u) : 0.f;
    }
    s[2] = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
}

// Rows of PIECES 32-byte pieces in LDS (16 columns each): piece p of row m in
// place p ^ turn(m), so that the 16 rows of a transposed read spread evenly
// over the banks.
template <int PIECES>
__device__ __forceinline__ int piece_at(int row, int piece) {
    const int turn = PIECES >= 4 ? row & 3 : PIECES == 2 ? row >> 1 & 1 : 0;
    return row * (32 * PIECES) + ((piece ^ turn) << 5);
}
// Fragment of 16 columns (lane % 16) by rows 8 (lane / 16) .. + 7 of 32 from row m0.
template <int PIECES>
__device__ __forceinline__ v4u read_transposed(const char *area, int m0, int piece, int lane) {
    typedef short v4s __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) v4s lds_v4s;
    const int row = m0 + 8 * (lane >> 4) + (lane & 15) / 4, at = (lane & 3) * 8;
    const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)(area + piece_at<PIECES>(row, piece) + at));
    const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)(area + piece_at<PIECES>(row + 4, piece) + at));
    const uint2 a = __builtin_bit_cast(uint2, lo), b = __builtin_bit_cast(uint2, hi);
    return v4u{a.x, a.y, b.x, b.y};
}

// acc = the sums of tiles begin .. end - 1: a wave's NC x NJ blocks of 16 x 16 of
// the 128 x 16 JB output, from pieces pc and pj.  FINITE: v's second and third
// parts meet the finite entries of y alone.
template <int JB, bool RANKS_FIRST, bool FINITE, int NC, int NJ>
__device__ __forceinline__ void outer_sums(v4f (&acc)[NC][NJ], const Outer &o, int col0, int pc, int pj, int64_t M,
                                           int L, int R, const int32_t *plan, int begin, int end, char *ys,
                                           char (&vs)[3][kTileRows * 32 * JB]) {
    constexpr int kThreads = 64 * kOuterWaves;
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[c][j] = v4f{0.f, 0.f, 0.f, 0.f};

    // lane i of every wave holds the entry of tile i of the 64 under way, so
    // that no scalar load (which would drain the LDS counter) is in the loop
    for (int c0 = begin; c0 < end; c0 += 64) {
        const int count = min(end - c0, 64);
        Tile mine = load_tile(plan, c0 + min(lane, count - 1), M, L);
        if (lane >= count) mine.rows = 0;
        const int entry_row = (int)mine.row0, entry_rows = mine.rows;
        v4u yd[2][4], vd[2][JB];
        // Past the last tile a fetch reads 0, without a branch, so that each
        // tile's loads are waited for by themselves.
        auto fetch = [&](int i, v4u (&y)[4], v4u (&v)[JB]) {
            const int row0 = __builtin_amdgcn_readlane(entry_row, min(i, 63));
            const int rows = i < count ? __builtin_amdgcn_readlane(entry_rows, min(i, 63)) : 0;
            // rows past the tile read 0 in both; columns past C are not stored
            const auto ry = rows_rsrc(o.y, row0, rows, o.ldy, o.C);
            const auto rv = v_rsrc(o.v, row0, rows, R);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                y[k] = load16(ry, (int)((k * 16 + (int)(threadIdx.x >> 4)) * o.ldy + col0 + 8 * (int)(threadIdx.x & 15)) * 2);
#pragma unroll
            for (int k = 0; k < JB; ++k) {
                const int q = k * kThreads + threadIdx.x, row = q / (4 * JB), j = q % (4 * JB) * 4;
                v[k] = load16(rv, j < R ? (row * R + j) * 4 : kOobOffset);
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        auto stage_y = [&](const v4u (&y)[4]) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int row = k * 16 + (threadIdx.x >> 4), c = threadIdx.x & 15;
                *reinterpret_cast<v4u *>(ys + piece_at<8>(row, c >> 1) + (c & 1) * 16) = y[k];
            }
        };
        auto stage_v = [&](const v4u (&v)[JB]) {
#pragma unroll
            for (int k = 0; k < JB; ++k) {
                const int q = k * kThreads + threadIdx.x, row = q / (4 * JB), j = q % (4 * JB) * 4;
                uint2 s[3];
                split3(__builtin_bit_cast(v4f, v[k]), s);
#pragma unroll
                for (int h = 0; h < 3; ++h)
                    *reinterpret_cast<uint2 *>(vs[h] + piece_at<JB>(row, j >> 4) + (j & 15) * 2) = s[h];
            }
        };
        // y times v's parts FROM .. TO - 1
        auto multiply = [&]<int FROM, int TO>() {
#pragma unroll
            for (int m0 = 0; m0 < kTileRows; m0 += 32) {
                v4u yf[NC];
#pragma unroll
                for (int c = 0; c < NC; ++c) yf[c] = read_transposed<8>(ys, m0, pc + c, lane);
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int h = FROM; h < TO; ++h) {
                        const v4u f = read_transposed<JB>(vs[h], m0, pj + j, lane);
#pragma unroll
                        for (int c = 0; c < NC; ++c)
                            acc[c][j] = RANKS_FIRST ? mfma(f, yf[c], acc[c][j]) : mfma(yf[c], f, acc[c][j]);
                    }
            }
        };
        if constexpr (FINITE) {  // seldom run: one tile in flight, for fewer registers
            for (int i = 0; i < count; ++i) {
                fetch(i, yd[0], vd[0]);
                __syncthreads();
                stage_y(yd[0]);
                stage_v(vd[0]);
                __syncthreads();
                multiply.template operator()<0, 1>();
                __syncthreads();
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int p = 0; p < 4; ++p) yd[0][k][p] = finite_halves(yd[0][k][p]);
                stage_y(yd[0]);
                __syncthreads();
                multiply.template operator()<1, 3>();
            }
        } else {
            fetch(0, yd[0], vd[0]);
            fetch(1, yd[1], vd[1]);
            for (int i = 0; i < count; i += 2) {
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    // (an odd count's last turn adds the 0 of a tile past the end)
                    __syncthreads();  // the last tile's fragments have been read
                    stage_y(yd[p]);
                    stage_v(vd[p]);
                    fetch(i + p + 2, yd[p], vd[p]);
                    __syncthreads();
                    multiply.template operator()<0, 3>();
                }
            }
        }
    }
}

// Block q of dA's or dB's: by adapter, split, columns.
template <int JB, bool RANKS_FIRST>
__device__ __forceinline__ void outer_block(const Outer &o, int q, int64_t M, int L, int R, const int32_t *ranks,
                                            const int32_t *plan, int T, int splits, char *ys,
                                            char (&vs)[3][kTileRows * 32 * JB]) {
    constexpr int NC = JB == 1 ? 2 : 4, NJ = JB == 1 ? 1 : JB / 2;
    const int col0 = q % o.groups * 128;
    q /= o.groups;
    const int split = q % splits, l = q / splits;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int pc = JB == 1 ? wave * 2 : (wave & 1) * 4, pj = JB == 1 ? 0 : (wave >> 1) * NJ;  // its first pieces
    const int r = rank_of(ranks, l, R);
    const int32_t *first = plan + 4 * (int64_t)T;
    const int t0 = T ? min(max(first[l], 0), T) : 0, t1 = T ? min(max(first[l + 1], t0), T) : 0;
    const int n = t1 - t0, begin = t0 + (int)((int64_t)n * split / splits);
    const int end = t0 + (int)((int64_t)n * (split + 1) / splits);
    v4f acc[NC][NJ];
    outer_sums<JB, RANKS_FIRST, false>(acc, o, col0, pc, pj, M, L, R, plan, begin, end, ys, vs);
    // Against an infinity of y the parts of v may give inf - inf or inf * 0 where v
    // gives an infinity: with a NaN among the results the block's sums are taken
    // again, the infinities meeting v's first part alone, which has v's sign.
    const int across = 4 * (lane >> 4), along = lane & 15;
    float any = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int b = 0; b < NJ; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int col = col0 + (pc + c) * 16 + (RANKS_FIRST ? along : across + e);
                const int j = (pj + b) * 16 + (RANKS_FIRST ? across + e : along);
                any = max_or_nan(any, col < o.C && j < r ? acc[c][b][e] : 0.f);
            }
    __syncthreads();  // every wave has read the last tile
    if (lane == 0) reinterpret_cast<int *>(ys)[wave] = 0;
    if (any != any) reinterpret_cast<int *>(ys)[wave] = 1;
    __syncthreads();
    const v4i flags = *reinterpret_cast<const v4i *>(ys);
    if (__builtin_expect((flags[0] | flags[1] | flags[2] | flags[3]) != 0, false)) {
        __syncthreads();
        outer_sums<JB, RANKS_FIRST, true>(acc, o, col0, pc, pj, M, L, R, plan, begin, end, ys, vs);
    }
    // the contiguous index of d along 16 lanes: rows of the product are ranks
    // (dA) or columns (dB)
    float *d = o.d + ((int64_t)split * L + l) * R * o.C;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int b = 0; b < NJ; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int col = col0 + (pc + c) * 16 + (RANKS_FIRST ? along : across + e);
                const int j = (pj + b) * 16 + (RANKS_FIRST ? across + e : along);
                if (col < o.C && j < R)
                    d[RANKS_FIRST ? (int64_t)j * o.C + col : (int64_t)col * R + j] = j < r ? acc[c][b][e] : 0.f;
            }
}

// Waves to a SIMD that the registers allow, with two tiles in flight.
constexpr int outer_simd_waves(int JB) { return JB == 1 ? 5 : JB == 2 ? 3 : 2; }

template <int JB>
__global__ __launch_bounds__(64 * kOuterWaves, outer_simd_waves(JB)) void lora_outer_kernel(
    OuterPair both, int64_t M, int L, int R, const int32_t *ranks, const int32_t *plan, int T, int splits, int q0) {
    __shared__ __attribute__((aligned(16))) char ys[kTileRows * 256], vs[3][kTileRows * 32 * JB];
    const int na = both.a.groups * L * splits, q = q0 + blockIdx.x;
    if (q < na) outer_block<JB, true>(both.a, q, M, L, R, ranks, plan, T, splits, ys, vs);
    else outer_block<JB, false>(both.b, q - na, M, L, R, ranks, plan, T, splits, ys, vs);
}

__global__ __launch_bounds__(256) void lora_sums_kernel(SplitSums sums) { add_splits(sums, blockIdx.x); }

// ---------------------------------------------------------------- host side
// Workgroups of a launch at most: with their threads far below HIP's 2^32.  A
// call that needs more makes several launches, each of a part of the plan's tiles.
constexpr int64_t kMaxBlocks = 1 << 20;

int rank_blocks(int64_t R) { return R <= 16 ? 1 : R <= 32 ? 2 : R <= 64 ? 4 : 8; }

// v [M, R] = scale x w^T, w [L, R, C] or, TR, [L, C, R].
template <bool TR>
void down_launch(const uint16_t *x, int64_t M, int64_t C, int64_t ldx, const uint16_t *w, int64_t L, int64_t R,
                 const float *scale, const int32_t *ranks, const int32_t *plan, int64_t T, float *v, hipStream_t stream) {
    // 16 rows a workgroup while those are no more than one to a CU, of which
    // mostly one fits a CU; else 32, which read the weights half as often
    // (C 4096, R 16 and 128: 4096 rows 14.3 and 27.5 us with 16, 14.4 and 30.2
    // with 32; 4500 rows 19.0 and 41.7, 15.7 and 32.3)
    const bool two = M > 16 * 256;
    // fewer still: the ranks in parts, since one CU takes long for a weight of
    // many (1 row, C 4096, R 128, with the up-projection: 19.2 us, 9.9 in 8 parts)
    int blocks = rank_blocks(R), parts = 1;
    if (!two)
        while (blocks > 1 && (M / 16 + T) * parts * 2 <= 256) blocks /= 2, parts *= 2;
    const int per_tile = (two ? 2 : 4) * parts;
#define W8A8_DOWN(JB, RB)                                                                                              \
    lora_down_kernel<JB, RB, TR><<<n * per_tile, 64 * down_waves(JB, RB), 0, stream>>>(                                \
        x, M, (int)C, ldx, w, (int)L, (int)R, scale, ranks, plan + 4 * t0, n, parts, v)
    for (int64_t t0 = 0; t0 < T; t0 += kMaxBlocks / per_tile) {
        const int n = (int)std::min(T - t0, kMaxBlocks / per_tile);
        switch (blocks) {
        case 1: two ? W8A8_DOWN(1, 2) : W8A8_DOWN(1, 1); break;
        case 2: two ? W8A8_DOWN(2, 2) : W8A8_DOWN(2, 1); break;
        case 4: two ? W8A8_DOWN(4, 2) : W8A8_DOWN(4, 1); break;
        default: two ? W8A8_DOWN(8, 2) : W8A8_DOWN(8, 1); break;
        }
    }
#undef W8A8_DOWN
}

template <bool TR>
void up_launch(const float *v, const uint16_t *w, int64_t M, int64_t C, int64_t L, int64_t R, const int32_t *ranks,
               const int32_t *plan, int64_t T, const uint16_t *base, int64_t ldbase, uint16_t *out, int64_t ldout,
               const SplitSums &sums, hipStream_t stream) {
    const int groups = (int)((C + 128 * kUpWaves - 1) / (128 * kUpWaves));
    // 64 rows a workgroup use the weights' fragments most often; 32 where that
    // would leave less than two workgroups to a CU (300 rows, K 2048, N 5120, R
    // 32, both launches: 9.3 us against 10.5)
    const bool half = T * groups < 512;
    const int per_tile = groups * (half ? 2 : 1);
    const int64_t most = std::max<int64_t>(kMaxBlocks / per_tile, 1);
#define W8A8_UP(JB, RB)                                                                                             \
    lora_up_kernel<JB, TR, RB><<<n * per_tile + part.blocks, 64 * kUpWaves, 0, stream>>>(                           \
        v, w, M, (int)C, (int)L, (int)R, ranks, plan + 4 * t0, groups, base, ldbase, out, ldout, part)
    for (int64_t t0 = 0; t0 < T; t0 += most) {
        const int n = (int)std::min(T - t0, most);
        const SplitSums part = t0 == 0 ? sums : SplitSums{};
        switch (rank_blocks(R)) {
        case 1: half ? W8A8_UP(1, 2) : W8A8_UP(1, 4); break;
        case 2: half ? W8A8_UP(2, 2) : W8A8_UP(2, 4); break;
        case 4: half ? W8A8_UP(4, 2) : W8A8_UP(4, 4); break;
        default: half ? W8A8_UP(8, 2) : W8A8_UP(8, 4); break;
        }
    }
#undef W8A8_UP
}

// Whether the down- and the up-projection go in one launch: where a workgroup
// of it for each CU is enough (its registers leave room for one), and the sums
// that each of a block's workgroups repeats do not add up.  K = 4096, R = 16,
// one launch against two: 1 token and 4096 columns 7.2 us against 7.8, 48
// requests of one 7.6 against 8.6, 1531 tokens and 2048 columns 8.5 against
// 11.5; but 4096 tokens 34 against 21, 48 requests and 12288 columns 16.7
// against 10.5.  Ranks past 16 do not fit the registers beside what is loaded
// ahead (32: 12.8 against 9.2 for 1 token).
bool one_launch(int64_t M, int64_t T, int64_t C2, int64_t R) {
    const int64_t groups = (C2 + 2047) / 2048, blocks = (M / 16 + T) * groups;
    return R <= 16 && blocks <= 256 && blocks * groups <= 512;
}
// out = base + (scale x w^T) w2^T; v [M, R] = scale x w^T is left where it is not null.
template <bool TR>
void both_launch(const uint16_t *x, int64_t M, int64_t C, int64_t ldx, const uint16_t *w, int64_t L, int64_t R,
                 const float *scale, const int32_t *ranks, const int32_t *plan, int64_t T, float *v, const uint16_t *w2,
                 int64_t C2, const uint16_t *base, int64_t ldbase, uint16_t *out, int64_t ldout, hipStream_t stream) {
    const int groups = (int)((C2 + 2047) / 2048);
    lora_both_kernel<TR><<<(int)(4 * T * groups), 1024, 0, stream>>>(x, M, (int)C, ldx, w, (int)L, (int)R, scale, ranks,
                                                                     plan, (int)T, v, w2, (int)C2, groups, base, ldbase,
                                                                     out, ldout);
}

// Over how many workgroups an adapter's rows are split: two workgroups for each
// CU, which overlap each other's loads, products and barriers, and no more,
// since each split's sums are written and read again.  Both gradients, with
// the down-projection, M 8192, K = N 4096, 1, 4, 8, 16 splits: R 32 116, 50,
// 51, 52 us; R 64 173, 68, 64, 73 us.  2039 rows of 4 adapters, K 4096, N 1024,
// R 16, the sums' kernel alone: 15.6 us with 1 split, 11.0 with 3.
int64_t outer_splits(int64_t T, int64_t K, int64_t N, int64_t L) {
    const int64_t one = ((K + 127) / 128 + (N + 127) / 128) * L, most = T / (2 * L);
    const int64_t s = 512 / one;
    return s < most ? (s < 1 ? 1 : s) : most < 1 ? 1 : most;
}

constexpr int64_t kMaxWidth = 1 << 22;

bool bad_width(int64_t w) { return w < 8 || w % 8 != 0 || w > kMaxWidth; }
bool bad_stride(int64_t ld, int64_t w) { return ld < w || ld % 8 != 0 || ld > kMaxWidth; }

w8a8_status lora_check(int64_t M, int64_t K, int64_t N, int64_t R, int64_t L, int64_t T, const uint16_t *a,
                       const uint16_t *b, const float *scale, const int32_t *ranks, const int32_t *plan) {
    if (M < 0 || T < 0 || L < 1 || R < 8 || R > kMaxR) return W8A8_ERR_INVALID_ARG;
    if (R % 8 != 0 || bad_width(K) || bad_width(N) || L > kMaxL || M > (1 << 30) || T > (1 << 24) ||
        T * ((K > N ? K : N) / 512 + 1) > INT32_MAX)
        return W8A8_ERR_SHAPE;
    if (!a || !b || !plan) return W8A8_ERR_INVALID_ARG;
    if (!aligned16(a) || !aligned16(b) || !aligned16(scale) || !aligned16(ranks) || !aligned16(plan))
        return W8A8_ERR_ALIGN;
    return W8A8_OK;
}

}  // namespace
}  // namespace w8a8

extern "C" w8a8_status lora_plan(const int64_t *lengths, const int32_t *adapters, int64_t S, int64_t L, int32_t *plan,
                                 int64_t capacity, int64_t *tiles) {
    using namespace w8a8;
    if (S < 0 || (S > 0 && (!lengths || !adapters)) || !tiles) return W8A8_ERR_INVALID_ARG;
    if (L < 1 || L > kMaxL) return W8A8_ERR_SHAPE;
    int64_t M = 0, T = 0;
    for (int64_t s = 0; s < S; ++s) {
        if (lengths[s] < 0 || adapters[s] < -1 || adapters[s] >= L) return W8A8_ERR_INVALID_ARG;
        if (lengths[s] > (1 << 30) - M) return W8A8_ERR_SHAPE;
        M += lengths[s];
        T += (lengths[s] + kTileRows - 1) / kTileRows;
    }
    if (T > (1 << 24)) return W8A8_ERR_SHAPE;
    *tiles = T;
    if (!plan) return W8A8_OK;
    if (capacity < 4 * T + L + 1) return W8A8_ERR_SHAPE;
    // counting sort by adapter: first[l] becomes the end of adapter l - 1's
    // tiles, then runs to l's own end while they are placed in row order
    int32_t *first = plan + 4 * T;
    for (int64_t l = 0; l <= L; ++l) first[l] = 0;
    int64_t none = 0;
    for (int64_t s = 0; s < S; ++s) {
        const int64_t n = (lengths[s] + kTileRows - 1) / kTileRows;
        if (adapters[s] < 0) none += n;
        else first[adapters[s] + 1] += (int32_t)n;
    }
    first[0] = (int32_t)none;
    for (int64_t l = 0; l < L; ++l) first[l + 1] += first[l];
    int64_t row = 0, at_none = 0;
    for (int64_t s = 0; s < S; ++s) {
        for (int64_t i = 0; i < lengths[s]; i += kTileRows) {
            const int64_t t = adapters[s] < 0 ? at_none++ : first[adapters[s]]++;
            plan[4 * t] = (int32_t)(row + i);
            plan[4 * t + 1] = (int32_t)(lengths[s] - i < kTileRows ? lengths[s] - i : kTileRows);
            plan[4 * t + 2] = adapters[s];
            plan[4 * t + 3] = 0;
        }
        row += lengths[s];
    }
    for (int64_t l = L; l > 0; --l) first[l] = first[l - 1];  // each had run to its own end
    first[0] = (int32_t)none;
    return W8A8_OK;
}

extern "C" size_t lora_forward_workspace_bytes(int64_t M, int64_t R) {
    if (M < 0 || R < 8 || R > w8a8::kMaxR) return 0;
    return (size_t)(M * R) * sizeof(float);
}

extern "C" w8a8_status lora_forward(const uint16_t *x, int64_t M, int64_t K, int64_t ldx, const uint16_t *a,
                                    const uint16_t *b, int64_t L, int64_t N, int64_t R, const float *scale,
                                    const int32_t *ranks, const int32_t *plan, int64_t T, const uint16_t *base,
                                    int64_t ldbase, uint16_t *out, int64_t ldout, float *u, void *workspace,
                                    hipStream_t stream) {
    using namespace w8a8;
    if (M == 0 || T == 0) return M < 0 || T < 0 ? W8A8_ERR_INVALID_ARG : W8A8_OK;
    const w8a8_status st = lora_check(M, K, N, R, L, T, a, b, scale, ranks, plan);
    if (st != W8A8_OK) return st;
    if (bad_stride(ldx, K) || bad_stride(ldout, N) || (base && bad_stride(ldbase, N))) return W8A8_ERR_SHAPE;
    if (!x || !out || (!u && !workspace)) return W8A8_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(base) || !aligned16(out) || !aligned16(u) || !aligned16(workspace))
        return W8A8_ERR_ALIGN;
    float *v = u ? u : static_cast<float *>(workspace);
    if (one_launch(M, T, N, R)) {
        both_launch<false>(x, M, K, ldx, a, L, R, scale, ranks, plan, T, v, b, N, base, ldbase, out, ldout, stream);
    } else {
        down_launch<false>(x, M, K, ldx, a, L, R, scale, ranks, plan, T, v, stream);
        up_launch<false>(v, b, M, N, L, R, ranks, plan, T, base, ldbase, out, ldout, SplitSums{}, stream);
    }
    return launch_status();
}

extern "C" size_t lora_backward_workspace_bytes(int64_t M, int64_t T, int64_t K, int64_t N, int64_t R, int64_t L) {
    using namespace w8a8;
    if (M < 0 || T < 0 || K < 8 || N < 8 || L < 1 || R < 8 || R > kMaxR) return 0;
    const int64_t splits = outer_splits(T, K, N, L);
    return (size_t)(M * R + (splits > 1 ? splits * L * R * (K + N) : 0)) * sizeof(float);
}

extern "C" w8a8_status lora_backward(const uint16_t *dy, int64_t M, int64_t N, int64_t lddy, const uint16_t *x,
                                     int64_t K, int64_t ldx, const float *u, const uint16_t *a, const uint16_t *b,
                                     int64_t L, int64_t R, const float *scale, const int32_t *ranks,
                                     const int32_t *plan, int64_t T, const uint16_t *base, int64_t ldbase,
                                     uint16_t *dx, int64_t lddx, float *da, float *db, void *workspace,
                                     hipStream_t stream) {
    using namespace w8a8;
    const w8a8_status st = lora_check(M, K, N, R, L, T, a, b, scale, ranks, plan);
    if (st != W8A8_OK) return st;
    if (bad_stride(ldx, K) || bad_stride(lddy, N) || (dx && bad_stride(lddx, K)) || (base && bad_stride(ldbase, K)))
        return W8A8_ERR_SHAPE;
    if (M == 0) T = 0;
    if (T > 0 && (!dy || (da && !x) || (db && !u) || !workspace)) return W8A8_ERR_INVALID_ARG;
    if ((da == nullptr) != (db == nullptr)) return W8A8_ERR_INVALID_ARG;
    if (!aligned16(dy) || !aligned16(x) || !aligned16(u) || !aligned16(base) || !aligned16(dx) || !aligned16(da) ||
        !aligned16(db) || !aligned16(workspace))
        return W8A8_ERR_ALIGN;
    float *g = static_cast<float *>(workspace), *parts = g + M * R;
    const int64_t splits = outer_splits(T, K, N, L), na = L * R * K, nb = L * R * N;
    const int ga = (int)((K + 127) / 128), gb = (int)((N + 127) / 128);
    const int64_t grid = (ga + gb) * L * splits;
    if (da && (grid > INT32_MAX || (na + nb) / 1024 >= INT32_MAX / 2)) return W8A8_ERR_SHAPE;
    SplitSums sums = {};
    if (da && splits > 1) {
        sums = {parts, parts + splits * na, da, db, na, nb, (int)splits, (int)(((na + nb) / 4 + 255) / 256)};
        if (sums.blocks + T * ((K + 511) / 512) > INT32_MAX) return W8A8_ERR_SHAPE;
    }
    // dx in one launch with g where that fits; else after the outer sums, whose
    // splits its launch adds up
    const bool one = T > 0 && dx && one_launch(M, T, K, R);
    if (one) both_launch<true>(dy, M, N, lddy, b, L, R, scale, ranks, plan, T, g, a, K, base, ldbase, dx, lddx, stream);
    else if (T > 0) down_launch<true>(dy, M, N, lddy, b, L, R, scale, ranks, plan, T, g, stream);
    if (da) {
        const OuterPair both = {{x, ldx, g, splits > 1 ? parts : da, (int)K, ga},
                                {dy, lddy, u, splits > 1 ? parts + splits * na : db, (int)N, gb}};
#define W8A8_OUTER(JB)                                                                                       \
    lora_outer_kernel<JB><<<n, 64 * kOuterWaves, 0, stream>>>(both, M, (int)L, (int)R, ranks, plan, (int)T,  \
                                                              (int)splits, (int)q0)
        for (int64_t q0 = 0; q0 < grid; q0 += kMaxBlocks) {
            const int n = (int)std::min(grid - q0, kMaxBlocks);
            switch (rank_blocks(R)) {
            case 1: W8A8_OUTER(1); break;
            case 2: W8A8_OUTER(2); break;
            case 4: W8A8_OUTER(4); break;
            default: W8A8_OUTER(8); break;
            }
        }
#undef W8A8_OUTER
    }
    if (T > 0 && dx && !one)
        up_launch<true>(g, a, M, K, L, R, ranks, plan, T, base, ldbase, dx, lddx, sums, stream);
    else if (sums.blocks > 0)
        lora_sums_kernel<<<sums.blocks, 256, 0, stream>>>(sums);
    return launch_status();
}
