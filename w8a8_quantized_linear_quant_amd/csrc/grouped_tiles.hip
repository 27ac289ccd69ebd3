// grouped_tiles.hip -- products of groups with many rows each: square output
// tiles, both operands staged in LDS, bound by the matrix cores and the power
// they draw or, for the smaller tile, by the latency of loads that miss L2 (8192
// x 12288 x 4096, 256 x 256: 4-bit 201 .. 220 us, 3.8 .. 4.1 PFLOP/s; int8 307 ..
// 330, 2.5 .. 2.7 POPS; e4m3 295 .. 305.  2048 x 4096 x 4096 in 4 bits, 128 x 128:
// 26 us, 2.6 PFLOP/s).
//
//  * Persistent: workgroups walk the tiles of all groups.  Which tiles there
//    are lies on the device (offsets), so each workgroup counts them itself,
//    64 groups at a time in the lanes of a wave.  Tiles are numbered so that
//    an XCD's workgroups share operand panels in its L2.
//  * 4 waves in a 2 x 2 grid, each WT x WT outputs: WT = 128 (256 accumulators
//    a lane, one workgroup a CU) or 64 (two workgroups a CU).  int8: blocks of
//    16 x 16 (v_mfma_i32_16x16x64_i8); e4m3 and the 4-bit format: blocks of
//    32 x 32 (v_mfma_scale_f32_32x32x64_f8f6f4).  The weight is the
//    instruction's first operand, so that a lane ends up with four consecutive
//    columns of one row.
//    (e4m3: eight neighbouring products are cut off 13 bits below the leading bit
//    of the greatest before they are added, by every instruction for e4m3.)
//  * Codes go from memory to LDS without registers, 128 bytes of every row a
//    stage, in a ring of two, or of four for 128 x 128 tiles where one a CU or
//    fewer are left (512 rows, N = K 4096: int8 24.4 us with two, 19.9 with four);
//    16-byte chunks are XOR-swizzled by row.  The ring runs ahead across tiles.
//    Gathered rows are a lane's own offset into x; their indices are loaded a
//    tile ahead, one a lane.
//  * 4-bit format: a stage is 256 values of K, 8 scales a row.  Lane half h of
//    a 32 x 32 x 64 product takes block 4 h + s of them at step s -- which
//    block goes with which step is free as long as both operands agree -- so
//    that the four scales a lane needs in a stage are one aligned word, and the
//    instruction's operand selector takes byte s.  Scales are staged for two
//    stages at a time, 16 bytes a row.
//  * Steps are laid out by hand: a step's fragment reads and loads are spread
//    over the products of the step before, the products being inline assembly
//    with tied accumulators (as builtins the compiler moves them together and
//    rotates the accumulators through copies).
#include <type_traits>
#include <utility>

#include "grouped.hpp"

namespace w8a8 {
namespace {

constexpr int kThreads = 256;
constexpr int kStageK = 128;  // bytes of a row a stage
constexpr int kXcds = 8;
constexpr int kTilesTogether = 4;  // row tiles that advance together along N

typedef __attribute__((address_space(3))) void *lds_ptr_t;

// s_waitcnt: at most n vector memory operations in flight; no LDS operation
constexpr int wait_vm(int n) { return (n & 15) | ((n >> 4) << 14) | (7 << 4) | (15 << 8); }
constexpr int kWaitVm0 = wait_vm(0);
constexpr int kWaitLgkm0 = 15 | (3 << 14) | (7 << 4);

// Which 16-byte chunk of a row's stage lies where: chunk c at c ^ swizzle(row).  Fragment reads of 16 or 32 rows, a
// chunk each, run at LDS's full rate with this one, 3.7 ns for a wave's 1 KB; with row & 7, or its exclusive or with
// row >> 3 & 1, 4.6 for one type or the other.
__device__ __forceinline__ int swizzle(int row) { return ((row >> 1) & 7) ^ (row & 1); }
constexpr int share_first(int g, int total, int groups) { return g * total / groups; }
constexpr int share_count(int g, int total, int groups) { return (g + 1) * total / groups - g * total / groups; }

// Number t of `tiles_m` x `tiles_n` tiles: each XCD (workgroup i runs on XCD
// i % 8) a contiguous range, kTilesTogether rows of tiles along N.
__device__ __forceinline__ void tile_at(int t, int tiles_m, int tiles_n, int &tm, int &tn) {
    const int total = tiles_m * tiles_n, per = total / kXcds;
    if (t < per * kXcds) t = (t % kXcds) * per + t / kXcds;
    const int group = kTilesTogether * tiles_n;
    const int g = t / group, first = g * kTilesTogether, together = min(tiles_m - first, kTilesTogether);
    const int in = t - g * group;
    tm = first + in % together;
    tn = in / together;
}

// An accumulator as a float.  As assembly, so that it is read where it is
// used: left alone, the compiler copies all 256 to ordinary registers at the
// loop's end and spills what the loop holds.
__device__ __forceinline__ float from_accumulator(float a) {
    float v;
    asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v) : "a"(a));
    return v;
}
__device__ __forceinline__ float from_accumulator(int a) {
    int v;
    asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v) : "a"(a));
    return (float)v;
}
// 8 values to a row that has `left` columns from dst on, at the alignment of one (rows of any N start anywhere).
__device__ __forceinline__ void store_row(uint16_t *dst, v4u d, int left) {
    if (left >= 8) {
        Bf16::store_chunk(dst, d);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) dst[i] = (uint16_t)(d[i >> 1] >> ((i & 1) * 16));
    }
}
// A buffer of a few bytes: reads past them are 0.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t small_rsrc(const void *p, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc((void *)p, (short)0, bytes, kBufferRsrcWord3);
}
// n clamped to [0, most], as scalars do it (as max and min it becomes v_med3, and descriptors vectors)
__device__ __forceinline__ int some(int n, int most) { return n <= 0 ? 0 : n < most ? n : most; }
__device__ __forceinline__ int load_i32(__amdgpu_buffer_rsrc_t r, int off) {
    return (int)__builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0);
}

// Of `all` tiles in rounds of `slots` workgroups, those of whole rounds if at
// most half a round would be left, else all.
__device__ __forceinline__ int kept_tiles(int all, int slots) {
    const int whole = all / slots * slots, rest = all - whole;
    return whole > 0 && 2 * rest <= slots ? whole : all;
}

// REST: the tiles of 256 that a launch of that size leaves, in quarters.
// `split`: in that launch, whether it leaves them (kept_tiles).
template <int QT, int WT, int NST, bool TAIL, bool REST>
__global__ __launch_bounds__(kThreads, WT == 64 && NST == 2 ? 2 : 1) void grouped_tiles_kernel(GroupedArgs p, int tiles_n,
                                                                                             int split) {
    static_assert(!REST || WT == 64, "quarters of 256 x 256 tiles");
    constexpr bool kInt8 = QT == kTypeInt8, kMx = QT == kTypeMx4;
    constexpr int BT = 2 * WT;                      // tile edge
    constexpr int CT = REST ? 2 * BT : BT;          // edge of the tiles that are counted
    constexpr int kOpBytes = BT * kStageK;          // one operand's stage
    constexpr int kRowsWave = BT / 4;               // rows of each operand that a wave loads
    constexpr int kLoadsOp = kRowsWave / 8;         // 8 rows an instruction
    constexpr int kLoads = 2 * kLoadsOp;
    constexpr int kSlabBytes = 2 * BT * 16;         // scales of both operands for two stages
    constexpr int kSlabLoads = 2 * BT / 64 / 4;     // a wave's share, 64 rows an instruction
    constexpr int kPassCols = WT == 128 ? 64 : 32;  // the epilogue's columns at a time, of 32 rows
    constexpr int kPassBytes = 32 * kPassCols * 2;
    __shared__ __attribute__((aligned(1024))) uint8_t lds0[2 * kOpBytes];
    __shared__ __attribute__((aligned(1024))) uint8_t lds1[2 * kOpBytes];
    __shared__ __attribute__((aligned(1024))) uint8_t lds2[NST == 4 ? 2 * kOpBytes : 16];
    __shared__ __attribute__((aligned(1024))) uint8_t lds3[NST == 4 ? 2 * kOpBytes : 16];
    __shared__ __attribute__((aligned(1024))) uint8_t slab0[kMx ? kSlabBytes : 16];
    __shared__ __attribute__((aligned(1024))) uint8_t slab1[kMx ? kSlabBytes : 16];
    __shared__ __attribute__((aligned(1024))) uint8_t obuf[4 * kPassBytes];
    constexpr int kEpBytes = 3 * WT * 4;
    __shared__ __attribute__((aligned(16))) uint8_t epbuf[kMx ? 16 : 4 * kEpBytes];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const int kb = p.kb, M = p.M, N = p.N;
    const bool gather = p.rows != nullptr;
    static_assert(NST == 2 || NST == 4, "stages in the ring");
    // stages of a tile: whole turns of the ring, so that every tile starts in the same buffer (those past K read zeros)
    const int stages = (kb + NST * kStageK - 1) / (NST * kStageK) * NST;

    GroupWindow win = {};
    load_window<CT>(win, p.offsets, p.E, M, lane);
    int tiles_m;
    {
        GroupWindow w = win;
        while (w.base + 64 < p.E) next_window<CT>(w, p.offsets, p.E, M, lane);
        tiles_m = __builtin_amdgcn_readlane(w.tiles, 63);
    }
    // this launch's tiles: numbers first .. first + total - 1 (REST: four quarters each)
    const int all = tiles_m * tiles_n, kept = split ? kept_tiles(all, split) : all;
    const int first = REST ? kept : 0, total = REST ? 4 * (all - kept) : kept;
    if ((int)blockIdx.x >= total) return;

    struct Tile {
        int group, m0, end, n0;
    };
    auto tile_of = [&](int t) __attribute__((always_inline)) {
        Tile c = {0, 0, 0, 0};
        if (t >= total) return c;
        int tm, tn;
        tile_at(REST ? first + t / 4 : t, tiles_m, tiles_n, tm, tn);
        if (tm < win.before) {
            win = GroupWindow{};
            load_window<CT>(win, p.offsets, p.E, M, lane);
        }
        const GroupTile g = find_tile<CT>(win, tm, p.offsets, p.E, M, lane);
        c.group = __builtin_amdgcn_readfirstlane(g.group);
        c.m0 = __builtin_amdgcn_readfirstlane(g.m0);
        c.end = __builtin_amdgcn_readfirstlane(g.end);
        c.n0 = __builtin_amdgcn_readfirstlane(tn * CT);
        if constexpr (REST) {
            // a quarter may lie past the group's rows or past N: nothing to do there
            c.m0 += (t & 2) ? BT : 0;
            c.n0 += (t & 1) ? BT : 0;
            if (c.m0 >= c.end || c.n0 >= N) c.end = c.m0 = 0;
            if (c.n0 >= N) c.n0 = 0;
        }
        return c;
    };

    // ---- loads.  Lane l of instruction i brings row 8 i + l / 8 of the wave's
    // rows, physical chunk l % 8; the instruction's immediate offset (i % 4 KB)
    // counts for the global address too and is taken back out of the lane's.
    int goff[kLoads];
    const int lrow8 = lane / 8;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
        const int i = j % kLoadsOp, row = wave * kRowsWave + i * 8 + lrow8;
        goff[j] = row * kb + (((lane & 7) ^ swizzle(row)) << 4) - (i & 3) * 1024;
    }
    // column of the lane's chunk: the swizzle is that of row % 16, so two cases
    const int gcol0 = ((lane & 7) ^ swizzle(lrow8)) << 4, gcol1 = ((lane & 7) ^ swizzle(8 + lrow8)) << 4;

    // the cursor: stage ld_kt of the tile ld_tile; `ahead` is the tile after it, ahead_row the lane's row of x in it
    int ld_tile = blockIdx.x, ld_kt = 0;
    Tile before, loading, ahead;  // the tiles before the cursor's, the cursor's own, after it
    int ahead_row = 0, ahead_srow = 0;
    __amdgpu_buffer_rsrc_t rx, rw, rxs, rws;
    // 4-bit format: scales of 64 rows an instruction.  Tiles of 256: each wave's own 64 rows of x, then of the
    // weight (two instructions); tiles of 128: waves 0 and 1 rows of x, 2 and 3 of the weight.
    int sgoff[kMx ? kSlabLoads : 1];
    auto slab_first = [&](int i) { return kSlabLoads == 2 ? i * BT + wave * 64 : wave * 64; };
    // The lane's row of x in a tile, loaded (lr) or scaled (sr) by this lane; -1: none.  (Buffer loads, here and for the
    // epilogue's inputs, instead of branches on the lane: what is uniform stays so for the compiler.)
    auto rows_of = [&](const Tile &c, int &lr, int &sr) __attribute__((always_inline)) {
        const int n = c.end - c.m0, i = wave * kRowsWave + lane;
        const __amdgpu_buffer_rsrc_t r = small_rsrc(p.rows + c.m0, min(n, BT) * 4);
        const int v = load_i32(r, i * 4);
        lr = lane < kRowsWave && i < n ? v : -1;
        if constexpr (kMx) {
            sr = lr;
            if constexpr (kSlabLoads == 1) {
                const int is = wave * 64 + lane, u = load_i32(r, is * 4);
                sr = wave < 2 && is < n ? u : -1;
            }
        }
    };
    auto look_ahead = [&]() __attribute__((always_inline)) {
        ahead = tile_of(ld_tile + gridDim.x);
        if (gather) rows_of(ahead, ahead_row, ahead_srow);
    };
    auto enter_tile = [&](const Tile &c, int row_index, int scale_index) __attribute__((always_inline)) {
        before = loading;
        loading = c;
        const int rows_w = min(N - c.n0, BT);
        const bool any = c.end > c.m0;
        const size_t w0 = (size_t)c.group * N + c.n0;
        const int rows_x = !any ? 0 : gather ? (int)p.X : min(c.end - c.m0, BT);
        const size_t x0 = gather ? 0 : c.m0;
        rx = __builtin_amdgcn_make_buffer_rsrc((void *)(p.xq + x0 * kb), (short)0, (int)((int64_t)rows_x * kb),
                                               kBufferRsrcWord3);
        rw = __builtin_amdgcn_make_buffer_rsrc((void *)(p.wq + w0 * kb), (short)0, any ? rows_w * kb : 0,
                                               kBufferRsrcWord3);
        if constexpr (kMx) {
            rxs = __builtin_amdgcn_make_buffer_rsrc((void *)(p.xs + x0 * p.stride), (short)0,
                                                    (int)((int64_t)rows_x * p.stride), kBufferRsrcWord3);
            rws = __builtin_amdgcn_make_buffer_rsrc((void *)(p.ws + w0 * p.stride), (short)0, any ? rows_w * p.stride : 0,
                                                    kBufferRsrcWord3);
        }
        if (gather) {
#pragma unroll
            for (int i = 0; i < kLoadsOp; ++i) {
                const int s = __builtin_amdgcn_ds_bpermute((i * 8 + lrow8) * 4, row_index);
                const bool ok = s >= 0 && s < rows_x;
                goff[i] = ok ? (int)((uint32_t)s * kb + ((i & 1) ? gcol1 : gcol0) - (i & 3) * 1024) : kOobOffset;
            }
        }
        if constexpr (kMx) {
#pragma unroll
            for (int i = 0; i < kSlabLoads; ++i) {
                const int r = slab_first(i) + lane;
                int s = r & (BT - 1);
                if (gather && r < BT) s = scale_index < rows_x ? scale_index : -1;
                sgoff[i] = s < 0 ? kOobOffset : (int)((uint32_t)s * p.stride);
            }
        }
    };
    auto load_one = [&](uint8_t *stage, auto jc) __attribute__((always_inline)) {
        constexpr int j = decltype(jc)::value;
        constexpr bool kX = j < kLoadsOp;
        constexpr int i = j % kLoadsOp, imm = (i & 3) * 1024;
        uint8_t *dst = stage + (kX ? 0 : kOpBytes) + wave * kRowsWave * kStageK + (i / 4) * 4096;
        const int k0 = ld_kt * kStageK;
        int o = goff[j] + k0;
        if constexpr (TAIL) {
            if (k0 + ((i & 1) ? gcol1 : gcol0) >= kb) o = kOobOffset;
        }
        __builtin_amdgcn_raw_ptr_buffer_load_lds(kX ? rx : rw, (lds_ptr_t)dst, 16, o, 0, imm, 0);
    };
    // the scales of this stage and the next
    auto load_slab = [&](uint8_t *slab) __attribute__((always_inline)) {
        if constexpr (kMx) {
#pragma unroll
            for (int i = 0; i < kSlabLoads; ++i) {
                const int r = slab_first(i);
                int o = sgoff[i] + ld_kt * 8;
                if (TAIL && ld_kt * 8 >= p.stride) o = kOobOffset;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(r < BT ? rxs : rws, (lds_ptr_t)(slab + r * 16), 16, o, 0, 0, 0);
            }
        }
    };
    auto advance = [&]() __attribute__((always_inline)) {
        if (++ld_kt == stages) {
            ld_kt = 0;
            ld_tile += gridDim.x;
            enter_tile(ahead, ahead_row, ahead_srow);
            look_ahead();
        }
    };

    // ---- fragments and products
    constexpr int kBlk = kInt8 ? 16 : 32;
    constexpr int kNB = WT / kBlk;
    constexpr int kQuads = kBlk * kBlk / 64 / 4;      // groups of 4 consecutive columns a lane has of a block
    constexpr int KSTEPS = kMx ? 4 : 2;
    constexpr int kRegs = kInt8 || kMx ? 1 : 2;       // 16-byte reads a fragment
    typedef typename std::conditional<kRegs == 1, v4i, v8i>::type frag_t;
    typedef typename std::conditional<kInt8, v4i, v16f>::type acc_t;
    acc_t acc[kNB][kNB];                              // [weight block][row block]
    frag_t fa[2][kNB], fb[2][kNB];
    int sa[2][kMx ? kNB : 1], sb[2][kMx ? kNB : 1];   // a stage's scale words of each block's rows
    const int frow = lane & (kBlk - 1), fq = lane / kBlk;  // the lane's row of a block, its part of the step's K
    // byte offset of the lane's 16-byte read h of step kk
    auto foff = [&](int kk, int h) {
        const int chunk = kInt8 ? kk * 4 + fq : kMx ? fq * 4 + kk : kk * 4 + fq * 2 + h;
        return frow * kStageK + ((chunk ^ swizzle(frow)) << 4);
    };
    constexpr int kReads = 2 * kNB * kRegs;
    auto read_one = [&](const uint8_t *lp0, const uint8_t *lp1, auto idx, frag_t *af, frag_t *bf) __attribute__((always_inline)) {
        constexpr int I = decltype(idx)::value, f = I / kRegs, h = I % kRegs;
        const uint8_t *lp = h ? lp1 : lp0;
        const v4i v = f < kNB ? *reinterpret_cast<const v4i *>(lp + kOpBytes + (wn * WT + (f % kNB) * kBlk) * kStageK)
                              : *reinterpret_cast<const v4i *>(lp + (wm * WT + (f % kNB) * kBlk) * kStageK);
        frag_t &dst = f < kNB ? af[f % kNB] : bf[f % kNB];
#pragma unroll
        for (int e = 0; e < 4; ++e) dst[4 * h + e] = v[e];
    };
    // scale word of block f (weight blocks first) for a stage of that parity
    auto read_scale = [&](const uint8_t *lp, auto idx, int *wa, int *wb) __attribute__((always_inline)) {
        constexpr int f = decltype(idx)::value;
        if constexpr (kMx) {
            if constexpr (f < kNB) wa[f] = *reinterpret_cast<const int *>(lp + (BT + wn * WT + f * 32) * 16);
            else wb[f - kNB] = *reinterpret_cast<const int *>(lp + (wm * WT + (f - kNB) * 32) * 16);
        }
    };
    if constexpr (!kMx) {
        // e4m3: the scale 1.  Opaque: its register is written here and not again next to a product, which as assembly
        // would not wait for that (nor does anything but the reads above write the other operands).
        int unit = 127;
        asm volatile("" : "+v"(unit));
        sa[0][0] = sa[1][0] = unit;
    }
    auto product = [&](acc_t &c, const frag_t &a, const frag_t &b, int wa, int wb, auto step, auto first) __attribute__((always_inline)) {
        // (the host's pass knows no 32-byte register operands, and would drop the kernel's launch stub without a word)
#ifdef __HIP_DEVICE_COMPILE__
        constexpr int s = decltype(step)::value;
        constexpr bool kFirst = decltype(first)::value;
        if constexpr (kInt8) {
            if constexpr (kFirst) asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, 0" : "=a"(c) : "v"(a), "v"(b));
            else asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
        } else if constexpr (!kMx) {
            if constexpr (kFirst)
                asm volatile("v_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, 0, %3, %3 op_sel_hi:[0,0,0]"
                             : "=a"(c) : "v"(a), "v"(b), "v"(wa));
            else
                asm volatile("v_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %3 op_sel_hi:[0,0,0]"
                             : "+a"(c) : "v"(a), "v"(b), "v"(wa));
        } else if constexpr (kFirst) {
            static_assert(!kFirst || s == 0, "a tile starts with step 0");
            asm volatile("v_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, 0, %3, %4 op_sel_hi:[0,0,0] cbsz:4 blgp:4"
                         : "=a"(c) : "v"(a), "v"(b), "v"(wa), "v"(wb));
        } else if constexpr (s == 0) {
            asm volatile("v_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel_hi:[0,0,0] cbsz:4 blgp:4"
                         : "+a"(c) : "v"(a), "v"(b), "v"(wa), "v"(wb));
        } else if constexpr (s == 1) {
            asm volatile("v_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[1,1,0] op_sel_hi:[0,0,0] cbsz:4 blgp:4"
                         : "+a"(c) : "v"(a), "v"(b), "v"(wa), "v"(wb));
        } else if constexpr (s == 2) {
            asm volatile("v_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel_hi:[1,1,0] cbsz:4 blgp:4"
                         : "+a"(c) : "v"(a), "v"(b), "v"(wa), "v"(wb));
        } else {
            asm volatile("v_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[1,1,0] op_sel_hi:[1,1,0] cbsz:4 blgp:4"
                         : "+a"(c) : "v"(a), "v"(b), "v"(wa), "v"(wb));
        }
#endif
    };
    auto buffer = [&](auto s) __attribute__((always_inline)) -> uint8_t * {
        constexpr int S = decltype(s)::value;
        if constexpr (S == 0) return lds0;
        else if constexpr (S == 1) return lds1;
        else if constexpr (S == 2) return lds2;
        else return lds3;
    };

    // Stage S of a turn.  While a step is multiplied, the next one's fragments
    // are read.  Before the stage's last step: the next stage has landed, and
    // every wave has read the last of this one (barrier).  Loads: with two
    // stages this buffer takes the stage two ahead, in its last step; with four
    // the buffer of the stage before takes the stage three ahead, in every step.
    // Scales.  Two stages: slab_cur holds this turn's, slab_next the next one's,
    // and they change places.  Four: slab0 holds those of stages 0 and 1, slab1
    // of 2 and 3, each loaded again for the next turn after the stage (1, 3)
    // during whose last step no wave reads it any more.
    constexpr int kPart = NST == 2 ? kLoads : kLoads / KSTEPS;  // loads of a step that has any
    // loads in flight that may be newer than the next stage's
    constexpr int kNewer = NST == 2 ? 0 : kLoads + (KSTEPS - 1) * kPart;
    static_assert(kLoads % KSTEPS == 0, "loads split evenly over a stage's steps");
    auto run_stage = [&](auto sc, auto first_c, const uint8_t *slab_cur, uint8_t *slab_next, int kt) __attribute__((always_inline)) {
        constexpr int S = decltype(sc)::value;
        constexpr bool FIRST = decltype(first_c)::value;
        uint8_t *cur = buffer(sc), *nxt = buffer(std::integral_constant<int, (S + 1) % NST>{});
        uint8_t *refill = NST == 2 ? cur : buffer(std::integral_constant<int, (S + 3) % NST>{});
        constexpr int Q = S & 1;  // which of the two sets of scale words
        if constexpr (kMx && TAIL) {
            // bytes past the row's scales count as 2^-127 (their codes are 0, but 0 times NaN is not)
            const int have = min(max(kb / 16 - kt * 8 - fq * 4, 0), 4);
            const int keep = have == 4 ? -1 : (1 << (8 * have)) - 1;
#pragma unroll
            for (int b = 0; b < kNB; ++b) {
                sa[Q][b] &= keep;
                sb[Q][b] &= keep;
            }
            asm volatile("s_nop 4" ::: "memory");  // the products are assembly: their wait for these words is this one
        }
        [&]<int... KK>(std::integer_sequence<int, KK...>) __attribute__((always_inline)) {
            (([&]() __attribute__((always_inline)) {
                 constexpr int kk = KK, P = kk & 1;
                 constexpr bool kLast = kk + 1 == KSTEPS;
                 if constexpr (kLast) {
                     __builtin_amdgcn_s_waitcnt(wait_vm(kNewer));
                     __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
                     // a bare barrier: __syncthreads() would also wait for what was issued for later stages
                     asm volatile("s_barrier" ::: "memory");
                 }
                 __builtin_amdgcn_sched_barrier(0);
                 // offsets of the next step's reads, opaque so that the compiler does not tie them to one
                 // buffer and wait for the loads into the other
                 int o0 = foff(kLast ? 0 : kk + 1, 0), o1 = foff(kLast ? 0 : kk + 1, kRegs - 1);
                 asm volatile("" : "+v"(o0), "+v"(o1));
                 const uint8_t *src = kLast ? nxt : cur;
                 const uint8_t *lp0 = src + o0, *lp1 = src + o1;
                 if constexpr (kMx && kLast) {
                     // The next stage's scale words.  Two stages: before this step's loads -- which buffer they are in
                     // is not known when compiling, so each read waits for the loads in flight; there are none here.
                     constexpr int n = (S + 1) % NST;
                     const uint8_t *slab = NST == 4 ? (n < 2 ? slab0 : slab1) : S == 0 ? slab_cur : slab_next;
                     int so = frow * 16 + (n & 1) * 8 + fq * 4;
                     asm volatile("" : "+v"(so));
                     [&]<int... R>(std::integer_sequence<int, R...>) __attribute__((always_inline)) {
                         (read_scale(slab + so, std::integral_constant<int, R>{}, sa[1 - Q], sb[1 - Q]), ...);
                     }(std::make_integer_sequence<int, 2 * kNB>{});
                     __builtin_amdgcn_sched_barrier(0);
                 }
                 constexpr int kPer = kInt8 ? 4 : 1;                // products of a group
                 constexpr int kGroups = kNB * kNB / kPer;
                 // reads in the first three quarters of a step: the last ones are there when the next step wants them (1%)
                 constexpr int kReadGroups = kGroups * 3 / 4;
                 constexpr int kL = NST == 4 ? kPart : kLast ? kLoads : 0, kL0 = NST == 4 ? kk * kPart : 0;
                 [&]<int... G>(std::integer_sequence<int, G...>) __attribute__((always_inline)) {
                     (([&]() __attribute__((always_inline)) {
                          constexpr int g = G;
                          constexpr auto first = std::integral_constant<bool, FIRST && S == 0 && kk == 0>{};
                          [&]<int... J>(std::integer_sequence<int, J...>) __attribute__((always_inline)) {
                              (product(acc[(g * kPer + J) / kNB][(g * kPer + J) % kNB], fa[P][(g * kPer + J) / kNB],
                                       fb[P][(g * kPer + J) % kNB], sa[Q][kMx ? (g * kPer + J) / kNB : 0],
                                       sb[Q][kMx ? (g * kPer + J) % kNB : 0], std::integral_constant<int, kk>{}, first),
                               ...);
                          }(std::make_integer_sequence<int, kPer>{});
                          [&]<int... R>(std::integer_sequence<int, R...>) __attribute__((always_inline)) {
                              (([&]() __attribute__((always_inline)) {
                                   constexpr int r = share_first(g, kReads, kReadGroups) + R;
                                   read_one(lp0, lp1, std::integral_constant<int, r>{}, fa[P ^ 1], fb[P ^ 1]);
                               }()),
                               ...);
                          }(std::make_integer_sequence<int, (g < kReadGroups ? share_count(g, kReads, kReadGroups) : 0)>{});
                          [&]<int... L>(std::integer_sequence<int, L...>) __attribute__((always_inline)) {
                              (load_one(refill, std::integral_constant<int, kL0 + share_first(g, kL, kGroups) + L>{}), ...);
                          }(std::make_integer_sequence<int, share_count(g, kL, kGroups)>{});
                          __builtin_amdgcn_sched_barrier(0);
                      }()),
                      ...);
                 }(std::make_integer_sequence<int, kGroups>{});
             }()),
             ...);
        }(std::make_integer_sequence<int, KSTEPS>{});
        if constexpr (NST == 4 && S == 1) load_slab(slab0);
        if constexpr (NST == 4 && S == 3) load_slab(slab1);
        advance();
    };

    // ---- prologue: stages 0 and 1 of the first tile, and their scales
    {
        const Tile c = tile_of(ld_tile);
        int lr = -1, sr = -1;
        if (gather) rows_of(c, lr, sr);
        loading = c;
        enter_tile(c, lr, sr);
        look_ahead();
    }
    auto load_stage = [&](uint8_t *stage) __attribute__((always_inline)) {
        [&]<int... J>(std::integer_sequence<int, J...>) __attribute__((always_inline)) {
            (load_one(stage, std::integral_constant<int, J>{}), ...);
        }(std::make_integer_sequence<int, kLoads>{});
        advance();
    };
    load_slab(slab0);
    load_stage(lds0);
    load_stage(lds1);
    if constexpr (NST == 4) {
        load_slab(slab1);
        load_stage(lds2);
        // stages 1 and 2 and the second scales may be in flight
        __builtin_amdgcn_s_waitcnt(wait_vm(2 * kLoads + (kMx ? kSlabLoads : 0)));
    } else {
        __builtin_amdgcn_s_waitcnt(kWaitVm0);
    }
    asm volatile("s_barrier" ::: "memory");

    uint8_t *slab_cur = slab0, *slab_next = slab1;
    // the first step's fragments; a tile's last step reads the next tile's
    {
        int o0 = foff(0, 0), o1 = foff(0, kRegs - 1), so = frow * 16 + fq * 4;
        asm volatile("" : "+v"(o0), "+v"(o1), "+v"(so));
        [&]<int... R>(std::integer_sequence<int, R...>) __attribute__((always_inline)) {
            (read_one(lds0 + o0, lds0 + o1, std::integral_constant<int, R>{}, fa[0], fb[0]), ...);
        }(std::make_integer_sequence<int, kReads>{});
        if constexpr (kMx) {
            [&]<int... R>(std::integer_sequence<int, R...>) __attribute__((always_inline)) {
                (read_scale(slab0 + so, std::integral_constant<int, R>{}, sa[0], sb[0]), ...);
            }(std::make_integer_sequence<int, 2 * kNB>{});
        }
    }
    for (int t = blockIdx.x; t < total; t += gridDim.x) {
        // the cursor is two stages on (three in a ring of four): in this tile, or past it if it has no more
        const Tile c = NST == 2 && stages == 2 ? before : loading;
        const int mw = c.m0 + wm * WT, nw = c.n0 + wn * WT;
        // Inputs of the epilogue, one or two rows and columns a lane: the rows' indices now, what they point to two
        // stages before the end, so that nothing waits for memory in between.
        constexpr int kSets = WT / 64;
        int erow[kMx ? 1 : kSets];
        float escale[kMx ? 1 : kSets], echannel[kMx ? 1 : kSets];
        uint16_t ebias[kSets];
        const size_t col0 = (size_t)c.group * N;
        float tensor_scale = 1.0f;
        if constexpr (!kMx) {
            const __amdgpu_buffer_rsrc_t r = small_rsrc(p.rows + mw, gather ? some(c.end - mw, WT) * 4 : 0);
#pragma unroll
            for (int i = 0; i < kSets; ++i) {
                const int m = i * 64 + lane;
                const int v = load_i32(r, m * 4);
                erow[i] = mw + m >= c.end ? -1 : gather ? v : m;
            }
        }
        auto fetch = [&]() __attribute__((always_inline)) {
            const int cols = some(N - nw, WT);
            const __amdgpu_buffer_rsrc_t rb = small_rsrc(p.bias + col0 + nw, p.bias ? cols * 2 : 0);
#pragma unroll
            for (int i = 0; i < kSets; ++i)
                ebias[i] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rb, (i * 64 + lane) * 2, 0, 0);
            if constexpr (!kMx) {
                // rows of x: all of it where they are gathered, the tile's own otherwise
                const __amdgpu_buffer_rsrc_t rs =
                    small_rsrc(p.sx + (gather ? 0 : mw), gather ? (int)p.X * 4 : some(c.end - mw, WT) * 4);
                const __amdgpu_buffer_rsrc_t rc = small_rsrc(p.sw + col0 + nw, p.per_channel ? cols * 4 : 0);
#pragma unroll
                for (int i = 0; i < kSets; ++i) {
                    const int off = erow[i] < 0 || erow[i] >= p.X ? kOobOffset : erow[i] * 4;
                    escale[i] = __int_as_float(load_i32(rs, off));
                    const float ch = __int_as_float(load_i32(rc, (i * 64 + lane) * 4));
                    echannel[i] = p.per_channel ? ch : 1.0f;
                }
                tensor_scale = p.per_channel ? 1.0f : p.sw[c.group];
            }
        };
        auto run_turn = [&](auto first, int kt) __attribute__((always_inline)) {
            if constexpr (NST == 2) load_slab(slab_next);  // the next turn's scales: the cursor stands at its first stage
            [&]<int... S>(std::integer_sequence<int, S...>) __attribute__((always_inline)) {
                (run_stage(std::integral_constant<int, S>{}, first, slab_cur, slab_next, kt + S), ...);
            }(std::make_integer_sequence<int, NST>{});
            uint8_t *s = slab_cur;
            slab_cur = slab_next;
            slab_next = s;
        };
        run_turn(std::true_type{}, 0);
        if (stages == NST) fetch();
        for (int kt = NST; kt < stages; kt += NST) {
            if (kt + NST == stages) fetch();
            run_turn(std::false_type{}, kt);
        }

        // ---- epilogue: y = bf16(acc * (sx * sw) + bias) through LDS, 32 rows by kPassCols columns at a time
        // (chunks of 16 bytes XOR-swizzled by row), so that it leaves in 16-byte stores along rows
        // the products are assembly: their results' wait before other instructions read them
        asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
        uint8_t *ob = obuf + wave * kPassBytes;
        // lane indices derived again here, so that the addresses below do not stay alive across the K loop
        int el = lane;
        asm volatile("" : "+v"(el));
        const int brow = el & (kBlk - 1), cq = 4 * (el / kBlk);
        // The epilogue's inputs go through LDS to the lanes that need them.  8 bits: f32, in an area of their own, read
        // where they are used.  4-bit format: the biases alone, as bf16, in the staging area, read beforehand.
        float *ep = reinterpret_cast<float *>(epbuf + wave * kEpBytes);  // [WT] row scales, [WT] biases, [WT] channel scales
#pragma unroll
        for (int i = 0; i < kSets; ++i) {
            if constexpr (kMx) {
                reinterpret_cast<uint16_t *>(ob)[i * 64 + el] = ebias[i];
            } else {
                ep[i * 64 + el] = escale[i] * tensor_scale;
                ep[WT + i * 64 + el] = bf16_bits_to_f32(ebias[i]);
                ep[2 * WT + i * 64 + el] = echannel[i];
            }
        }
        __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
        asm volatile("" ::: "memory");
        uint2 bias2[kMx ? kNB : 1][kMx ? kQuads : 1];
        if constexpr (kMx) {
#pragma unroll
            for (int b = 0; b < kNB; ++b)
#pragma unroll
                for (int q = 0; q < kQuads; ++q)
                    bias2[b][q] = *reinterpret_cast<const uint2 *>(ob + (b * kBlk + 8 * q + cq) * 2);
        }
        float tm[kMx ? 1 : kNB];
        if constexpr (!kMx) {
#pragma unroll
            for (int b = 0; b < kNB; ++b) tm[b] = ep[b * kBlk + brow];
        }
        __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
        asm volatile("" ::: "memory");
        constexpr int kCB = kPassCols / kBlk, kRB = 32 / kBlk;  // blocks of a pass
        constexpr int kOutChunks = kPassCols / 8, kOutRows = 64 / kOutChunks;
#pragma unroll
        for (int cp = 0; cp < WT / kPassCols; ++cp) {
            v4f bias[kMx ? 1 : kCB][kMx ? 1 : kQuads], channel[kMx ? 1 : kCB][kMx ? 1 : kQuads];
            if constexpr (!kMx) {
#pragma unroll
                for (int cb = 0; cb < kCB; ++cb)
#pragma unroll
                    for (int q = 0; q < kQuads; ++q) {
                        const float *at = ep + WT + (cp * kCB + cb) * kBlk + 8 * q + cq;
                        bias[cb][q] = *reinterpret_cast<const v4f *>(at);
                        channel[cb][q] = *reinterpret_cast<const v4f *>(at + WT);
                    }
            }
#pragma unroll
            for (int ps = 0; ps < WT / 32; ++ps) {
                __builtin_amdgcn_sched_barrier(0);  // one pass's accumulators in ordinary registers at a time
#pragma unroll
                for (int rb = 0; rb < kRB; ++rb)
#pragma unroll
                    for (int cb = 0; cb < kCB; ++cb) {
                        const int mb = ps * kRB + rb, nb = cp * kCB + cb;
                        float v[4 * kQuads];
#pragma unroll
                        for (int e = 0; e < 4 * kQuads; ++e) v[e] = from_accumulator(acc[nb][mb][e]);
                        // (branches on the call's arguments spare an instruction a value each; int8 lost 2% with its own)
                        if constexpr (kMx) {
                            if (p.bias) {
#pragma unroll
                                for (int e = 0; e < 4 * kQuads; ++e) {
                                    const uint32_t w = (e & 2) ? bias2[nb][e / 4].y : bias2[nb][e / 4].x;
                                    v[e] += bf16_bits_to_f32((e & 1) ? w >> 16 : w & 0xFFFFu);
                                }
                            }
                        } else if (kInt8 || p.per_channel) {
#pragma unroll
                            for (int e = 0; e < 4 * kQuads; ++e)
                                v[e] = __builtin_fmaf(v[e], tm[mb] * channel[cb][e / 4][e % 4], bias[cb][e / 4][e % 4]);
                        } else {
#pragma unroll
                            for (int e = 0; e < 4 * kQuads; ++e) v[e] = __builtin_fmaf(v[e], tm[mb], bias[cb][e / 4][e % 4]);
                        }
#pragma unroll
                        for (int q = 0; q < kQuads; ++q) {
                            const int row = rb * kBlk + brow, col = cb * kBlk + 8 * q + cq;
                            const int chunk = (col >> 3) ^ (row & (kOutChunks - 1));
                            *reinterpret_cast<uint2 *>(ob + row * kPassCols * 2 + chunk * 16 + (col & 7) * 2) =
                                make_uint2(pack_bf16x2(v[4 * q], v[4 * q + 1]), pack_bf16x2(v[4 * q + 2], v[4 * q + 3]));
                        }
                    }
                __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
#pragma unroll
                for (int it = 0; it < 32 / kOutRows; ++it) {
                    const int row = it * kOutRows + el / kOutChunks, ch = el % kOutChunks;
                    const v4u d = *reinterpret_cast<const v4u *>(ob + row * kPassCols * 2 + ((ch ^ (row & (kOutChunks - 1))) << 4));
                    const int m = mw + ps * 32 + row, n = nw + cp * kPassCols + ch * 8;
                    if (m >= c.end) continue;
                    uint16_t *dst = p.out + (size_t)m * N + n;
                    // whole 128-byte lines past the caches; parts of lines through them, to be merged there
                    if ((N & 63) == 0) {
                        if (n < N) __builtin_nontemporal_store(d, reinterpret_cast<v4u *>(dst));
                    } else {
                        store_row(dst, d, N - n);
                    }
                }
                __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
            }
        }
    }
    // loads for stages past the last tile may still be in flight
    __builtin_amdgcn_s_waitcnt(kWaitVm0);
}

template <int QT, int WT, int NST, bool REST>
void launch(const GroupedArgs &a, int split, hipStream_t stream) {
    constexpr int BT = 2 * WT, CT = REST ? 2 * BT : BT;
    const int tiles_n = (a.N + CT - 1) / CT;
    int64_t most = rows_tiles(a, CT) * tiles_n;
    if (REST && most > split / 2) most = split / 2;
    if (REST) most *= 4;
    const int64_t slots = (int64_t)device_cu_count() * (WT == 64 && NST == 2 ? 2 : 1);
    const unsigned grid = (unsigned)(most < slots ? most : slots);
    if (a.kb % (NST * kStageK) == 0)
        grouped_tiles_kernel<QT, WT, NST, false, REST><<<grid, kThreads, 0, stream>>>(a, tiles_n, split);
    else
        grouped_tiles_kernel<QT, WT, NST, true, REST><<<grid, kThreads, 0, stream>>>(a, tiles_n, split);
}

}  // namespace

template <int QT>
void launch_grouped_tiles(const GroupedArgs &a, GroupedKind kind, hipStream_t stream) {
    if (kind == kTile256Split) {
        const int slots = device_cu_count();
        launch<QT, 128, 2, false>(a, slots, stream);
        launch<QT, 64, 2, true>(a, slots, stream);
    } else if (kind == kTile256) {
        launch<QT, 128, 2, false>(a, 0, stream);
    } else if (kind == kTile128) {
        launch<QT, 64, 2, false>(a, 0, stream);
    } else {
        launch<QT, 64, 4, false>(a, 0, stream);
    }
}
template void launch_grouped_tiles<kTypeInt8>(const GroupedArgs &, GroupedKind, hipStream_t);
template void launch_grouped_tiles<kTypeE4m3>(const GroupedArgs &, GroupedKind, hipStream_t);
template void launch_grouped_tiles<kTypeMx4>(const GroupedArgs &, GroupedKind, hipStream_t);

}  // namespace w8a8
