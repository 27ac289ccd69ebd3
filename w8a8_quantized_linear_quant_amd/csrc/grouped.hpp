// grouped.hpp -- arguments of the products of groups of rows, and the search
// for the group that a tile of rows belongs to.
#pragma once

#include "../../include/w8a8_experts.h"
#include "block.hpp"
#include "internal.hpp"

namespace w8a8 {

// Code types of a product: the two of w8a8_qtype, and the 4-bit format.
enum { kTypeInt8 = W8A8_INT8, kTypeE4m3 = W8A8_FP8_E4M3, kTypeMx4 = 2 };

struct GroupedArgs {
    const uint8_t *xq;       // [X, kb] codes
    const uint8_t *wq;       // [E, N, kb]
    const uint8_t *xs, *ws;  // 4-bit format: scale bytes, `stride` a row
    const float *sx, *sw;    // 8 bits: [X]; [E] or [E, N]
    const uint16_t *bias;    // [E, N] or null
    const int32_t *offsets;  // [E + 1], or null: one group of M rows
    const int32_t *rows;     // [M], or null
    uint16_t *out;           // [M, N]
    int64_t X;
    int M, N, E;
    int kb;      // bytes of a row's codes, a multiple of 16
    int stride;  // bytes of a row's scales, a multiple of 16
    int per_channel;
};

// Prefix sum and prefix maximum over the 64 lanes (inclusive): DPP row shifts
// within the rows of 16 lanes, then each row's last lane to the rows after it.
__device__ __forceinline__ int scan_step(int v, int ctrl) {
    switch (ctrl) {  // lanes without a source, and rows outside the mask, read 0
    case 1: return __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);
    case 2: return __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
    case 4: return __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
    case 8: return __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
    case 15: return __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast:15, rows 1 and 3
    default: return __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast:31, rows 2 and 3
    }
}
constexpr int kScanSteps[6] = {1, 2, 4, 8, 15, 31};
__device__ __forceinline__ int wave_scan_sum(int v) {
#pragma unroll
    for (int i = 0; i < 6; ++i) v += scan_step(v, kScanSteps[i]);
    return v;
}
__device__ __forceinline__ int wave_scan_max(int v) {  // of values >= 0
#pragma unroll
    for (int i = 0; i < 6; ++i) v = max(v, scan_step(v, kScanSteps[i]));
    return v;
}

// A wave's view of 64 consecutive groups: lane i holds group base + i.
struct GroupWindow {
    int start, end;  // the group's rows
    int tiles;       // inclusive prefix sum of the groups' tiles of kRows rows, those of earlier windows included
    int base;        // first group of the window
    int before;      // tiles of earlier windows
    int floor_row;   // where the window's first group can begin at the earliest
};

// Loads the window of groups base .. base + 63.  Offsets are clamped to
// [0, M] and to the greatest before them, so that no two groups share a row
// whatever the caller's integers are.
template <int kRows>
__device__ __forceinline__ void load_window(GroupWindow &w, const int32_t *offsets, int E, int M, int lane) {
    const int g = w.base + lane;
    int o0 = 0, o1 = M;
    if (offsets) {
        o0 = offsets[min(g, E)];
        o1 = offsets[min(g + 1, E)];
    }
    o0 = max(min(o0, M), w.floor_row);
    w.start = wave_scan_max(o0);
    w.end = max(w.start, min(o1, M));
    if (g >= E) w.end = w.start;
    w.tiles = w.before + wave_scan_sum((w.end - w.start + kRows - 1) / kRows);
}
template <int kRows>
__device__ __forceinline__ void next_window(GroupWindow &w, const int32_t *offsets, int E, int M, int lane) {
    w.before = __builtin_amdgcn_readlane(w.tiles, 63);
    w.floor_row = __builtin_amdgcn_readlane(w.end, 63);
    w.base += 64;
    load_window<kRows>(w, offsets, E, M, lane);
}

struct GroupTile {
    int group, m0, end;  // rows m0 .. min(m0 + kRows, end) - 1; group -1: there is no such tile
};

// The tile of that number among all groups' tiles; `w` moves forward as needed.
template <int kRows>
__device__ __forceinline__ GroupTile find_tile(GroupWindow &w, int tile, const int32_t *offsets, int E, int M, int lane) {
    GroupTile t = {-1, 0, 0};
    while (__builtin_amdgcn_readlane(w.tiles, 63) <= tile) {
        if (w.base + 64 >= E) return t;
        next_window<kRows>(w, offsets, E, M, lane);
    }
    const int i = __builtin_popcountll(__ballot(w.tiles <= tile));
    const int before = i ? __builtin_amdgcn_readlane(w.tiles, i - 1) : w.before;
    t.group = w.base + i;
    t.end = __builtin_amdgcn_readlane(w.end, i);
    t.m0 = __builtin_amdgcn_readlane(w.start, i) + (tile - before) * kRows;
    return t;
}

// Tiles of `rows` rows that M rows in E groups can have: every group may leave one partly filled.
inline int64_t rows_tiles(const GroupedArgs &a, int rows) { return a.M / rows + (int64_t)(a.E < a.M ? a.E : a.M); }

// Kernels and their tiles; grouped.hip chooses.  Those of grouped_rows.hip take
// what fits 2^23 workgroups (2^31 threads), the others every size.
enum GroupedKind {
    kRows16x16,    // grouped_rows.hip: rows x columns
    kRows16x32,
    kRows32x32,
    kRows64x64,
    kTile128Deep,  // grouped_tiles.hip: 128 x 128, a ring of four stages, one workgroup a CU
    kTile128,      // 128 x 128, a ring of two, two workgroups a CU
    kTile256,      // 256 x 256, a ring of two, one workgroup a CU
    kTile256Split, // the same for whole rounds; a rest of at most half a round in a second launch, in 128 x 128
    kGroupedKinds
};
template <int QT>
void launch_grouped_rows(const GroupedArgs &a, GroupedKind kind, hipStream_t stream);
template <int QT>
void launch_grouped_tiles(const GroupedArgs &a, GroupedKind kind, hipStream_t stream);

}  // namespace w8a8
