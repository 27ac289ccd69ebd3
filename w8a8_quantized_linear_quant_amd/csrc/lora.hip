// lora.hip -- low-rank adapters of many requests beside a shared projection.
//
// Row m of X belongs to a request that uses adapter l (or none):
//   u = s_l x A_l^T           (down, over K)       out = base + u B_l^T   (up)
//   g = s_l dy B_l            (down, over N)       dx  = base + g A_l     (up)
//   dA_l = sum_m g^T x        dB_l = sum_m dy^T u  (over the rows of l)
// Three forms in all: a down-projection of the rows, an up-projection added to
// a base, and a sum of outer products over an adapter's rows.  The weight of a
// form is A [R, K] or B [N, R]; the strides (sj, sc) of the rank index j and
// the wide index c tell them apart.
#include "block.hpp"

namespace w8a8 {
namespace {

constexpr int kThreads = 256;
constexpr int kTileRows = W8A8_LORA_TILE_ROWS;
constexpr int kMaxR = 128;
constexpr int64_t kMaxL = 65535;

struct Tile {
    int64_t row0;
    int rows, adapter;
};

// Tile t of the plan; rows = 0 where the entry does not fit M and L.
__device__ __forceinline__ Tile load_tile(const int32_t *plan, int t, int64_t M, int L) {
    const int4 e = reinterpret_cast<const int4 *>(plan)[t];
    Tile r = {e.x, e.y, e.z};
    if (r.row0 < 0 || r.rows < 0 || r.rows > kTileRows || r.row0 + r.rows > M || r.adapter < -1 || r.adapter >= L)
        r = {0, 0, -1};
    return r;
}

__device__ __forceinline__ int rank_of(const int32_t *ranks, int l, int R) {
    return ranks ? min(max(ranks[l], 0), R) : R;
}

// One workgroup per tile: p[t][row][j], and u[m][j] if wanted.
__global__ __launch_bounds__(kThreads) void lora_down_kernel(const uint16_t *x, int64_t M, int C, int64_t ldx,
                                                             const uint16_t *w, int64_t wl, int64_t sj, int64_t sc,
                                                             int L, int R, const float *scale, const int32_t *ranks,
                                                             const int32_t *plan, float *p, float *u) {
    const Tile tile = load_tile(plan, blockIdx.x, M, L);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = tile.adapter < 0 ? 0 : rank_of(ranks, tile.adapter, R);
    for (int i = wave; i < kTileRows * R; i += kThreads / 64) {
        const int row = i / R, j = i % R;
        float s = 0.f;
        if (row < tile.rows && j < r) {
            const uint16_t *xr = x + (tile.row0 + row) * ldx;
            const uint16_t *wr = w + tile.adapter * wl + j * sj;
            for (int c = lane; c < C; c += 64) s = __builtin_fmaf(bf16_bits_to_f32(xr[c]), bf16_bits_to_f32(wr[c * sc]), s);
            s = wave_sum(s) * (scale ? scale[tile.adapter] : 1.f);
        }
        if (lane == 0) {
            p[((int64_t)blockIdx.x * kTileRows + row) * R + j] = s;
            if (u && row < tile.rows) u[(tile.row0 + row) * R + j] = s;
        }
    }
}

// One workgroup per tile and 256 columns.
__global__ __launch_bounds__(kThreads) void lora_up_kernel(const float *p, const uint16_t *w, int64_t wl, int64_t sj,
                                                           int64_t sc, int64_t M, int C, int L, int R,
                                                           const int32_t *ranks, const int32_t *plan,
                                                           const uint16_t *base, int64_t ldbase, uint16_t *out,
                                                           int64_t ldout) {
    const Tile tile = load_tile(plan, blockIdx.x, M, L);
    const int c = blockIdx.y * kThreads + threadIdx.x;
    if (c >= C) return;
    const int r = tile.adapter < 0 ? 0 : rank_of(ranks, tile.adapter, R);
    for (int row = 0; row < tile.rows; ++row) {
        const float *pr = p + ((int64_t)blockIdx.x * kTileRows + row) * R;
        float s = base ? bf16_bits_to_f32(base[(tile.row0 + row) * ldbase + c]) : 0.f;
        for (int j = 0; j < r; ++j) s = __builtin_fmaf(pr[j], bf16_bits_to_f32(w[tile.adapter * wl + j * sj + c * sc]), s);
        Bf16::store(out + (tile.row0 + row) * ldout + c, s);
    }
}

// One thread per (j, c) of an adapter: the sum over its rows of v[m][j] y[m][c],
// v = u[m][j] (by row) or the down-projection's p[t][row][j] (by tile).
__global__ __launch_bounds__(kThreads) void lora_outer_kernel(const float *u, const float *p, const uint16_t *y,
                                                              int64_t M, int C, int64_t ldy, int L, int R,
                                                              const int32_t *ranks, const int32_t *plan, int T,
                                                              int64_t sj, int64_t sc, float *d) {
    const int l = blockIdx.z, j = blockIdx.y, c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= C) return;
    const int32_t *first = plan + 4 * (int64_t)T;
    float s = 0.f;
    if (j < rank_of(ranks, l, R)) {
        const int t1 = min(first[l + 1], T);
        for (int t = max(first[l], 0); t < t1; ++t) {
            const Tile tile = load_tile(plan, t, M, L);
            for (int row = 0; row < tile.rows; ++row) {
                const int64_t m = tile.row0 + row;
                const float v = u ? u[m * R + j] : p[((int64_t)t * kTileRows + row) * R + j];
                s = __builtin_fmaf(v, bf16_bits_to_f32(y[m * ldy + c]), s);
            }
        }
    }
    d[(int64_t)l * R * C + j * sj + c * sc] = s;
}

constexpr int64_t kMaxWidth = 1 << 22;

bool bad_width(int64_t w) { return w < 8 || w % 8 != 0 || w > kMaxWidth; }
bool bad_stride(int64_t ld, int64_t w) { return ld < w || ld % 8 != 0 || ld > kMaxWidth; }

w8a8_status lora_check(int64_t M, int64_t K, int64_t N, int64_t R, int64_t L, int64_t T, const uint16_t *a,
                       const uint16_t *b, const float *scale, const int32_t *ranks, const int32_t *plan,
                       const void *workspace) {
    if (M < 0 || T < 0 || L < 1 || R < 8 || R > kMaxR) return W8A8_ERR_INVALID_ARG;
    if (R % 8 != 0 || bad_width(K) || bad_width(N) || L > kMaxL || M > (1 << 30) || T > (1 << 24))
        return W8A8_ERR_SHAPE;
    if (!a || !b || !plan || !workspace) return W8A8_ERR_INVALID_ARG;
    if (!aligned16(a) || !aligned16(b) || !aligned16(scale) || !aligned16(ranks) || !aligned16(plan) ||
        !aligned16(workspace))
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

extern "C" size_t lora_forward_workspace_bytes(int64_t T, int64_t K, int64_t R) {
    if (T < 0 || K < 8 || R < 8 || R > w8a8::kMaxR) return 0;
    return (size_t)T * w8a8::kTileRows * R * sizeof(float);
}

extern "C" w8a8_status lora_forward(const uint16_t *x, int64_t M, int64_t K, int64_t ldx, const uint16_t *a,
                                    const uint16_t *b, int64_t L, int64_t N, int64_t R, const float *scale,
                                    const int32_t *ranks, const int32_t *plan, int64_t T, const uint16_t *base,
                                    int64_t ldbase, uint16_t *out, int64_t ldout, float *u, void *workspace,
                                    hipStream_t stream) {
    using namespace w8a8;
    if (M == 0 || T == 0) return M < 0 || T < 0 ? W8A8_ERR_INVALID_ARG : W8A8_OK;
    const w8a8_status st = lora_check(M, K, N, R, L, T, a, b, scale, ranks, plan, workspace);
    if (st != W8A8_OK) return st;
    if (bad_stride(ldx, K) || bad_stride(ldout, N) || (base && bad_stride(ldbase, N))) return W8A8_ERR_SHAPE;
    if (!x || !out) return W8A8_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(base) || !aligned16(out) || !aligned16(u)) return W8A8_ERR_ALIGN;
    float *p = static_cast<float *>(workspace);
    lora_down_kernel<<<(int)T, kThreads, 0, stream>>>(x, M, (int)K, ldx, a, R * K, K, 1, (int)L, (int)R, scale, ranks, plan, p, u);
    const dim3 grid((unsigned)T, (unsigned)((N + kThreads - 1) / kThreads));
    lora_up_kernel<<<grid, kThreads, 0, stream>>>(p, b, N * R, 1, R, M, (int)N, (int)L, (int)R, ranks, plan, base, ldbase, out, ldout);
    return launch_status();
}

extern "C" size_t lora_backward_workspace_bytes(int64_t T, int64_t K, int64_t N, int64_t R, int64_t L) {
    if (T < 0 || K < 8 || N < 8 || L < 1 || R < 8 || R > w8a8::kMaxR) return 0;
    return (size_t)(T * w8a8::kTileRows * R * sizeof(float) + 16);
}

extern "C" w8a8_status lora_backward(const uint16_t *dy, int64_t M, int64_t N, int64_t lddy, const uint16_t *x,
                                     int64_t K, int64_t ldx, const float *u, const uint16_t *a, const uint16_t *b,
                                     int64_t L, int64_t R, const float *scale, const int32_t *ranks,
                                     const int32_t *plan, int64_t T, const uint16_t *base, int64_t ldbase,
                                     uint16_t *dx, int64_t lddx, float *da, float *db, void *workspace,
                                     hipStream_t stream) {
    using namespace w8a8;
    const w8a8_status st = lora_check(M, K, N, R, L, T, a, b, scale, ranks, plan, workspace);
    if (st != W8A8_OK) return st;
    if (bad_stride(ldx, K) || bad_stride(lddy, N) || (dx && bad_stride(lddx, K)) || (base && bad_stride(ldbase, K)))
        return W8A8_ERR_SHAPE;
    if (M > 0 && T > 0 && (!dy || (da && !x) || (db && !u))) return W8A8_ERR_INVALID_ARG;
    if ((da == nullptr) != (db == nullptr)) return W8A8_ERR_INVALID_ARG;
    if (!aligned16(dy) || !aligned16(x) || !aligned16(u) || !aligned16(base) || !aligned16(dx) || !aligned16(da) ||
        !aligned16(db))
        return W8A8_ERR_ALIGN;
    if (M == 0) T = 0;
    float *p = static_cast<float *>(workspace);
    if (T > 0) {
        lora_down_kernel<<<(int)T, kThreads, 0, stream>>>(dy, M, (int)N, lddy, b, N * R, 1, R, (int)L, (int)R, scale, ranks, plan, p, nullptr);
        if (dx) {
            const dim3 grid((unsigned)T, (unsigned)((K + kThreads - 1) / kThreads));
            lora_up_kernel<<<grid, kThreads, 0, stream>>>(p, a, R * K, K, 1, M, (int)K, (int)L, (int)R, ranks, plan, base, ldbase, dx, lddx);
        }
    }
    if (da) {
        const dim3 ga((unsigned)((K + kThreads - 1) / kThreads), (unsigned)R, (unsigned)L);
        lora_outer_kernel<<<ga, kThreads, 0, stream>>>(nullptr, p, x, M, (int)K, ldx, (int)L, (int)R, ranks, plan, (int)T, K, 1, da);
        const dim3 gb((unsigned)((N + kThreads - 1) / kThreads), (unsigned)R, (unsigned)L);
        lora_outer_kernel<<<gb, kThreads, 0, stream>>>(u, nullptr, dy, M, (int)N, lddy, (int)L, (int)R, ranks, plan, (int)T, 1, R, db);
    }
    return launch_status();
}
