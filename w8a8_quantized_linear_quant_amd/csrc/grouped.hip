// grouped.hip -- entry points of the products of groups of rows, and of the
// 4-bit product (one group): argument checks and the choice of the kernel.
#include <cmath>

#include "grouped.hpp"

namespace w8a8 {
namespace {

constexpr int64_t kMaxGroups = 4096;

w8a8_status check(const void *xq, int64_t X, const void *wq, const void *out, const int32_t *offsets, int64_t E,
                  const int32_t *rows, const uint16_t *bias, int64_t M, int64_t N, int64_t kb) {
    if (M < 0 || N < 0 || X < 0 || kb < 0) return W8A8_ERR_INVALID_ARG;
    if (kb < 16 || kb % 16 != 0 || kb > (1 << 22)) return W8A8_ERR_SHAPE;
    if (M > (1 << 30) || N > (1 << 30) || X > (1 << 30) || E < 1 || E > kMaxGroups) return W8A8_ERR_SHAPE;
    if (!rows && X != M && M > 0) return W8A8_ERR_SHAPE;
    if (rows && X * kb > ((int64_t)1 << 31)) return W8A8_ERR_SHAPE;
    if ((M / 16 + E) * ((N + 15) / 16) > 0x7FFFFFFF) return W8A8_ERR_SHAPE;
    if (M == 0 || N == 0) return W8A8_OK;
    if ((!xq && X > 0) || !wq || !out) return W8A8_ERR_INVALID_ARG;
    if (!aligned16(xq) || !aligned16(wq) || !aligned16(out) || !aligned16(offsets) || !aligned16(rows) ||
        !aligned16(bias))
        return W8A8_ERR_ALIGN;
    return W8A8_OK;
}

// Which kernel: the one of least estimated time (us).  What each takes is
// fitted to measurements over E 1 .. 64, N 768 .. 12288, K 1024 .. 4096 and 2 ..
// 2048 rows a group; on 270 shapes drawn from E 1 .. 61, N 137 .. 6144, K
// 256 .. 5056 and 1 .. 16384 rows the choice took 3% more than the best of all,
// geometric mean (a quarter more at worst, among calls of 4 to 8 us).
// Some measurements (best; another):
//   one group, 4-bit:  N = K 4096, 24 rows 16 x 32 5.8 (128 deep 11.8);  192 rows
//     64 x 64 10.9 (128 deep 12.2);  1024 rows 128 deep 15.3 (128 17.9);  N 12288
//     K 4096, 48 rows 64 x 64 11.6 (16 x 32 15.2)
//   8 experts, N = K 4096, e4m3:  8 rows each 16 x 32 24.3 (32 x 32 27.1);  64 each
//     128 deep 33.9 (128 38.1);  400 each 256 61.7 (128 85.9)
//   32 experts of 25 rows, N 2048, K 4096, int8:  64 x 64 61.6 (128 75.7)
//   8 experts of 2048 rows, N 1280, K 4096, int8:  256 with a rest 93.6 (256 101.0)
// An estimate has two parts, joined so that the greater one counts and a near
// second adds to it: the weights' bytes at the rate the kernel reaches, and
// rounds of its tiles over the chip, each with a start and a time for each 128
// bytes of K (a partly filled round of the tile kernels is faster: fewer
// workgroups share the memory and the power).
template <int QT>
GroupedKind choose(const GroupedArgs &a) {
    constexpr bool kMx = QT == kTypeMx4;
    const double cus = device_cu_count(), M = a.M, E = a.E, N = a.N;
    const double steps = (a.kb + 127) / 128;
    // groups with rows, if the rows fall at random; a group leaves half a tile empty on average
    const double active = a.E == 1 ? 1.0 : E * (1.0 - std::exp(-M / E));
    auto tiles = [&](double rows, double columns) {
        const double tm = a.E == 1 ? std::ceil(M / rows) : std::fmax(active, M / rows + 0.5 * active);
        return tm * std::ceil(N / columns);
    };
    const double bytes = active * N * a.kb * (kMx ? 1.0625 : 1.0);
    // (compared as cubes)
    auto joined = [](double work, double memory) { return work * work * work + memory * memory * memory; };
    // rows kernels: first round, later ones, workgroups a CU; a
    // group's weights are read again for each of its row tiles, from closer memory
    auto rows = [&](double rows, double columns, double a_cu, double t0, double t1, double r0, double r1) {
        if ((double)rows_tiles(a, (int)rows) * (N / columns + 8.0) > (1 << 23)) return 1e60;  // a launch's workgroups
        // (the busiest XCD's share: column tiles go to XCDs in turn)
        const double share = tiles(rows, 8.0 * columns) * 8.0 / (a_cu * cus), again = tiles(rows, N) / active - 1.0;
        // a round begun counts whole with one workgroup a CU, by half with more
        const double rounds = a_cu > 1.0 ? 0.5 * (share + std::ceil(share)) : std::ceil(share);
        return joined(t0 + t1 * steps + (rounds > 1.0 ? (rounds - 1.0) * (r0 + r1 * steps) : 0.0),
                      bytes / (kMx ? 4.2e6 : 4.8e6) + again * bytes / (kMx ? 8.0e6 : 9.0e6));
    };
    // n workgroups at once, `full` a full round's time, `few` one's of up to `free` of them
    auto persistent = [](double n, double slots, double free, double few, double full) {
        const double whole = std::floor(n / slots), rest = n - whole * slots;
        return whole * full + (rest < 1.0 ? 0.0 : rest <= free ? few : few + (full - few) * (rest - free) / (slots - free));
    };
    double t[kGroupedKinds];
    t[kRows16x16] = rows(16, 16, 5, 4.2, 0.05, 4.0, 0.13);
    t[kRows16x32] = rows(16, 32, 3, 4.5, 0.05, 3.7, 0.115);
    t[kRows32x32] = rows(32, 32, 2, 4.6, 0.08, 3.6, 0.13);
    t[kRows64x64] = rows(64, 64, 1, 6.5, 0.17, 6.0, 0.16);
    const double n128 = tiles(128, 128);
    // (of groups of unknown lengths, beyond half a tile on average, the tiles may be a few more or fewer)
    const double deep = n128 / cus, around = a.E > 1 && M / 128.0 > 0.5 * active ? 0.07 : 0.0;
    const double rounds_deep = 0.5 * (std::ceil((1.0 - around) * deep) + std::ceil((1.0 + around) * deep));
    t[kTile128Deep] = joined(rounds_deep * (kMx ? 6.0 + 0.4 * steps : 4.7 + 0.43 * steps), bytes / (kMx ? 5.2e6 : 4.2e6));
    // tile kernels: a start, then rounds
    const double few128 = kMx ? 0.9 + 0.65 * steps : 0.4 + 0.6 * steps, full128 = kMx ? 3.2 + 1.3 * steps : 2.0 + 1.1 * steps;
    t[kTile128] = joined(4.0 + persistent(n128, 2 * cus, cus, few128, full128), bytes / (kMx ? 5.2e6 : 3.9e6));
    const double n256 = tiles(256, 256) * (a.E == 1 ? 1.0 : 0.97);
    const double few256 = kMx ? 5.0 + 1.1 * steps : 4.0 + 1.02 * steps, full256 = kMx ? 8.5 + 1.55 * steps : 8.0 + 1.4 * steps;
    const double work256 = 7.0 + persistent(n256, cus, 0.0, few256, full256);
    t[kTile256] = joined(work256, bytes / 4.2e6);
    // Whole rounds of 256, the rest in quarters: 3 us for the second launch, 5 where it may find nothing.  Groups of
    // unknown lengths: the rest may be anything, so half the time it is what the first launch does by itself.
    const double whole = std::floor(n256 / cus), rest = n256 - whole * cus;
    t[kTile256Split] = 1e60;
    if (whole >= 1.0 && a.E == 1 && 2.0 * rest <= cus && rest > 0.0) {
        const double quarters = persistent(4.0 * rest, 2 * cus, cus, few128, full128);
        t[kTile256Split] = joined(10.0 + whole * full256 + quarters, bytes / 4.2e6);
    } else if (whole >= 1.0 && a.E > 1) {
        const double plain = few256 + (full256 - few256) * 0.5, split = 5.0 + few128 + (full128 - few128) * 0.5;
        t[kTile256Split] = joined(work256 + 5.0 - (split < plain ? 0.5 * (plain - split) : 0.0), bytes / 4.2e6);
    }
    int best = 0;
    for (int k = 1; k < kGroupedKinds; ++k)
        if (t[k] < t[best]) best = k;
    return static_cast<GroupedKind>(best);
}

template <int QT>
w8a8_status launch_grouped(const GroupedArgs &a, hipStream_t stream) {
    if (a.M == 0 || a.N == 0) return W8A8_OK;
    const GroupedKind kind = choose<QT>(a);
    if (kind >= kTile128Deep) launch_grouped_tiles<QT>(a, kind, stream);
    else launch_grouped_rows<QT>(a, kind, stream);
    return launch_status();
}

w8a8_status mx_product(const uint8_t *xq, int64_t X, const uint8_t *xs, const uint8_t *wq, const uint8_t *ws,
                       const uint16_t *bias, const int32_t *offsets, int64_t E, const int32_t *rows, int64_t M,
                       int64_t N, int64_t K, uint16_t *y, hipStream_t stream) {
    if (K < 0) return W8A8_ERR_INVALID_ARG;
    if (K < 32 || K % 32 != 0 || K > (1 << 22)) return W8A8_ERR_SHAPE;
    const w8a8_status st = check(xq, X, wq, y, offsets, E, rows, bias, M, N, K / 2);
    if (st != W8A8_OK) return st;
    if (M == 0 || N == 0) return W8A8_OK;
    if ((!xs && X > 0) || !ws) return W8A8_ERR_INVALID_ARG;
    if (!aligned16(xs) || !aligned16(ws)) return W8A8_ERR_ALIGN;
    GroupedArgs a = {};
    a.xq = xq;
    a.wq = wq;
    a.xs = xs;
    a.ws = ws;
    a.bias = bias;
    a.offsets = offsets;
    a.rows = rows;
    a.out = y;
    a.X = X;
    a.M = (int)M;
    a.N = (int)N;
    a.E = (int)E;
    a.kb = (int)(K / 2);
    a.stride = (int)mxfp4_scale_stride(K);
    return launch_grouped<kTypeMx4>(a, stream);
}

}  // namespace
}  // namespace w8a8

extern "C" w8a8_status w8a8_linear_grouped(w8a8_qtype qtype, const void *xq, int64_t X, const float *x_scale,
                                           const void *wq, const float *w_scale, int per_channel, const uint16_t *bias,
                                           const int32_t *offsets, int64_t E, const int32_t *rows, int64_t M, int64_t N,
                                           int64_t K, uint16_t *y, hipStream_t stream) {
    using namespace w8a8;
    if (!valid_qtype(qtype)) return W8A8_ERR_INVALID_ARG;
    const w8a8_status st = check(xq, X, wq, y, offsets, E, rows, bias, M, N, K);
    if (st != W8A8_OK) return st;
    if (M == 0 || N == 0) return W8A8_OK;
    if (!offsets || (!x_scale && X > 0) || !w_scale) return W8A8_ERR_INVALID_ARG;
    if (!aligned16(x_scale) || !aligned16(w_scale)) return W8A8_ERR_ALIGN;
    GroupedArgs a = {};
    a.xq = static_cast<const uint8_t *>(xq);
    a.wq = static_cast<const uint8_t *>(wq);
    a.sx = x_scale;
    a.sw = w_scale;
    a.per_channel = per_channel != 0;
    a.bias = bias;
    a.offsets = offsets;
    a.rows = rows;
    a.out = y;
    a.X = X;
    a.M = (int)M;
    a.N = (int)N;
    a.E = (int)E;
    a.kb = (int)K;
    return qtype == W8A8_INT8 ? launch_grouped<kTypeInt8>(a, stream) : launch_grouped<kTypeE4m3>(a, stream);
}

extern "C" w8a8_status w8a8_linear_grouped_backward_dx(w8a8_qtype qtype, const void *dyq, const float *dy_scale,
                                                       const void *wq_t, const float *w_scale, const int32_t *offsets,
                                                       int64_t E, int64_t M, int64_t N, int64_t K, uint16_t *dx,
                                                       hipStream_t stream) {
    // dX[p] = dYq[p] . Wq[g] = the product of dYq's rows with Wq^T [K, N] over the reduction length N
    return w8a8_linear_grouped(qtype, dyq, M, dy_scale, wq_t, w_scale, 0, nullptr, offsets, E, nullptr, M, K, N, dx,
                               stream);
}

extern "C" w8a8_status mxfp4_linear_grouped(const uint8_t *xq, int64_t X, const uint8_t *xs, const uint8_t *wq,
                                            const uint8_t *ws, const uint16_t *bias, const int32_t *offsets, int64_t E,
                                            const int32_t *rows, int64_t M, int64_t N, int64_t K, uint16_t *y,
                                            hipStream_t stream) {
    if (M > 0 && N > 0 && !offsets) return W8A8_ERR_INVALID_ARG;
    return w8a8::mx_product(xq, X, xs, wq, ws, bias, offsets, E, rows, M, N, K, y, stream);
}

extern "C" w8a8_status mxfp4_linear_grouped_backward_dx(const uint8_t *dyq, const uint8_t *dys, const uint8_t *wq_t,
                                                        const uint8_t *ws_t, const int32_t *offsets, int64_t E,
                                                        int64_t M, int64_t N, int64_t K, uint16_t *dx,
                                                        hipStream_t stream) {
    return mxfp4_linear_grouped(dyq, M, dys, wq_t, ws_t, nullptr, offsets, E, nullptr, M, K, N, dx, stream);
}

extern "C" w8a8_status mxfp4_linear(const uint8_t *xq, const uint8_t *xs, const uint8_t *wq, const uint8_t *ws,
                                    const uint16_t *bias, int64_t M, int64_t N, int64_t K, uint16_t *y,
                                    hipStream_t stream) {
    return w8a8::mx_product(xq, M, xs, wq, ws, bias, nullptr, 1, nullptr, M, N, K, y, stream);
}

extern "C" w8a8_status mxfp4_linear_backward_dx(const uint8_t *dyq, const uint8_t *dys, const uint8_t *wq_t,
                                                const uint8_t *ws_t, int64_t M, int64_t N, int64_t K, uint16_t *dx,
                                                hipStream_t stream) {
    return w8a8::mx_product(dyq, M, dys, wq_t, ws_t, nullptr, nullptr, 1, nullptr, M, K, N, dx, stream);
}

extern "C" int w8a8_probe_grouped_kernel(int type, int64_t M, int64_t N, int64_t K, int64_t E) {
    using namespace w8a8;
    if (M < 1 || N < 1 || K < 1 || E < 1 || M > (1 << 30) || N > (1 << 30) || K > (1 << 22) || E > kMaxGroups) return -1;
    GroupedArgs a = {};
    a.M = (int)M;
    a.N = (int)N;
    a.E = (int)E;
    a.kb = (int)(type == kTypeMx4 ? K / 2 : K);
    if (type == kTypeInt8) return choose<kTypeInt8>(a);
    if (type == kTypeE4m3) return choose<kTypeE4m3>(a);
    return type == kTypeMx4 ? choose<kTypeMx4>(a) : -1;
}
