// grouped.hip -- entry points of the products of groups of rows, and of the
// 4-bit product (one group): argument checks and the choice of the kernel.
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

template <int QT>
w8a8_status launch_grouped(const GroupedArgs &a, hipStream_t stream) {
    if (a.M == 0 || a.N == 0) return W8A8_OK;
    if (a.M > 64 * (int64_t)a.E) {
        const int64_t tiles = ((a.M + 255) / 256) * (((int64_t)a.N + 255) / 256);
        launch_grouped_tiles<QT>(a, tiles >= device_cu_count() ? kTile256 : kTile128Deep, stream);
    } else {
        launch_grouped_rows<QT>(a, stream);
    }
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
