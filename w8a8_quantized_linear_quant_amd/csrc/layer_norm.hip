// layer_norm.hip -- layer norm over the rows of X, its backward pass, and
// layer norm fused with the row-wise activation quantizer.
//
//   mean = <x>,  var = <(x - mean)^2>,  rstd = 1 / sqrt(var + eps)
//   h = (x - mean) rstd,  y = h w + b
// With t = dy w the input gradient is
//   dx = rstd (t - <t> - h <t h>),  dw = sum_m dy h,  db = sum_m dy
// (<.>: mean over a row).  The variance is taken about the mean, never as
// <x^2> - mean^2, which loses every digit where |mean| >> the deviation.
#include "block.hpp"

namespace w8a8 {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int64_t kMaxK = 1 << 24;

// One workgroup per row, the row read again for each pass.
template <class X>
__device__ __forceinline__ void row_stats(const typename X::type *x, int K, float eps, float *part, float &mean,
                                          float &rstd) {
    float s = 0.f;
    for (int k = threadIdx.x; k < K; k += kThreads) s += X::load(x + k);
    mean = group_sum<kWaves>(s, part) / (float)K;
    float q = 0.f;
    for (int k = threadIdx.x; k < K; k += kThreads) {
        const float d = X::load(x + k) - mean;
        q = __builtin_fmaf(d, d, q);
    }
    rstd = 1.0f / sqrtf(group_sum<kWaves>(q, part) / (float)K + eps);
}

template <class X>
__global__ __launch_bounds__(kThreads) void ln_forward_kernel(const void *xv, int64_t ldx, int K, int wt, const void *w,
                                                              const void *b, float eps, void *yv, int64_t ldy,
                                                              float *mean_out, float *rstd_out) {
    __shared__ float part[kWaves];
    const int64_t m = blockIdx.x;
    const auto *x = static_cast<const typename X::type *>(xv) + m * ldx;
    auto *y = static_cast<typename X::type *>(yv) + m * ldy;
    float mean, rstd;
    row_stats<X>(x, K, eps, part, mean, rstd);
    for (int k = threadIdx.x; k < K; k += kThreads) {
        const float h = (X::load(x + k) - mean) * rstd;
        X::store(y + k, __builtin_fmaf(h, load_param(w, wt, k, 1.f), load_param(b, wt, k, 0.f)));
    }
    if (threadIdx.x == 0) {
        if (mean_out) mean_out[m] = mean;
        if (rstd_out) rstd_out[m] = rstd;
    }
}

// Code of one f32 value with the shared rule.
template <int QT>
__device__ __forceinline__ uint8_t code1(float v, float s, float r) {
    if constexpr (QT == W8A8_INT8) {
        return (uint8_t)(__float_as_uint(quotient_nosign(v, s, r) + 12582912.0f));  // 1.5 * 2^23: rounds half to even
    } else {
        const float q = __builtin_amdgcn_fmed3f(quotient(v, s, r), -448.0f, 448.0f);
        return (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(q, q, 0, false);
    }
}

template <class X, int QT>
__global__ __launch_bounds__(kThreads) void ln_quant_kernel(const void *xv, int64_t ldx, int K, int wt, const void *w,
                                                            const void *b, float eps, uint8_t *xq, int64_t ldq,
                                                            float *sx, float *mean_out, float *rstd_out) {
    __shared__ float part[kWaves];
    const int64_t m = blockIdx.x;
    const auto *x = static_cast<const typename X::type *>(xv) + m * ldx;
    float mean, rstd;
    row_stats<X>(x, K, eps, part, mean, rstd);
    float top = 0.f;
    for (int k = threadIdx.x; k < K; k += kThreads) {
        const float h = (X::load(x + k) - mean) * rstd;
        top = fmaxf(top, fabsf(__builtin_fmaf(h, load_param(w, wt, k, 1.f), load_param(b, wt, k, 0.f))));
    }
    const float s = absmax_scale(group_max<kWaves>(top, part), QT == W8A8_INT8 ? 127.0f : 448.0f);
    const float r = 1.0f / s;
    for (int64_t k = threadIdx.x; k < ldq; k += kThreads) {
        uint8_t c = 0;
        if (k < K) {
            const float h = (X::load(x + k) - mean) * rstd;
            c = code1<QT>(__builtin_fmaf(h, load_param(w, wt, k, 1.f), load_param(b, wt, k, 0.f)), s, r);
        }
        xq[m * ldq + k] = c;
    }
    if (threadIdx.x == 0) {
        sx[m] = s;
        if (mean_out) mean_out[m] = mean;
        if (rstd_out) rstd_out[m] = rstd;
    }
}

template <class X>
__global__ __launch_bounds__(kThreads) void ln_backward_dx_kernel(const void *dyv, int64_t lddy, const void *xv,
                                                                  int64_t ldx, const float *mean, const float *rstd,
                                                                  int K, int wt, const void *w, void *dxv,
                                                                  int64_t lddx) {
    __shared__ float part[kWaves];
    const int64_t m = blockIdx.x;
    const auto *dy = static_cast<const typename X::type *>(dyv) + m * lddy;
    const auto *x = static_cast<const typename X::type *>(xv) + m * ldx;
    auto *dx = static_cast<typename X::type *>(dxv) + m * lddx;
    const float mu = mean[m], rs = rstd[m];
    float s1 = 0.f, s2 = 0.f;
    for (int k = threadIdx.x; k < K; k += kThreads) {
        const float t = X::load(dy + k) * load_param(w, wt, k, 1.f);
        s1 += t;
        s2 = __builtin_fmaf(t, (X::load(x + k) - mu) * rs, s2);
    }
    const float c1 = group_sum<kWaves>(s1, part) / (float)K;
    const float c2 = group_sum<kWaves>(s2, part) / (float)K;
    for (int k = threadIdx.x; k < K; k += kThreads) {
        const float t = X::load(dy + k) * load_param(w, wt, k, 1.f);
        const float h = (X::load(x + k) - mu) * rs;
        X::store(dx + k, rs * (t - c1 - h * c2));
    }
}

// One thread per column.
template <class X>
__global__ __launch_bounds__(kThreads) void ln_backward_params_kernel(const void *dyv, int64_t lddy, const void *xv,
                                                                      int64_t ldx, const float *mean,
                                                                      const float *rstd, int64_t M, int K, float *dw,
                                                                      float *db) {
    const int k = blockIdx.x * kThreads + threadIdx.x;
    if (k >= K) return;
    const auto *dy = static_cast<const typename X::type *>(dyv) + k;
    const auto *x = static_cast<const typename X::type *>(xv) + k;
    float sw = 0.f, sb = 0.f;
    for (int64_t m = 0; m < M; ++m) {
        const float g = X::load(dy + m * lddy);
        sb += g;
        sw = __builtin_fmaf(g, (X::load(x + m * ldx) - mean[m]) * rstd[m], sw);
    }
    if (dw) dw[k] = sw;
    if (db) db[k] = sb;
}

w8a8_status ln_check(w8a8_dtype xt, const void *x, int64_t M, int64_t K, int64_t ldx, w8a8_dtype wt,
                     const void *weight, const void *bias, float eps, const float *mean, const float *rstd) {
    if (!valid_dtype(xt) || !valid_dtype(wt) || M < 0 || !(eps >= 0.f && eps <= 3.402823466e38f))
        return W8A8_ERR_INVALID_ARG;
    if (K < 1 || K > kMaxK || ldx < K || ldx > kMaxK || M > (1 << 30)) return W8A8_ERR_SHAPE;
    if (M > 0 && !x) return W8A8_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(weight) || !aligned16(bias) || !aligned16(mean) || !aligned16(rstd))
        return W8A8_ERR_ALIGN;
    return W8A8_OK;
}

}  // namespace
}  // namespace w8a8

extern "C" w8a8_status layer_norm_forward(w8a8_dtype xt, const void *x, int64_t M, int64_t K, int64_t ldx,
                                          w8a8_dtype wt, const void *weight, const void *bias, float eps, void *y,
                                          int64_t ldy, float *mean, float *rstd, hipStream_t stream) {
    using namespace w8a8;
    const w8a8_status st = ln_check(xt, x, M, K, ldx, wt, weight, bias, eps, mean, rstd);
    if (st != W8A8_OK) return st;
    if (ldy < K || ldy > kMaxK) return W8A8_ERR_SHAPE;
    if (M > 0 && !y) return W8A8_ERR_INVALID_ARG;
    if (!aligned16(y)) return W8A8_ERR_ALIGN;
    if (M == 0) return W8A8_OK;
    if (xt == W8A8_BF16)
        ln_forward_kernel<Bf16><<<(int)M, kThreads, 0, stream>>>(x, ldx, (int)K, wt, weight, bias, eps, y, ldy, mean, rstd);
    else
        ln_forward_kernel<F32><<<(int)M, kThreads, 0, stream>>>(x, ldx, (int)K, wt, weight, bias, eps, y, ldy, mean, rstd);
    return launch_status();
}

extern "C" w8a8_status w8a8_quant_act_rowwise_layer_norm(w8a8_qtype qtype, w8a8_dtype xt, const void *x, int64_t M,
                                                         int64_t K, int64_t ldx, w8a8_dtype wt, const void *weight,
                                                         const void *bias, float eps, void *xq, int64_t ldq,
                                                         float *x_scale, float *mean, float *rstd,
                                                         hipStream_t stream) {
    using namespace w8a8;
    if (!valid_qtype(qtype)) return W8A8_ERR_INVALID_ARG;
    const w8a8_status st = ln_check(xt, x, M, K, ldx, wt, weight, bias, eps, mean, rstd);
    if (st != W8A8_OK) return st;
    if (ldq < K || ldq % 16 != 0 || ldq > kMaxK) return W8A8_ERR_SHAPE;
    if (M > 0 && (!xq || !x_scale)) return W8A8_ERR_INVALID_ARG;
    if (!aligned16(xq) || !aligned16(x_scale)) return W8A8_ERR_ALIGN;
    if (M == 0) return W8A8_OK;
    uint8_t *q = static_cast<uint8_t *>(xq);
#define W8A8_LN_QUANT(X, QT) \
    ln_quant_kernel<X, QT><<<(int)M, kThreads, 0, stream>>>(x, ldx, (int)K, wt, weight, bias, eps, q, ldq, x_scale, mean, rstd)
    if (xt == W8A8_BF16) {
        if (qtype == W8A8_INT8) W8A8_LN_QUANT(Bf16, W8A8_INT8);
        else W8A8_LN_QUANT(Bf16, W8A8_FP8_E4M3);
    } else {
        if (qtype == W8A8_INT8) W8A8_LN_QUANT(F32, W8A8_INT8);
        else W8A8_LN_QUANT(F32, W8A8_FP8_E4M3);
    }
#undef W8A8_LN_QUANT
    return launch_status();
}

extern "C" size_t layer_norm_backward_workspace_bytes(int64_t M, int64_t K) {
    if (M < 0 || K < 1 || K > w8a8::kMaxK) return 0;
    return 16;
}

extern "C" w8a8_status layer_norm_backward(w8a8_dtype xt, const void *dy, int64_t lddy, const void *x, int64_t ldx,
                                           const float *mean, const float *rstd, int64_t M, int64_t K, w8a8_dtype wt,
                                           const void *weight, void *dx, int64_t lddx, float *dweight, float *dbias,
                                           void *workspace, hipStream_t stream) {
    using namespace w8a8;
    const w8a8_status st = ln_check(xt, x, M, K, ldx, wt, weight, nullptr, 0.f, mean, rstd);
    if (st != W8A8_OK) return st;
    if (lddy < K || lddy > kMaxK || (dx && (lddx < K || lddx > kMaxK))) return W8A8_ERR_SHAPE;
    if (M > 0 && (!dy || !mean || !rstd)) return W8A8_ERR_INVALID_ARG;
    if ((dweight || dbias) && !workspace) return W8A8_ERR_INVALID_ARG;
    if (!aligned16(dy) || !aligned16(dx) || !aligned16(dweight) || !aligned16(dbias) || !aligned16(workspace))
        return W8A8_ERR_ALIGN;
    const int cols = (int)((K + kThreads - 1) / kThreads);
    // the parameters' gradients first: dx may be dy
#define W8A8_LN_BACKWARD(X)                                                                                        \
    if (dweight || dbias)                                                                                          \
        ln_backward_params_kernel<X><<<cols, kThreads, 0, stream>>>(dy, lddy, x, ldx, mean, rstd, M, (int)K,        \
                                                                    dweight, dbias);                               \
    if (dx && M > 0)                                                                                               \
    ln_backward_dx_kernel<X><<<(int)M, kThreads, 0, stream>>>(dy, lddy, x, ldx, mean, rstd, (int)K, wt, weight, dx, lddx)
    if (xt == W8A8_BF16) {
        W8A8_LN_BACKWARD(Bf16);
    } else {
        W8A8_LN_BACKWARD(F32);
    }
#undef W8A8_LN_BACKWARD
    return launch_status();
}
