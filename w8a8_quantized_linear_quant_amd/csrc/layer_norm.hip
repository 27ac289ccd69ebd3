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
constexpr int kMaxGroups = 256;      // workgroups of the backward kernel: one for each CU
constexpr int kStreamSplits = 64;    // row splits of the streaming column sums
// Workgroups of a launch at most: with their threads below HIP's 2^32.  More
// rows than these have are taken by them in turn.  (Streamed rows are more than
// 16384 wide: 2^24 of them, a workgroup each, fit no memory.)
constexpr int64_t kMaxGrid = 1 << 22;

// Rows too wide for registers: one workgroup per row, the row read again for
// each pass, an element at a time (2048 rows of 20000 bf16: the norm 130 us, to
// codes 171 us, the backward pass 57 + 146 + 5 us; a floor of 31, 23 and 46 us
// at the rate of a large copy).
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

// What the codes of a row are computed with.  A row that holds a NaN has a NaN
// scale, from which every quotient is NaN.  An infinite scale s has x / s = 0
// with x's sign, NaN for an infinite x: the quotient's correction would make
// NaN of all (0 * inf); divisor 1 and reciprocal 0 give these values.  int8 has
// no NaN: every code beside a scale that is not finite is 0.
struct RowScale {
    float s, r;      // divisor and its reciprocal
    uint32_t keep;   // int8: the codes' bits that stay
};
__device__ __forceinline__ RowScale row_scale(float s) {
    return {__builtin_isinf(s) ? 1.0f : s, 1.0f / s, __builtin_isfinite(s) ? ~0u : 0u};
}

// Codes of 4 f32 values (one word, element order) with the shared rule.
template <int QT>
__device__ __forceinline__ uint32_t codes4(const float *v, const RowScale &s) {
    if constexpr (QT == W8A8_INT8) {
        const float magic = 12582912.0f;  // 1.5 * 2^23: the add rounds half to even
        uint32_t b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(quotient_nosign(v[i], s.s, s.r) + magic);
        return (__builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u) | __builtin_amdgcn_perm(b[3], b[2], 0x04000c0cu)) & s.keep;
    } else {
        // |v| <= absmax gives |v / s| <= 448 (1 + 2^-23), which converts to 448:
        // the clamp of the definition cannot bind
        float q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = quotient(v[i], s.s, s.r);
        const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
        return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
    }
}
// ---------------------------------------------------------------- resident
// Rows that fit the registers of one workgroup are read once: W waves share a
// row, thread t of the row's 64 W holds its chunks t, t + 64 W, ... (16 bytes
// each).  A workgroup takes several rows, the next one's loads in flight while a
// row is worked on, the weights in registers.  Bound by memory: 8192 rows of
// 4096 in f32 43.7 us (268 MB, 6.1 TB/s with what the caches keep), in bf16
// 23.2 us (134 MB, 5.8 TB/s); to codes by memory and about 25 vector instructions
// an element alike (bf16 24.8 us, 101 MB, 4.1 TB/s).  (These and the backward
// kernel's times: medians under rocprofv3, inputs rotated over three sets.  The
// comparisons of layouts further down: inputs rotated over more memory than the
// caches hold, the launches of a call together.)
// OUT: what leaves (the norm in X's type, int8 codes or e4m3 codes).  EVEN: K
// is a whole number of chunks, so that a chunk is either there or not.
enum { kOutNorm = 0, kOutInt8 = 1, kOutE4m3 = 2 };

// 1 / sqrt(a) to about one unit in the last place: the hardware's estimate
// with one Newton step.
__device__ __forceinline__ float inverse_sqrt(float a) {
    if (!(a > 1e-30f)) return 1.0f / sqrtf(a);  // 0, where eps = 0
    const float r = __builtin_amdgcn_rsqf(a);
    const float e = __builtin_fmaf(-a * r, r, 1.0f);
    const float y = __builtin_fmaf(0.5f * r, e, r);
    return a > 1e30f ? r : y;  // a * r * r would not stay finite
}

// One chunk of a weight vector as it lies in memory (WT: its type): `none`
// (its bits, of WT) in every element where there is no vector.
template <int WT, int VEC>
struct ParamChunk {
    v4u d[WT == W8A8_BF16 ? 1 : VEC / 4];
};
template <int WT, int VEC, bool EVEN>
__device__ __forceinline__ ParamChunk<WT, VEC> fetch_params(const void *p, int col, int K, float none) {
    const uint32_t bits = WT == W8A8_F32 ? __float_as_uint(none) : __float_as_uint(none) >> 16 | __float_as_uint(none);
    ParamChunk<WT, VEC> c;
#pragma unroll
    for (v4u &d : c.d) d = p ? v4u{0u, 0u, 0u, 0u} : v4u{bits, bits, bits, bits};
    if (!p || col >= K) return c;
    if constexpr (EVEN) {
        if constexpr (WT == W8A8_F32) {
#pragma unroll
            for (int i = 0; i < VEC / 4; ++i)
                c.d[i] = *reinterpret_cast<const v4u *>(static_cast<const float *>(p) + col + 4 * i);
        } else if constexpr (VEC == 8) {
            c.d[0] = *reinterpret_cast<const v4u *>(static_cast<const uint16_t *>(p) + col);
        } else {
            const uint2 q = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + col);
            c.d[0][0] = q.x, c.d[0][1] = q.y;
        }
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            if (col + e >= K) continue;
            if constexpr (WT == W8A8_F32) c.d[e / 4][e % 4] = static_cast<const uint32_t *>(p)[col + e];
            else c.d[0][e / 2] |= (uint32_t)static_cast<const uint16_t *>(p)[col + e] << (16 * (e & 1));
        }
    }
    return c;
}
template <int WT, int VEC>
__device__ __forceinline__ float param(const ParamChunk<WT, VEC> &c, int e) {
    if constexpr (WT == W8A8_F32) return __uint_as_float(c.d[e / 4][e % 4]);
    else return __uint_as_float(e & 1 ? c.d[0][e / 2] & 0xFFFF0000u : c.d[0][e / 2] << 16);
}

template <class X, bool EVEN>
__device__ __forceinline__ v4u fetch_chunk(const typename X::type *row, int col, int K) {
    if constexpr (EVEN) return col < K ? X::load_chunk(row + col) : v4u{0u, 0u, 0u, 0u};
    return col < K ? load_row_chunk<X>(row, col, K) : v4u{0u, 0u, 0u, 0u};
}

// Elements of wave w of a row: whole chunk strides, then what the last stride
// holds of it.
template <int V, int W>
__device__ __forceinline__ int wave_elements(int K, int w) {
    constexpr int stride = 64 * W * V;
    return K / stride * (64 * V) + min(max(K % stride - w * 64 * V, 0), 64 * V);
}

// Mean and rstd of a row from the chunks of its W waves.  Each wave takes the
// mean and the squared deviations of its own n elements; the waves' parts meet
// by  M2 = sum_w M2_w + n_w (mean_w - mean)^2,  which needs one exchange and,
// like the two-pass form, never subtracts large sums.  counts: n_w of each
// wave; part: this row's, used again two rows later.
template <class X, int W, int NCH, bool EVEN>
__device__ __forceinline__ void resident_stats(const float (&v)[NCH][X::kVec], int K, int tid, float own_n, float eps,
                                               const float *counts, float2 *part, float &mean, float &rstd) {
    constexpr int V = X::kVec, T = 64 * W;
    // chunk by chunk in pairs: fewer roundings on each element's way than one
    // running sum, which counts where the mean is near 0
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        float c[V];
#pragma unroll
        for (int e = 0; e < V; ++e) c[e] = v[i][e];
#pragma unroll
        for (int h = V / 2; h > 0; h /= 2)
#pragma unroll
            for (int e = 0; e < h; ++e) c[e] += c[e + h];
        s += c[0];
    }
    const float mu = wave_sum(s) / own_n;
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int col = (i * T + tid) * V;
        float p = 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            float d = v[i][e] - mu;
            if constexpr (!EVEN) d = col + e < K ? d : 0.f;
            p = __builtin_fmaf(d, d, p);
        }
        q += col < K ? p : 0.f;
    }
    float m2 = wave_sum(q);
    mean = mu;
    if constexpr (W > 1) {
        if ((tid & 63) == 0) part[tid >> 6] = make_float2(mu, m2);
        __syncthreads();
        float total = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) total = __builtin_fmaf(part[w].x, counts[w], total);
        mean = total / (float)K;
        m2 = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float d = part[w].x - mean;
            m2 += __builtin_fmaf(counts[w] * d, d, part[w].y);
        }
    }
    rstd = inverse_sqrt(m2 / (float)K + eps);
}

template <int W>
constexpr int kResidentThreads = 64 * W > kThreads ? 64 * W : kThreads;

template <class X, int WT, bool EVEN, int W, int NCH, int OUT>
__global__ __launch_bounds__(kResidentThreads<W>) void ln_resident_kernel(const void *xv, int64_t M, int64_t ldx, int K,
                                                                          const void *w, const void *b, float eps,
                                                                          void *yv, int64_t ldy, float *sx,
                                                                          float *mean_out, float *rstd_out) {
    constexpr int V = X::kVec, T = 64 * W, G = kResidentThreads<W> / T;
    typedef typename X::type E;
    __shared__ float2 part[2][G][W];
    __shared__ float top_part[2][G][W];
    const int group = threadIdx.x / T, tid = threadIdx.x % T;
    const int64_t step = (int64_t)gridDim.x * G;
    float counts[W];  // a wave without elements has count 0 and takes 0 / 1 for its mean
#pragma unroll
    for (int k = 0; k < W; ++k) counts[k] = (float)wave_elements<V, W>(K, k);
    const float own_n = fmaxf((float)wave_elements<V, W>(K, tid >> 6), 1.f);
    int64_t m = (int64_t)blockIdx.x * G + group;
    v4u raw[NCH];
    auto fetch = [&](int64_t row) {
        // a group without a row of its own still meets the others at the barriers
        const E *x = static_cast<const E *>(xv) + (row < M ? row : M - 1) * ldx;
#pragma unroll
        for (int i = 0; i < NCH; ++i) raw[i] = fetch_chunk<X, EVEN>(x, (i * T + tid) * V, K);
    };
    fetch(m);
    ParamChunk<WT, V> wc[NCH], bc[NCH];
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        wc[i] = fetch_params<WT, V, EVEN>(w, (i * T + tid) * V, K, 1.f);
        bc[i] = fetch_params<WT, V, EVEN>(b, (i * T + tid) * V, K, 0.f);
    }
    int flip = 0;
    for (int64_t m0 = (int64_t)blockIdx.x * G; m0 < M; m0 += step, m += step, flip ^= 1) {
        float v[NCH][V];
#pragma unroll
        for (int i = 0; i < NCH; ++i) X::unpack(raw[i], v[i]);
        if (m0 + step < M) fetch(m + step);
        float mean, rstd;
        resident_stats<X, W, NCH, EVEN>(v, K, tid, own_n, eps, counts, part[flip][group], mean, rstd);
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int col = (i * T + tid) * V;
            float most = 0.f;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float y = __builtin_fmaf((v[i][e] - mean) * rstd, param(wc[i], e), param(bc[i], e));
                if constexpr (OUT != kOutNorm) {
                    if constexpr (!EVEN) y = col + e < K ? y : 0.f;
                    most = max_or_nan(most, fabsf(y));
                }
                v[i][e] = y;
            }
            if constexpr (OUT != kOutNorm) top = max_or_nan(top, col < K ? most : 0.f);
            if constexpr (OUT == kOutNorm) {
                E *y = static_cast<E *>(yv) + m * ldy;
                if (m < M && col < K) {
                    if constexpr (EVEN) X::store_chunk(y + col, X::pack(v[i]));
                    else store_row_chunk<X>(y, col, K, v[i]);
                }
            }
        }
        if (tid == 0 && m < M) {
            if (mean_out) mean_out[m] = mean;
            if (rstd_out) rstd_out[m] = rstd;
        }
        if constexpr (OUT != kOutNorm) {
            constexpr int QT = OUT == kOutInt8 ? W8A8_INT8 : W8A8_FP8_E4M3;
            top = wave_max(top);
            if constexpr (W > 1) {
                if ((tid & 63) == 0) top_part[flip][group][tid >> 6] = top;
                __syncthreads();
#pragma unroll
                for (int k = 0; k < W; ++k) top = max_or_nan(top, top_part[flip][group][k]);
            }
            if (m >= M) continue;
            const float s = absmax_scale(top, QT == W8A8_INT8 ? 127.0f : 448.0f);
            const RowScale rs = row_scale(s);
            uint8_t *q = static_cast<uint8_t *>(yv) + m * ldy;
#pragma unroll
            for (int i = 0; i < NCH; ++i) {
                const int col = (i * T + tid) * V;
                if (col >= ldy) continue;
                uint32_t c[V / 4];
#pragma unroll
                for (int e = 0; e < V; e += 4) c[e / 4] = col < K ? codes4<QT>(&v[i][e], rs) : 0u;
                if constexpr (V == 8) *reinterpret_cast<uint2 *>(q + col) = make_uint2(c[0], c[1]);
                else *reinterpret_cast<uint32_t *>(q + col) = c[0];
            }
            if constexpr (!EVEN && QT == W8A8_FP8_E4M3) {
                // beside a NaN the chunk over K's end got NaN past K too: its own thread clears them
                if (s != s && tid == K / V % T)
                    for (int col = K; col % V != 0; ++col) q[col] = 0;
            }
            for (int64_t col = (int64_t)(NCH * T + tid) * V; col < ldy; col += T * V) {
                if constexpr (V == 8) *reinterpret_cast<uint2 *>(q + col) = make_uint2(0u, 0u);
                else *reinterpret_cast<uint32_t *>(q + col) = 0u;
            }
            if (tid == 0) sx[m] = s;
        }
    }
}

// Code of one f32 value with the shared rule.
template <int QT>
__device__ __forceinline__ uint8_t code1(float v, const RowScale &s) {
    if constexpr (QT == W8A8_INT8) {
        return (uint8_t)(__float_as_uint(quotient_nosign(v, s.s, s.r) + 12582912.0f) & s.keep);  // as codes4
    } else {
        const float q = quotient(v, s.s, s.r);
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
        top = max_or_nan(top, fabsf(__builtin_fmaf(h, load_param(w, wt, k, 1.f), load_param(b, wt, k, 0.f))));
    }
    const float s = absmax_scale(group_max<kWaves>(top, part), QT == W8A8_INT8 ? 127.0f : 448.0f);
    const RowScale rs = row_scale(s);
    for (int64_t k = threadIdx.x; k < ldq; k += kThreads) {
        uint8_t c = 0;
        if (k < K) {
            const float h = (X::load(x + k) - mean) * rstd;
            c = code1<QT>(__builtin_fmaf(h, load_param(w, wt, k, 1.f), load_param(b, wt, k, 0.f)), rs);
        }
        xq[m * ldq + k] = c;
    }
    if (threadIdx.x == 0) {
        sx[m] = s;
        if (mean_out) mean_out[m] = mean;
        if (rstd_out) rstd_out[m] = rstd;
    }
}

// -------------------------------------------------------- resident, backward
// Threads a backward workgroup may have: 128 registers for each with 8 elements, else 256.
constexpr int backward_threads(int ept) { return ept <= 8 ? 1024 : 512; }

// As the forward kernel, and each thread keeps the sums over its workgroup's
// rows of dy h and dy for its own columns.  A workgroup of `groups` row groups
// takes every gridDim.x * groups-th row (8192 x 4096: bf16 37.5 us for 201 MB,
// 5.4 TB/s; f32 74.7 us for 403 MB); the next row's loads are in flight while a
// row is worked on.  At the end the groups' sums meet in LDS and leave as partials
// [workgroup][dw, db][position]; ln_reduce_kernel adds them.
// Position p of column c = (i T + t) V + e:  p = (i V + e) T + t.
template <class X, int WT, bool EVEN, int W, int NCH, bool PARAMS>
__global__ __launch_bounds__(backward_threads(NCH * X::kVec)) void ln_backward_kernel(
    const void *dyv, int64_t lddy, const void *xv, int64_t ldx, const float *mean, const float *rstd, int64_t M, int K,
    const void *w, void *dxv, int64_t lddx, float *partials) {
    constexpr int V = X::kVec, T = 64 * W;
    typedef typename X::type E;
    __shared__ float2 part[2][backward_threads(NCH * V) / T][W];
    __shared__ float sums[PARAMS ? backward_threads(NCH * V) * V : 1];
    const int group = threadIdx.x / T, tid = threadIdx.x % T, groups = blockDim.x / T;
    const int64_t step = (int64_t)gridDim.x * groups;
    float aw[NCH][V], ab[NCH][V];
    ParamChunk<WT, V> wc[NCH];
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        wc[i] = fetch_params<WT, V, EVEN>(w, (i * T + tid) * V, K, 1.f);
#pragma unroll
        for (int e = 0; e < V; ++e) aw[i][e] = ab[i][e] = 0.f;
    }
    v4u rx[NCH], ry[NCH];
    float mu = 0.f, rs = 0.f;
    auto fetch = [&](int64_t m) {
        mu = rs = 0.f;
#pragma unroll
        for (int i = 0; i < NCH; ++i) rx[i] = ry[i] = v4u{0u, 0u, 0u, 0u};
        if (m >= M) return;  // x = dy = 0 with mean = rstd = 0 add nothing
        const E *x = static_cast<const E *>(xv) + m * ldx, *dy = static_cast<const E *>(dyv) + m * lddy;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int col = (i * T + tid) * V;
            rx[i] = fetch_chunk<X, EVEN>(x, col, K), ry[i] = fetch_chunk<X, EVEN>(dy, col, K);
        }
        mu = mean[m], rs = rstd[m];
    };
    fetch((int64_t)blockIdx.x * groups + group);
    int flip = 0;
    for (int64_t m0 = (int64_t)blockIdx.x * groups; m0 < M; m0 += step, flip ^= 1) {
        const int64_t m = m0 + group;
        float h[NCH][V], t[NCH][V];
        const float rstd_m = rs;
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            X::unpack(rx[i], h[i]);
            X::unpack(ry[i], t[i]);
            // columns past K hold x = dy = 0: t = 0 there, and h must be finite,
            // which -mean rstd need not be
            const int col = (i * T + tid) * V;
            const float mean_i = EVEN && col >= K ? 0.f : mu, rstd_i = EVEN && col >= K ? 0.f : rs;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                h[i][e] = (h[i][e] - mean_i) * rstd_i;
                if constexpr (!EVEN) h[i][e] = col + e < K ? h[i][e] : 0.f;
                if constexpr (PARAMS) {
                    aw[i][e] = __builtin_fmaf(t[i][e], h[i][e], aw[i][e]);
                    ab[i][e] += t[i][e];
                }
                t[i][e] *= param(wc[i], e);
                s1 += t[i][e];
                s2 = __builtin_fmaf(t[i][e], h[i][e], s2);
            }
        }
        fetch(m + step);
        if (!dxv) continue;
        s1 = wave_sum(s1);
        s2 = wave_sum(s2);
        if constexpr (W > 1) {
            if ((tid & 63) == 0) part[flip][group][tid >> 6] = make_float2(s1, s2);
            __syncthreads();  // the other half of `part` is the next row's
            s1 = s2 = 0.f;
#pragma unroll
            for (int k = 0; k < W; ++k) s1 += part[flip][group][k].x, s2 += part[flip][group][k].y;
        }
        const float c1 = s1 / (float)K, c2 = s2 / (float)K;
        if (m >= M) continue;
        E *dx = static_cast<E *>(dxv) + m * lddx;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int col = (i * T + tid) * V;
            float d[V];
#pragma unroll
            for (int e = 0; e < V; ++e) d[e] = rstd_m * __builtin_fmaf(-h[i][e], c2, t[i][e] - c1);
            if constexpr (EVEN) {
                if (col < K) X::store_chunk(dx + col, X::pack(d));
            } else {
                if (col < K) store_row_chunk<X>(dx, col, K, d);
            }
        }
    }
    if constexpr (PARAMS) {
        float *out = partials + (int64_t)blockIdx.x * 2 * (NCH * V * T);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int i = 0; i < NCH; ++i) {
                __syncthreads();
#pragma unroll
                for (int e = 0; e < V; ++e) sums[(group * V + e) * T + tid] = k ? ab[i][e] : aw[i][e];
                __syncthreads();
                for (int p = threadIdx.x; p < V * T; p += blockDim.x) {
                    float a = sums[p];
                    for (int g = 1; g < groups; ++g) a += sums[g * V * T + p];
                    out[(k * NCH + i) * V * T + p] = a;
                }
            }
        }
    }
}

// dw and db from `count` partials [2][positions]: 32 positions a workgroup, the
// partials split over its 32 threads for each.  T = 0: position = column.
__global__ __launch_bounds__(1024) void ln_reduce_kernel(const float *partials, int count, int64_t positions, int T,
                                                         int V, int K, float *dw, float *db) {
    __shared__ float part[32][33];
    const int lane = threadIdx.x & 31, split = threadIdx.x >> 5;
    const int64_t p = (int64_t)blockIdx.x * 32 + lane;
    float a = 0.f;
    if (p < 2 * positions) {
        float v[kMaxGroups / 32];
#pragma unroll
        for (int i = 0; i < kMaxGroups / 32; ++i) {
            const int g = split + 32 * i;
            v[i] = g < count ? partials[g * 2 * positions + p] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < kMaxGroups / 32; ++i) a += v[i];
    }
    part[split][lane] = a;
    __syncthreads();
    if (threadIdx.x >= 64) return;
    a = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) a += part[split * 16 + k][lane];
    a += __shfl_xor(a, 32);
    if (split != 0 || p >= 2 * positions) return;
    const int64_t q = p < positions ? p : p - positions;
    const int64_t col = T ? (q / ((int64_t)T * V) * T + q % T) * V + q / T % V : q;
    float *out = p < positions ? dw : db;
    if (out && col < K) out[col] = a;
}

// ------------------------------------------------------- streaming, backward
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

// One thread per column, the rows split over gridDim.y: partials [split][dw, db][K].
template <class X>
__global__ __launch_bounds__(kThreads) void ln_backward_params_kernel(const void *dyv, int64_t lddy, const void *xv,
                                                                      int64_t ldx, const float *mean,
                                                                      const float *rstd, int64_t M, int K,
                                                                      float *partials) {
    const int k = blockIdx.x * kThreads + threadIdx.x;
    if (k >= K) return;
    const auto *dy = static_cast<const typename X::type *>(dyv) + k;
    const auto *x = static_cast<const typename X::type *>(xv) + k;
    float sw = 0.f, sb = 0.f;
    for (int64_t m = blockIdx.y; m < M; m += gridDim.y) {
        const float g = X::load(dy + m * lddy);
        sb += g;
        sw = __builtin_fmaf(g, (X::load(x + m * ldx) - mean[m]) * rstd[m], sw);
    }
    float *out = partials + (int64_t)blockIdx.y * 2 * K;
    out[k] = sw;
    out[K + k] = sb;
}

// ---------------------------------------------------------------- host side
// How a row is shared: W waves, EPT elements per thread.  0 waves: the row
// does not fit and is streamed.
struct Layout {
    int W, ept;
};
// Forward: as few waves as 32 elements per thread allow.  The statistics cost
// each wave about 150 instructions and an exchange a row, whatever its length:
// at 8192 rows of 4096 bf16, 2 waves of 32 elements take 25.6 us (codes 26.0),
// 4 of 16 25.7 (26.3), 8 of 8 31 (38), 16 waves 52 (74).  24 elements fill
// widths between powers of two: 5120 takes 20.2 us with them, 21.3 with 32.
Layout forward_layout(int64_t K) {
    if (K <= 512) return {1, 8};
    if (K <= 1024) return {1, 16};
    for (int W = 1; W <= 8; W *= 2)
        for (int ept = 24; ept <= 32; ept += 8)
            if (K <= 64 * W * ept) return {W, ept};
    return {0, 0};
}
// Backward with the parameters' sums: 8 elements per thread, whose sums, rows
// in flight and weights fit 128 registers, 16 waves to a CU (8192 rows of 4096
// bf16: 43 us; 16 elements and 8 waves to a CU: 45).  5 waves fill widths a
// little past 2048 (2560: 30 us, 37 with 8).
Layout backward_layout(int64_t K) {
    for (int W : {1, 2, 4, 5, 8, 16})
        if (K <= 64 * W * 8) return {W, 8};
    return {0, 0};
}
// The input gradient alone keeps no sums: 16 elements per thread (8192 rows of
// 2048: 18.9 us against 26.8 with 8; of 4096: 36.4 against 38.1), 32 for the
// widest.
Layout backward_dx_layout(int64_t K) {
    if (K <= 512) return {1, 8};
    for (int W = 1; W <= 8; W *= 2)
        if (K <= 64 * W * 16) return {W, 16};
    return K <= 64 * 8 * 32 ? Layout{8, 32} : Layout{0, 0};
}

// Row groups per workgroup and workgroups of the backward kernel: few rows
// spread over all CUs first, many rows fill workgroups.
void backward_grid(int64_t M, Layout lay, int &groups, int &count) {
    const int most = backward_threads(lay.ept) / (64 * lay.W);
    const int64_t per = (M + kMaxGroups - 1) / kMaxGroups;
    groups = (int)(per < 1 ? 1 : per < most ? per : most);
    const int64_t n = (M + groups - 1) / groups;
    count = (int)(n < kMaxGroups ? (n < 1 ? 1 : n) : kMaxGroups);
}

template <class X, bool EVEN, int W, int EPT, int OUT>
void resident_launch(const void *x, int64_t M, int64_t K, int64_t ldx, int wt, const void *weight, const void *bias,
                     float eps, void *y, int64_t ldy, float *sx, float *mean, float *rstd, hipStream_t stream) {
    constexpr int per = kResidentThreads<W> / (64 * W);
    // 8 workgroups to a CU, each with the same number of rows
    constexpr int64_t most = 2048;
    const int64_t n = (M + per - 1) / per, rows = (n + most - 1) / most;
    const int grid = (int)((n + rows - 1) / rows);
    if (wt == W8A8_BF16)
        ln_resident_kernel<X, W8A8_BF16, EVEN, W, EPT / X::kVec, OUT><<<grid, kResidentThreads<W>, 0, stream>>>(
            x, M, ldx, (int)K, weight, bias, eps, y, ldy, sx, mean, rstd);
    else
        ln_resident_kernel<X, W8A8_F32, EVEN, W, EPT / X::kVec, OUT><<<grid, kResidentThreads<W>, 0, stream>>>(
            x, M, ldx, (int)K, weight, bias, eps, y, ldy, sx, mean, rstd);
}

template <class X, int OUT>
w8a8_status forward_launch(const void *x, int64_t M, int64_t K, int64_t ldx, int wt, const void *weight,
                           const void *bias, float eps, void *y, int64_t ldy, float *sx, float *mean, float *rstd,
                           hipStream_t stream) {
    const Layout lay = forward_layout(K);
#define W8A8_LN(W_, E_)                                                                                            \
    if (lay.W == W_ && lay.ept == E_) {                                                                            \
        if (K % X::kVec == 0)                                                                                      \
            resident_launch<X, true, W_, E_, OUT>(x, M, K, ldx, wt, weight, bias, eps, y, ldy, sx, mean, rstd, stream);  \
        else                                                                                                       \
            resident_launch<X, false, W_, E_, OUT>(x, M, K, ldx, wt, weight, bias, eps, y, ldy, sx, mean, rstd, stream); \
        return launch_status();                                                                                    \
    }
    W8A8_LN(1, 8) W8A8_LN(1, 16) W8A8_LN(1, 24) W8A8_LN(1, 32) W8A8_LN(2, 24) W8A8_LN(2, 32)
    W8A8_LN(4, 24) W8A8_LN(4, 32) W8A8_LN(8, 24) W8A8_LN(8, 32)
#undef W8A8_LN
    if constexpr (OUT == kOutNorm)
        ln_forward_kernel<X><<<(int)M, kThreads, 0, stream>>>(x, ldx, (int)K, wt, weight, bias, eps, y, ldy, mean, rstd);
    else
        ln_quant_kernel<X, OUT == kOutInt8 ? W8A8_INT8 : W8A8_FP8_E4M3><<<(int)M, kThreads, 0, stream>>>(
            x, ldx, (int)K, wt, weight, bias, eps, static_cast<uint8_t *>(y), ldy, sx, mean, rstd);
    return launch_status();
}

// Everything a backward launch takes.
struct BackwardArgs {
    const void *dy, *x, *weight;
    void *dx;
    const float *mean, *rstd;
    float *dweight, *dbias, *partials;
    int64_t lddy, ldx, lddx, M;
    int K, wt;
};

template <class X, int W, int EPT, bool PARAMS>
void backward_resident(const BackwardArgs &a, int grid, int groups, hipStream_t stream) {
    constexpr int NCH = EPT / X::kVec;
#define W8A8_LN(WT, EVEN)                                                                               \
    ln_backward_kernel<X, WT, EVEN, W, NCH, PARAMS><<<grid, 64 * W * groups, 0, stream>>>(              \
        a.dy, a.lddy, a.x, a.ldx, a.mean, a.rstd, a.M, a.K, a.weight, a.dx, a.lddx, a.partials)
    if (a.wt == W8A8_BF16) {
        if (a.K % X::kVec == 0) W8A8_LN(W8A8_BF16, true);
        else W8A8_LN(W8A8_BF16, false);
    } else {
        if (a.K % X::kVec == 0) W8A8_LN(W8A8_F32, true);
        else W8A8_LN(W8A8_F32, false);
    }
#undef W8A8_LN
}

// dx alone.
template <class X>
void backward_dx_launch(const BackwardArgs &a, hipStream_t stream) {
    if (a.M == 0) return;
    const Layout lay = backward_dx_layout(a.K);
#define W8A8_LN(W_, E_)                                                                                     \
    if (lay.W == W_ && lay.ept == E_) {                                                                     \
        constexpr int groups = W_ < 4 ? 4 / W_ : 1;                                                         \
        const int64_t n = (a.M + groups - 1) / groups;                                                      \
        return backward_resident<X, W_, E_, false>(a, (int)(n < kMaxGrid ? n : kMaxGrid), groups, stream);  \
    }
    W8A8_LN(1, 8) W8A8_LN(1, 16) W8A8_LN(2, 16) W8A8_LN(4, 16) W8A8_LN(8, 16) W8A8_LN(8, 32)
#undef W8A8_LN
    ln_backward_dx_kernel<X><<<(int)a.M, kThreads, 0, stream>>>(a.dy, a.lddy, a.x, a.ldx, a.mean, a.rstd, a.K, a.wt,
                                                                a.weight, a.dx, a.lddx);
}

template <class X>
w8a8_status backward_launch(const BackwardArgs &a, hipStream_t stream) {
    if (!a.dweight && !a.dbias) {
        if (a.dx) backward_dx_launch<X>(a, stream);
        return launch_status();
    }
    const Layout lay = backward_layout(a.K);
    int count = kStreamSplits, T = 0;
    int64_t positions = a.K;
    if (lay.W > 0) {
        int groups;
        backward_grid(a.M, lay, groups, count);
        T = 64 * lay.W;
        positions = (int64_t)T * lay.ept;
#define W8A8_LN(W_) \
    if (lay.W == W_) backward_resident<X, W_, 8, true>(a, count, groups, stream);
        W8A8_LN(1) W8A8_LN(2) W8A8_LN(4) W8A8_LN(5) W8A8_LN(8) W8A8_LN(16)
#undef W8A8_LN
    } else {
        // the parameters' sums first: dx may be dy
        const dim3 grid((unsigned)((a.K + kThreads - 1) / kThreads), (unsigned)count);
        ln_backward_params_kernel<X><<<grid, kThreads, 0, stream>>>(a.dy, a.lddy, a.x, a.ldx, a.mean, a.rstd, a.M, a.K,
                                                                    a.partials);
        if (a.dx) backward_dx_launch<X>(a, stream);
    }
    const w8a8_status st = launch_status();
    if (st != W8A8_OK) return st;
    ln_reduce_kernel<<<(int)((2 * positions + 31) / 32), 1024, 0, stream>>>(a.partials, count, positions, T, X::kVec, a.K,
                                                                           a.dweight, a.dbias);
    return launch_status();
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
        return forward_launch<Bf16, kOutNorm>(x, M, K, ldx, wt, weight, bias, eps, y, ldy, nullptr, mean, rstd, stream);
    return forward_launch<F32, kOutNorm>(x, M, K, ldx, wt, weight, bias, eps, y, ldy, nullptr, mean, rstd, stream);
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
#define W8A8_LN_QUANT(X, OUT) \
    forward_launch<X, OUT>(x, M, K, ldx, wt, weight, bias, eps, xq, ldq, x_scale, mean, rstd, stream)
    if (xt == W8A8_BF16) return qtype == W8A8_INT8 ? W8A8_LN_QUANT(Bf16, kOutInt8) : W8A8_LN_QUANT(Bf16, kOutE4m3);
    return qtype == W8A8_INT8 ? W8A8_LN_QUANT(F32, kOutInt8) : W8A8_LN_QUANT(F32, kOutE4m3);
#undef W8A8_LN_QUANT
}

extern "C" size_t layer_norm_backward_workspace_bytes(int64_t M, int64_t K) {
    using namespace w8a8;
    if (M < 0 || K < 1 || K > kMaxK) return 0;
    const Layout lay = backward_layout(K);
    if (lay.W == 0) return (size_t)(kStreamSplits * 2 * K * sizeof(float));
    int groups, count;
    backward_grid(M, lay, groups, count);
    return (size_t)count * 2 * (64 * lay.W * lay.ept) * sizeof(float);
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
    const BackwardArgs a = {dy,   x,   weight, dx, mean,   rstd, dweight, dbias, static_cast<float *>(workspace),
                            lddy, ldx, lddx,   M,  (int)K, wt};
    return xt == W8A8_BF16 ? backward_launch<Bf16>(a, stream) : backward_launch<F32>(a, stream);
}
