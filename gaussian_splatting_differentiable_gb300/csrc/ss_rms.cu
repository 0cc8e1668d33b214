// Root-mean-square norm, and the gradients of both norms from rows kept in 8
// bits (model: include/ss_rms.h).
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "ss_internal.h"
#include "ss_launch.cuh"
#include "ss_profile.h"
#include "ss_rms.h"
#include "ss_rows8.cuh"

namespace ss {
namespace {

constexpr int kThreads = 256;

template <typename T>
struct Rows {
    T *base;
    int64_t stride;
};

// Sum over the CTA, the same value in every thread (fixed order).
__device__ __forceinline__ float block_sum(float v, float *s_red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.0f;
    for (int w = 0; w < kThreads / 32; ++w) t += s_red[w];
    return t;
}

// What a warp's 32 consecutive columns hold, into 8 bits (v: 0 past the row).
template <int FMT>
__device__ __forceinline__ void put_group(const Rows8 &out, int64_t row, int j, int32_t held, float v) {
    const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(v) & 0x7fffffffu);
    const uint32_t e = exponent_of<FMT>(most);
    const float z = e == kNanExponent ? 0.0f : v * inverse_of(e);
    if (j < held) out.q[row * out.stride + j] = uint8_t(encode4<FMT>(z, 0.0f, 0.0f, 0.0f));
    if ((threadIdx.x & 31) == 0 && j < held) out.scales[row * out.scale_stride + j / kGroup] = uint8_t(e);
}
__device__ __forceinline__ void put_group(int fmt, const Rows8 &out, int64_t row, int j, int32_t held, float v) {
    if (fmt == SS_INT8)
        put_group<SS_INT8>(out, row, j, held, v);
    else
        put_group<SS_E4M3>(out, row, j, held, v);
}

struct FwdArgs {
    const void *x;
    int64_t xs;
    const void *residual;
    int64_t rs, n;
    int32_t D;
    const void *gamma;
    int pdt;
    float eps;
    void *sum;
    int64_t ss_;
    void *y;
    int64_t ys;
    Rows8 out, kept;
    int out_fmt, kept_fmt;     // -1: not wanted
    float *rstd;
};

// A CTA a row, an element a thread, the row read again for its result.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_rms_fwd_wide(FwdArgs a) {
    __shared__ float s_red[kThreads / 32];
    const int32_t held = (a.D + 7) / 8 * 8, padded = (a.D + 31) / 32 * 32;
    for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
        const T *x = static_cast<const T *>(a.x) + row * a.xs;
        T *sum = a.sum ? static_cast<T *>(a.sum) + row * a.ss_ : nullptr;
        const T *h = sum ? sum : x;
        float q = 0.0f;
        for (int j = threadIdx.x; j < a.D; j += kThreads) {
            float v = to_float(x[j]);
            if (sum) {
                sum[j] = from_float<T>(v + to_float(static_cast<const T *>(a.residual)[row * a.rs + j]));
                v = to_float(sum[j]);
            }
            q = fmaf(v, v, q);
        }
        const float r = __frsqrt_rn(block_sum(q, s_red) / float(a.D) + a.eps);
        for (int j0 = 0; j0 < padded; j0 += kThreads) {
            const int j = j0 + threadIdx.x;
            const bool here = j < a.D;
            const float v = here ? to_float(h[j]) : 0.0f;
            const float y = here ? v * r * (a.gamma ? load_param(a.gamma, a.pdt, j) : 1.0f) : 0.0f;
            if (a.y && here) static_cast<T *>(a.y)[row * a.ys + j] = from_float<T>(y);
            if (a.kept_fmt >= 0) put_group(a.kept_fmt, a.kept, row, j, held, v);
            if (a.out_fmt >= 0) put_group(a.out_fmt, a.out, row, j, held, y);
        }
        if (threadIdx.x == 0 && a.rstd) a.rstd[row] = r;
    }
}

struct BwdArgs {
    const void *dy;
    int64_t dys;
    const void *h;      // or kept
    int64_t hs;
    Rows8 kept;
    int fmt;            // -1: h
    int64_t n;
    int32_t D;
    const void *gamma;
    int pdt;
    const float *mean, *rstd;      // mean: the layer norm's
    const void *dsum;
    int64_t dss;
    void *dx;
    int64_t dxs;
    void *dgamma, *dbeta;
    float *part;
    bool centred;
};

template <typename T>
__device__ __forceinline__ float kept_value(const BwdArgs &a, int64_t row, int j) {
    if (a.fmt < 0) return to_float(static_cast<const T *>(a.h)[row * a.hs + j]);
    const uint8_t q = a.kept.q[row * a.kept.stride + j];
    const float s = scale_of(a.kept.scales[row * a.kept.scale_stride + j / kGroup]);
    return (a.fmt == SS_INT8 ? decode1<SS_INT8>(q) : decode1<SS_E4M3>(q)) * s;
}

// The weights' partial sums: thread = column, CTA y = a slice of the rows.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_norm8_bwd_weights_wide(BwdArgs a) {
    const int j = blockIdx.x * kThreads + threadIdx.x;
    if (j >= a.D) return;
    float dg = 0.0f, db = 0.0f;
    for (int64_t row = blockIdx.y; row < a.n; row += gridDim.y) {
        const float d = to_float(static_cast<const T *>(a.dy)[row * a.dys + j]);
        const float mu = a.centred ? a.mean[row] : 0.0f;
        dg = fmaf(d, (kept_value<T>(a, row, j) - mu) * a.rstd[row], dg);
        db += d;
    }
    a.part[size_t(blockIdx.y) * 2 * a.D + j] = dg;
    a.part[size_t(blockIdx.y) * 2 * a.D + a.D + j] = db;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_norm8_bwd_rows_wide(BwdArgs a) {
    __shared__ float s_red[kThreads / 32];
    for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
        const T *dy = static_cast<const T *>(a.dy) + row * a.dys;
        const float mu = a.centred ? a.mean[row] : 0.0f, r = a.rstd[row];
        float sa = 0.0f, sah = 0.0f;
        for (int j = threadIdx.x; j < a.D; j += kThreads) {
            const float v = to_float(dy[j]) * (a.gamma ? load_param(a.gamma, a.pdt, j) : 1.0f);
            sa += v;
            sah = fmaf(v, (kept_value<T>(a, row, j) - mu) * r, sah);
        }
        const float ma = a.centred ? block_sum(sa, s_red) / float(a.D) : 0.0f;
        const float mah = block_sum(sah, s_red) / float(a.D);
        for (int j = threadIdx.x; j < a.D; j += kThreads) {
            const float v = to_float(dy[j]) * (a.gamma ? load_param(a.gamma, a.pdt, j) : 1.0f);
            const float g = (kept_value<T>(a, row, j) - mu) * r;
            float d = r * (v - ma - g * mah);
            if (a.dsum) d += to_float(static_cast<const T *>(a.dsum)[row * a.dss + j]);
            static_cast<T *>(a.dx)[row * a.dxs + j] = from_float<T>(d);
        }
    }
}

// The partial sums of 32 columns of [dgamma | dbeta]: 32 slices of them side by
// side, then the slices in order.
__global__ void __launch_bounds__(1024) k_norm8_bwd_final(const float *part, int parts, int32_t D, void *dgamma,
                                                          void *dbeta, int pdt) {
    __shared__ float s_t[32][33];
    wait_for_previous();
    const int c = threadIdx.x & 31, q = threadIdx.x >> 5;
    const int j = blockIdx.x * 32 + c;
    float t = 0.0f;
    if (j < 2 * D)
#pragma unroll 4
        for (int p = q; p < parts; p += 32) t += part[size_t(p) * 2 * D + j];
    s_t[q][c] = t;
    __syncthreads();
    t = s_t[c][q];                         // column q of the 32, slice c
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    const int col = blockIdx.x * 32 + q;
    if (c != 0 || col >= 2 * D) return;
    if (col < D)
        store_param(dgamma, pdt, col, t);
    else if (dbeta)
        store_param(dbeta, pdt, col - D, t);
}

// Partial sums of the weights' gradients that the workspace has room for.
constexpr int kMaxParts = 1024;
int64_t weight_parts(int64_t n) { return n < 1 ? 1 : (n < kMaxParts ? n : kMaxParts); }
int wide_grid(int64_t n, int sms) { return int(n < int64_t(sms) * 8 ? n : int64_t(sms) * 8); }

ss_status backward(const char *who, const BwdArgs &a, int dtype, int sms, cudaStream_t s) {
    with_type(dtype, [&](auto t) {
        using T = decltype(t);
        // the weights first: dx may overwrite dy, dsum or h
        if (a.dgamma) {
            const dim3 g((a.D + kThreads - 1) / kThreads, unsigned(a.n < 64 ? (a.n < 1 ? 1 : a.n) : 64));
            SS_LAUNCH("k_norm8_bwd_weights_wide", s, k_norm8_bwd_weights_wide<T><<<g, kThreads, 0, s>>>(a));
            SS_LAUNCH("k_norm8_bwd_final", s,
                      launch_after(k_norm8_bwd_final, dim3((2 * a.D + 31) / 32), 1024, 0, s, a.part, int(g.y), a.D,
                                   a.dgamma, a.dbeta, a.pdt));
        }
        if (a.n > 0)
            SS_LAUNCH("k_norm8_bwd_rows_wide", s, k_norm8_bwd_rows_wide<T><<<wide_grid(a.n, sms), kThreads, 0, s>>>(a));
    });
    return check_launch(who);
}

}  // namespace
}  // namespace ss

using namespace ss;

extern "C" {

ss_status ss_rms_norm_fwd(const void *x, ss_dtype dtype, int64_t x_stride, const void *residual,
                          int64_t residual_stride, int64_t n, int32_t D, const void *gamma, ss_dtype param_dtype,
                          float eps, void *sum, int64_t sum_stride, void *y, int64_t y_stride, const ss_rows8 *out,
                          const ss_rows8 *kept, float *rstd, ss_stream_t stream) {
    clear_error();
    const char *who = "ss_rms_norm_fwd";
    ss_status st = check_row_sizes(who, n, D);
    if (st != SS_OK) return st;
    if ((st = check_row_types(who, dtype, param_dtype)) != SS_OK) return st;
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(SS_ERR_INVALID_ARG, "%s: eps negative or not finite", who);
    if (n == 0) return SS_OK;
    if ((st = check_row_tensor(who, "x", x, x_stride, D, dtype)) != SS_OK) return st;
    if ((residual == nullptr) != (sum == nullptr))
        return fail(SS_ERR_INVALID_ARG, "%s: one of residual and sum is NULL", who);
    if (residual) {
        if ((st = check_row_tensor(who, "residual", residual, residual_stride, D, dtype)) != SS_OK) return st;
        if ((st = check_row_tensor(who, "sum", sum, sum_stride, D, dtype)) != SS_OK) return st;
        if (sum == y) return fail(SS_ERR_INVALID_ARG, "%s: sum and y are the same rows", who);
    }
    if (y && (st = check_row_tensor(who, "y", y, y_stride, D, dtype)) != SS_OK) return st;
    if (out && (st = check_rows8(who, "out", out, D)) != SS_OK) return st;
    if (kept && (st = check_rows8(who, "kept", kept, D)) != SS_OK) return st;
    if (out && kept && out->q == kept->q) return fail(SS_ERR_INVALID_ARG, "%s: out and kept are the same rows", who);
    if ((st = check_aligned(who, "gamma", gamma, param_dtype)) != SS_OK) return st;
    if ((st = check_aligned(who, "rstd", rstd, SS_F32)) != SS_OK) return st;
    int dev = 0, sms = 0;
    if ((st = current_device(&dev, &sms, "ss_rms_norm_fwd: device query")) != SS_OK) return st;
    cudaStream_t s = (cudaStream_t)stream;
    const FwdArgs a{x, x_stride, residual, residual_stride, n, D, gamma, int(param_dtype), eps, sum, sum_stride, y,
                    y_stride, rows8_of(out), rows8_of(kept), out ? out->format : -1, kept ? kept->format : -1, rstd};
    with_type(dtype, [&](auto t) {
        using T = decltype(t);
        SS_LAUNCH("k_rms_fwd_wide", s, k_rms_fwd_wide<T><<<wide_grid(n, sms), kThreads, 0, s>>>(a));
    });
    return check_launch(who);
}

size_t ss_rms_norm_workspace_bytes(int64_t n, int32_t D) {
    return row_sizes_ok(n, D) ? size_t(weight_parts(n)) * 2 * D * sizeof(float) : 0;
}

size_t ss_layer_norm_bwd8_workspace_bytes(int64_t n, int32_t D) { return ss_rms_norm_workspace_bytes(n, D); }

ss_status ss_rms_norm_bwd(const void *dy, int64_t dy_stride, const void *h, int64_t h_stride, const ss_rows8 *kept,
                          ss_dtype dtype, int64_t n, int32_t D, const void *gamma, ss_dtype param_dtype,
                          const float *rstd, const void *dsum, int64_t dsum_stride, void *dx, int64_t dx_stride,
                          void *dgamma, void *workspace, size_t workspace_bytes, ss_stream_t stream) {
    clear_error();
    const char *who = "ss_rms_norm_bwd";
    ss_status st = check_row_sizes(who, n, D);
    if (st != SS_OK) return st;
    if ((st = check_row_types(who, dtype, param_dtype)) != SS_OK) return st;
    if (n > 0) {
        if ((st = check_row_tensor(who, "dy", dy, dy_stride, D, dtype)) != SS_OK) return st;
        if ((h == nullptr) == (kept == nullptr))
            return fail(SS_ERR_INVALID_ARG, "%s: one of h and kept is wanted, and not both", who);
        if (h && (st = check_row_tensor(who, "h", h, h_stride, D, dtype)) != SS_OK) return st;
        if (kept && (st = check_rows8(who, "kept", kept, D)) != SS_OK) return st;
        if (dsum && (st = check_row_tensor(who, "dsum", dsum, dsum_stride, D, dtype)) != SS_OK) return st;
        if ((st = check_row_tensor(who, "dx", dx, dx_stride, D, dtype)) != SS_OK) return st;
        if (!rstd) return fail(SS_ERR_INVALID_ARG, "%s: rstd is NULL", who);
        if ((st = check_aligned(who, "rstd", rstd, SS_F32)) != SS_OK) return st;
        if ((st = check_aligned(who, "gamma", gamma, param_dtype)) != SS_OK) return st;
    }
    if ((st = check_aligned(who, "dgamma", dgamma, param_dtype)) != SS_OK) return st;
    if (dgamma && (st = check_workspace(who, workspace, workspace_bytes, ss_rms_norm_workspace_bytes(n, D))) != SS_OK)
        return st;
    int dev = 0, sms = 0;
    if ((st = current_device(&dev, &sms, "ss_rms_norm_bwd: device query")) != SS_OK) return st;
    const BwdArgs a{dy, dy_stride, h, h_stride, rows8_of(kept), kept ? kept->format : -1, n, D, gamma,
                    int(param_dtype), nullptr, rstd, dsum, dsum_stride, dx, dx_stride, dgamma, nullptr,
                    static_cast<float *>(workspace), false};
    return backward(who, a, dtype, sms, (cudaStream_t)stream);
}

ss_status ss_layer_norm_bwd8(const void *dy, int64_t dy_stride, const ss_rows8 *kept, ss_dtype dtype, int64_t n,
                             int32_t D, const void *gamma, ss_dtype param_dtype, const float *mean, const float *rstd,
                             void *dx, int64_t dx_stride, void *dgamma, void *dbeta, void *workspace,
                             size_t workspace_bytes, ss_stream_t stream) {
    clear_error();
    const char *who = "ss_layer_norm_bwd8";
    ss_status st = check_row_sizes(who, n, D);
    if (st != SS_OK) return st;
    if ((st = check_row_types(who, dtype, param_dtype)) != SS_OK) return st;
    if (n > 0) {
        if ((st = check_row_tensor(who, "dy", dy, dy_stride, D, dtype)) != SS_OK) return st;
        if ((st = check_rows8(who, "kept", kept, D)) != SS_OK) return st;
        if ((st = check_row_tensor(who, "dx", dx, dx_stride, D, dtype)) != SS_OK) return st;
        if (!mean || !rstd) return fail(SS_ERR_INVALID_ARG, "%s: mean or rstd is NULL", who);
        if ((st = check_aligned(who, "mean", mean, SS_F32)) != SS_OK) return st;
        if ((st = check_aligned(who, "rstd", rstd, SS_F32)) != SS_OK) return st;
        if ((st = check_aligned(who, "gamma", gamma, param_dtype)) != SS_OK) return st;
    }
    if ((dgamma == nullptr) != (dbeta == nullptr))
        return fail(SS_ERR_INVALID_ARG, "%s: one of dgamma and dbeta is NULL", who);
    if ((st = check_aligned(who, "dgamma", dgamma, param_dtype)) != SS_OK) return st;
    if ((st = check_aligned(who, "dbeta", dbeta, param_dtype)) != SS_OK) return st;
    if (dgamma &&
        (st = check_workspace(who, workspace, workspace_bytes, ss_layer_norm_bwd8_workspace_bytes(n, D))) != SS_OK)
        return st;
    int dev = 0, sms = 0;
    if ((st = current_device(&dev, &sms, "ss_layer_norm_bwd8: device query")) != SS_OK) return st;
    const BwdArgs a{dy, dy_stride, nullptr, 0, rows8_of(kept), kept ? kept->format : -1, n, D, gamma,
                    int(param_dtype), mean, rstd, nullptr, 0, dx, dx_stride, dgamma, dbeta,
                    static_cast<float *>(workspace), true};
    return backward(who, a, dtype, sms, (cudaStream_t)stream);
}

}  // extern "C"
