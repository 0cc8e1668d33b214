// Layer normalisation of rows and its gradient (model: include/ss_norm.h).
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "ss_internal.h"
#include "ss_norm.h"
#include "ss_profile.h"
#include "ss_vec.cuh"

namespace ss {
namespace {

constexpr int kThreads = 256;
constexpr int32_t kMaxD = 65536;

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

template <typename T>
__global__ void __launch_bounds__(kThreads) k_norm_fwd(const T *__restrict__ x, int64_t xs, int64_t n, int32_t D,
                                                       const void *gamma, const void *beta, int pdt, float eps, T *y,
                                                       int64_t ys, float *mean, float *rstd) {
    __shared__ float s_red[kThreads / 32];
    for (int64_t row = blockIdx.x; row < n; row += gridDim.x) {
        const T *xr = x + row * xs;
        float s = 0.0f;
        for (int j = threadIdx.x; j < D; j += kThreads) s += to_float(xr[j]);
        const float mu = block_sum(s, s_red) / float(D);
        s = 0.0f;
        for (int j = threadIdx.x; j < D; j += kThreads) {
            const float c = to_float(xr[j]) - mu;
            s += c * c;
        }
        const float r = 1.0f / sqrtf(block_sum(s, s_red) / float(D) + eps);
        for (int j = threadIdx.x; j < D; j += kThreads) {
            const float g = gamma ? load_param(gamma, pdt, j) : 1.0f;
            const float b = beta ? load_param(beta, pdt, j) : 0.0f;
            y[row * ys + j] = from_float<T>((to_float(xr[j]) - mu) * r * g + b);
        }
        if (threadIdx.x == 0) {
            if (mean) mean[row] = mu;
            if (rstd) rstd[row] = r;
        }
    }
}

// The weights' partial sums: thread = column, CTA y = a slice of the rows.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_norm_bwd_weights(const T *__restrict__ dy, int64_t dys,
                                                               const T *__restrict__ x, int64_t xs, int64_t n,
                                                               int32_t D, const float *mean, const float *rstd,
                                                               float *part) {
    const int j = blockIdx.x * kThreads + threadIdx.x;
    if (j >= D) return;
    float dg = 0.0f, db = 0.0f;
    for (int64_t row = blockIdx.y; row < n; row += gridDim.y) {
        const float d = to_float(dy[row * dys + j]);
        dg = fmaf(d, (to_float(x[row * xs + j]) - mean[row]) * rstd[row], dg);
        db += d;
    }
    part[size_t(blockIdx.y) * 2 * D + j] = dg;
    part[size_t(blockIdx.y) * 2 * D + D + j] = db;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_norm_bwd_rows(const T *dy, int64_t dys, const T *x, int64_t xs,
                                                            int64_t n, int32_t D, const void *gamma, int pdt,
                                                            const float *mean, const float *rstd, T *dx,
                                                            int64_t dxs) {
    __shared__ float s_red[kThreads / 32];
    for (int64_t row = blockIdx.x; row < n; row += gridDim.x) {
        const float mu = mean[row], r = rstd[row];
        float sa = 0.0f, sah = 0.0f;
        for (int j = threadIdx.x; j < D; j += kThreads) {
            const float a = to_float(dy[row * dys + j]) * (gamma ? load_param(gamma, pdt, j) : 1.0f);
            sa += a;
            sah = fmaf(a, (to_float(x[row * xs + j]) - mu) * r, sah);
        }
        const float ma = block_sum(sa, s_red) / float(D);
        const float mah = block_sum(sah, s_red) / float(D);
        for (int j = threadIdx.x; j < D; j += kThreads) {
            const float a = to_float(dy[row * dys + j]) * (gamma ? load_param(gamma, pdt, j) : 1.0f);
            const float h = (to_float(x[row * xs + j]) - mu) * r;
            dx[row * dxs + j] = from_float<T>(r * (a - ma - h * mah));
        }
    }
}

__global__ void __launch_bounds__(kThreads) k_norm_bwd_final(const float *part, int parts, int32_t D, void *dgamma,
                                                             void *dbeta, int pdt) {
    const int j = blockIdx.x * kThreads + threadIdx.x;
    if (j >= D) return;
    float dg = 0.0f, db = 0.0f;
    for (int p = 0; p < parts; ++p) {
        dg += part[size_t(p) * 2 * D + j];
        db += part[size_t(p) * 2 * D + D + j];
    }
    if (dgamma) store_param(dgamma, pdt, j, dg);
    if (dbeta) store_param(dbeta, pdt, j, db);
}

int64_t weight_parts(int64_t n) { return n < 1 ? 1 : (n < 512 ? n : 512); }

bool sizes_ok(int64_t n, int32_t D) { return n >= 0 && n < (int64_t(1) << 31) && D >= 1 && D <= kMaxD; }

ss_status check_rows(const char *who, const char *what, const void *p, int64_t stride, int32_t D, int dtype) {
    if (!p) return fail(SS_ERR_INVALID_ARG, "%s: %s is NULL", who, what);
    if (!aligned_to(p, dtype_bytes(dtype)))
        return fail(SS_ERR_INVALID_ARG, "%s: %s is not aligned to its type", who, what);
    if (stride < D || stride > (int64_t(1) << 31))
        return fail(SS_ERR_INVALID_ARG, "%s: %s stride %lld below D or above 2^31", who, what, (long long)stride);
    return SS_OK;
}

ss_status check_param(const char *who, const char *what, const void *p, int dtype) {
    if (p && !aligned_to(p, dtype_bytes(dtype)))
        return fail(SS_ERR_INVALID_ARG, "%s: %s is not aligned to its type", who, what);
    return SS_OK;
}

ss_status check_common(const char *who, int64_t n, int32_t D, int dtype, int pdt) {
    if (!sizes_ok(n, D))
        return fail(SS_ERR_UNSUPPORTED, "%s: %lld rows of %d outside 0..2^31-1 x 1..%d", who, (long long)n, D, kMaxD);
    if (!dtype_known(dtype)) return fail(SS_ERR_INVALID_ARG, "%s: unknown dtype %d", who, dtype);
    if (pdt != SS_F32 && pdt != dtype)
        return fail(SS_ERR_INVALID_ARG, "%s: param_dtype %d is neither SS_F32 nor the rows' type", who, pdt);
    return SS_OK;
}

template <typename T>
void launch_fwd(const void *x, int64_t xs, int64_t n, int32_t D, const void *gamma, const void *beta, int pdt,
                float eps, void *y, int64_t ys, float *mean, float *rstd, int sms, cudaStream_t s) {
    const int grid = int(n < int64_t(sms) * 8 ? n : int64_t(sms) * 8);
    SS_LAUNCH("k_norm_fwd", s,
              k_norm_fwd<T><<<grid, kThreads, 0, s>>>(static_cast<const T *>(x), xs, n, D, gamma, beta, pdt, eps,
                                                      static_cast<T *>(y), ys, mean, rstd));
}

template <typename T>
void launch_bwd(const void *dy, int64_t dys, const void *x, int64_t xs, int64_t n, int32_t D, const void *gamma,
                int pdt, const float *mean, const float *rstd, void *dx, int64_t dxs, void *dgamma, void *dbeta,
                float *part, int sms, cudaStream_t s) {
    // the weights first: dx may overwrite dy or x
    if (dgamma || dbeta) {
        const dim3 g((D + kThreads - 1) / kThreads, unsigned(weight_parts(n)));
        SS_LAUNCH("k_norm_bwd_weights", s,
                  k_norm_bwd_weights<T><<<g, kThreads, 0, s>>>(static_cast<const T *>(dy), dys,
                                                               static_cast<const T *>(x), xs, n, D, mean, rstd, part));
        SS_LAUNCH("k_norm_bwd_final", s,
                  k_norm_bwd_final<<<g.x, kThreads, 0, s>>>(part, int(g.y), D, dgamma, dbeta, pdt));
    }
    if (n == 0) return;
    const int grid = int(n < int64_t(sms) * 8 ? n : int64_t(sms) * 8);
    SS_LAUNCH("k_norm_bwd_rows", s,
              k_norm_bwd_rows<T><<<grid, kThreads, 0, s>>>(static_cast<const T *>(dy), dys,
                                                           static_cast<const T *>(x), xs, n, D, gamma, pdt, mean,
                                                           rstd, static_cast<T *>(dx), dxs));
}

}  // namespace
}  // namespace ss

using namespace ss;

extern "C" {

ss_status ss_layer_norm_fwd(const void *x, ss_dtype dtype, int64_t x_stride, int64_t n, int32_t D, const void *gamma,
                            const void *beta, ss_dtype param_dtype, float eps, void *y, int64_t y_stride, float *mean,
                            float *rstd, ss_stream_t stream) {
    clear_error();
    const char *who = "ss_layer_norm_fwd";
    ss_status st = check_common(who, n, D, dtype, param_dtype);
    if (st != SS_OK) return st;
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(SS_ERR_INVALID_ARG, "%s: eps negative or not finite", who);
    if (n == 0) return SS_OK;
    if ((st = check_rows(who, "x", x, x_stride, D, dtype)) != SS_OK) return st;
    if ((st = check_rows(who, "y", y, y_stride, D, dtype)) != SS_OK) return st;
    if ((st = check_param(who, "gamma", gamma, param_dtype)) != SS_OK) return st;
    if ((st = check_param(who, "beta", beta, param_dtype)) != SS_OK) return st;
    if ((st = check_param(who, "mean", mean, SS_F32)) != SS_OK) return st;
    if ((st = check_param(who, "rstd", rstd, SS_F32)) != SS_OK) return st;
    int dev = 0, sms = 0;
    if ((st = current_device(&dev, &sms, "ss_layer_norm_fwd: device query")) != SS_OK) return st;
    cudaStream_t s = (cudaStream_t)stream;
    if (dtype == SS_F32)
        launch_fwd<float>(x, x_stride, n, D, gamma, beta, param_dtype, eps, y, y_stride, mean, rstd, sms, s);
    else if (dtype == SS_F16)
        launch_fwd<__half>(x, x_stride, n, D, gamma, beta, param_dtype, eps, y, y_stride, mean, rstd, sms, s);
    else
        launch_fwd<__nv_bfloat16>(x, x_stride, n, D, gamma, beta, param_dtype, eps, y, y_stride, mean, rstd, sms, s);
    return check_launch(who);
}

size_t ss_layer_norm_workspace_bytes(int64_t n, int32_t D) {
    if (!sizes_ok(n, D)) return 0;
    return size_t(weight_parts(n)) * 2 * D * sizeof(float);
}

ss_status ss_layer_norm_bwd(const void *dy, int64_t dy_stride, const void *x, int64_t x_stride, ss_dtype dtype,
                            int64_t n, int32_t D, const void *gamma, ss_dtype param_dtype, const float *mean,
                            const float *rstd, void *dx, int64_t dx_stride, void *dgamma, void *dbeta,
                            void *workspace, size_t workspace_bytes, ss_stream_t stream) {
    clear_error();
    const char *who = "ss_layer_norm_bwd";
    ss_status st = check_common(who, n, D, dtype, param_dtype);
    if (st != SS_OK) return st;
    if (n > 0) {
        if ((st = check_rows(who, "dy", dy, dy_stride, D, dtype)) != SS_OK) return st;
        if ((st = check_rows(who, "x", x, x_stride, D, dtype)) != SS_OK) return st;
        if ((st = check_rows(who, "dx", dx, dx_stride, D, dtype)) != SS_OK) return st;
        if (!mean || !rstd) return fail(SS_ERR_INVALID_ARG, "%s: mean or rstd is NULL", who);
        if ((st = check_param(who, "mean", mean, SS_F32)) != SS_OK) return st;
        if ((st = check_param(who, "rstd", rstd, SS_F32)) != SS_OK) return st;
        if ((st = check_param(who, "gamma", gamma, param_dtype)) != SS_OK) return st;
    }
    if ((dgamma == nullptr) != (dbeta == nullptr))
        return fail(SS_ERR_INVALID_ARG, "%s: one of dgamma and dbeta is NULL", who);
    if ((st = check_param(who, "dgamma", dgamma, param_dtype)) != SS_OK) return st;
    if ((st = check_param(who, "dbeta", dbeta, param_dtype)) != SS_OK) return st;
    if (dgamma) {
        if (!workspace || !aligned_to(workspace, 256))
            return fail(SS_ERR_INVALID_ARG, "%s: workspace NULL or not 256-byte aligned", who);
        const size_t need = ss_layer_norm_workspace_bytes(n, D);
        if (workspace_bytes < need)
            return fail(SS_ERR_INVALID_ARG, "%s: workspace %zu bytes < %zu", who, workspace_bytes, need);
    }
    int dev = 0, sms = 0;
    if ((st = current_device(&dev, &sms, "ss_layer_norm_bwd: device query")) != SS_OK) return st;
    cudaStream_t s = (cudaStream_t)stream;
    float *part = static_cast<float *>(workspace);
    if (dtype == SS_F32)
        launch_bwd<float>(dy, dy_stride, x, x_stride, n, D, gamma, param_dtype, mean, rstd, dx, dx_stride, dgamma,
                          dbeta, part, sms, s);
    else if (dtype == SS_F16)
        launch_bwd<__half>(dy, dy_stride, x, x_stride, n, D, gamma, param_dtype, mean, rstd, dx, dx_stride, dgamma,
                           dbeta, part, sms, s);
    else
        launch_bwd<__nv_bfloat16>(dy, dy_stride, x, x_stride, n, D, gamma, param_dtype, mean, rstd, dx, dx_stride,
                                  dgamma, dbeta, part, sms, s);
    return check_launch(who);
}

}  // extern "C"
