// The norm of all gradients and their scaling by it (model: include/ss_clip.h).
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "ss_clip.h"
#include "ss_internal.h"
#include "ss_profile.h"
#include "ss_vec.cuh"

namespace ss {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 64;           // tensors in one launch's parameters
constexpr int kGrid = 512;
constexpr int kTile = kThreads * 16; // elements of one CTA's step
constexpr int32_t kMaxTensors = 65536;

struct Table {
    const void *in[kBatch];
    void *out[kBatch];
    int64_t numel[kBatch];
    int64_t first[kBatch + 1];   // first tile of each tensor
    int dtype[kBatch];
    int count;
};

template <typename T>
__device__ float tile_squares(const T *p, int64_t lo, int64_t hi) {
    float s = 0.0f;
    for (int64_t i = lo + threadIdx.x; i < hi; i += kThreads) {
        const float v = to_float(p[i]);
        s = fmaf(v, v, s);
    }
    return s;
}

template <typename T>
__device__ void tile_scale(const T *in, T *out, int64_t lo, int64_t hi, float c) {
    for (int64_t i = lo + threadIdx.x; i < hi; i += kThreads) out[i] = c == 1.0f ? in[i] : from_float<T>(to_float(in[i]) * c);
}

__global__ void __launch_bounds__(kThreads) k_clip_squares(Table t, double *part) {
    __shared__ double s_red[kThreads / 32];
    double sum = 0.0;
    int k = 0;
    for (int64_t tile = blockIdx.x; tile < t.first[t.count]; tile += gridDim.x) {
        while (tile >= t.first[k + 1]) ++k;
        const int64_t lo = (tile - t.first[k]) * kTile;
        const int64_t hi = lo + kTile < t.numel[k] ? lo + kTile : t.numel[k];
        float s;
        if (t.dtype[k] == SS_F32)
            s = tile_squares(static_cast<const float *>(t.in[k]), lo, hi);
        else if (t.dtype[k] == SS_F16)
            s = tile_squares(static_cast<const __half *>(t.in[k]), lo, hi);
        else
            s = tile_squares(static_cast<const __nv_bfloat16 *>(t.in[k]), lo, hi);
        sum += s;
    }
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kThreads / 32; ++w) sum += s_red[w];
        part[blockIdx.x] = sum;
    }
}

__global__ void __launch_bounds__(kThreads) k_clip_result(const double *part, int parts, float max_norm, float eps,
                                                          bool clip, float *result) {
    __shared__ double s_red[kThreads / 32];
    double sum = 0.0;
    for (int i = threadIdx.x; i < parts; i += kThreads) sum += part[i];
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kThreads / 32; ++w) sum += s_red[w];
        const float norm = float(sqrt(sum));
        const bool fine = isfinite(norm);
        result[0] = norm;
        result[1] = !fine ? 0.0f : (clip ? fminf(1.0f, max_norm / (norm + eps)) : 1.0f);
    }
}

__global__ void __launch_bounds__(kThreads) k_clip_scale(Table t, const float *result) {
    const bool fine = isfinite(result[0]);
    const float c = fine ? result[1] : 1.0f;
    int k = 0;
    for (int64_t tile = blockIdx.x; tile < t.first[t.count]; tile += gridDim.x) {
        while (tile >= t.first[k + 1]) ++k;
        if (c == 1.0f && t.in[k] == t.out[k]) continue;
        const int64_t lo = (tile - t.first[k]) * kTile;
        const int64_t hi = lo + kTile < t.numel[k] ? lo + kTile : t.numel[k];
        if (t.dtype[k] == SS_F32)
            tile_scale(static_cast<const float *>(t.in[k]), static_cast<float *>(t.out[k]), lo, hi, c);
        else if (t.dtype[k] == SS_F16)
            tile_scale(static_cast<const __half *>(t.in[k]), static_cast<__half *>(t.out[k]), lo, hi, c);
        else
            tile_scale(static_cast<const __nv_bfloat16 *>(t.in[k]), static_cast<__nv_bfloat16 *>(t.out[k]), lo, hi, c);
    }
}

int batches(int32_t n) { return n < 1 ? 1 : (n + kBatch - 1) / kBatch; }

void fill(Table *t, const ss_tensor *h, int32_t n, int b) {
    t->count = 0;
    t->first[0] = 0;
    for (int32_t i = b * kBatch; i < n && i < (b + 1) * kBatch; ++i) {
        const int k = t->count++;
        t->in[k] = h[i].in, t->out[k] = h[i].out, t->numel[k] = h[i].numel, t->dtype[k] = h[i].dtype;
        t->first[k + 1] = t->first[k] + (h[i].numel + kTile - 1) / kTile;
    }
}

ss_status run(const char *who, const ss_tensor *h, int32_t n, bool clip, float max_norm, float eps, float *result,
              void *workspace, size_t bytes, cudaStream_t s) {
    clear_error();
    if (n < 0 || n > kMaxTensors)
        return fail(SS_ERR_UNSUPPORTED, "%s: %d tensors outside 0..%d", who, n, kMaxTensors);
    if (n > 0 && !h) return fail(SS_ERR_INVALID_ARG, "%s: the tensor list is NULL", who);
    if (!result || !aligned_to(result, 4)) return fail(SS_ERR_INVALID_ARG, "%s: result NULL or misaligned", who);
    if (clip && (!(max_norm >= 0.0f) || !(eps >= 0.0f)))
        return fail(SS_ERR_INVALID_ARG, "%s: max_norm or eps negative or NaN", who);
    int64_t total = 0;
    for (int32_t i = 0; i < n; ++i) {
        const ss_tensor &t = h[i];
        if (!dtype_known(t.dtype) || t.reserved != 0)
            return fail(SS_ERR_INVALID_ARG, "%s: tensor %d: unknown dtype or reserved not 0", who, i);
        if (t.numel < 0) return fail(SS_ERR_INVALID_ARG, "%s: tensor %d: numel < 0", who, i);
        if (t.numel == 0) continue;
        const size_t a = dtype_bytes(t.dtype);
        if (!t.in || !aligned_to(t.in, a) || (clip && (!t.out || !aligned_to(t.out, a))))
            return fail(SS_ERR_INVALID_ARG, "%s: tensor %d: a pointer is NULL or misaligned", who, i);
        if (t.numel >= (int64_t(1) << 40) || (total += t.numel) >= (int64_t(1) << 40))
            return fail(SS_ERR_UNSUPPORTED, "%s: 2^40 elements or more", who);
    }
    if (!workspace || !aligned_to(workspace, 256))
        return fail(SS_ERR_INVALID_ARG, "%s: workspace NULL or not 256-byte aligned", who);
    const size_t need = ss_clip_workspace_bytes(n);
    if (bytes < need) return fail(SS_ERR_INVALID_ARG, "%s: workspace %zu bytes < %zu", who, bytes, need);
    double *part = static_cast<double *>(workspace);
    Table t;
    for (int b = 0; b < batches(n); ++b) {
        fill(&t, h, n, b);
        SS_LAUNCH("k_clip_squares", s, k_clip_squares<<<kGrid, kThreads, 0, s>>>(t, part + size_t(b) * kGrid));
    }
    SS_LAUNCH("k_clip_result", s,
              k_clip_result<<<1, kThreads, 0, s>>>(part, batches(n) * kGrid, max_norm, eps, clip, result));
    if (clip)
        for (int b = 0; b < batches(n); ++b) {
            fill(&t, h, n, b);
            SS_LAUNCH("k_clip_scale", s, k_clip_scale<<<kGrid, kThreads, 0, s>>>(t, result));
        }
    return check_launch(who);
}

}  // namespace
}  // namespace ss

using namespace ss;

extern "C" {

size_t ss_clip_workspace_bytes(int32_t n_tensors) {
    if (n_tensors < 0 || n_tensors > kMaxTensors) return 0;
    return size_t(batches(n_tensors)) * kGrid * sizeof(double);
}

ss_status ss_grad_clip(const ss_tensor *h_tensors, int32_t n_tensors, float max_norm, float eps, float *result,
                       void *workspace, size_t workspace_bytes, ss_stream_t stream) {
    return run("ss_grad_clip", h_tensors, n_tensors, true, max_norm, eps, result, workspace, workspace_bytes,
               (cudaStream_t)stream);
}

ss_status ss_grad_norm(const ss_tensor *h_tensors, int32_t n_tensors, float *result, void *workspace,
                       size_t workspace_bytes, ss_stream_t stream) {
    return run("ss_grad_norm", h_tensors, n_tensors, false, 0.0f, 0.0f, result, workspace, workspace_bytes,
               (cudaStream_t)stream);
}

}  // extern "C"
