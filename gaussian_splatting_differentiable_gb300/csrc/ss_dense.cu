// The weight gradient of a dense layer from its input kept in 8 bits (model:
// include/ss_dense.h).
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "ss_dense.h"
#include "ss_internal.h"
#include "ss_profile.h"
#include "ss_rows8.cuh"

namespace ss {
namespace {

constexpr int kThreads = 256;
constexpr int kSide = 64;       // of a CTA's tile of the weight
constexpr int kDepth = 16;      // rows at a time

struct DenseArgs {
    const void *dy;
    int64_t dys;
    Rows8 x;
    int fmt;
    int64_t n;
    int32_t N, D;
    int64_t rows;         // of a split
    float *part;          // [splits][N][D], then [splits][N]
    float *part_bias;
};

// CTA (tile of D, tile of N, split): 4 x 4 values a thread, in float32.
template <typename T, int FMT>
__global__ void __launch_bounds__(kThreads) k_dense_part(DenseArgs a) {
    __shared__ float s_d[kDepth][kSide], s_x[kDepth][kSide];
    const int i0 = blockIdx.y * kSide, j0 = blockIdx.x * kSide;
    const int ti = threadIdx.x >> 4, tj = threadIdx.x & 15;
    float acc[4][4] = {}, bias = 0.0f;
    const int64_t first = int64_t(blockIdx.z) * a.rows, last = first + a.rows < a.n ? first + a.rows : a.n;
    for (int64_t m0 = first; m0 < last; m0 += kDepth) {
        __syncthreads();
        for (int k = threadIdx.x; k < kDepth * kSide; k += kThreads) {
            const int r = k / kSide, c = k % kSide;
            const int64_t m = m0 + r;
            s_d[r][c] = m < last && i0 + c < a.N ? to_float(static_cast<const T *>(a.dy)[m * a.dys + i0 + c]) : 0.0f;
            s_x[r][c] = m < last && j0 + c < a.D
                            ? decode1<FMT>(a.x.q[m * a.x.stride + j0 + c]) *
                                  scale_of(a.x.scales[m * a.x.scale_stride + (j0 + c) / kGroup])
                            : 0.0f;
        }
        __syncthreads();
        if (threadIdx.x < kSide)
            for (int r = 0; r < kDepth; ++r) bias += s_d[r][threadIdx.x];
        for (int r = 0; r < kDepth; ++r)
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[u][v] = fmaf(s_d[r][ti + 16 * u], s_x[r][tj + 16 * v], acc[u][v]);
    }
    float *part = a.part + size_t(blockIdx.z) * a.N * a.D;
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int i = i0 + ti + 16 * u, j = j0 + tj + 16 * v;
            if (i < a.N && j < a.D) part[size_t(i) * a.D + j] = acc[u][v];
        }
    if (blockIdx.x == 0 && threadIdx.x < kSide && i0 + threadIdx.x < a.N)
        a.part_bias[size_t(blockIdx.z) * a.N + i0 + threadIdx.x] = bias;
}

// The splits' sums in order; [N][D], then the bias.
__global__ void __launch_bounds__(kThreads) k_dense_join(DenseArgs a, int splits, void *dw, int64_t dws, void *db,
                                                         int gdt) {
    const int64_t all = int64_t(a.N) * a.D, count = all + (db ? a.N : 0);
    for (int64_t k = int64_t(blockIdx.x) * kThreads + threadIdx.x; k < count; k += int64_t(gridDim.x) * kThreads) {
        float t = 0.0f;
        for (int p = 0; p < splits; ++p) t += k < all ? a.part[size_t(p) * all + k] : a.part_bias[size_t(p) * a.N + (k - all)];
        if (k < all)
            store_param(dw, gdt, k / a.D * dws + k % a.D, t);
        else
            store_param(db, gdt, k - all, t);
    }
}

// How many ranges of rows have sums of their own: as many as give the device's
// SMs two tiles each, of 256 rows at least.
constexpr int kWanted = 304;
int splits_of(int64_t n, int32_t N, int32_t D) {
    const int64_t tiles = int64_t((N + kSide - 1) / kSide) * ((D + kSide - 1) / kSide);
    int64_t s = (kWanted + tiles - 1) / tiles;
    const int64_t most = (n + 255) / 256;
    if (s > most) s = most;
    return int(s < 1 ? 1 : s);
}

bool dense_sizes_ok(int64_t n, int32_t N, int32_t D) { return row_sizes_ok(n, D) && N >= 1 && N <= kMaxWidth; }

}  // namespace
}  // namespace ss

using namespace ss;

extern "C" {

size_t ss_dense_grad8_workspace_bytes(int64_t n, int32_t N, int32_t D) {
    if (!dense_sizes_ok(n, N, D)) return 0;
    return size_t(splits_of(n, N, D)) * N * (size_t(D) + 1) * sizeof(float);
}

ss_status ss_dense_grad8(const void *dy, ss_dtype dtype, int64_t dy_stride, const ss_rows8 *x, int64_t n, int32_t N,
                         int32_t D, void *dweight, int64_t dweight_stride, void *dbias, ss_dtype grad_dtype,
                         void *workspace, size_t workspace_bytes, ss_stream_t stream) {
    clear_error();
    const char *who = "ss_dense_grad8";
    if (!dense_sizes_ok(n, N, D))
        return fail(SS_ERR_UNSUPPORTED, "%s: %lld rows, %d x %d outside 0..2^31-1, 1..%d", who, (long long)n, N, D,
                    kMaxWidth);
    ss_status st = check_row_types(who, dtype, grad_dtype);
    if (st != SS_OK) return st;
    if (n > 0) {
        if ((st = check_row_tensor(who, "dy", dy, dy_stride, N, dtype)) != SS_OK) return st;
        if ((st = check_rows8(who, "x", x, D)) != SS_OK) return st;
    }
    if ((st = check_row_tensor(who, "dweight", dweight, dweight_stride, D, grad_dtype)) != SS_OK) return st;
    if ((st = check_aligned(who, "dbias", dbias, grad_dtype)) != SS_OK) return st;
    if ((st = check_workspace(who, workspace, workspace_bytes, ss_dense_grad8_workspace_bytes(n, N, D))) != SS_OK)
        return st;
    int dev = 0, sms = 0;
    if ((st = current_device(&dev, &sms, "ss_dense_grad8: device query")) != SS_OK) return st;
    cudaStream_t s = (cudaStream_t)stream;
    const int splits = splits_of(n, N, D);
    float *part = static_cast<float *>(workspace);
    const int64_t each = (n + splits - 1) / splits;
    const DenseArgs a{dy, dy_stride, rows8_of(x), x ? x->format : 0, n, N, D, (each + kDepth - 1) / kDepth * kDepth,
                      part, part + size_t(splits) * N * D};
    const dim3 grid((D + kSide - 1) / kSide, (N + kSide - 1) / kSide, splits);
    with_type(dtype, [&](auto t) {
        using T = decltype(t);
        SS_LAUNCH("k_dense_part", s,
                  (a.fmt == SS_INT8 ? k_dense_part<T, SS_INT8> : k_dense_part<T, SS_E4M3>)<<<grid, kThreads, 0, s>>>(a));
    });
    const int64_t ctas = (int64_t(N) * D + N + kThreads - 1) / kThreads;
    SS_LAUNCH("k_dense_join", s,
              k_dense_join<<<int(ctas < sms * 8 ? ctas : sms * 8), kThreads, 0, s>>>(a, splits, dweight, dweight_stride,
                                                                                    dbias, grad_dtype));
    return check_launch(who);
}

}  // extern "C"
