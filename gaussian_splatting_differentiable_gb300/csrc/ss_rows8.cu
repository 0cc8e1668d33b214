// Rows packed into 8 bits and unpacked (model: include/ss_rows8.h).
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "ss_internal.h"
#include "ss_profile.h"
#include "ss_rows8.cuh"

namespace ss {
namespace {

constexpr int kThreads = 256;

// A warp a group, a lane a column.
template <typename T, int FMT>
__global__ void __launch_bounds__(kThreads) k_rows8_pack(const T *x, int64_t xs, int64_t n, int32_t D, Rows8 out) {
    const int G = groups_of(D), lane = threadIdx.x & 31;
    const int64_t warps = int64_t(gridDim.x) * (kThreads / 32);
    const int32_t held = (D + 7) / 8 * 8;
    for (int64_t k = int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); k < n * G; k += warps) {
        const int64_t row = k / G;
        const int g = int(k - row * G), j = g * kGroup + lane;
        const float v = j < D ? to_float(x[row * xs + j]) : 0.0f;
        const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(v) & 0x7fffffffu);
        const uint32_t e = exponent_of<FMT>(most);
        const float z = e == kNanExponent ? 0.0f : v * inverse_of(e);
        if (j < held) out.q[row * out.stride + j] = uint8_t(encode4<FMT>(z, 0.0f, 0.0f, 0.0f));
        if (lane == 0) out.scales[row * out.scale_stride + g] = uint8_t(e);
    }
}

template <typename T>
__device__ __forceinline__ T held_to(float v) { return from_float<T>(v); }
// Finite values stay finite.
template <>
__device__ __forceinline__ __half held_to<__half>(float v) {
    return __float2half_rn(isnan(v) ? v : fminf(fmaxf(v, -65504.0f), 65504.0f));
}

template <typename T, int FMT>
__global__ void __launch_bounds__(kThreads) k_rows8_unpack(Rows8 in, int64_t n, int32_t D, T *x, int64_t xs) {
    for (int64_t row = blockIdx.x; row < n; row += gridDim.x)
        for (int j = threadIdx.x; j < D; j += kThreads)
            x[row * xs + j] = held_to<T>(decode1<FMT>(in.q[row * in.stride + j]) *
                                         scale_of(in.scales[row * in.scale_stride + j / kGroup]));
}

}  // namespace
}  // namespace ss

using namespace ss;

extern "C" {

ss_status ss_rows8_pack(const void *x, ss_dtype dtype, int64_t x_stride, int64_t n, int32_t D, const ss_rows8 *out,
                        ss_stream_t stream) {
    clear_error();
    const char *who = "ss_rows8_pack";
    ss_status st = check_row_sizes(who, n, D);
    if (st != SS_OK) return st;
    if ((st = check_row_types(who, dtype, SS_F32)) != SS_OK) return st;
    if (n == 0) return SS_OK;
    if ((st = check_row_tensor(who, "x", x, x_stride, D, dtype)) != SS_OK) return st;
    if ((st = check_rows8(who, "out", out, D)) != SS_OK) return st;
    int dev = 0, sms = 0;
    if ((st = current_device(&dev, &sms, "ss_rows8_pack: device query")) != SS_OK) return st;
    cudaStream_t s = (cudaStream_t)stream;
    const int64_t ctas = (n * groups_of(D) + kThreads / 32 - 1) / (kThreads / 32);
    const int grid = int(ctas < int64_t(sms) * 8 ? ctas : int64_t(sms) * 8);
    with_type(dtype, [&](auto t) {
        using T = decltype(t);
        SS_LAUNCH("k_rows8_pack", s,
                  (out->format == SS_INT8 ? k_rows8_pack<T, SS_INT8> : k_rows8_pack<T, SS_E4M3>)<<<grid, kThreads, 0, s>>>(
                      static_cast<const T *>(x), x_stride, n, D, rows8_of(out)));
    });
    return check_launch(who);
}

ss_status ss_rows8_unpack(const ss_rows8 *in, int64_t n, int32_t D, void *x, ss_dtype dtype, int64_t x_stride,
                          ss_stream_t stream) {
    clear_error();
    const char *who = "ss_rows8_unpack";
    ss_status st = check_row_sizes(who, n, D);
    if (st != SS_OK) return st;
    if ((st = check_row_types(who, dtype, SS_F32)) != SS_OK) return st;
    if (n == 0) return SS_OK;
    if ((st = check_rows8(who, "in", in, D)) != SS_OK) return st;
    if ((st = check_row_tensor(who, "x", x, x_stride, D, dtype)) != SS_OK) return st;
    int dev = 0, sms = 0;
    if ((st = current_device(&dev, &sms, "ss_rows8_unpack: device query")) != SS_OK) return st;
    cudaStream_t s = (cudaStream_t)stream;
    const int grid = int(n < int64_t(sms) * 8 ? n : int64_t(sms) * 8);
    with_type(dtype, [&](auto t) {
        using T = decltype(t);
        SS_LAUNCH("k_rows8_unpack", s,
                  (in->format == SS_INT8 ? k_rows8_unpack<T, SS_INT8> : k_rows8_unpack<T, SS_E4M3>)<<<grid, kThreads, 0, s>>>(
                      rows8_of(in), n, D, static_cast<T *>(x), x_stride));
    });
    return check_launch(who);
}

}  // extern "C"
