// Element types and 16-byte vectors of the training operators.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "ss_dtype.h"

namespace ss {

inline size_t dtype_bytes(int dt) { return dt == SS_F32 ? 4 : 2; }
inline bool dtype_known(int dt) { return dt == SS_F32 || dt == SS_F16 || dt == SS_BF16; }
inline bool aligned_to(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// N elements of T, loaded and stored as one access (N * sizeof(T) <= 16
// bytes, address aligned to it) or, with 32 bytes, as two.
template <typename T, int N>
struct alignas(N * sizeof(T) > 16 ? 16 : N * sizeof(T)) Vec {
    T v[N];
};

template <typename T, int N>
__device__ __forceinline__ Vec<T, N> load_vec(const T *p) {
    return *reinterpret_cast<const Vec<T, N> *>(p);
}
template <typename T, int N>
__device__ __forceinline__ void store_vec(T *p, const Vec<T, N> &x) {
    *reinterpret_cast<Vec<T, N> *>(p) = x;
}

// Stores N floats rounded to T.
template <typename T, int N>
__device__ __forceinline__ void store_floats(T *p, const float (&f)[N]) {
    Vec<T, N> x;
#pragma unroll
    for (int k = 0; k < N; ++k) x.v[k] = from_float<T>(f[k]);
    store_vec<T, N>(p, x);
}

// One element of a parameter vector whose type is known at run time.
__device__ __forceinline__ float load_param(const void *p, int dtype, int64_t i) {
    if (dtype == SS_F32) return static_cast<const float *>(p)[i];
    if (dtype == SS_F16) return __half2float(static_cast<const __half *>(p)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}
__device__ __forceinline__ void store_param(void *p, int dtype, int64_t i, float v) {
    if (dtype == SS_F32)
        static_cast<float *>(p)[i] = v;
    else if (dtype == SS_F16)
        static_cast<__half *>(p)[i] = __float2half_rn(v);
    else
        static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
}

}  // namespace ss
