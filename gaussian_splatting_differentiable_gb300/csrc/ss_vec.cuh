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

// N elements of T as they lie in memory: one of them, or 4, 8 or 16 bytes held
// as words (an array of 16-bit class types would be loaded element by
// element).
template <typename T, int N>
struct Vec {
    static constexpr int kWords = N * int(sizeof(T)) / 4;
    static_assert(kWords == 1 || kWords == 2 || kWords == 4, "a vector is 4, 8 or 16 bytes");
    uint32_t w[kWords];
    __device__ __forceinline__ float get(int i) const { return get_as(i, T()); }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0u;
    }
    // Element i as it is.
    __device__ __forceinline__ T elem(int i) const { return elem_as(i, T()); }
    // Puts element i in place (after clear()).
    __device__ __forceinline__ void set(int i, T v) { set_as(i, v); }

  private:
    __device__ __forceinline__ float elem_as(int i, float) const { return __uint_as_float(w[i]); }
    __device__ __forceinline__ __nv_bfloat16 elem_as(int i, __nv_bfloat16) const {
        return __ushort_as_bfloat16(static_cast<unsigned short>(w[i >> 1] >> (16 * (i & 1))));
    }
    __device__ __forceinline__ __half elem_as(int i, __half) const {
        return __ushort_as_half(static_cast<unsigned short>(w[i >> 1] >> (16 * (i & 1))));
    }
    __device__ __forceinline__ void set_as(int i, float v) { w[i] = __float_as_uint(v); }
    __device__ __forceinline__ void set_as(int i, __nv_bfloat16 v) {
        w[i >> 1] |= uint32_t(__bfloat16_as_ushort(v)) << (16 * (i & 1));
    }
    __device__ __forceinline__ void set_as(int i, __half v) {
        w[i >> 1] |= uint32_t(__half_as_ushort(v)) << (16 * (i & 1));
    }
    __device__ __forceinline__ float get_as(int i, float) const { return __uint_as_float(w[i]); }
    __device__ __forceinline__ float get_as(int i, __nv_bfloat16) const {
        return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    }
    __device__ __forceinline__ float get_as(int i, __half) const {
        return __half2float(__ushort_as_half(static_cast<unsigned short>(i & 1 ? w[i >> 1] >> 16 : w[i >> 1] & 0xffffu)));
    }
};
template <typename T>
struct Vec<T, 1> {
    T v;
    __device__ __forceinline__ float get(int) const { return to_float(v); }
    __device__ __forceinline__ void clear() { v = from_float<T>(0.0f); }
};

template <typename T, int N>
__device__ __forceinline__ Vec<T, N> load_vec(const T *p) {
    Vec<T, N> x;
    if constexpr (N == 1) {
        x.v = *p;
    } else if constexpr (Vec<T, N>::kWords == 1) {
        x.w[0] = *reinterpret_cast<const uint32_t *>(p);
    } else if constexpr (Vec<T, N>::kWords == 2) {
        const uint2 u = *reinterpret_cast<const uint2 *>(p);
        x.w[0] = u.x, x.w[1] = u.y;
    } else {
        const uint4 u = *reinterpret_cast<const uint4 *>(p);
        x.w[0] = u.x, x.w[1] = u.y, x.w[2] = u.z, x.w[3] = u.w;
    }
    return x;
}

// The same, and a store of it, marked to leave the caches first.
template <typename T, int N>
__device__ __forceinline__ Vec<T, N> load_vec_cs(const T *p) {
    const uint4 u = __ldcs(reinterpret_cast<const uint4 *>(p));
    Vec<T, N> x;
    x.w[0] = u.x, x.w[1] = u.y, x.w[2] = u.z, x.w[3] = u.w;
    return x;
}
template <typename T, int N>
__device__ __forceinline__ void store_vec_cs(T *p, const Vec<T, N> &x) {
    __stcs(reinterpret_cast<uint4 *>(p), make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]));
}

// Two floats rounded to T, the first in the low half.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// Stores N floats rounded to T: one of them, 4 or 8 bytes, or 16-byte pieces.
template <typename T, int N>
__device__ __forceinline__ void store_floats(T *p, const float (&f)[N]) {
    if constexpr (N == 1) {
        *p = from_float<T>(f[0]);
    } else if constexpr (N == 2 && sizeof(T) == 4) {
        *reinterpret_cast<float2 *>(p) = make_float2(f[0], f[1]);
    } else if constexpr (N == 2) {
        *reinterpret_cast<uint32_t *>(p) = pack2<T>(f[0], f[1]);
    } else if constexpr (N == 4 && sizeof(T) == 2) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]));
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int k = 0; k < N; k += 4)
            *reinterpret_cast<float4 *>(p + k) = make_float4(f[k], f[k + 1], f[k + 2], f[k + 3]);
    } else {
#pragma unroll
        for (int k = 0; k < N; k += 8)
            *reinterpret_cast<uint4 *>(p + k) =
                make_uint4(pack2<T>(f[k], f[k + 1]), pack2<T>(f[k + 2], f[k + 3]), pack2<T>(f[k + 4], f[k + 5]),
                           pack2<T>(f[k + 6], f[k + 7]));
    }
}

// Two float32 values in a register pair; sums, products and fused products
// of pairs take one instruction each.
using F2 = float2;
__device__ __forceinline__ F2 add2(F2 a, F2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ F2 mul2(F2 a, F2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ F2 both(float a) { return make_float2(a, a); }
__device__ __forceinline__ float sum_of(F2 a) {
    return a.x + a.y;
}

// The four words of a vector as pairs of floats, and back.
template <typename T, int N>
__device__ __forceinline__ void widen(F2 (&f)[N / 2], const Vec<T, N> &x) {
#pragma unroll
    for (int i = 0; i < N; i += 2) f[i / 2] = make_float2(x.get(i), x.get(i + 1));
}
template <typename T, int N>
__device__ __forceinline__ void store_pairs(T *p, const F2 (&f)[N / 2]) {
    float o[N];
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        o[i] = f[i / 2].x, o[i + 1] = f[i / 2].y;
    }
    store_floats<T, N>(p, o);
}

// The same marked to leave the caches first (16-byte pieces; others as they are).
template <typename T, int N>
__device__ __forceinline__ void store_floats_cs(T *p, const float (&f)[N]) {
    if constexpr (N * sizeof(T) == 16 && sizeof(T) == 4) {
        __stcs(reinterpret_cast<float4 *>(p), make_float4(f[0], f[1], f[2], f[3]));
    } else if constexpr (N * sizeof(T) == 16) {
        __stcs(reinterpret_cast<uint4 *>(p), make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]),
                                                        pack2<T>(f[6], f[7])));
    } else {
        store_floats<T, N>(p, f);
    }
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
