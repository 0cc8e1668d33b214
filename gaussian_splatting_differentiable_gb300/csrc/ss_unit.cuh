// Eight consecutive elements of a row, the piece that a thread works on in the
// operators for activations in 8 bits: 8 bytes of a row in 8 bits, 16 of a
// 16-bit row, 32 of a float32 row; four of them, in four lanes side by side,
// share a scale.
//
// Rows start anywhere (to their type's alignment).  kAligned: every unit starts on
// a boundary of its size, and is one load or store.  kShifted: rows do not, but all tensors'
// rows alike; units lie on the boundaries, and the first and the last of a row are partly its.
// kAnyhow: units begin with the row, and a unit is cut out of
// the 16-byte vectors that hold it, the lanes of a warp side by side reading each
// vector twice (the second time from L1); and a store goes by vectors too, each
// put together from a lane's first elements and the lane before's last.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "ss_vec.cuh"

namespace ss {

constexpr int kUnit = 8;
__host__ __device__ inline int units_of(int32_t D) { return (D + kUnit - 1) / kUnit; }

enum Lie { kAligned, kShifted, kAnyhow };

template <typename T>
struct Raw {
    static constexpr int kWords = kUnit * int(sizeof(T)) / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0u;
    }
};

__device__ __forceinline__ void load_words(uint32_t (&w)[4], const void *p) {
    const uint4 u = *static_cast<const uint4 *>(p);
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
}
__device__ __forceinline__ void load_words(uint32_t (&w)[8], const void *p) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p) : "memory");
}
__device__ __forceinline__ void store_words(void *p, const uint32_t (&w)[4]) {
    *static_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store_words(void *p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

__device__ __forceinline__ void floats_of(F2 (&f)[4], const Raw<float> &r) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = make_float2(__uint_as_float(r.w[2 * i]), __uint_as_float(r.w[2 * i + 1]));
}
__device__ __forceinline__ void floats_of(F2 (&f)[4], const Raw<__half> &r) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __half22float2(*reinterpret_cast<const __half2 *>(&r.w[i]));
}
__device__ __forceinline__ void floats_of(F2 (&f)[4], const Raw<__nv_bfloat16> &r) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = make_float2(__uint_as_float(r.w[i] << 16), __uint_as_float(r.w[i] & 0xffff0000u));
}
template <typename T>
__device__ __forceinline__ Raw<T> raw_of(const F2 (&f)[4]) {
    Raw<T> r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4)
            r.w[2 * i] = __float_as_uint(f[i].x), r.w[2 * i + 1] = __float_as_uint(f[i].y);
        else
            r.w[i] = pack2<T>(f[i].x, f[i].y);
    }
    return r;
}

// Clears what lies past the first `count` elements.
template <typename T>
__device__ __forceinline__ void cut(Raw<T> &r, int count) {
#pragma unroll
    for (int i = 0; i < Raw<T>::kWords; ++i) {
        if constexpr (sizeof(T) == 4) {
            if (i >= count) r.w[i] = 0u;
        } else {
            if (2 * i >= count)
                r.w[i] = 0u;
            else if (2 * i + 1 >= count)
                r.w[i] &= 0xffffu;
        }
    }
}

// W words that begin `bytes` (0 .. 15) into the words of `a`.
template <int W, int N>
__device__ __forceinline__ void cut_out(uint32_t (&out)[W], uint32_t (&a)[N], int bytes) {
    static_assert(N >= W + 4, "");
    const bool two = bytes & 8, one = bytes & 4;
#pragma unroll
    for (int i = 0; i < W + 2; ++i)
        if (two) a[i] = a[i + 2];
#pragma unroll
    for (int i = 0; i < W + 1; ++i)
        if (one) a[i] = a[i + 1];
    const int bits = 8 * (bytes & 3);
#pragma unroll
    for (int i = 0; i < W; ++i) out[i] = __funnelshift_r(a[i], a[i + 1], bits);
}

// The unit at p, of which the first `count` elements (0 .. 8) are the row's; the
// others read as zeros, and no 16-byte block is touched that holds none of the row's.
template <typename T, bool ALIGNED>
__device__ __forceinline__ Raw<T> load_unit(const T *p, int count) {
    constexpr int W = Raw<T>::kWords;
    Raw<T> r;
    if (ALIGNED && count == kUnit) {
        load_words(r.w, p);
        return r;
    }
    if (count <= 0) {
        r.clear();
        return r;
    }
    const int o = int(reinterpret_cast<uintptr_t>(p) & 15);
    const uint4 *v = reinterpret_cast<const uint4 *>(reinterpret_cast<uintptr_t>(p) - o);
    const int bytes = o + count * int(sizeof(T));
    uint32_t a[W + 4];
#pragma unroll
    for (int k = 0; k < W / 4 + 1; ++k) {
        uint4 u = make_uint4(0u, 0u, 0u, 0u);
        if (bytes > 16 * k) u = v[k];
        a[4 * k] = u.x, a[4 * k + 1] = u.y, a[4 * k + 2] = u.z, a[4 * k + 3] = u.w;
    }
    cut_out<W>(r.w, a, o);
    if (count < kUnit) cut(r, count);
    return r;
}

// One element of a unit to memory.
template <typename T>
__device__ __forceinline__ void store_element(T *p, const Raw<T> &r, int i) {
    if constexpr (sizeof(T) == 4) {
        uint32_t w = r.w[0];
#pragma unroll
        for (int k = 1; k < Raw<T>::kWords; ++k)
            if (i == k) w = r.w[k];
        reinterpret_cast<uint32_t *>(p)[i] = w;
    } else {
        uint32_t w = r.w[0];
#pragma unroll
        for (int k = 1; k < Raw<T>::kWords; ++k)
            if ((i >> 1) == k) w = r.w[k];
        reinterpret_cast<uint16_t *>(p)[i] = static_cast<uint16_t>(i & 1 ? w >> 16 : w);
    }
}

// Four, two and one elements from element i on, a multiple of as many, at a place aligned for them.
template <typename T>
__device__ __forceinline__ void store_four(T *p, const Raw<T> &r, bool upper) {
    constexpr int H = Raw<T>::kWords / 2;
    if constexpr (H == 4)
        *reinterpret_cast<uint4 *>(p) = upper ? make_uint4(r.w[4], r.w[5], r.w[6], r.w[7]) : make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
    else
        *reinterpret_cast<uint2 *>(p) = upper ? make_uint2(r.w[2], r.w[3]) : make_uint2(r.w[0], r.w[1]);
}
template <typename T>
__device__ __forceinline__ void store_two(T *p, const Raw<T> &r, int i) {
    const bool u = i & 4, m = i & 2;
    if constexpr (sizeof(T) == 4) {
        const uint32_t a = m ? (u ? r.w[6] : r.w[2]) : (u ? r.w[4] : r.w[0]), b = m ? (u ? r.w[7] : r.w[3]) : (u ? r.w[5] : r.w[1]);
        *reinterpret_cast<uint2 *>(p) = make_uint2(a, b);
    } else {
        *reinterpret_cast<uint32_t *>(p) = m ? (u ? r.w[3] : r.w[1]) : (u ? r.w[2] : r.w[0]);
    }
}
// Elements [lo, hi) of the unit on the boundary p: of a part that begins or ends with the unit at most
// three pieces.
template <typename T>
__device__ __forceinline__ void store_range(T *p, const Raw<T> &r, int lo, int hi) {
    if (lo == 0) {
        if (hi & 4) store_four(p, r, false);
        if (hi & 2) store_two(p + (hi & 4), r, hi & 4);
        if (hi & 1) store_element(p, r, hi - 1);
    } else if (hi == kUnit) {
        if (lo & 1) store_element(p, r, lo);
        const int two = (lo + 1) & 6;                 // the even element from lo on
        if ((two & 2) != 0) store_two(p + two, r, two);
        if (lo <= 4) store_four(p + 4, r, true);
    } else {
        for (int i = lo; i < hi; ++i) store_element(p, r, i);
    }
}

// Stores the first `count` elements (0 .. 8) of the unit to p.  Every lane of the warp
// calls it, lanes without a unit with count 0.  prev, next: the lane before holds
// the row's unit before this one, the lane after the one after (with count > 0).
template <typename T, bool ALIGNED>
__device__ __forceinline__ void store_unit(T *p, const Raw<T> &r, int count, bool prev, bool next) {
    constexpr int W = Raw<T>::kWords, kSize = int(sizeof(T));
    if (ALIGNED) {
        if (count == kUnit)
            store_words(p, r.w);
        else if (count > 0)
            store_range(p, r, 0, count);
        return;
    }
    uint32_t before[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) before[i] = __shfl_up_sync(0xffffffffu, r.w[W - 4 + i], 1);
    if (count <= 0) return;
    const int o = int(reinterpret_cast<uintptr_t>(p) & 15), mine = count * kSize;
    if (o == 0) {
        uint4 *v = reinterpret_cast<uint4 *>(p);
        int done = 0;
#pragma unroll
        for (int k = 0; k < W / 4; ++k)
            if (mine >= 16 * (k + 1)) {
                v[k] = make_uint4(r.w[4 * k], r.w[4 * k + 1], r.w[4 * k + 2], r.w[4 * k + 3]);
                done = (k + 1) * 16 / kSize;
            }
        for (int i = done; i < count; ++i) store_element(p, r, i);
        return;
    }
    // the vectors that begin o bytes before p: the first takes the last o bytes of the unit before
    uint32_t a[W + 8], out[W];
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = before[i];
#pragma unroll
    for (int i = 0; i < W; ++i) a[4 + i] = r.w[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) a[W + 4 + i] = 0u;
    cut_out<W>(out, a, 16 - o);
    uint4 *v = reinterpret_cast<uint4 *>(reinterpret_cast<uintptr_t>(p) - o);
    int first = 0;                              // elements of this unit stored so far
#pragma unroll
    for (int k = 0; k < W / 4; ++k) {
        const int end = 16 * (k + 1) - o;       // bytes of this unit up to the vector's end
        if (mine >= end && (k > 0 || prev)) {
            v[k] = make_uint4(out[4 * k], out[4 * k + 1], out[4 * k + 2], out[4 * k + 3]);
            first = end / kSize;
        } else if (k == 0) {                    // in pieces: the unit before's end, where there is one, and this one's start
            if (prev) {
                Raw<T> u;
                u.clear();
#pragma unroll
                for (int i = 0; i < 4; ++i) u.w[W - 4 + i] = before[i];
                for (int i = kUnit - o / kSize; i < kUnit; ++i) store_element(p - kUnit, u, i);
            }
            const int stop = end / kSize < count ? end / kSize : count;
            for (int i = 0; i < stop; ++i) store_element(p, r, i);
            first = stop;
        }
    }
    // what is left: up to the unit's last o bytes, which the lane after stores where it holds the
    // next unit, and all of a short unit's
    const int last = next ? kUnit - o / kSize : count;
    for (int i = first; i < last; ++i) store_element(p, r, i);
}

// Clears all but elements [lo, hi).
template <typename T>
__device__ __forceinline__ void cut(Raw<T> &r, int lo, int hi) {
#pragma unroll
    for (int i = 0; i < Raw<T>::kWords; ++i) {
        if constexpr (sizeof(T) == 4) {
            if (i < lo || i >= hi) r.w[i] = 0u;
        } else {
            if (2 * i < lo || 2 * i >= hi) r.w[i] &= 0xffff0000u;
            if (2 * i + 1 < lo || 2 * i + 1 >= hi) r.w[i] &= 0xffffu;
        }
    }
}
// The unit on the boundary p, of which elements [lo, hi) are the row's; the others read as zeros.
template <typename T>
__device__ __forceinline__ Raw<T> load_block(const T *p, int lo, int hi) {
    Raw<T> r;
    if (lo >= hi) {
        r.clear();
        return r;
    }
    load_words(r.w, p);
    if (hi - lo < kUnit) cut(r, lo, hi);
    return r;
}
template <typename T>
__device__ __forceinline__ void store_block(T *p, const Raw<T> &r, int lo, int hi) {
    if (hi - lo == kUnit)
        store_words(p, r.w);
    else if (lo < hi)
        store_range(p, r, lo, hi);
}

// How far into its block of a unit's bytes p lies, in elements.
template <typename T>
__host__ __device__ inline int head_of(const void *p) {
    return int(reinterpret_cast<uintptr_t>(p) & (kUnit * sizeof(T) - 1)) / int(sizeof(T));
}
// Whether the rows of both start alike within blocks, and the rows after which starts repeat.
template <typename T>
inline bool start_alike(const void *a, int64_t as, const void *b, int64_t bs) {
    return head_of<T>(a) == head_of<T>(b) && (as - bs) % kUnit == 0;
}
inline int period_of(int64_t stride) {
    const int r = int(stride % kUnit);
    return r == 0 ? 1 : kUnit / (r & -r);
}

// Where rows of T allow units of one load or store.
template <typename T>
inline bool units_aligned(const void *p, int64_t stride) {
    constexpr int kBytes = kUnit * int(sizeof(T));
    return aligned_to(p, kBytes) && stride * int64_t(sizeof(T)) % kBytes == 0;
}

}  // namespace ss
