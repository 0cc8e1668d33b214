// Rows in 8 bits (model: include/ss_rows8.h): scales, encoding and decoding on
// the device, and the checks of arguments that their entry points share.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "ss_internal.h"
#include "ss_rows8.h"
#include "ss_unit.cuh"
#include "ss_vec.cuh"

namespace ss {

constexpr int kGroup = SS_ROWS8_GROUP;
constexpr uint32_t kLeastExponent = 16;    // 2^-111: what q s can be stays clear of subnormals
constexpr uint32_t kNanExponent = 255;

// An ss_rows8 as kernels take it.
struct Rows8 {
    uint8_t *q;
    int64_t stride;
    uint8_t *scales;
    int64_t scale_stride;
};
inline Rows8 rows8_of(const ss_rows8 *r) {
    return r ? Rows8{static_cast<uint8_t *>(r->q), r->q_stride, r->scales, r->scale_stride} : Rows8{};
}
__host__ __device__ inline int groups_of(int32_t D) { return (D + kGroup - 1) / kGroup; }

// The biased exponent of a group's scale, from the bits of its largest
// magnitude: the bits' exponent less Q's, one more where the mantissa is above
// Q's (which the addition carries into the exponent).
template <int FMT>
__device__ __forceinline__ uint32_t exponent_of(uint32_t bits) {
    constexpr uint32_t carry = FMT == SS_INT8 ? 0x7fffffu - 0x7e0000u : 0x7fffffu - 0x600000u;   // 127 = 1.984375 2^6, 448 = 1.75 2^8
    constexpr int top = FMT == SS_INT8 ? 6 : 8;
    const int e = int((bits + carry) >> 23) - top;
    return bits >= 0x7f800000u ? kNanExponent : uint32_t(e < int(kLeastExponent) ? int(kLeastExponent) : e);
}

// 1 / s for a scale that exponent_of gave and is not NaN's.
__device__ __forceinline__ float inverse_of(uint32_t e) { return __uint_as_float((254u - e) << 23); }
// s for any byte.
__device__ __forceinline__ float scale_of(uint32_t e) {
    return __uint_as_float(e == kNanExponent ? 0x7fffffffu : (e == 0 ? 0x400000u : e << 23));
}

// Four values, already divided by their scale, as bytes.  SS_INT8: 1.5 2^23 added in
// float32 rounds to a whole number, to nearest even, and leaves it in the low
// byte as two's complement.
template <int FMT>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
    if (FMT == SS_INT8) {
        const float m = 12582912.0f;
        const uint32_t u = __byte_perm(__float_as_uint(__fadd_rn(a, m)), __float_as_uint(__fadd_rn(b, m)), 0x0040);
        const uint32_t v = __byte_perm(__float_as_uint(__fadd_rn(c, m)), __float_as_uint(__fadd_rn(d, m)), 0x0040);
        return __byte_perm(u, v, 0x5410);
    }
    uint16_t u, v;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(u) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(v) : "f"(d), "f"(c));
    return uint32_t(u) | uint32_t(v) << 16;
}

// Four bytes as the float32 values that they hold before their scale.
// SS_INT8: the byte plus 128 below 2^23's exponent is 2^23 + q + 128.
template <int FMT>
__device__ __forceinline__ void decode4(F2 &a, F2 &b, uint32_t w) {
    if (FMT == SS_INT8) {
        const uint32_t u = w ^ 0x80808080u;
        const F2 off = both(-8388736.0f);
        a = add2(make_float2(__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440)),
                             __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7441))), off);
        b = add2(make_float2(__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7442)),
                             __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7443))), off);
        return;
    }
    uint32_t lo, hi;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"(uint16_t(w)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"(uint16_t(w >> 16)));
    a = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
    b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
}

template <int FMT>
__device__ __forceinline__ float decode1(uint8_t q) {
    F2 a, b;
    decode4<FMT>(a, b, q);
    return a.x;
}

// Of a group whose 32 values four lanes side by side hold, 8 each (zeros past the row; fewer
// lanes where the row has fewer columns): the biased exponent of its scale, in all of them.
template <int FMT>
__device__ __forceinline__ uint32_t group_exponent(const F2 (&f)[4], int lanes = 4) {
    // as whole numbers: NaN is the largest magnitude of all
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        m = max(m, max(__float_as_uint(f[i].x) & 0x7fffffffu, __float_as_uint(f[i].y) & 0x7fffffffu));
    if (lanes > 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    if (lanes > 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    return exponent_of<FMT>(m);
}

// Unit u of a row into 8 bits, with its group's exponent beside the first of the group.
template <int FMT>
__device__ __forceinline__ void put_unit(const Rows8 &out, int64_t row, int u, uint32_t e, const F2 (&f)[4]) {
    uint2 q = make_uint2(0u, 0u);
    if (e != kNanExponent) {
        const F2 inv = both(inverse_of(e));
        F2 z[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = mul2(f[i], inv);
        q = make_uint2(encode4<FMT>(z[0].x, z[0].y, z[1].x, z[1].y), encode4<FMT>(z[2].x, z[2].y, z[3].x, z[3].y));
    }
    *reinterpret_cast<uint2 *>(out.q + row * out.stride + u * kUnit) = q;
    if (u % (kGroup / kUnit) == 0) out.scales[row * out.scale_stride + u / (kGroup / kUnit)] = uint8_t(e);
}

// A unit as it is held.
struct Held {
    uint2 q;
    uint32_t e;
    __device__ __forceinline__ void load(const Rows8 &in, int64_t row, int u, bool here) {
        load(in.q + row * in.stride + u * kUnit, in.scales + row * in.scale_stride + u / (kGroup / kUnit), here);
    }
    __device__ __forceinline__ void load(const uint8_t *pq, const uint8_t *ps, bool here) {
        q = make_uint2(0u, 0u), e = 127u;
        if (!here) return;
        q = *reinterpret_cast<const uint2 *>(pq);
        e = *ps;
    }
    template <int FMT>
    __device__ __forceinline__ void values(F2 (&f)[4]) const {
        decode4<FMT>(f[0], f[1], q.x);
        decode4<FMT>(f[2], f[3], q.y);
        const F2 s = both(scale_of(e));
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = mul2(f[i], s);
    }
};

// Eight elements from column j on (j down to -7, where the first are not the row's and read as anything
// finite that the row's first group holds), which need not begin with a unit: bytes of two
// units, and scales of two groups where `edge`, the column where the second begins, is among them.
struct HeldAcross {
    uint2 a, b;
    uint32_t e0, e1;
    __device__ __forceinline__ void load(const Rows8 &in, int64_t row, int j, int32_t D, bool here) {
        a = b = make_uint2(0u, 0u), e0 = e1 = 127u;
        if (!here) return;
        const uint8_t *q = in.q + row * in.stride, *s = in.scales + row * in.scale_stride;
        const int u = j >> 3, last = (D - 1) / kUnit;              // units u and u + 1
        if (u >= 0) a = *reinterpret_cast<const uint2 *>(q + u * kUnit);
        if ((j & 7) && u < last) b = *reinterpret_cast<const uint2 *>(q + (u + 1) * kUnit);
        const int g = j < 0 ? 0 : j / kGroup, h = (j + kUnit - 1) / kGroup, most = (D - 1) / kGroup;
        e0 = s[g], e1 = s[h < most ? h : most];
    }
    template <int FMT>
    __device__ __forceinline__ void values(F2 (&f)[4], int j) const {
        const int off = j & 7, bits = 8 * (off & 3);
        const bool up = off & 4;
        const uint32_t w0 = up ? a.y : a.x, w1 = up ? b.x : a.y, w2 = up ? b.y : b.x;
        decode4<FMT>(f[0], f[1], __funnelshift_r(w0, w1, bits));
        decode4<FMT>(f[2], f[3], __funnelshift_r(w1, w2, bits));
        const float s0 = scale_of(e0), s1 = scale_of(e1);
        const int edge = kGroup - (j & (kGroup - 1));              // elements from here on are the second group's
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = mul2(f[i], make_float2(2 * i < edge ? s0 : s1, 2 * i + 1 < edge ? s0 : s1));
    }
};

// ------------------------------------------------------------------ checks

constexpr int32_t kMaxWidth = 65536;
inline bool row_sizes_ok(int64_t n, int32_t D) { return n >= 0 && n < (int64_t(1) << 31) && D >= 1 && D <= kMaxWidth; }

inline ss_status check_row_sizes(const char *who, int64_t n, int32_t D) {
    if (!row_sizes_ok(n, D))
        return fail(SS_ERR_UNSUPPORTED, "%s: %lld rows of %d outside 0..2^31-1 x 1..%d", who, (long long)n, D, kMaxWidth);
    return SS_OK;
}
inline ss_status check_row_types(const char *who, int dtype, int pdt) {
    if (!dtype_known(dtype)) return fail(SS_ERR_INVALID_ARG, "%s: unknown dtype %d", who, dtype);
    if (pdt != SS_F32 && pdt != dtype)
        return fail(SS_ERR_INVALID_ARG, "%s: type %d of the weights is neither SS_F32 nor the rows' type", who, pdt);
    return SS_OK;
}
inline ss_status check_row_tensor(const char *who, const char *what, const void *p, int64_t stride, int32_t D, int dtype) {
    if (!p) return fail(SS_ERR_INVALID_ARG, "%s: %s is NULL", who, what);
    if (!aligned_to(p, dtype_bytes(dtype)))
        return fail(SS_ERR_INVALID_ARG, "%s: %s is not aligned to its type", who, what);
    if (stride < D || stride > (int64_t(1) << 31))
        return fail(SS_ERR_INVALID_ARG, "%s: %s stride %lld below %d or above 2^31", who, what, (long long)stride, D);
    return SS_OK;
}
inline ss_status check_aligned(const char *who, const char *what, const void *p, int dtype) {
    if (p && !aligned_to(p, dtype_bytes(dtype)))
        return fail(SS_ERR_INVALID_ARG, "%s: %s is not aligned to its type", who, what);
    return SS_OK;
}
inline ss_status check_rows8(const char *who, const char *what, const ss_rows8 *r, int32_t D) {
    if (!r) return fail(SS_ERR_INVALID_ARG, "%s: %s is NULL", who, what);
    if (r->format != SS_INT8 && r->format != SS_E4M3)
        return fail(SS_ERR_INVALID_ARG, "%s: %s has the unknown format %d", who, what, r->format);
    if (r->reserved != 0) return fail(SS_ERR_INVALID_ARG, "%s: %s: reserved is not 0", who, what);
    if (!r->q || !r->scales) return fail(SS_ERR_INVALID_ARG, "%s: %s: q or scales is NULL", who, what);
    if (!aligned_to(r->q, 8)) return fail(SS_ERR_INVALID_ARG, "%s: %s: q is not 8-byte aligned", who, what);
    if (r->q_stride % 8 != 0 || r->q_stride < (D + 7) / 8 * 8 || r->q_stride > (int64_t(1) << 31))
        return fail(SS_ERR_INVALID_ARG, "%s: %s: q_stride %lld is no multiple of 8 that holds %d, or above 2^31", who,
                    what, (long long)r->q_stride, D);
    if (r->scale_stride < groups_of(D) || r->scale_stride > (int64_t(1) << 31))
        return fail(SS_ERR_INVALID_ARG, "%s: %s: scale_stride %lld below %d or above 2^31", who, what,
                    (long long)r->scale_stride, groups_of(D));
    return SS_OK;
}
inline ss_status check_workspace(const char *who, const void *ws, size_t have, size_t need) {
    if (!ws || !aligned_to(ws, 256))
        return fail(SS_ERR_INVALID_ARG, "%s: workspace NULL or not 256-byte aligned", who);
    if (have < need) return fail(SS_ERR_INVALID_ARG, "%s: workspace %zu bytes < %zu", who, have, need);
    return SS_OK;
}

// f of a type, of a format, for run-time codes.
template <typename F>
void with_type(int dtype, F &&f) {
    if (dtype == SS_F32)
        f(float());
    else if (dtype == SS_F16)
        f(__half());
    else
        f(__nv_bfloat16());
}

template <typename F>
void with_format(int format, F &&f) {
    if (format == SS_INT8)
        f(std::integral_constant<int, SS_INT8>());
    else
        f(std::integral_constant<int, SS_E4M3>());
}

}  // namespace ss
