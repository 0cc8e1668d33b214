// What the kernels of a dense layer's weight gradient share.
//
// dW = dy^T x on the tensor cores, the rows being the sum's index: both operands
// lie in memory with their columns side by side ("MN-major"), and go into shared memory
// as they lie, 64 columns (128 bytes) to a row of a swizzled 8-row atom of 1 KB.
// x becomes bfloat16 on the way, which holds it exactly.  dy is one bfloat16, or is cut into
// as many as hold it exactly: hi, mid and lo of a float32's 24 bits, hi and lo of
// a float16's 11.  The tensor cores add a step's 16 products to a sum and cut it off at float32's last place, towards
// zero, so a long chain of steps loses a little of each sum: of summands of one sign and of many exponents 3.0e-6 after
// 2048 rows, in step with their number (of a few bits 1.7e-6 after 2048, 2.5e-6 after 2816, 7.6e-6 after 5632), of
// random signs 4.8e-7 after 2048 and 1.2e-6 after 4096; a float32 product by PyTorch is off by 1.0e-6 at most, to either
// side.  So the products of mid and lo have sums of their own (with hi's they would cut those off three times as
// often), and no sum stays in the tensor memory for more than a chain of rows, kChain32 where dW is float32; what it held
// then is added in float32.  That takes time: 150 us for 145 with chains of 2816 rows (2M x 48 x 48 float32), 249 for
// 228 (8191 x 4096 x 4096 bfloat16 into float32).  Where dW has 16 bits, chains of kChain16 lose up to 2.4e-5, which
// the rounding to 16 bits hides but for one value in several hundred that lies next to a border.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "ss_rows8.cuh"
#include "ss_unit.cuh"

namespace ss {

constexpr int kStep = 16;              // rows of one product
constexpr int kWide = 16;              // columns of x that a thread converts at a time
constexpr int kChain32 = 2048, kChain16 = 16384;    // rows of a chain; dW in float32, in 16 bits
// The split of the rows goes by this device's SMs as written down, and not as asked for: so the workspace's
// size, which is asked for without a device, and a result's bits depend on the sizes and types alone.
constexpr int kSms = 152;

template <typename T>
constexpr int parts_of() { return sizeof(T) == 4 ? 3 : (std::is_same<T, __half>::value ? 2 : 1); }

struct DenseArgs {
    const void *dy;
    int64_t dys;
    Rows8 x;
    int64_t n;
    int32_t N, D;
    int splits, bias_splits;
    int chain;            // stages of a chain of sums (weights past one tile)
    float *part;          // [splits][N][D], where sums leave the tensor memory before they are done
    float *part_bias;     // [bias_splits][N]
    void *dw;
    int64_t dws;
    void *db;
    int gdt;
    uint32_t tries;       // of a wait, after which it has run out
    int sent;             // stages that the copies stop after (a test's: none for all others)
};

// A bfloat16 holds the upper half of a float32's bits; what is left of the value is exact.
__device__ __forceinline__ uint32_t tops(F2 v) { return __byte_perm(__float_as_uint(v.x), __float_as_uint(v.y), 0x7632); }
__device__ __forceinline__ F2 rests(F2 v) {
    return add2(v, make_float2(-__uint_as_float(__float_as_uint(v.x) & 0xffff0000u),
                               -__uint_as_float(__float_as_uint(v.y) & 0xffff0000u)));
}
// An infinity or a NaN among them?  0 x is neither for all other values.
__device__ __forceinline__ bool any_special(const F2 (&f)[4]) {
    const F2 o = both(0.0f);
    const F2 z = fma2(f[0], o, fma2(f[1], o, fma2(f[2], o, mul2(f[3], o))));
    return !(z.x + z.y == 0.0f);
}

__device__ __forceinline__ void store16(uint32_t at, const uint32_t (&w)[4]) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
}
// A unit of dy as bfloat16s.  Of an infinity or a NaN hi holds all, a NaN with a bit that hi has, and
// there is no rest.
__device__ __forceinline__ void cut_parts(uint32_t (&w)[1][4], const Raw<__nv_bfloat16> &r) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[0][i] = r.w[i];
}
template <typename T>
__device__ __forceinline__ void cut_parts_special(uint32_t (&w)[parts_of<T>()][4], const Raw<T> &r) {
    F2 f[4];
    floats_of(f, r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float v[2] = {f[i].x, f[i].y};
#pragma unroll
        for (int p = 0; p < parts_of<T>(); ++p) {
            uint32_t top[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t u = __float_as_uint(v[k]);
                if ((u & 0x7fffffffu) > 0x7f800000u) u = 0x7fffffffu;
                top[k] = u >> 16;
                v[k] = (u & 0x7f800000u) == 0x7f800000u ? 0.0f : v[k] - __uint_as_float(u & 0xffff0000u);
            }
            w[p][i] = top[0] | top[1] << 16;
        }
    }
}
template <typename T>
__device__ __forceinline__ void cut_parts(uint32_t (&w)[parts_of<T>()][4], const Raw<T> &r) {
    F2 f[4];
    floats_of(f, r);
    if (any_special(f)) {
        cut_parts_special(w, r);
        return;
    }
#pragma unroll
    for (int p = 0; p < parts_of<T>(); ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[p][i] = tops(f[i]);
            if (p + 1 < parts_of<T>()) f[i] = rests(f[i]);
        }
}

// 16 columns of x as they are held, of which 8 or all are the row's.
struct Wide {
    uint32_t w[4], e;
    template <bool FAST>
    __device__ __forceinline__ void load(const uint8_t *pq, const uint8_t *ps, bool all) {
        if (FAST && all) {
            load_words(w, pq);
        } else {
            const uint2 u = *reinterpret_cast<const uint2 *>(pq);
            uint2 v = make_uint2(0u, 0u);
            if (all) v = *reinterpret_cast<const uint2 *>(pq + 8);
            w[0] = u.x, w[1] = u.y, w[2] = v.x, w[3] = v.y;
        }
        e = *ps;
    }
};
__device__ __forceinline__ uint32_t times(uint32_t a, uint32_t b) {      // pairs of bfloat16
    const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t minus(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}
// x in bfloat16, every step exact.  SS_E4M3: the byte's exponent and mantissa in a bfloat16's places are
// the value times 2^-120, subnormals too, which the scale makes good (in two factors where one
// would be past bfloat16's range); the format's NaN, seven ones, would be 480 so, and is put in afterwards, where a
// carry into bit 7 shows that there is one.  SS_INT8: the byte's lower seven bits as 128 .. 255, less 128, or
// 256 with the sign bit.
template <int FMT>
__device__ __forceinline__ void convert(uint32_t (&out)[8], const Wide &h) {
    uint32_t factor, more = 0, carries = 0;
    if (FMT == SS_INT8) {
        factor = h.e == kNanExponent ? 0x7fffu : (h.e == 0 ? 0x40u : h.e << 7);
    } else {
        const uint32_t e = h.e + 120u;
        factor = e > 254u ? 254u << 7 : e << 7;
        if (e > 254u) more = h.e == kNanExponent ? 0x7fffu : (e - 127u) << 7;
#pragma unroll
        for (int i = 0; i < 4; ++i) carries |= (h.w[i] & 0x7f7f7f7fu) + 0x01010101u;
    }
    factor |= factor << 16, more |= more << 16;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t w = h.w[i / 2];
        if (FMT == SS_INT8) {
            const uint32_t x = __byte_perm(w, 0u, i & 1 ? 0x4342 : 0x4140);
            out[i] = minus((x & 0x007f007fu) | 0x43004300u, (x & 0x00800080u) | 0x43004300u);
        } else {
            const uint32_t x = __byte_perm(w, 0u, i & 1 ? 0x3424 : 0x1404);
            out[i] = (x & 0x80008000u) | ((x & 0x7f007f00u) >> 4);
        }
        out[i] = times(out[i], factor);
    }
    if (FMT == SS_E4M3 && more)
#pragma unroll
        for (int i = 0; i < 8; ++i) out[i] = times(out[i], more);
    if (FMT == SS_E4M3 && (carries & 0x80808080u))
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t c = ((h.w[i / 2] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
            const uint32_t x = __byte_perm(c, 0u, i & 1 ? 0x3424 : 0x1404);    // 0x8000 in the NaNs' places
            out[i] |= x - (x >> 9);
        }
}

// A sum of products with dy's hi and those with its rests together.  A rest that is 0 makes NaN of an infinite x,
// where dy x is infinite; hi, which is 0, infinite or NaN where dy is (below 2^-133 it is 0), has it right, and
// whatever its sum reads as that is not finite, dW does too.
__device__ __forceinline__ float joined(float hi, float rests) { return isfinite(hi) ? hi + rests : hi; }

// 8 sums of a row of the tile (`count` of them the weight's) to float32 values at p, added to
// what is there or in its place.  No other thread has these, and a thread's additions to one
// address come in its own order, so the sum's order is fixed, and nobody waits for what was there.
__device__ __forceinline__ void put_sums(float *p, int count, const uint32_t (&v)[8], bool add) {
    const bool vectors = count == 8 && (reinterpret_cast<uintptr_t>(p) & 15) == 0;
    if (vectors) {
#pragma unroll
        for (int k = 0; k < 8; k += 4)
            if (add)
                asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p + k), "f"(__uint_as_float(v[k])),
                             "f"(__uint_as_float(v[k + 1])), "f"(__uint_as_float(v[k + 2])), "f"(__uint_as_float(v[k + 3]))
                             : "memory");
            else
                *reinterpret_cast<uint4 *>(p + k) = make_uint4(v[k], v[k + 1], v[k + 2], v[k + 3]);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < count) {
                if (add)
                    asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" ::"l"(p + k), "f"(__uint_as_float(v[k])) : "memory");
                else
                    p[k] = __uint_as_float(v[k]);
            }
    }
}
// The same as dW of 16 bits, with what is in `part` added where there is something.
__device__ __forceinline__ void put_rounded(const DenseArgs &a, int64_t e, const float *part, int count, uint32_t (&v)[8],
                                            bool add) {
    if (add)
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < count) v[k] = __float_as_uint(__uint_as_float(v[k]) + part[k]);
    uint16_t *at = static_cast<uint16_t *>(a.dw) + e;
    if (count == 8 && (reinterpret_cast<uintptr_t>(at) & 15) == 0) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float x = __uint_as_float(v[2 * k]), y = __uint_as_float(v[2 * k + 1]);
            w[k] = a.gdt == SS_F16 ? pack2<__half>(x, y) : pack2<__nv_bfloat16>(x, y);
        }
        *reinterpret_cast<uint4 *>(at) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < count) store_param(a.dw, a.gdt, e + k, __uint_as_float(v[k]));
    }
}

// Where 8 sums of a chain go: row i, columns from j on, of range `split`.
__device__ __forceinline__ void put(const DenseArgs &a, int split, int i, int j, int count, uint32_t (&v)[8], bool first, bool last) {
    const int64_t e = int64_t(i) * a.dws + j;
    float *part = a.part + (size_t(split) * a.N + i) * a.D + j;
    if (a.splits == 1 && a.gdt == SS_F32)
        put_sums(static_cast<float *>(a.dw) + e, count, v, !first);
    else if (a.splits == 1 && last)
        put_rounded(a, e, part, count, v, !first);
    else
        put_sums(part, count, v, !first);
}

// For weights past one tile (ss_dense_big.cu).
size_t dense_big_workspace(int64_t n, int32_t N, int32_t D, int dtype, int gdt);
ss_status dense_big(const char *who, DenseArgs a, int dtype, int format, void *workspace, cudaStream_t s, int sms);
// Adds up a.part and a.part_bias into the results, where they are there.
void dense_join(const DenseArgs &a, bool weight, cudaStream_t s, int sms);

}  // namespace ss
