// The weight gradient of a dense layer from its input kept in 8 bits (model:
// include/ss_dense.h).
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <type_traits>

#include "ss_dense.h"
#include "ss_internal.h"
#include "ss_profile.h"
#include "ss_rows8.cuh"
#include "ss_unit.cuh"

namespace ss {
namespace {

// dW = dy^T x on the tensor cores, the rows being the sum's index: both operands
// lie in memory with their columns side by side ("MN-major"), and go into shared memory
// as they lie, 64 columns (128 bytes) to a row of a swizzled 8-row atom of 1 KB.
// x becomes bfloat16 on the way, which holds it exactly.  dy is one bfloat16, or is cut into
// as many as hold it exactly: hi, mid and lo of a float32's 24 bits, hi and lo of
// a float16's 11.  The tensor cores cut every addition off at float32's last place, towards
// zero, so a long chain of them loses a little of each sum: after 2048 rows 5e-7 of it.
// So the products of mid and lo have sums of their own (with hi's they would cut those off
// three times as often), and where dW is float32 the sums leave the tensor memory every
// kChain32 rows and are added in float32.
//
// A CTA has a tile TI x TJ of dW over a range of rows, stages of which go through a ring
// in shared memory.  A bfloat16 dy needs no change: where it lies on 16-byte boundaries (FAST), a
// thread has the copy engine bring it.  All else passes through the registers of
// the loader warps, kAhead stages before it is converted and stored.  One thread of another
// warp issues the products; at the end of a chain the loaders read the sums out of the tensor memory.
constexpr int kStep = 16;              // rows of one product
constexpr int kWide = 16;              // columns of x that a thread converts at a time

template <typename T>
constexpr int parts_of() { return sizeof(T) == 4 ? 3 : (std::is_same<T, __half>::value ? 2 : 1); }

template <typename T, int TI, int TJ>
struct Config {
    static constexpr int kParts = parts_of<T>();
    static constexpr bool kLarge = TJ == 256;
    static constexpr int kSums = kParts > 1 ? 2 : 1;
    static constexpr int kLoaders = kLarge ? 512 : 256;
    static constexpr int kThreads = kLoaders + 64;                  // and the warps of the products and of the copies
    static constexpr int kRows = kParts == 3 && TJ > 64 ? 32 : 64;  // of a stage
    static constexpr int kBlock = kRows * 128;                      // bytes of 64 columns of a stage
    static constexpr int kABytes = TI / 64 * kBlock, kBBytes = TJ / 64 * kBlock;
    static constexpr int kStageBytes = kParts * kABytes + kBBytes;
    static constexpr int kStages = kLarge ? 200 * 1024 / kStageBytes : (kParts == 1 ? 3 : 2);
    static constexpr int kSmem = kStages * kStageBytes + 1024;      // and up to the first 1 KB boundary
    static constexpr int kAhead = kParts == 3 && !kLarge ? 1 : 2;
    static constexpr int kTurnsA = kRows * (TI / kUnit) / kLoaders;
    static constexpr int kTurnsB = kRows * (TJ / kWide) / kLoaders < 1 ? 1 : kRows * (TJ / kWide) / kLoaders;
    static constexpr int kTile = TI / 128 * TJ;                     // columns of tensor memory for one set of sums
    static constexpr int kColumns = kSums * kTile;
    static constexpr int kMinCtas = kLarge ? 1 : 2;
};

struct DenseArgs {
    const void *dy;
    int64_t dys;
    Rows8 x;
    int64_t n;
    int32_t N, D;
    int64_t rows;         // of a split
    int splits;
    int chain;            // stages of a chain of sums, a multiple of kAhead
    float *part;          // [splits][N][D], then [splits][N]; not used by one split of one chain, or into float32
    float *part_bias;
    void *dw;
    int64_t dws;
    void *db;
    int gdt;
};

// ---- tensor core and barrier instructions

__device__ __forceinline__ uint32_t smem_of(const void *p) { return uint32_t(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void barrier_init(uint64_t *b, uint32_t count) {
    asm volatile("mbarrier.init.shared.b64 [%0], %1;" ::"r"(smem_of(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void barrier_arrive(uint64_t *b) {
    asm volatile("mbarrier.arrive.shared.b64 _, [%0];" ::"r"(smem_of(b)) : "memory");
}
// Waits for the phase of that parity to end; false after some seconds, when something has gone
// wrong.
__device__ __forceinline__ bool barrier_wait(uint64_t *b, uint32_t parity) {
    for (uint32_t k = 0; k < (1u << 20); ++k) {
        uint32_t done;
        asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
                     : "=r"(done) : "r"(smem_of(b)), "r"(parity) : "memory");
        if (done) return true;
    }
    return false;
}
__device__ __forceinline__ void writes_to_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// A box of 64 columns (kRows rows) at (column, row), zeros outside the matrix.
__device__ __forceinline__ void copy_box(uint32_t smem, const CUtensorMap *map, int column, int row, uint64_t *b) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
                 ::"r"(smem), "l"(map), "r"(column), "r"(row), "r"(smem_of(b)) : "memory");
}
__device__ __forceinline__ void barrier_expect(uint64_t *b, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared.b64 _, [%0], %1;" ::"r"(smem_of(b)), "r"(bytes) : "memory");
}

// 64 columns of 128 bytes a row, swizzled, columns side by side: blocks of 64
// columns BLOCK apart, groups of 8 rows 1 KB apart.
template <int BLOCK>
__device__ __forceinline__ uint64_t operand_at(uint32_t smem) {
    return uint64_t((smem & 0x3ffff) >> 4) | uint64_t(BLOCK >> 4) << 16 | uint64_t(1024 >> 4) << 32 | uint64_t(1) << 46 |
           uint64_t(2) << 61;
}
// bfloat16 x bfloat16 into float32, both operands MN-major, 128 x n.
__device__ __forceinline__ uint32_t product_of(int n) {
    return 1u << 4 | 1u << 7 | 1u << 10 | 1u << 15 | 1u << 16 | uint32_t(n >> 3) << 17 | uint32_t(128 >> 4) << 24;
}
__device__ __forceinline__ void product(uint32_t d, uint64_t a, uint64_t b, uint32_t what, bool add) {
    asm volatile("{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\n"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d), "l"(a), "l"(b), "r"(what),
                 "r"(uint32_t(add)) : "memory");
}
__device__ __forceinline__ void products_arrive(uint64_t *b) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_of(b)) : "memory");
}
__device__ __forceinline__ void tensor_load8(uint32_t (&v)[8], uint32_t at) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(at));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// ---- conversion

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
// Such a unit: hi holds all of them, a NaN with a bit that hi has, and there is no rest.
template <int APART, int PARTS>
__device__ __noinline__ void store_special(uint32_t at, float2 f0, float2 f1, float2 f2, float2 f3) {
    float f[8] = {f0.x, f0.y, f1.x, f1.y, f2.x, f2.y, f3.x, f3.y};
    for (int p = 0; p < PARTS; ++p) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t u = __float_as_uint(f[i]);
            if ((u & 0x7fffffffu) > 0x7f800000u) u = 0x7fffffffu;
            const bool special = (u & 0x7f800000u) == 0x7f800000u;
            w[i / 2] = i & 1 ? (w[i / 2] & 0xffffu) | (u & 0xffff0000u) : u >> 16;
            f[i] = special ? 0.0f : f[i] - __uint_as_float(u & 0xffff0000u);
        }
        store16(at + p * APART, w);
    }
}
template <int APART>
__device__ __forceinline__ void store_parts(uint32_t at, const Raw<__nv_bfloat16> &r) { store16(at, r.w); }
template <int APART, typename T>
__device__ __forceinline__ void store_parts(uint32_t at, const Raw<T> &r) {
    F2 f[4];
    floats_of(f, r);
    if (any_special(f)) {
        store_special<APART, parts_of<T>()>(at, f[0], f[1], f[2], f[3]);
        return;
    }
#pragma unroll
    for (int p = 0; p < parts_of<T>(); ++p) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = tops(f[i]);
            if (p + 1 < parts_of<T>()) f[i] = rests(f[i]);
        }
        store16(at + p * APART, w);
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
// would be past bfloat16's range).  SS_INT8: the byte's lower seven bits as 128 .. 255, less 128, or
// 256 with the sign bit.
template <int FMT>
__device__ __forceinline__ void store_held(uint32_t at, const Wide &h) {
    uint32_t factor, more = 0;
    if (FMT == SS_INT8) {
        factor = h.e == kNanExponent ? 0x7fffu : (h.e == 0 ? 0x40u : h.e << 7);
    } else {
        const uint32_t e = h.e + 120u;
        factor = e > 254u ? 254u << 7 : e << 7;
        if (e > 254u) more = h.e == kNanExponent ? 0x7fffu : (e - 127u) << 7;
    }
    factor |= factor << 16, more |= more << 16;
    uint32_t out[8];
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
    const uint32_t a[4] = {out[0], out[1], out[2], out[3]}, b[4] = {out[4], out[5], out[6], out[7]};
    store16(at, a);
    store16(at ^ 16u, b);
}

// Where a thread's pieces of W columns of a stage lie: `valid` of them a row, the threads
// one after the other along them, rows after rows; turn k's are k * rows rows on.  A
// thread without a piece has row ROWS.
template <int ROWS, int W>
struct Turns {
    int piece, row, rows;     // rows: of a turn
    __device__ __forceinline__ Turns(int threads, int valid) {
        rows = threads / valid;
        row = threadIdx.x / valid, piece = threadIdx.x - row * valid;
        if (row >= rows) piece = 0, row = ROWS;
    }
    // Of turn k's piece in an operand: 64 columns of a row, swizzled by 16 bytes.
    __device__ __forceinline__ uint32_t place(int k) const {
        const int r = row + k * rows, u = piece * (W / kUnit);
        return (u >> 3) * (ROWS * 128) + r * 128 + (((u ^ r) & 7) << 4);
    }
    __device__ __forceinline__ bool has(int k, int of) const { return row + k * rows < of; }
};

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

template <typename T, int TI, int TJ, int FMT, bool FAST>
__global__ void __launch_bounds__(Config<T, TI, TJ>::kThreads, Config<T, TI, TJ>::kMinCtas)
    k_dense(DenseArgs a, const __grid_constant__ CUtensorMap map) {
    using C = Config<T, TI, TJ>;
    constexpr bool kCopies = FAST && C::kParts == 1;
    extern __shared__ uint8_t s_raw[];
    __shared__ uint64_t s_full[C::kStages], s_copied[C::kStages], s_empty[C::kStages], s_done, s_drained;
    __shared__ uint32_t s_tensor, s_failed;
    const uint32_t ring = (smem_of(s_raw) + 1023u) & ~1023u;
    uint8_t *ring_ptr = s_raw + (ring - smem_of(s_raw));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int i0 = blockIdx.z * TI, j0 = blockIdx.y * TJ;
    const int ni = a.N - i0 < TI ? a.N - i0 : TI, nj = a.D - j0 < TJ ? a.D - j0 : TJ;
    const int64_t first = int64_t(blockIdx.x) * a.rows;
    const int64_t last = first + a.rows < a.n ? first + a.rows : a.n;
    const int stages = last > first ? int((last - first + C::kRows - 1) / C::kRows) : 0;
    const bool bias = blockIdx.y == 0 && a.db;

    if (threadIdx.x == 0) {
        s_failed = 0;
        for (int k = 0; k < C::kStages; ++k) {
            barrier_init(&s_full[k], C::kLoaders / 32);
            barrier_init(&s_copied[k], 1);
            barrier_init(&s_empty[k], 1);
        }
        barrier_init(&s_done, 1);
        barrier_init(&s_drained, C::kLoaders / 32);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == C::kLoaders / 32) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_of(&s_tensor)),
                     "n"(C::kColumns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    // columns past the matrices stay zeros
    if (ni < TI || nj < TJ)
        for (int k = threadIdx.x; k < C::kStages * C::kStageBytes / 16; k += C::kThreads)
            reinterpret_cast<uint4 *>(ring_ptr)[k] = make_uint4(0u, 0u, 0u, 0u);
    writes_to_async();
    asm volatile("tcgen05.fence::before_thread_sync;");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;");
    const uint32_t tensor = s_tensor;

    F2 sums[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[i] = both(0.0f);
    const Turns<C::kRows, kUnit> ta(C::kLoaders, (ni + kUnit - 1) / kUnit);
    const Turns<C::kRows, kWide> tb(C::kLoaders, (nj + kWide - 1) / kWide);

    // The sums of a chain out of the tensor memory: added to what the chains before left, and to their
    // place if it is the last.  A warp reads the 32 lanes (rows of dW) of its quarter, the warps of a
    // quarter 8 columns in turn.
    auto drain = [&](bool first_chain, bool last_chain) {
        const int quarter = warp & 3;
        const bool failed = *static_cast<volatile uint32_t *>(&s_failed) != 0;
#pragma unroll 1
        for (int h = 0; h < TI / 128 && h * 128 < ni; ++h) {
            const int i = i0 + h * 128 + quarter * 32 + lane;
#pragma unroll 1
            for (int c = (warp >> 2) * 8; c < nj; c += C::kLoaders / 128 * 8) {
                uint32_t v[8];
                const uint32_t at = tensor + (uint32_t(quarter * 32) << 16) + h * TJ + c;
                __syncwarp();
                tensor_load8(v, at);
                if (C::kSums > 1) {
                    uint32_t w[8];
                    tensor_load8(w, at + C::kTile);
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) + __uint_as_float(w[k]));
                }
                if (stages == 0 || failed)      // a wait that ran out leaves NaN
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] = failed ? 0x7fffffffu : 0u;
                if (i >= a.N) continue;
                const int count = nj - c < 8 ? nj - c : 8;
                const int64_t e = int64_t(i) * a.dws + j0 + c;
                float *part = a.part + (size_t(blockIdx.x) * a.N + i) * a.D + j0 + c;
                if (a.splits == 1 && a.gdt == SS_F32)
                    put_sums(static_cast<float *>(a.dw) + e, count, v, !first_chain);
                else if (a.splits == 1 && last_chain)
                    put_rounded(a, e, part, count, v, !first_chain);
                else
                    put_sums(part, count, v, !first_chain);
            }
        }
    };
    if (warp < C::kLoaders / 32) {
        Raw<T> ra[C::kAhead][C::kTurnsA];
        Wide rb[C::kAhead][C::kTurnsB];
        const int ca = ni - ta.piece * kUnit < kUnit ? ni - ta.piece * kUnit : kUnit;
        const bool all = nj - tb.piece * kWide > kUnit;
        // the next stage to load: its pieces, and how many of its rows there are
        const T *pa = static_cast<const T *>(a.dy) + (first + ta.row) * a.dys + i0 + ta.piece * kUnit;
        const uint8_t *pq = a.x.q + (first + tb.row) * a.x.stride + j0 + tb.piece * kWide;
        const uint8_t *ps = a.x.scales + (first + tb.row) * a.x.scale_stride + j0 / kGroup + tb.piece / (kGroup / kWide);
        int64_t left = last - first;
        auto load = [&](Raw<T> (&va)[C::kTurnsA], Wide (&vb)[C::kTurnsB]) {
            const int rows = left < C::kRows ? int(left) : C::kRows;
            if (!kCopies)
#pragma unroll
                for (int k = 0; k < C::kTurnsA; ++k)
                    if (ta.has(k, rows))
                        va[k] = load_unit<T, FAST>(pa + k * ta.rows * a.dys, ca);
                    else
                        va[k].clear();
#pragma unroll
            for (int k = 0; k < C::kTurnsB; ++k)
                if (tb.has(k, rows))
                    vb[k].template load<FAST>(pq + k * tb.rows * a.x.stride, ps + k * tb.rows * a.x.scale_stride, all);
                else
                    vb[k] = Wide{{0u, 0u, 0u, 0u}, 127u};
            pa += C::kRows * a.dys, pq += C::kRows * a.x.stride, ps += C::kRows * a.x.scale_stride;
            left -= C::kRows;
        };
#pragma unroll
        for (int q = 0; q < C::kAhead; ++q) load(ra[q], rb[q]);
        auto add_bias = [&](const Raw<T> &r) {
            F2 f[4];
            floats_of(f, r);
#pragma unroll
            for (int i = 0; i < 4; ++i) sums[i] = add2(sums[i], f[i]);
        };
        int slot = 0, chains = 0;
        uint32_t parity = 1;
        bool ok = true, end;
        int base = 0;
        do {
#pragma unroll
            for (int q = 0; q < C::kAhead; ++q) {
                if (base + q >= stages) break;
                if (!barrier_wait(&s_empty[slot], parity)) {
                    ok = false;
                    break;
                }
                const uint32_t at = ring + slot * C::kStageBytes;
                if (!kCopies)
#pragma unroll
                    for (int k = 0; k < C::kTurnsA; ++k) {
                        if (!ta.has(k, C::kRows)) continue;
                        store_parts<C::kABytes>(at + ta.place(k), ra[q][k]);
                        if (bias) add_bias(ra[q][k]);
                    }
#pragma unroll
                for (int k = 0; k < C::kTurnsB; ++k)
                    if (tb.has(k, C::kRows)) store_held<FMT>(at + C::kParts * C::kABytes + tb.place(k), rb[q][k]);
                if constexpr (kCopies) if (bias) {       // the copy engine's rows, before the slot may be filled again
                    if (!barrier_wait(&s_copied[slot], parity ^ 1)) {
                        ok = false;
                        break;
                    }
#pragma unroll
                    for (int k = 0; k < C::kTurnsA; ++k)
                        if (ta.has(k, C::kRows)) {
                            load_words(ra[q][k].w, ring_ptr + slot * C::kStageBytes + ta.place(k));
                            add_bias(ra[q][k]);
                        }
                }
                writes_to_async();
                __syncwarp();
                if (lane == 0) barrier_arrive(&s_full[slot]);
                load(ra[q], rb[q]);
                if (++slot == C::kStages) slot = 0, parity ^= 1;
            }
            base += C::kAhead;
            end = !ok || base >= stages;
            if (end || base % a.chain == 0) {
                if (!ok || !barrier_wait(&s_done, chains & 1)) s_failed = 1;
                asm volatile("tcgen05.fence::after_thread_sync;");
                drain(chains == 0, end);
                asm volatile("tcgen05.fence::before_thread_sync;");
                __syncwarp();
                if (lane == 0) barrier_arrive(&s_drained);
                ++chains;
            }
        } while (!end);
    } else if (warp == C::kLoaders / 32) {
        if (lane == 0) {
            const uint32_t what = product_of((nj + 15) / 16 * 16);
            int slot = 0, chains = 0, link = 0;
            uint32_t parity = 0;
            for (int stage = 0; stage < stages; ++stage) {
                if (!barrier_wait(&s_full[slot], parity) || (kCopies && !barrier_wait(&s_copied[slot], parity))) {
                    s_failed = 1;
                    break;
                }
                asm volatile("tcgen05.fence::after_thread_sync;");
                const uint32_t at = ring + slot * C::kStageBytes, bt = at + C::kParts * C::kABytes;
#pragma unroll
                for (int k = 0; k < C::kRows / kStep; ++k)
#pragma unroll
                    for (int p = 0; p < C::kParts; ++p)
#pragma unroll
                        for (int h = 0; h < TI / 128; ++h)
                            if (h * 128 < ni)
                                product(tensor + (p > 0 ? C::kTile : 0) + h * TJ,
                                        operand_at<C::kBlock>(at + p * C::kABytes + h * 2 * C::kBlock + k * kStep * 128),
                                        operand_at<C::kBlock>(bt + k * kStep * 128), what, link > 0 || k > 0 || p > 1);
                products_arrive(&s_empty[slot]);
                if (++slot == C::kStages) slot = 0, parity ^= 1;
                if (++link == a.chain && stage + 1 < stages) {
                    products_arrive(&s_done);
                    if (!barrier_wait(&s_drained, chains & 1)) {
                        s_failed = 1;
                        break;
                    }
                    link = 0, ++chains;
                }
            }
            products_arrive(&s_done);
            if (!barrier_wait(&s_done, chains & 1)) s_failed = 1;    // the tensor memory is freed after them
        }
        __syncwarp();
    } else {
        if (kCopies && lane == 0) {
            const int boxes = (ni + 63) / 64;
            int slot = 0, stage = 0;
            uint32_t parity = 1;
            for (; stage < stages; ++stage) {
                if (!barrier_wait(&s_empty[slot], parity)) {
                    s_failed = 1;
                    break;
                }
                barrier_expect(&s_copied[slot], boxes * C::kBlock);
                for (int k = 0; k < boxes; ++k)
                    copy_box(ring + slot * C::kStageBytes + k * C::kBlock, &map, i0 + 64 * k,
                             int(first + int64_t(stage) * C::kRows), &s_copied[slot]);
                if (++slot == C::kStages) slot = 0, parity ^= 1;
            }
            // every copy has come before the block ends
            for (int k = stage < C::kStages ? stage : C::kStages; k > 0; --k) {
                const int s = (stage - k) % C::kStages;
                if (!barrier_wait(&s_copied[s], (stage - k) / C::kStages & 1)) s_failed = 1;
            }
        }
        __syncwarp();
    }
    __syncthreads();
    if (bias) {
        // the threads' sums of a column, in the order of their rows
        float *s = reinterpret_cast<float *>(ring_ptr);
        const int width = (ni + kUnit - 1) / kUnit * kUnit;
        if (warp < C::kLoaders / 32 && ta.row < C::kRows)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                reinterpret_cast<float2 *>(s + size_t(ta.row) * width + ta.piece * kUnit)[i] = sums[i];
        __syncthreads();
        for (int j = threadIdx.x; j < ni; j += C::kThreads) {
            float t = 0.0f;
            for (int r = 0; r < ta.rows && r < C::kRows; ++r) t += s[size_t(r) * width + j];
            if (a.splits > 1)
                a.part_bias[size_t(blockIdx.x) * a.N + i0 + j] = t;
            else
                store_param(a.db, a.gdt, i0 + j, t);
        }
    }
    asm volatile("tcgen05.fence::before_thread_sync;");
    __syncthreads();
    if (warp == C::kLoaders / 32)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tensor), "n"(C::kColumns));
}

__device__ __forceinline__ void put_result(const DenseArgs &a, int64_t all, int64_t k, float t) {
    if (k < all)
        store_param(a.dw, a.gdt, k / a.D * a.dws + k % a.D, t);
    else
        store_param(a.db, a.gdt, k - all, t);
}

// The splits' sums, of [N][D] and then of the bias.  Few splits: a thread a value.
__global__ void __launch_bounds__(256) k_dense_join(DenseArgs a) {
    const int64_t all = int64_t(a.N) * a.D, count = all + (a.db ? a.N : 0);
    for (int64_t k = int64_t(blockIdx.x) * 256 + threadIdx.x; k < count; k += int64_t(gridDim.x) * 256) {
        const float *p = k < all ? a.part + k : a.part_bias + (k - all);
        const int64_t apart = k < all ? all : a.N;
        float t = 0.0f;
#pragma unroll 4
        for (int v = 0; v < a.splits; ++v) t += p[v * apart];
        put_result(a, all, k, t);
    }
}

// Many splits: 32 values by 32 slices of the splits side by side, then the slices in order.
__global__ void __launch_bounds__(1024) k_dense_join_many(DenseArgs a) {
    __shared__ float s_t[32][33];
    const int64_t all = int64_t(a.N) * a.D, count = all + (a.db ? a.N : 0);
    const int c = threadIdx.x & 31, q = threadIdx.x >> 5;
    for (int64_t base = int64_t(blockIdx.x) * 32; base < count; base += int64_t(gridDim.x) * 32) {
        const int64_t k = base + c;
        float t = 0.0f;
        if (k < count) {
            const float *p = k < all ? a.part + k : a.part_bias + (k - all);
            const int64_t apart = k < all ? all : a.N;
#pragma unroll 4
            for (int v = q; v < a.splits; v += 32) t += p[v * apart];
        }
        __syncthreads();
        s_t[q][c] = t;
        __syncthreads();
        t = s_t[c][q];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
        const int64_t e = base + q;
        if (c == 0 && e < count) put_result(a, all, e, t);
    }
}

// The tile's sides for a weight's.
struct Tile {
    int i, j, ctas;    // ctas: of an SM
};
Tile tile_of(int32_t N, int32_t D, int dtype) {
    if (N <= 128 && D <= 64) return {128, 64, 3};
    if (N <= 128 && D <= 128) return {128, 128, 2};
    if (dtype == SS_BF16) return {256, 256, 1};
    return {128, 256, 1};      // two sets of sums
}

// How the rows are shared out: ranges with sums of their own, as many as fill the device; and the chains of sums within a range.
constexpr int kSms = 152;
constexpr int kLeastRows = 256;     // of a range
constexpr int kChain32 = 2048, kChain16 = 16384;    // rows; dW in float32, in 16 bits
struct Shares {
    int splits, chain;     // chain: rows
    bool part;         // sums leave the tensor memory before they are done
};
Shares shares_of(int64_t n, int32_t N, int32_t D, int dtype, int gdt) {
    const Tile t = tile_of(N, D, dtype);
    const int64_t tiles = int64_t((N + t.i - 1) / t.i) * ((D + t.j - 1) / t.j);
    int64_t s = kSms * t.ctas / tiles;
    const int64_t most = (n + kLeastRows - 1) / kLeastRows;
    if (s > most) s = most;
    if (s < 1) s = 1;
    const int rows = gdt == SS_F32 ? kChain32 : kChain16;
    return {int(s), rows, s > 1 || (gdt != SS_F32 && n > rows)};
}

// The driver's function that describes a matrix to the copy engine.
using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                              const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
ss_status encoder(EncodeFn *fn, const char *who) {
    static std::atomic<EncodeFn> known{nullptr};
    *fn = known.load(std::memory_order_acquire);
    if (*fn) return SS_OK;
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    const ss_status st =
        check_cuda(cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q), who);
    if (st != SS_OK) return st;
    if (q != cudaDriverEntryPointSuccess || !p) return fail(SS_ERR_CUDA, "%s: the driver has no cuTensorMapEncodeTiled", who);
    *fn = reinterpret_cast<EncodeFn>(p);
    known.store(*fn, std::memory_order_release);
    return SS_OK;
}

// dy [n][N] of bfloat16 in boxes of 64 columns x `rows` rows, swizzled as the products read them.
ss_status map_of(CUtensorMap *map, const DenseArgs &a, int rows, const char *who) {
    EncodeFn encode;
    const ss_status st = encoder(&encode, who);
    if (st != SS_OK) return st;
    const cuuint64_t dims[2] = {cuuint64_t(a.N), cuuint64_t(a.n)}, strides[1] = {cuuint64_t(a.dys) * 2};
    const cuuint32_t box[2] = {64, cuuint32_t(rows)}, each[2] = {1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(a.dy), dims, strides, box, each,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? SS_OK : fail(SS_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed (%d)", who, int(r));
}

template <typename T, int TI, int TJ, int FMT>
ss_status launch(DenseArgs a, cudaStream_t s, const char *who) {
    using C = Config<T, TI, TJ>;
    const int64_t each = (a.n + a.splits - 1) / a.splits;
    a.rows = (each + C::kRows - 1) / C::kRows * C::kRows;
    a.chain /= C::kRows;
    const dim3 grid(a.splits, (a.D + TJ - 1) / TJ, (a.N + TI - 1) / TI);
    const bool fast = a.n > 0 && units_aligned<T>(a.dy, a.dys) && aligned_to(a.x.q, 16) && a.x.stride % 16 == 0;
    static std::atomic<unsigned long long> smem_ctx[kMaxDevices];   // see ensure_dyn_smem
    const void *fn[2] = {(const void *)k_dense<T, TI, TJ, FMT, true>, (const void *)k_dense<T, TI, TJ, FMT, false>};
    ss_status st = ensure_dyn_smem(smem_ctx, fn, 2, C::kSmem, who);
    if (st != SS_OK) return st;
    CUtensorMap map = {};
    if (fast && C::kParts == 1 && (st = map_of(&map, a, C::kRows, who)) != SS_OK) return st;
    auto kernel = fast ? k_dense<T, TI, TJ, FMT, true> : k_dense<T, TI, TJ, FMT, false>;
    SS_LAUNCH("k_dense", s, kernel<<<grid, C::kThreads, C::kSmem, s>>>(a, map));
    return SS_OK;
}

bool dense_sizes_ok(int64_t n, int32_t N, int32_t D) { return row_sizes_ok(n, D) && N >= 1 && N <= kMaxWidth; }

}  // namespace
}  // namespace ss

using namespace ss;

extern "C" {

size_t ss_dense_grad8_workspace_bytes(int64_t n, int32_t N, int32_t D, ss_dtype dtype, ss_dtype grad_dtype) {
    if (!dense_sizes_ok(n, N, D) || !dtype_known(dtype) || (grad_dtype != SS_F32 && grad_dtype != dtype)) return 0;
    const Shares sh = shares_of(n, N, D, dtype, grad_dtype);
    return sh.part ? size_t(sh.splits) * N * (size_t(D) + 1) * sizeof(float) : 256;
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
    if ((st = check_workspace(who, workspace, workspace_bytes, ss_dense_grad8_workspace_bytes(n, N, D, dtype, grad_dtype))) != SS_OK)
        return st;
    int dev = 0, sms = 0;
    if ((st = current_device(&dev, &sms, "ss_dense_grad8: device query")) != SS_OK) return st;
    cudaStream_t s = (cudaStream_t)stream;
    const Shares sh = shares_of(n, N, D, dtype, grad_dtype);
    float *part = static_cast<float *>(workspace);
    const DenseArgs a{dy, dy_stride, rows8_of(x), n, N, D, 0, sh.splits, sh.chain, part,
                      part + size_t(sh.splits) * N * D, dweight, dweight_stride, dbias, int(grad_dtype)};
    const Tile tile = tile_of(N, D, dtype);
    with_type(dtype, [&](auto t) {
        using T = decltype(t);
        constexpr int kLargeI = std::is_same<T, __nv_bfloat16>::value ? 256 : 128;
        with_format(x ? x->format : SS_INT8, [&](auto F) {
            constexpr int FMT = decltype(F)::value;
            if (tile.j == 256)
                st = launch<T, kLargeI, 256, FMT>(a, s, who);
            else if (tile.j == 128)
                st = launch<T, 128, 128, FMT>(a, s, who);
            else
                st = launch<T, 128, 64, FMT>(a, s, who);
        });
    });
    if (st != SS_OK) return st;
    if (sh.splits > 1) {
        const int64_t values = int64_t(N) * D + N;
        if (sh.splits >= 16) {
            const int64_t ctas = (values + 31) / 32;
            SS_LAUNCH("k_dense_join_many", s,
                      k_dense_join_many<<<int(ctas < sms * 16 ? ctas : sms * 16), 1024, 0, s>>>(a));
        } else {
            const int64_t ctas = (values + 255) / 256;
            SS_LAUNCH("k_dense_join", s, k_dense_join<<<int(ctas < sms * 16 ? ctas : sms * 16), 256, 0, s>>>(a));
        }
    }
    return check_launch(who);
}

}  // extern "C"
