// Root-mean-square norm, and the gradients of both norms from rows kept in 8
// bits (model: include/ss_rms.h).  Times that stand alone are a kernel's by ncu; where two
// are compared they are both calls', some microseconds more.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "ss_internal.h"
#include "ss_launch.cuh"
#include "ss_norm.cuh"
#include "ss_profile.h"
#include "ss_rms.h"
#include "ss_rows8.cuh"
#include "ss_unit.cuh"

namespace ss {
namespace {

constexpr int kThreads = kNormThreads;

template <typename T>
struct Rows {
    T *base;
    int64_t stride;
};

// A row's place in the threads.  `lanes` threads share it, thread l of them
// holding units l, l + lanes, ... (NV of them) in registers, so the row is read
// once.  Narrow rows (MULTI false) take a power of two of lanes inside a warp and reduce
// by shuffles; wide ones take whole warps and reduce through
// shared memory and a barrier of their own.  Groups of 32 columns are four lanes side
// by side in both (fewer where the row ends with them).
//
// Rows that start off their blocks' boundaries, all tensors' alike (kShifted): units lie on the
// boundaries, head elements of the first not being the row's; a group of lanes takes every
// step-th row with step a multiple of the rows after which starts repeat, so its columns stay
// fixed.
constexpr int kMaxGroups = 4;          // rows of several warps side by side in a CTA: of two warps at least

struct Place {
    int lanes, shift;   // lanes = 1 << shift where !MULTI
    int units;          // of a row
    int groups;         // rows side by side in a CTA
};

bool in_registers(int32_t D) { return D <= kMaxRowThreads * 2 * kUnit; }
bool shifted_in_registers(int32_t D) { return D + 2 * (kUnit - 1) < kMaxRowThreads * 2 * kUnit; }

// Up to 32 lanes a unit each; a warp with two units a lane up to 64; from there on
// whole warps.  `single`: whole warps with a unit a lane as far as they go, for the gradients of float32 rows, whose
// two units take more registers than there are (8191 x 4096: 131 us for 80; of 16-bit rows 49 for 66).
Place place_of(int32_t D, bool shifted, bool single, int *nv, bool *multi) {
    Place pl{};
    pl.units = units_of(shifted ? D + kUnit - 1 : D);
    *nv = pl.units <= 32 ? 1 : 2;
    *multi = pl.units > 64;
    if (single && pl.units > 32 && pl.units <= kMaxRowThreads) *nv = 1, *multi = true;
    if (*multi) {
        pl.lanes = (pl.units + 32 * *nv - 1) / (32 * *nv) * 32;
        pl.groups = pl.lanes < kThreads ? kThreads / pl.lanes : 1;
    } else {
        pl.lanes = 1, pl.shift = 0;
        while (pl.lanes * *nv < pl.units) pl.lanes <<= 1, ++pl.shift;
        pl.groups = kThreads / pl.lanes;
    }
    return pl;
}

// Where a thread's units lie.
struct Units {
    int lane, lanes, head;
    int32_t D;
    bool first, last;    // of the lanes of a warp that share a row
    __device__ __forceinline__ int at(int k) const { return lane + k * lanes; }
    // Elements of unit k that are the row's: from lo on, up to hi.
    __device__ __forceinline__ int lo(int k) const { return at(k) == 0 ? head : 0; }
    __device__ __forceinline__ int hi(int k) const {
        const int c = D + head - at(k) * kUnit;
        return c <= 0 ? 0 : (c < kUnit ? c : kUnit);
    }
    // The column of its element 0.
    __device__ __forceinline__ int column(int k) const { return at(k) * kUnit - head; }
    __device__ __forceinline__ bool next(int k) const { return !last && (at(k) + 1) * kUnit < D; }
};
template <bool MULTI>
__device__ __forceinline__ Units units_at(int lane, const Place &pl, int32_t D, int head) {
    const int l = MULTI ? lane & 31 : lane;
    return Units{lane, pl.lanes, head, D, l == 0, l == (MULTI ? 31 : pl.lanes - 1)};
}

// Unit k of the row at p (`here`: there is such a row).
template <typename T, Lie LIE>
__device__ __forceinline__ Raw<T> load_of(const T *p, const Units &c, int k, bool here) {
    if constexpr (LIE == kShifted) return load_block(p + c.column(k), c.lo(k), here ? c.hi(k) : 0);
    return load_unit<T, LIE == kAligned>(p + c.column(k), here ? c.hi(k) : 0);
}
template <typename T, Lie LIE>
__device__ __forceinline__ void store_of(T *p, const Raw<T> &r, const Units &c, int k, bool here) {
    if constexpr (LIE == kShifted)
        store_block(p + c.column(k), r, here ? c.lo(k) : 0, here ? c.hi(k) : 0);
    else
        store_unit<T, LIE == kAligned>(p + c.column(k), r, here ? c.hi(k) : 0, !c.first, c.next(k));
}

// A thread's weights in float32 (1 where there are none, and past the row).
template <int NV>
__device__ __forceinline__ void load_weights(F2 (&g)[NV][4], const void *w, int pdt, const Units &c) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        float f[kUnit];
        const int j = c.column(k), lo = c.lo(k), hi = w ? c.hi(k) : 0;
#pragma unroll
        for (int i = 0; i < kUnit; ++i) f[i] = i >= lo && i < hi ? load_param(w, pdt, j + i) : 1.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) g[k][i] = make_float2(f[2 * i], f[2 * i + 1]);
    }
}

// What a warp's 32 consecutive columns hold, into 8 bits (v: 0 past the row).
template <int FMT>
__device__ __forceinline__ void put_group(const Rows8 &out, int64_t row, int j, int32_t held, float v) {
    const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(v) & 0x7fffffffu);
    const uint32_t e = exponent_of<FMT>(most);
    const float z = e == kNanExponent ? 0.0f : v * inverse_of(e);
    if (j < held) out.q[row * out.stride + j] = uint8_t(encode4<FMT>(z, 0.0f, 0.0f, 0.0f));
    if ((threadIdx.x & 31) == 0 && j < held) out.scales[row * out.scale_stride + j / kGroup] = uint8_t(e);
}
__device__ __forceinline__ void put_group(int fmt, const Rows8 &out, int64_t row, int j, int32_t held, float v) {
    if (fmt == SS_INT8)
        put_group<SS_INT8>(out, row, j, held, v);
    else
        put_group<SS_E4M3>(out, row, j, held, v);
}

// A unit into 8 bits; all lanes of a warp together.  What lies past the row is whatever the
// unit has there, and counts for nothing.
template <int FMT>
__device__ __forceinline__ void put_held(const Rows8 &out, int64_t row, int u, int count, const F2 (&v)[4], int lanes) {
    F2 f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f[i] = make_float2(2 * i < count ? v[i].x : 0.0f, 2 * i + 1 < count ? v[i].y : 0.0f);
    const uint32_t e = group_exponent<FMT>(f, lanes);
    if (count > 0) put_unit<FMT>(out, row, u, e, f);
}
__device__ __forceinline__ void put_held(int fmt, const Rows8 &out, int64_t row, int u, int count, const F2 (&v)[4], int lanes) {
    if (fmt == SS_INT8)
        put_held<SS_INT8>(out, row, u, count, v, lanes);
    else
        put_held<SS_E4M3>(out, row, u, count, v, lanes);
}

struct FwdArgs {
    const void *x;
    int64_t xs;
    const void *residual;
    int64_t rs, n;
    int32_t D;
    const void *gamma;
    int pdt;
    float eps;
    void *sum;
    int64_t ss_;
    void *y;
    int64_t ys;
    Rows8 out, kept;
    int out_fmt, kept_fmt;     // -1: not wanted
    float *rstd;
};

// CTAs an SM that the registers are held down for, of narrow rows (0: wide ones as the compiler has them in CTAs of
// up to 512).  Forward, us: 700,000 x 87 float16 with five 193, with four 207; 2M x 48 float32 with four 228, with
// five 236; two units a lane with three, two and four: 60,000 x 500 float32 89, 97 and 95 (three spill 72 to 232
// bytes, two none), 60,000 x 512 float32 86, 83 and 92, 60,000 x 500 float16 60, 73 and 61, 60,000 x 501 bfloat16 79,
// 101 and 74.
constexpr int fwd_ctas(int bytes, int nv, bool multi) { return multi ? 0 : (nv == 2 ? 3 : (bytes == 2 ? 5 : 4)); }
// Backward: 2M x 48 float32 with two 224, with three 282 (spills); 2M x 48 bfloat16 with three 142, with two
// 169; two units a lane (16 bits) with two, three and one: 60,000 x 500 float16 57, 116 and 78, 60,000 x 512
// bfloat16 47, 79 and 56, the layer norm's 41, 93 and 52.
constexpr int bwd_ctas(int bytes, int nv, bool multi) { return multi ? 0 : (bytes == 4 || nv == 2 ? 2 : 3); }

// A row from registers: its sum with the residual, its square's mean, and every
// output that is wanted.  The next row's loads are in flight meanwhile.  (kShifted: without
// outputs in 8 bits, whose groups begin with the row.)  2M x 48 float32 (1.54 GB): 222 us, at a
// copy's rate; 8191 x 4096 bfloat16 into e4m3 (235 MB) 52 (35), with 57 % of the issue slots taken by 15 warps
// an SM; 16384 x 1001 bfloat16 a call 33 (20).
template <typename T, int NV, bool MULTI, Lie LIE, bool RES>
__global__ void __launch_bounds__(MULTI ? kMaxRowThreads : kThreads, fwd_ctas(sizeof(T), NV, MULTI)) k_rms_fwd(FwdArgs a, Place pl) {
    __shared__ alignas(16) float s_red[MULTI ? kMaxGroups : 1][2][1][kRowWarps];
    const int group = MULTI ? threadIdx.x / pl.lanes : threadIdx.x >> pl.shift;
    const int lane = MULTI ? threadIdx.x - group * pl.lanes : threadIdx.x & (pl.lanes - 1);
    const int64_t step = int64_t(gridDim.x) * pl.groups, row0 = int64_t(blockIdx.x) * pl.groups + group;
    const Units c = units_at<MULTI>(lane, pl, a.D, LIE == kShifted ? head_of<T>(static_cast<const T *>(a.x) + row0 * a.xs) : 0);
    Raw<T> x[NV], res[NV];
    auto load = [&](int64_t row) {
        const T *px = static_cast<const T *>(a.x) + row * a.xs, *pr = static_cast<const T *>(a.residual) + row * a.rs;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            x[k] = load_of<T, LIE>(px, c, k, row < a.n);
            if (RES) res[k] = load_of<T, LIE>(pr, c, k, row < a.n);
        }
    };
    load(row0);
    F2 g[NV][4];
    load_weights<NV>(g, a.gamma, a.pdt, c);
    if (MULTI) {
        for (int e = threadIdx.x; e < kMaxGroups * 2 * kRowWarps; e += blockDim.x) (&s_red[0][0][0][0])[e] = 0.0f;
        __syncthreads();
    }
    const float width = float(a.D);
    int flip = 0;
    // a warp's lanes leave together: they shuffle with one another; a row past the
    // last is zeros, and not stored
    const int64_t lead = MULTI ? row0 : row0 - ((threadIdx.x & 31) >> pl.shift);
    for (int64_t base = lead; base < a.n; base += step) {
        const int64_t row = base + (row0 - lead);
        const bool here = row < a.n;
        F2 h[NV][4], acc = both(0.0f);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            floats_of(h[k], x[k]);
            if (RES) {
                F2 q[4];
                floats_of(q, res[k]);
#pragma unroll
                for (int i = 0; i < 4; ++i) h[k][i] = add2(h[k][i], q[i]);
                const Raw<T> r = raw_of<T>(h[k]);
                store_of<T, LIE>(static_cast<T *>(a.sum) + row * a.ss_, r, c, k, here);
                floats_of(h[k], r);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) acc = fma2(h[k][i], h[k][i], acc);
        }
        load(row + step);
        float sum[1] = {sum_of(acc)};
        row_sum<1, MULTI>(sum, pl.lanes, group, lane, s_red[MULTI ? group : 0], flip);
        const float r = __frsqrt_rn(__fdiv_rn(sum[0], width) + a.eps);
        const F2 rr = both(r);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (LIE != kShifted && a.kept_fmt >= 0)
                put_held(a.kept_fmt, a.kept, row, c.at(k), here ? c.hi(k) : 0, h[k], pl.lanes);
#pragma unroll
            for (int i = 0; i < 4; ++i) h[k][i] = mul2(mul2(h[k][i], rr), g[k][i]);
            if (a.y) store_of<T, LIE>(static_cast<T *>(a.y) + row * a.ys, raw_of<T>(h[k]), c, k, here);
            if (LIE != kShifted && a.out_fmt >= 0)
                put_held(a.out_fmt, a.out, row, c.at(k), here ? c.hi(k) : 0, h[k], pl.lanes);
        }
        if (here && lane == 0 && a.rstd) a.rstd[row] = r;
    }
}

// A CTA a row, an element a thread, the row read again for its result.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_rms_fwd_wide(FwdArgs a) {
    __shared__ float s_red[kThreads / 32];
    const int32_t held = (a.D + 7) / 8 * 8, padded = (a.D + 31) / 32 * 32;
    for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
        const T *x = static_cast<const T *>(a.x) + row * a.xs;
        T *sum = a.sum ? static_cast<T *>(a.sum) + row * a.ss_ : nullptr;
        const T *h = sum ? sum : x;
        float q = 0.0f;
        for (int j = threadIdx.x; j < a.D; j += kThreads) {
            float v = to_float(x[j]);
            if (sum) {
                sum[j] = from_float<T>(v + to_float(static_cast<const T *>(a.residual)[row * a.rs + j]));
                v = to_float(sum[j]);
            }
            q = fmaf(v, v, q);
        }
        const float r = __frsqrt_rn(block_sum(q, s_red) / float(a.D) + a.eps);
        for (int j0 = 0; j0 < padded; j0 += kThreads) {
            const int j = j0 + threadIdx.x;
            const bool here = j < a.D;
            const float v = here ? to_float(h[j]) : 0.0f;
            const float y = here ? v * r * (a.gamma ? load_param(a.gamma, a.pdt, j) : 1.0f) : 0.0f;
            if (a.y && here) static_cast<T *>(a.y)[row * a.ys + j] = from_float<T>(y);
            if (a.kept_fmt >= 0) put_group(a.kept_fmt, a.kept, row, j, held, v);
            if (a.out_fmt >= 0) put_group(a.out_fmt, a.out, row, j, held, y);
        }
        if (threadIdx.x == 0 && a.rstd) a.rstd[row] = r;
    }
}

struct BwdArgs {
    const void *dy;
    int64_t dys;
    const void *h;      // or kept
    int64_t hs;
    Rows8 kept;
    int fmt;            // -1: h
    int64_t n;
    int32_t D;
    const void *gamma;
    int pdt;
    const float *mean, *rstd;      // mean: the layer norm's
    const void *dsum;
    int64_t dss;
    void *dx;
    int64_t dxs;
    void *dgamma, *dbeta;
    float *part;
    bool centred;
};

template <typename T>
__device__ __forceinline__ float kept_value(const BwdArgs &a, int64_t row, int j) {
    if (a.fmt < 0) return to_float(static_cast<const T *>(a.h)[row * a.hs + j]);
    const uint8_t q = a.kept.q[row * a.kept.stride + j];
    const float s = scale_of(a.kept.scales[row * a.kept.scale_stride + j / kGroup]);
    return (a.fmt == SS_INT8 ? decode1<SS_INT8>(q) : decode1<SS_E4M3>(q)) * s;
}

// The weights' partial sums: thread = column, CTA y = a slice of the rows.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_norm8_bwd_weights_wide(BwdArgs a) {
    const int j = blockIdx.x * kThreads + threadIdx.x;
    if (j >= a.D) return;
    float dg = 0.0f, db = 0.0f;
    for (int64_t row = blockIdx.y; row < a.n; row += gridDim.y) {
        const float d = to_float(static_cast<const T *>(a.dy)[row * a.dys + j]);
        const float mu = a.centred ? a.mean[row] : 0.0f;
        dg = fmaf(d, (kept_value<T>(a, row, j) - mu) * a.rstd[row], dg);
        db += d;
    }
    const int cols = a.centred ? 2 * a.D : a.D;
    a.part[size_t(blockIdx.y) * cols + j] = dg;
    if (a.centred) a.part[size_t(blockIdx.y) * cols + a.D + j] = db;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_norm8_bwd_rows_wide(BwdArgs a) {
    __shared__ float s_red[kThreads / 32];
    for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
        const T *dy = static_cast<const T *>(a.dy) + row * a.dys;
        const float mu = a.centred ? a.mean[row] : 0.0f, r = a.rstd[row];
        float sa = 0.0f, sah = 0.0f;
        for (int j = threadIdx.x; j < a.D; j += kThreads) {
            const float v = to_float(dy[j]) * (a.gamma ? load_param(a.gamma, a.pdt, j) : 1.0f);
            sa += v;
            sah = fmaf(v, (kept_value<T>(a, row, j) - mu) * r, sah);
        }
        const float ma = a.centred ? block_sum(sa, s_red) / float(a.D) : 0.0f;
        const float mah = block_sum(sah, s_red) / float(a.D);
        for (int j = threadIdx.x; j < a.D; j += kThreads) {
            const float v = to_float(dy[j]) * (a.gamma ? load_param(a.gamma, a.pdt, j) : 1.0f);
            const float g = (kept_value<T>(a, row, j) - mu) * r;
            float d = r * (v - ma - g * mah);
            if (a.dsum) d += to_float(static_cast<const T *>(a.dsum)[row * a.dss + j]);
            static_cast<T *>(a.dx)[row * a.dxs + j] = from_float<T>(d);
        }
    }
}

__device__ __forceinline__ void copy8(uint32_t smem, const void *p) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem), "l"(p) : "memory");
}
// What a stage of the backward's ring has of each thread, tensor after tensor, [units][16 bytes][threads]:
// dy, dsum (not CENTRED), and h or what is held of it (two units' bytes where they are shifted).
template <typename T, int NV, Lie LIE, bool CENTRED, bool HELD>
struct Ring {
    static constexpr int kVecs = kUnit * int(sizeof(T)) / 16;       // of a unit
    static constexpr int kRows = NV * kVecs * (CENTRED ? 1 : 2);
    static constexpr int kHeld = HELD ? (LIE == kShifted ? 2 * NV : NV) * 8 : NV * kVecs * 16;   // bytes a thread
    static constexpr bool kUsed = sizeof(T) == 2;                   // (float32: see below)
    static constexpr int kBytes = kUsed ? kRows * 16 + kHeld : 0;   // a thread and stage
    static constexpr int kStages = kBytes > 96 ? 2 : 3;
};

// A row's dy and h (FMT >= 0: kept in 8 bits) through a ring in shared memory, asynchronously, kStages
// - 1 rows ahead: every thread copies into slots of its own and reads only those, so the
// ring needs no barrier and the copies in flight no registers.  A unit of float32 would be two
// such copies, each of half of every 32-byte sector, which L2 reads twice; these come by
// one load of 32 bytes into registers, a row ahead (2M x 48: 227 us a call for 283).  The weights' sums stay in
// registers over all of a CTA's rows and leave one partial sum a CTA in a.part (none where it is
// NULL), or, where one CTA has all rows, the gradients themselves.
//
// 2M x 48 float32 from int8 (1.26 GB): 222 us at 5.6 TB/s; 8191 x 4096 bfloat16 from e4m3 (236 MB) 46 (35 at a
// copy's rate), 16384 x 1001 bfloat16 from int8 (83 MB) 34 (12): both have 15 warps an SM for the registers that
// x, dy and the weights' sums take, and wait on one another's instructions, 52 and 58 % of the issue slots taken.
template <typename T, int NV, bool MULTI, Lie LIE, bool CENTRED, int FMT>
__global__ void __launch_bounds__(MULTI ? kMaxRowThreads : kThreads, bwd_ctas(sizeof(T), NV, MULTI)) k_norm8_bwd(BwdArgs a, Place pl, bool alone) {
    constexpr int kSums = CENTRED ? 2 : 1;
    constexpr bool HELD = FMT >= 0;
    using R = Ring<T, NV, LIE, CENTRED, HELD>;
    constexpr int kStages = R::kStages;
    extern __shared__ uint4 s_ring[];        // the ring, then gamma [2 NV][threads]; at the end the sums
    __shared__ alignas(16) float s_red[MULTI ? kMaxGroups : 1][2][kSums][kRowWarps];
    const int group = MULTI ? threadIdx.x / pl.lanes : threadIdx.x >> pl.shift;
    const int lane = MULTI ? threadIdx.x - group * pl.lanes : threadIdx.x & (pl.lanes - 1);
    const int64_t step = int64_t(gridDim.x) * pl.groups, row0 = int64_t(blockIdx.x) * pl.groups + group;
    const Units c =
        units_at<MULTI>(lane, pl, a.D, LIE == kShifted ? head_of<T>(static_cast<const T *>(a.dy) + row0 * a.dys) : 0);
    const int apart = blockDim.x;
    const int stage_vecs = R::kBytes / 8 * apart / 2;        // 16-byte vectors of a stage
    uint4 *slot = s_ring + threadIdx.x;
    int lo[NV], hi[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) lo[k] = c.lo(k), hi[k] = c.hi(k);
    // the rows to fetch next
    const T *pd = static_cast<const T *>(a.dy) + row0 * a.dys + c.column(0),
            *ps = static_cast<const T *>(a.dsum) + row0 * a.dss + c.column(0),
            *px = static_cast<const T *>(a.h) + row0 * a.hs + c.column(0);
    const uint8_t *pq = a.kept.q + row0 * a.kept.stride;
    const int held_units = units_of(a.D);
    // unit k of a tensor into its slot
    auto fetch_unit = [&](uint4 *to, const T *p, int k) {
        if (LIE == kAnyhow) {
            const Raw<T> r = load_unit<T, false>(p + k * c.lanes * kUnit, hi[k]);
#pragma unroll
            for (int v = 0; v < R::kVecs; ++v)
                to[v * apart] = make_uint4(r.w[4 * v], r.w[4 * v + 1], r.w[4 * v + 2], r.w[4 * v + 3]);
        } else if (hi[k] > lo[k]) {
#pragma unroll
            for (int v = 0; v < R::kVecs; ++v)
                copy16(to + v * apart, reinterpret_cast<const uint4 *>(p + k * c.lanes * kUnit) + v);
        }
    };
    using HeldUnit = typename std::conditional<LIE == kShifted, HeldAcross, Held>::type;
    struct Ahead {
        Raw<T> dy[NV], dsum[NV], x[HELD ? 1 : NV];
        HeldUnit q[HELD ? NV : 1];
    };
    Ahead ahead;
    // Row `row` of all tensors into a stage (or registers); a row past the last as zeros.
    auto fetch = [&](int stage, int64_t row) {
        if constexpr (!R::kUsed) {
            const bool here = row < a.n;
            const int64_t skip = c.column(0);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                ahead.dy[k] = load_of<T, LIE>(pd - skip, c, k, here);
                if (!CENTRED && a.dsum) ahead.dsum[k] = load_of<T, LIE>(ps - skip, c, k, here);
                if constexpr (!HELD)
                    ahead.x[k] = load_of<T, LIE>(px - skip, c, k, here);
                else if constexpr (LIE == kShifted)
                    ahead.q[k].load(a.kept, row, c.column(k), a.D, here && hi[k] > 0);
                else
                    ahead.q[k].load(a.kept, row, c.at(k), here && hi[k] > 0);
            }
            pd += step * a.dys, ps += step * a.dss, px += step * a.hs;
            return;
        }
        uint4 *to = slot + stage * stage_vecs;
        uint2 *held = reinterpret_cast<uint2 *>(s_ring + stage * stage_vecs + R::kRows * apart) + threadIdx.x;
        if (row < a.n) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                fetch_unit(to + k * R::kVecs * apart, pd, k);
                if (!CENTRED && a.dsum) fetch_unit(to + (NV + k) * R::kVecs * apart, ps, k);
                if constexpr (!HELD) {
                    fetch_unit(to + (R::kRows + k * R::kVecs) * apart, px, k);
                } else if constexpr (LIE == kShifted) {
                    const int j = c.column(k), u = j >> 3;
                    if (hi[k] > 0 && u >= 0)
                        copy8(uint32_t(__cvta_generic_to_shared(held + 2 * k * apart)), pq + u * kUnit);
                    if (hi[k] > 0 && (j & 7) && u + 1 < held_units)
                        copy8(uint32_t(__cvta_generic_to_shared(held + (2 * k + 1) * apart)), pq + (u + 1) * kUnit);
                } else {
                    if (hi[k] > 0) copy8(uint32_t(__cvta_generic_to_shared(held + k * apart)), pq + c.at(k) * kUnit);
                }
            }
        } else {
            for (int v = 0; v < R::kRows + (HELD ? 0 : NV * R::kVecs); ++v) to[v * apart] = make_uint4(0u, 0u, 0u, 0u);
            if (HELD)
                for (int v = 0; v < R::kHeld / 8; ++v) held[v * apart] = make_uint2(0u, 0u);
        }
        copies_commit();
        pd += step * a.dys, ps += step * a.dss, px += step * a.hs, pq += step * a.kept.stride;
    };
    // slots that no copy fills stay zeros (a copy is not ordered after a store before it)
#pragma unroll
    for (int q = 0; q < (R::kUsed ? kStages : 0); ++q) {
        uint4 *to = slot + q * stage_vecs;
        uint2 *held = reinterpret_cast<uint2 *>(s_ring + q * stage_vecs + R::kRows * apart) + threadIdx.x;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (LIE != kAnyhow && hi[k] <= lo[k])
#pragma unroll
                for (int v = 0; v < R::kVecs; ++v) {
                    to[(k * R::kVecs + v) * apart] = make_uint4(0u, 0u, 0u, 0u);
                    if (!CENTRED) to[((NV + k) * R::kVecs + v) * apart] = make_uint4(0u, 0u, 0u, 0u);
                    if (!HELD) to[(R::kRows + k * R::kVecs + v) * apart] = make_uint4(0u, 0u, 0u, 0u);
                }
            if constexpr (HELD && LIE == kShifted) {
                const int j = c.column(k), u = j >> 3;
                if (hi[k] <= 0 || u < 0) held[2 * k * apart] = make_uint2(0u, 0u);
                if (hi[k] <= 0 || !(j & 7) || u + 1 >= held_units) held[(2 * k + 1) * apart] = make_uint2(0u, 0u);
            } else if constexpr (HELD) {
                if (hi[k] <= 0) held[k * apart] = make_uint2(0u, 0u);
            }
        }
    }
#pragma unroll
    for (int q = 0; q < (R::kUsed ? kStages - 1 : 1); ++q) fetch(q, row0 + q * step);
    // what a row needs beside them, a row ahead
    float mu, r;
    uint32_t e0[NV], e1[NV];
    auto load = [&](int64_t row) {
        const bool here = row < a.n;
        mu = CENTRED && here ? a.mean[row] : 0.0f, r = here ? a.rstd[row] : 0.0f;
        if (HELD && R::kUsed) {
            const uint8_t *s = a.kept.scales + row * a.kept.scale_stride;
            const int most = (a.D - 1) / kGroup;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int j = c.column(k), g = j < 0 ? 0 : j / kGroup, h = (j + kUnit - 1) / kGroup;
                e0[k] = here && hi[k] > 0 ? s[g] : 127u;
                if (LIE == kShifted) e1[k] = here && hi[k] > 0 ? s[h < most ? h : most] : 127u;
            }
        }
    };
    load(row0);
    float4 *plane = reinterpret_cast<float4 *>(s_ring + kStages * stage_vecs) + threadIdx.x;
    {
        F2 g[NV][4];
        load_weights<NV>(g, a.gamma, a.pdt, c);
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                plane[(2 * k + i) * apart] = make_float4(g[k][2 * i].x, g[k][2 * i].y, g[k][2 * i + 1].x, g[k][2 * i + 1].y);
    }
    if (MULTI) {
        for (int e = threadIdx.x; e < kMaxGroups * 2 * kSums * kRowWarps; e += blockDim.x) (&s_red[0][0][0][0])[e] = 0.0f;
        __syncthreads();
    }
    const float inv = 1.0f / float(a.D);
    F2 dg[NV][4], db[NV][4];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) dg[k][i] = db[k][i] = both(0.0f);
    int flip = 0, stage = 0;
    const int64_t lead = MULTI ? row0 : row0 - ((threadIdx.x & 31) >> pl.shift);
    T *pdx = static_cast<T *>(a.dx) + row0 * a.dxs;
    // unit k as a stage has it, of which [lo, hi) are the row's; others as zeros
    auto unit_in = [&](const uint4 *at, int k) {
        Raw<T> u;
#pragma unroll
        for (int v = 0; v < R::kVecs; ++v) {
            const uint4 q = at[v * apart];
            u.w[4 * v] = q.x, u.w[4 * v + 1] = q.y, u.w[4 * v + 2] = q.z, u.w[4 * v + 3] = q.w;
        }
        if (LIE != kAnyhow && hi[k] - lo[k] < kUnit) cut(u, lo[k], hi[k]);
        return u;
    };
    for (int64_t base = lead; base < a.n; base += step, pdx += step * a.dxs) {
        const int64_t row = base + (row0 - lead);
        Ahead now;
        if constexpr (R::kUsed) {
            copies_wait<kStages - 2>();
        } else {
            now = ahead;
            fetch(0, row + step);
        }
        const uint4 *from = slot + stage * stage_vecs;
        const uint2 *held = reinterpret_cast<const uint2 *>(s_ring + stage * stage_vecs + R::kRows * apart) + threadIdx.x;
        F2 d[NV][4], g[NV][4], s0 = both(0.0f), s1 = both(0.0f);
        const F2 rr = both(r), neg = both(-mu);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            F2 wt[4];
            floats_of(d[k], R::kUsed ? unit_in(from + k * R::kVecs * apart, k) : now.dy[k]);
            // g = (h - mean) r; what is not the row's meets zeros of dy
            if constexpr (!HELD) {
                floats_of(g[k], R::kUsed ? unit_in(from + (R::kRows + k * R::kVecs) * apart, k) : now.x[k]);
            } else if constexpr (!R::kUsed && LIE == kShifted) {
                now.q[k].template values<FMT>(g[k], c.column(k));
            } else if constexpr (!R::kUsed) {
                now.q[k].template values<FMT>(g[k]);
            } else if constexpr (LIE == kShifted) {
                const HeldAcross h{held[2 * k * apart], held[(2 * k + 1) * apart], e0[k], e1[k]};
                h.template values<FMT>(g[k], c.column(k));
            } else {
                const Held h{held[k * apart], e0[k]};
                h.template values<FMT>(g[k]);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float4 q = plane[(2 * k + i) * apart];
                wt[2 * i] = make_float2(q.x, q.y), wt[2 * i + 1] = make_float2(q.z, q.w);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                g[k][i] = mul2(CENTRED ? add2(g[k][i], neg) : g[k][i], rr);
                dg[k][i] = fma2(d[k][i], g[k][i], dg[k][i]);
                if (CENTRED) db[k][i] = add2(db[k][i], d[k][i]);
                d[k][i] = mul2(d[k][i], wt[i]);
                if (CENTRED) s1 = add2(s1, d[k][i]);
                s0 = fma2(d[k][i], g[k][i], s0);
            }
        }
        Raw<T> up[NV];
        const bool sums = !CENTRED && a.dsum;
        if (sums)
#pragma unroll
            for (int k = 0; k < NV; ++k) up[k] = R::kUsed ? unit_in(from + (NV + k) * R::kVecs * apart, k) : now.dsum[k];
        float sum[kSums];
        sum[0] = sum_of(s0);
        if (CENTRED) sum[kSums - 1] = sum_of(s1);
        load(row + step);
        if (R::kUsed) fetch(stage == 0 ? kStages - 1 : stage - 1, row + (kStages - 1) * step);   // the slots read one row ago
        stage = stage == kStages - 1 ? 0 : stage + 1;
        row_sum<kSums, MULTI>(sum, pl.lanes, group, lane, s_red[MULTI ? group : 0], flip);
        const F2 mag = both(-sum[0] * inv), ma = both(CENTRED ? -sum[kSums - 1] * inv : 0.0f);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (CENTRED) d[k][i] = add2(d[k][i], ma);
                d[k][i] = mul2(fma2(g[k][i], mag, d[k][i]), rr);
            }
            if (sums) {
                F2 u[4];
                floats_of(u, up[k]);
#pragma unroll
                for (int i = 0; i < 4; ++i) d[k][i] = add2(d[k][i], u[i]);
            }
            store_of<T, LIE>(pdx, raw_of<T>(d[k]), c, k, row < a.n);
        }
    }
    copies_wait<0>();
    start_dependents();
    if (!a.part) return;
    // The CTA's sums, in fixed order: the rows of a warp are joined by shuffles where their columns
    // are the same (!MULTI, not kShifted), then the warps or groups in turn, in the ring's place.
    __syncthreads();                       // the last rows' slots and gamma have been read
    constexpr bool kFold = !MULTI && LIE != kShifted;
    const int cols = kSums * a.D;
    const int slots = kFold ? kThreads / 32 : pl.groups;
    float *s_sum = reinterpret_cast<float *>(s_ring);
    float *part = a.part + size_t(blockIdx.x) * cols;
    const bool direct = slots == 1 && !alone;
    float *mine = direct ? part : s_sum + size_t(kFold ? threadIdx.x >> 5 : group) * cols;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int q = 0; q < kSums; ++q)
#pragma unroll
            for (int i = 0; i < kUnit; ++i) {
                const F2 t = q ? db[k][i / 2] : dg[k][i / 2];
                float v = i & 1 ? t.y : t.x;
                if (kFold)
                    for (int o = pl.lanes; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                if (i >= c.lo(k) && i < c.hi(k) && (!kFold || (threadIdx.x & 31) < pl.lanes))
                    mine[q * a.D + c.column(k) + i] = v;
            }
    if (direct) return;
    __syncthreads();
    for (int j = threadIdx.x; j < cols; j += blockDim.x) {
        float t = 0.0f;
        for (int v = 0; v < slots; ++v) t += s_sum[size_t(v) * cols + j];
        if (!alone)
            part[j] = t;
        else if (j < a.D)
            store_param(a.dgamma, a.pdt, j, t);
        else
            store_param(a.dbeta, a.pdt, j - a.D, t);
    }
}

// The partial sums of 32 columns of [dgamma | dbeta], or of dgamma alone.
__global__ void __launch_bounds__(1024) k_norm8_bwd_final(const float *part, int parts, int32_t D, int cols,
                                                          void *dgamma, void *dbeta, int pdt) {
    add_up_parts(part, parts, D, cols, dgamma, dbeta, pdt);
}

constexpr int kMaxSmem = 225 * 1024;   // 227 KB less 2 KB of static buffers
static_assert(kUnit == kMaxPeriod, "rows' starts repeat after a unit's elements at most");

// f(NV, MULTI) of a place, as constants.
template <bool SINGLE, typename F>
void with_place(int nv, bool multi, F &&f) {
    if (multi && nv == 2) {
        f(std::integral_constant<int, 2>(), std::true_type());
        return;
    }
    if constexpr (SINGLE) {
        if (multi) return f(std::integral_constant<int, 1>(), std::true_type());
    } else {
        if (nv == 2) return f(std::integral_constant<int, 2>(), std::false_type());
    }
    f(std::integral_constant<int, 1>(), std::false_type());
}
template <typename F>
void with_lie(Lie lie, F &&f) {
    if (lie == kAligned)
        f(std::integral_constant<Lie, kAligned>());
    else if (lie == kShifted)
        f(std::integral_constant<Lie, kShifted>());
    else
        f(std::integral_constant<Lie, kAnyhow>());
}
template <typename F>
void with_flag(bool b, F &&f) {
    if (b)
        f(std::true_type());
    else
        f(std::false_type());
}

template <typename T>
void launch_fwd(const FwdArgs &a, int sms, cudaStream_t s) {
    if (!in_registers(a.D)) {
        SS_LAUNCH("k_rms_fwd_wide", s, k_rms_fwd_wide<T><<<wide_grid(a.n, sms), kThreads, 0, s>>>(a));
        return;
    }
    const bool aligned = units_aligned<T>(a.x, a.xs) &&
                         (!a.residual || (units_aligned<T>(a.residual, a.rs) && units_aligned<T>(a.sum, a.ss_))) &&
                         (!a.y || units_aligned<T>(a.y, a.ys));
    const bool alike = (!a.residual || (start_alike<T>(a.x, a.xs, a.residual, a.rs) && start_alike<T>(a.x, a.xs, a.sum, a.ss_))) &&
                       (!a.y || start_alike<T>(a.x, a.xs, a.y, a.ys)) && a.kept_fmt < 0 && a.out_fmt < 0;
    const Lie lie = aligned ? kAligned : (alike && shifted_in_registers(a.D) ? kShifted : kAnyhow);
    int nv;
    bool multi;
    const Place pl = place_of(a.D, lie == kShifted, false, &nv, &multi);
    const int threads = multi ? pl.lanes * pl.groups : kThreads, period = lie == kShifted ? period_of(a.xs) : 1;
    with_place<false>(nv, multi, [&](auto NV, auto MULTI) {
        with_lie(lie, [&](auto LIE) {
            with_flag(a.residual != nullptr, [&](auto RES) {
                auto kernel = k_rms_fwd<T, NV(), MULTI(), LIE(), RES()>;
                static std::atomic<unsigned long long> known{0};
                const int grid = grid_of(&known, kernel, threads, 0, a.n, pl.groups, period, multi ? 1 : 8, 1 << 30, sms);
                SS_LAUNCH("k_rms_fwd", s, kernel<<<grid, threads, 0, s>>>(a, pl));
            });
        });
    });
}

template <typename T, bool CENTRED, int FMT>
ss_status launch_bwd(const BwdArgs &a, int sms, cudaStream_t s) {
    constexpr bool HELD = FMT >= 0;
    const int cols = CENTRED ? 2 * a.D : a.D;
    const dim3 final_grid((cols + 31) / 32);
    if (a.n == 0 || !in_registers(a.D)) {
        // the weights first: dx may overwrite dy, dsum or h
        if (a.dgamma) {
            const dim3 g((a.D + kThreads - 1) / kThreads, unsigned(a.n < 64 ? (a.n < 1 ? 1 : a.n) : 64));
            SS_LAUNCH("k_norm8_bwd_weights_wide", s, k_norm8_bwd_weights_wide<T><<<g, kThreads, 0, s>>>(a));
            SS_LAUNCH("k_norm8_bwd_final", s,
                      launch_after(k_norm8_bwd_final, final_grid, 1024, 0, s, a.part, int(g.y), a.D, cols, a.dgamma,
                                   a.dbeta, a.pdt));
        }
        if (a.n > 0)
            SS_LAUNCH("k_norm8_bwd_rows_wide", s, k_norm8_bwd_rows_wide<T><<<wide_grid(a.n, sms), kThreads, 0, s>>>(a));
        return SS_OK;
    }
    const bool aligned = units_aligned<T>(a.dy, a.dys) && units_aligned<T>(a.dx, a.dxs) &&
                         (HELD || units_aligned<T>(a.h, a.hs)) && (!a.dsum || units_aligned<T>(a.dsum, a.dss));
    const bool alike = start_alike<T>(a.dy, a.dys, a.dx, a.dxs) && (HELD || start_alike<T>(a.dy, a.dys, a.h, a.hs)) &&
                       (!a.dsum || start_alike<T>(a.dy, a.dys, a.dsum, a.dss));
    const Lie lie = aligned ? kAligned : (alike && shifted_in_registers(a.D) ? kShifted : kAnyhow);
    int nv;
    bool multi;
    const Place pl = place_of(a.D, lie == kShifted, sizeof(T) == 4, &nv, &multi);
    const int threads = multi ? pl.lanes * pl.groups : kThreads, period = lie == kShifted ? period_of(a.dys) : 1;
    // what one CTA takes at once needs no launch that adds up several CTAs' sums
    const bool alone = a.n <= pl.groups;
    ss_status st = SS_OK;
    with_place<sizeof(T) == 4>(nv, multi, [&](auto NV, auto MULTI) {
        with_lie(lie, [&](auto LIE) {
            auto kernel = k_norm8_bwd<T, NV(), MULTI(), LIE(), CENTRED, FMT>;
            using R = Ring<T, NV(), LIE(), CENTRED, HELD>;
            const int slots = MULTI() || LIE() == kShifted ? pl.groups : kThreads / 32;
            size_t smem = (size_t(R::kStages) * R::kBytes + 2 * NV() * sizeof(float4)) * threads;
            const size_t sums = a.dgamma && (slots > 1 || alone) ? size_t(slots) * cols * sizeof(float) : 0;
            if (smem < sums) smem = sums;
            static std::atomic<unsigned long long> smem_ctx[kMaxDevices];   // see ensure_dyn_smem
            const void *fn = (const void *)kernel;
            if ((st = ensure_dyn_smem(smem_ctx, &fn, 1, kMaxSmem, "k_norm8_bwd")) != SS_OK) return;
            static std::atomic<unsigned long long> known{0};
            const int grid = alone ? 1 : grid_of(&known, kernel, threads, smem, a.n, pl.groups, period, 1, kMaxParts - kMaxPeriod, sms);
            BwdArgs b = a;
            if (!a.dgamma) b.part = nullptr;
            SS_LAUNCH("k_norm8_bwd", s, kernel<<<grid, threads, smem, s>>>(b, pl, alone));
            if (a.dgamma && !alone)
                SS_LAUNCH("k_norm8_bwd_final", s,
                          launch_after(k_norm8_bwd_final, final_grid, 1024, 0, s, a.part, grid, a.D, cols, a.dgamma,
                                       a.dbeta, a.pdt));
        });
    });
    return st;
}

ss_status backward(const char *who, const BwdArgs &a, int dtype, int sms, cudaStream_t s) {
    ss_status st = SS_OK;
    with_type(dtype, [&](auto t) {
        using T = decltype(t);
        if (a.centred)
            with_format(a.fmt, [&](auto F) { st = launch_bwd<T, true, decltype(F)::value>(a, sms, s); });
        else if (a.fmt >= 0)
            with_format(a.fmt, [&](auto F) { st = launch_bwd<T, false, decltype(F)::value>(a, sms, s); });
        else
            st = launch_bwd<T, false, -1>(a, sms, s);
    });
    return st != SS_OK ? st : check_launch(who);
}

}  // namespace
}  // namespace ss

using namespace ss;

extern "C" {

ss_status ss_rms_norm_fwd(const void *x, ss_dtype dtype, int64_t x_stride, const void *residual,
                          int64_t residual_stride, int64_t n, int32_t D, const void *gamma, ss_dtype param_dtype,
                          float eps, void *sum, int64_t sum_stride, void *y, int64_t y_stride, const ss_rows8 *out,
                          const ss_rows8 *kept, float *rstd, ss_stream_t stream) {
    clear_error();
    const char *who = "ss_rms_norm_fwd";
    ss_status st = check_row_sizes(who, n, D);
    if (st != SS_OK) return st;
    if ((st = check_row_types(who, dtype, param_dtype)) != SS_OK) return st;
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(SS_ERR_INVALID_ARG, "%s: eps negative or not finite", who);
    if (n == 0) return SS_OK;
    if ((st = check_row_tensor(who, "x", x, x_stride, D, dtype)) != SS_OK) return st;
    if ((residual == nullptr) != (sum == nullptr))
        return fail(SS_ERR_INVALID_ARG, "%s: one of residual and sum is NULL", who);
    if (residual) {
        if ((st = check_row_tensor(who, "residual", residual, residual_stride, D, dtype)) != SS_OK) return st;
        if ((st = check_row_tensor(who, "sum", sum, sum_stride, D, dtype)) != SS_OK) return st;
        if (sum == y) return fail(SS_ERR_INVALID_ARG, "%s: sum and y are the same rows", who);
    }
    if (y && (st = check_row_tensor(who, "y", y, y_stride, D, dtype)) != SS_OK) return st;
    if (out && (st = check_rows8(who, "out", out, D)) != SS_OK) return st;
    if (kept && (st = check_rows8(who, "kept", kept, D)) != SS_OK) return st;
    if (out && kept && out->q == kept->q) return fail(SS_ERR_INVALID_ARG, "%s: out and kept are the same rows", who);
    if ((st = check_aligned(who, "gamma", gamma, param_dtype)) != SS_OK) return st;
    if ((st = check_aligned(who, "rstd", rstd, SS_F32)) != SS_OK) return st;
    int dev = 0, sms = 0;
    if ((st = current_device(&dev, &sms, "ss_rms_norm_fwd: device query")) != SS_OK) return st;
    cudaStream_t s = (cudaStream_t)stream;
    const FwdArgs a{x, x_stride, residual, residual_stride, n, D, gamma, int(param_dtype), eps, sum, sum_stride, y,
                    y_stride, rows8_of(out), rows8_of(kept), out ? out->format : -1, kept ? kept->format : -1, rstd};
    with_type(dtype, [&](auto t) { launch_fwd<decltype(t)>(a, sms, s); });
    return check_launch(who);
}

size_t ss_rms_norm_workspace_bytes(int64_t n, int32_t D) {
    return row_sizes_ok(n, D) ? size_t(weight_parts(n)) * 2 * D * sizeof(float) : 0;
}

size_t ss_layer_norm_bwd8_workspace_bytes(int64_t n, int32_t D) { return ss_rms_norm_workspace_bytes(n, D); }

ss_status ss_rms_norm_bwd(const void *dy, int64_t dy_stride, const void *h, int64_t h_stride, const ss_rows8 *kept,
                          ss_dtype dtype, int64_t n, int32_t D, const void *gamma, ss_dtype param_dtype,
                          const float *rstd, const void *dsum, int64_t dsum_stride, void *dx, int64_t dx_stride,
                          void *dgamma, void *workspace, size_t workspace_bytes, ss_stream_t stream) {
    clear_error();
    const char *who = "ss_rms_norm_bwd";
    ss_status st = check_row_sizes(who, n, D);
    if (st != SS_OK) return st;
    if ((st = check_row_types(who, dtype, param_dtype)) != SS_OK) return st;
    if (n > 0) {
        if ((st = check_row_tensor(who, "dy", dy, dy_stride, D, dtype)) != SS_OK) return st;
        if ((h == nullptr) == (kept == nullptr))
            return fail(SS_ERR_INVALID_ARG, "%s: one of h and kept is wanted, and not both", who);
        if (h && (st = check_row_tensor(who, "h", h, h_stride, D, dtype)) != SS_OK) return st;
        if (kept && (st = check_rows8(who, "kept", kept, D)) != SS_OK) return st;
        if (dsum && (st = check_row_tensor(who, "dsum", dsum, dsum_stride, D, dtype)) != SS_OK) return st;
        if ((st = check_row_tensor(who, "dx", dx, dx_stride, D, dtype)) != SS_OK) return st;
        if (!rstd) return fail(SS_ERR_INVALID_ARG, "%s: rstd is NULL", who);
        if ((st = check_aligned(who, "rstd", rstd, SS_F32)) != SS_OK) return st;
        if ((st = check_aligned(who, "gamma", gamma, param_dtype)) != SS_OK) return st;
    }
    if ((st = check_aligned(who, "dgamma", dgamma, param_dtype)) != SS_OK) return st;
    if (dgamma && (st = check_workspace(who, workspace, workspace_bytes, ss_rms_norm_workspace_bytes(n, D))) != SS_OK)
        return st;
    int dev = 0, sms = 0;
    if ((st = current_device(&dev, &sms, "ss_rms_norm_bwd: device query")) != SS_OK) return st;
    const BwdArgs a{dy, dy_stride, h, h_stride, rows8_of(kept), kept ? kept->format : -1, n, D, gamma,
                    int(param_dtype), nullptr, rstd, dsum, dsum_stride, dx, dx_stride, dgamma, nullptr,
                    static_cast<float *>(workspace), false};
    return backward(who, a, dtype, sms, (cudaStream_t)stream);
}

ss_status ss_layer_norm_bwd8(const void *dy, int64_t dy_stride, const ss_rows8 *kept, ss_dtype dtype, int64_t n,
                             int32_t D, const void *gamma, ss_dtype param_dtype, const float *mean, const float *rstd,
                             void *dx, int64_t dx_stride, void *dgamma, void *dbeta, void *workspace,
                             size_t workspace_bytes, ss_stream_t stream) {
    clear_error();
    const char *who = "ss_layer_norm_bwd8";
    ss_status st = check_row_sizes(who, n, D);
    if (st != SS_OK) return st;
    if ((st = check_row_types(who, dtype, param_dtype)) != SS_OK) return st;
    if (n > 0) {
        if ((st = check_row_tensor(who, "dy", dy, dy_stride, D, dtype)) != SS_OK) return st;
        if ((st = check_rows8(who, "kept", kept, D)) != SS_OK) return st;
        if ((st = check_row_tensor(who, "dx", dx, dx_stride, D, dtype)) != SS_OK) return st;
        if (!mean || !rstd) return fail(SS_ERR_INVALID_ARG, "%s: mean or rstd is NULL", who);
        if ((st = check_aligned(who, "mean", mean, SS_F32)) != SS_OK) return st;
        if ((st = check_aligned(who, "rstd", rstd, SS_F32)) != SS_OK) return st;
        if ((st = check_aligned(who, "gamma", gamma, param_dtype)) != SS_OK) return st;
    }
    if ((dgamma == nullptr) != (dbeta == nullptr))
        return fail(SS_ERR_INVALID_ARG, "%s: one of dgamma and dbeta is NULL", who);
    if ((st = check_aligned(who, "dgamma", dgamma, param_dtype)) != SS_OK) return st;
    if ((st = check_aligned(who, "dbeta", dbeta, param_dtype)) != SS_OK) return st;
    if (dgamma &&
        (st = check_workspace(who, workspace, workspace_bytes, ss_layer_norm_bwd8_workspace_bytes(n, D))) != SS_OK)
        return st;
    int dev = 0, sms = 0;
    if ((st = current_device(&dev, &sms, "ss_layer_norm_bwd8: device query")) != SS_OK) return st;
    const BwdArgs a{dy, dy_stride, nullptr, 0, rows8_of(kept), kept ? kept->format : -1, n, D, gamma,
                    int(param_dtype), mean, rstd, nullptr, 0, dx, dx_stride, dgamma, dbeta,
                    static_cast<float *>(workspace), true};
    return backward(who, a, dtype, sms, (cudaStream_t)stream);
}

}  // extern "C"
