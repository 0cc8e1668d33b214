// Layer normalisation of rows and its gradient (model: include/ss_norm.h).
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "ss_internal.h"
#include "ss_launch.cuh"
#include "ss_norm.cuh"
#include "ss_norm.h"
#include "ss_profile.h"
#include "ss_vec.cuh"

namespace ss {
namespace {

constexpr int kThreads = kNormThreads;
constexpr int32_t kMaxD = 65536;

// A row's place in the threads.  `lanes` threads share it, thread l of them
// holding 16-byte vectors l, l + lanes, ... (NV of them) in registers, so the
// row is read once for the mean, the centred squares and the result.  Narrow
// rows (MULTI false) take a power of two of lanes inside a warp and reduce by
// shuffles; wide ones take whole warps and reduce through shared memory and a
// barrier of their own.
//
// Rows arrive through a ring in shared memory, asynchronously, kStages - 1
// rows ahead: every thread copies into slots of its own and reads only
// those, so the ring needs no barrier and the copies in flight no registers.
//
// Rows need not start on 16-byte boundaries (SHIFT): vectors lie on the
// boundaries, and the few elements of a row before its first and after its
// last vector go to the lanes, X at most to each.  A group of lanes takes every
// step-th row with step a multiple of the period after which rows start
// alike, so its columns stay fixed.
constexpr int kPerThread = 16;       // elements of a row in one thread's vectors
constexpr int kMaxGroups = 8;        // of two warps at least

struct Place {
    int lanes, shift;   // lanes = 1 << shift where !MULTI
    int vecs;           // vectors of a row, where it starts on a boundary
    int groups;         // rows side by side in a CTA
};

// Rows of one tensor; `same`: they start as far from a boundary as x's.
template <typename T>
struct Rows {
    T *base;
    int64_t stride;
    bool same;
};

// Rows ahead by what they take: 16 bytes a vector, thread and tensor.
constexpr int stages_of(int vectors) { return vectors <= 2 ? 4 : 3; }

// Rounding of the mean.  1 / sqrt(var + eps) multiplies it: a row of one value
// 1e4 and a mean one unit of its last place off give y = 0.3 for 0.
// A float32 sum of 16-bit values that are all alike is exact (in float16 up to
// 8192 of them), so there the quotient sum / D is rounded once and no more.
// Sums of float32 values are not; where the mean is `far` from the row's spread
// the deviations from it, which are nearly exact there, are averaged and the
// average taken off.  Nearer, a few units of the mean's last place are no more
// than a few roundings of a result of that size.
constexpr float kFar = 8.0f;
// v = var + eps: by the squares, so that it need not wait for the root.
__device__ __forceinline__ bool far_off(float mu, float v) { return mu * mu > kFar * kFar * v; }
// a / width, correctly rounded, from inv = 1 / width: the product, and its
// remainder, which a fused product gives exactly, times inv (P. Markstein, IBM
// J. Res. Dev. 34, 1990).
__device__ __forceinline__ float quotient(float a, float width, float inv) {
    const float q = a * inv, r = fmaf(-q, width, a);
    return isfinite(q) ? fmaf(r, inv, q) : q;
}

template <int K>
__device__ __forceinline__ void clear_sums(float *s_red, int count) {
    for (int e = threadIdx.x; e < count * 2 * K * kRowWarps; e += blockDim.x) s_red[e] = 0.0f;
}

// Where a thread's columns lie: vectors lane, lane + lanes, ... of the `vecs`
// whole ones that begin after `head` elements, and, of the elements before
// and after them, lane, lane + lanes, ... (column extra(u), -1: none).
struct Cols {
    int lane, lanes, vecs, head, tail;
    int32_t D;
    __device__ __forceinline__ int extra(int u) const {
        const int q = lane + u * lanes;
        return q < head ? q : (q < head + tail ? D - tail + q - head : -1);
    }
};

template <typename T, int VEC, bool SHIFT>
__device__ __forceinline__ Cols cols_of(const Rows<const T> &x, int64_t row, int lane, const Place &pl, int32_t D) {
    Cols c{lane, pl.lanes, pl.vecs, 0, 0, D};
    if (SHIFT) {
        const int h = int((16 - (reinterpret_cast<uintptr_t>(x.base + row * x.stride) & 15)) & 15) / int(sizeof(T));
        c.head = h < D ? h : D;
        c.vecs = (D - c.head) / VEC;
        c.tail = D - c.head - c.vecs * VEC;
    }
    return c;
}

// Starts the copies of a row's vectors into this thread's slots (slots `apart`
// vectors from one another).  p: the row's start.  A tensor whose rows start
// otherwise than x's is read element by element.
template <typename T, int VEC, int NV, bool SHIFT>
__device__ __forceinline__ void fetch_row(uint4 *slot, int apart, const T *p, bool same, const Cols &c) {
    if (SHIFT) p += c.head;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int v = c.lane + k * c.lanes;
        if (v >= c.vecs) continue;
        if (!SHIFT || same) {
            copy16(slot + k * apart, p + v * VEC);
        } else {
            Vec<T, VEC> r;
            r.clear();
#pragma unroll
            for (int i = 0; i < VEC; ++i) r.set(i, p[v * VEC + i]);
            slot[k * apart] = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
        }
    }
}

template <typename T, int VEC>
__device__ __forceinline__ Vec<T, VEC> from_slot(const uint4 *slot) {
    const uint4 u = *slot;
    Vec<T, VEC> x;
    x.w[0] = u.x, x.w[1] = u.y, x.w[2] = u.z, x.w[3] = u.w;
    return x;
}

template <typename T, int VEC, bool SHIFT>
__device__ __forceinline__ void store_row(T *p, bool same, int v, const Cols &c, const F2 (&o)[VEC / 2]) {
    p += (SHIFT ? c.head : 0) + v * VEC;
    if (!SHIFT || same) {
        store_pairs<T, VEC>(p, o);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; i += 2) {
            p[i] = from_float<T>(o[i / 2].x), p[i + 1] = from_float<T>(o[i / 2].y);
        }
    }
}

// A thread's weights, in float32 registers; `absent` where there are none.
// All its loads are in flight together.
template <int VEC, int NV, bool SHIFT, typename P>
__device__ __forceinline__ void load_weights_as(F2 (&g)[NV][VEC / 2], const P *w, float absent, const Cols &c) {
    constexpr int kVec = 16 / sizeof(P);
    if constexpr (VEC % kVec == 0)
    if (w && !SHIFT && (reinterpret_cast<uintptr_t>(w) & 15) == 0) {
        Vec<P, kVec> q[NV][VEC / kVec];
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < VEC / kVec; ++i) {
                q[k][i].clear();
                if (c.lane + k * c.lanes < c.vecs) q[k][i] = load_vec<P, kVec>(w + (c.lane + k * c.lanes) * VEC + i * kVec);
            }
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < VEC; i += 2)
                g[k][i / 2] = make_float2(q[k][i / kVec].get(i % kVec), q[k][i / kVec].get(i % kVec + 1));
        return;
    }
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < VEC; i += 2) {
            float q[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int v = c.lane + k * c.lanes;
                q[u] = w && v < c.vecs ? to_float(w[c.head + v * VEC + i + u]) : absent;
            }
            g[k][i / 2] = make_float2(q[0], q[1]);
        }
}

template <int VEC, int NV, bool SHIFT>
__device__ __forceinline__ void load_weights(F2 (&g)[NV][VEC / 2], const void *w, int pdt, float absent, const Cols &c) {
    if (pdt == SS_F32)
        load_weights_as<VEC, NV, SHIFT>(g, static_cast<const float *>(w), absent, c);
    else if (pdt == SS_F16)
        load_weights_as<VEC, NV, SHIFT>(g, static_cast<const __half *>(w), absent, c);
    else
        load_weights_as<VEC, NV, SHIFT>(g, static_cast<const __nv_bfloat16 *>(w), absent, c);
}

// The weight of a column (-1: none).
__device__ __forceinline__ float weight_of(const void *w, int pdt, float absent, int col) {
    return w && col >= 0 ? load_param(w, pdt, col) : absent;
}

// The backward has no registers left for gamma: a thread's vectors lie in
// shared memory, one plane for every four columns of a vector, so that the
// lanes of a warp read side by side (as two vectors of one thread, one after
// the other, they would meet in the banks).
template <int VEC, int NV>
__device__ __forceinline__ void put_weights(float4 *plane, int apart, const F2 (&g)[NV][VEC / 2]) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) {
            const F2 a = g[k][2 * i], b = g[k][2 * i + 1];
            plane[(k * (VEC / 4) + i) * apart] = make_float4(a.x, a.y, b.x, b.y);
        }
}
template <int VEC>
__device__ __forceinline__ void weights_of(F2 (&g)[VEC / 2], const float4 *plane, int apart, int k) {
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
        const float4 q = plane[(k * (VEC / 4) + i) * apart];
        g[2 * i] = make_float2(q.x, q.y), g[2 * i + 1] = make_float2(q.z, q.w);
    }
}

// CTAs an SM that the registers are held down for: a row's chain of sums is
// long, and more rows at a time hide it while they leave the rows' own registers
// alone (1.5M x 7 bfloat16: 58 us with two or three, 45 with four; 1.73M x 35: 112
// with two, 89 with three, 104 with four; 500,000 x 50 float32: 37 with two, 38
// with three, 47 with four).
constexpr int fwd_ctas(int vec, int nv, bool multi, int x) {
    return multi ? 1 : (nv == 1 && x <= 2 ? 4 : (x > 0 && nv * vec > 8 ? 2 : 3));
}

// mean, centred squares and result of a row from registers.  Float32 rows whose
// mean is far_off take one sum more, and one branch for every row: 2M x 48
// 113.8 -> 114.0 us, 2M x 3 47 -> 50 (in 16 bits, where the quotient does, the
// branch would cost 1 to 5 us of 20 to 100).  Bound by memory:
// 2M x 48 float32 (768 MB and the statistics) 114 us, at copy bandwidth (116);
// 8191 x 4096 bfloat16 29 (20); 8191 x 8192 float32 83 (79); 1,731,207 x 35
// bfloat16 89 (38: seven of eight rows start off a 16-byte boundary, and their
// three or four vectors leave up to 14 elements that are loaded one by one).
template <typename T, int VEC, int NV, bool MULTI, int X>
__global__ void __launch_bounds__(MULTI ? kMaxRowThreads : kThreads, fwd_ctas(VEC, NV, MULTI, X))
    k_norm_fwd(Rows<const T> x, int64_t n, int32_t D, Place pl, const void *gamma, const void *beta, int pdt, float eps,
               Rows<T> y, float *mean, float *rstd) {
    extern __shared__ uint4 s_ring[];    // [stages][NV][threads]
    __shared__ alignas(16) float s_red[MULTI ? kMaxGroups : 1][2][1][kRowWarps];
    constexpr bool SHIFT = X > 0;
    constexpr bool kAgain = sizeof(T) == 4;
    constexpr int kStages = stages_of(NV), kHalf = VEC / 2, kX = SHIFT ? X : 1;
    const int group = MULTI ? threadIdx.x / pl.lanes : threadIdx.x >> pl.shift;
    const int lane = MULTI ? threadIdx.x - group * pl.lanes : threadIdx.x & (pl.lanes - 1);
    const int64_t step = int64_t(gridDim.x) * pl.groups;
    const int64_t row0 = int64_t(blockIdx.x) * pl.groups + group;
    const Cols c = cols_of<T, VEC, SHIFT>(x, row0, lane, pl, D);
    const int apart = blockDim.x;
    uint4 *slot = s_ring + threadIdx.x;
    const T *px = x.base + row0 * x.stride, *pe = px;   // the rows to fetch next: its vectors, its other elements
    const int64_t xstep = step * x.stride;
#pragma unroll
    for (int q = 0; q < kStages; ++q) {
        if (q < kStages - 1) {
            if (row0 + q * step < n) fetch_row<T, VEC, NV, SHIFT>(slot + q * NV * apart, apart, px, true, c);
            copies_commit();
            px += xstep;
        }
#pragma unroll
        for (int k = 0; k < NV; ++k)       // slots that no copy fills stay zero
            if (c.lane + k * c.lanes >= c.vecs) slot[(q * NV + k) * apart] = make_uint4(0, 0, 0, 0);
    }
    float e[kX], ge[kX], be[kX];
    int col[kX];
#pragma unroll
    for (int u = 0; u < kX; ++u) {
        col[u] = SHIFT ? c.extra(u) : -1;
        e[u] = SHIFT && col[u] >= 0 && row0 < n ? to_float(pe[col[u]]) : 0.0f;
        ge[u] = SHIFT ? weight_of(gamma, pdt, 1.0f, col[u]) : 1.0f;
        be[u] = SHIFT ? weight_of(beta, pdt, 0.0f, col[u]) : 0.0f;
    }
    pe += xstep;
    F2 g[NV][kHalf], b[NV][kHalf];
    load_weights<VEC, NV, SHIFT>(g, gamma, pdt, 1.0f, c);
    load_weights<VEC, NV, SHIFT>(b, beta, pdt, 0.0f, c);
    if (MULTI) clear_sums<1>(&s_red[0][0][0][0], kMaxGroups);
    __syncthreads();
    const float width = float(D), inv = 1.0f / width;
    int flip = 0, stage = 0;
    T *py = y.base + row0 * y.stride;
    const int64_t ystep = step * y.stride;
    // a warp's lanes leave together: they shuffle with one another; a row past
    // the last is worked on as it lies in the ring and not stored
    const int64_t lead = MULTI ? row0 : row0 - ((threadIdx.x & 31) >> pl.shift);
    for (int64_t base = lead; base < n; base += step, py += ystep) {
        const int64_t row = base + (row0 - lead);
        copies_wait<kStages - 2>();
        F2 f[NV][kHalf], acc = both(0.0f);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            widen<T, VEC>(f[k], from_slot<T, VEC>(slot + (stage * NV + k) * apart));
#pragma unroll
            for (int i = 0; i < kHalf; ++i) acc = add2(acc, f[k][i]);
        }
        const int last = stage == 0 ? kStages - 1 : stage - 1;   // the slots read one row ago
        if (row + (kStages - 1) * step < n)
            fetch_row<T, VEC, NV, SHIFT>(slot + last * NV * apart, apart, px, true, c);
        copies_commit();
        px += xstep;
        stage = stage == kStages - 1 ? 0 : stage + 1;
        float sum[1] = {sum_of(acc)}, ec[kX];
        if (SHIFT) {
#pragma unroll
            for (int u = 0; u < kX; ++u) {
                ec[u] = e[u];
                sum[0] += e[u];
                if (col[u] >= 0 && row + step < n) e[u] = to_float(pe[col[u]]);
            }
            pe += xstep;
        }
        row_sum<1, MULTI>(sum, pl.lanes, group, c.lane, s_red[MULTI ? group : 0], flip);
        float mu = kAgain ? sum[0] * inv : quotient(sum[0], width, inv);
        const F2 neg = both(-mu);
        acc = both(0.0f);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (c.lane + k * pl.lanes < c.vecs) {
#pragma unroll
                for (int i = 0; i < kHalf; ++i) {
                    f[k][i] = add2(f[k][i], neg);
                    acc = fma2(f[k][i], f[k][i], acc);
                }
            }
        }
        sum[0] = sum_of(acc);
        if (SHIFT)
#pragma unroll
            for (int u = 0; u < kX; ++u) {
                ec[u] = col[u] >= 0 ? ec[u] - mu : 0.0f;
                sum[0] = fmaf(ec[u], ec[u], sum[0]);
            }
        row_sum<1, MULTI>(sum, pl.lanes, group, c.lane, s_red[MULTI ? group : 0], flip);
        float v = fmaf(sum[0], inv, eps);
        const bool again = kAgain && far_off(mu, v);
        // (a row's lanes agree; and one branch for what few rows are)
        if (kAgain && (MULTI ? again : __any_sync(0xffffffffu, again || row >= n))) {
            const float var = sum[0] * inv;
            acc = both(0.0f);
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (c.lane + k * c.lanes < c.vecs)
#pragma unroll
                    for (int i = 0; i < kHalf; ++i) acc = add2(acc, f[k][i]);
            sum[0] = sum_of(acc);
            if (SHIFT)
#pragma unroll
                for (int u = 0; u < kX; ++u) sum[0] += ec[u];
            row_sum<1, MULTI>(sum, pl.lanes, group, c.lane, s_red[MULTI ? group : 0], flip);
            const float off = again ? sum[0] / width : 0.0f;    // (a product with 1 / D would leave a rounding)
            if (again) v = fmaxf(fmaf(-off, off, var), 0.0f) + eps;
            mu += off;
            const F2 less = both(-off);
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int i = 0; i < kHalf; ++i) f[k][i] = add2(f[k][i], less);
            if (SHIFT)
#pragma unroll
                for (int u = 0; u < kX; ++u) ec[u] -= off;
            if (!MULTI && row >= n) continue;
        }
        const float r = __frsqrt_rn(v);
        if (!kAgain && row >= n) continue;
        const F2 rr = both(r);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int v = c.lane + k * pl.lanes;
            if (v >= c.vecs) continue;
#pragma unroll
            for (int i = 0; i < kHalf; ++i) f[k][i] = fma2(mul2(f[k][i], rr), g[k][i], b[k][i]);
            store_row<T, VEC, SHIFT>(py, y.same, v, c, f[k]);
        }
        if (SHIFT)
#pragma unroll
            for (int u = 0; u < kX; ++u)
                if (col[u] >= 0) py[col[u]] = from_float<T>(fmaf(ec[u] * r, ge[u], be[u]));
        if (c.lane == 0) {
            if (mean) mean[row] = mu;
            if (rstd) rstd[row] = r;
        }
    }
}

// As the forward, with dy and x of a row in registers; the weights' sums stay
// in the threads' registers over all of a CTA's rows and leave one partial
// sum a CTA in `part` [CTAs][2][D] (none where part is NULL), or, where one
// CTA has all rows, the gradients themselves.  8191 x 4096 bfloat16 (201 MB):
// 42 us, 30 at copy bandwidth; two rows of 256 threads are all that the
// registers of an SM hold (x, dy and two sums a column, 127 a thread), and 16
// warps issue every other cycle.  (16-bit rows of 40 to 71 elements that start off
// 16-byte boundaries, with up to four elements a lane outside two vectors, spill
// 148 bytes.)  1M x 48 float32 (576 MB): 89 us (86).
// 76,363 x 48 (44 MB): 10.2 with the last launch, both bound by latency.
template <typename T, int VEC, int NV, bool MULTI, int X>
__global__ void __launch_bounds__(MULTI ? kMaxRowThreads : kThreads, MULTI ? 1 : (NV == 1 && X <= 1 ? 3 : 2))
    k_norm_bwd(Rows<const T> dy, Rows<const T> x, int64_t n, int32_t D, Place pl, const void *gamma, int pdt,
               const float *mean, const float *rstd, Rows<T> dx, float *part, void *dgamma, void *dbeta) {
    extern __shared__ uint4 s_ring[];    // [stages][dy | x][NV][threads], then gamma; at the end the sums
    __shared__ alignas(16) float s_red[MULTI ? kMaxGroups : 1][2][2][kRowWarps];
    constexpr bool SHIFT = X > 0;
    constexpr int kStages = stages_of(2 * NV), kHalf = VEC / 2, kX = SHIFT ? X : 1;
    const int group = MULTI ? threadIdx.x / pl.lanes : threadIdx.x >> pl.shift;
    const int lane = MULTI ? threadIdx.x - group * pl.lanes : threadIdx.x & (pl.lanes - 1);
    const int64_t step = int64_t(gridDim.x) * pl.groups;
    const int64_t row0 = int64_t(blockIdx.x) * pl.groups + group;
    const Cols c = cols_of<T, VEC, SHIFT>(x, row0, lane, pl, D);
    const int apart = blockDim.x;
    uint4 *slot = s_ring + threadIdx.x;
    // Row `row` of both tensors into a stage; a row past the last as zeros.
    auto fetch = [&](int stage, int64_t row) {
        uint4 *sd = slot + stage * 2 * NV * apart, *sx = sd + NV * apart;
        if (row < n) {
            fetch_row<T, VEC, NV, SHIFT>(sd, apart, dy.base + row * dy.stride, dy.same, c);
            fetch_row<T, VEC, NV, SHIFT>(sx, apart, x.base + row * x.stride, true, c);
        } else {
#pragma unroll
            for (int k = 0; k < 2 * NV; ++k) sd[k * apart] = make_uint4(0, 0, 0, 0);
        }
        copies_commit();
    };
#pragma unroll
    for (int q = 0; q < kStages - 1; ++q) fetch(q, row0 + q * step);
    // what a row needs beside its vectors, a row ahead
    float mu, r, ed[kX], ex[kX], ge[kX], dge[kX], dbe[kX];
    int col[kX];
#pragma unroll
    for (int u = 0; u < kX; ++u) {
        col[u] = SHIFT ? c.extra(u) : -1;
        ge[u] = SHIFT ? weight_of(gamma, pdt, 1.0f, col[u]) : 1.0f;
        dge[u] = dbe[u] = 0.0f;
    }
    auto load = [&](int64_t row) {
        const bool here = row < n;
        mu = here ? mean[row] : 0.0f, r = here ? rstd[row] : 0.0f;
        if (SHIFT)
#pragma unroll
            for (int u = 0; u < kX; ++u) {
                ed[u] = here && col[u] >= 0 ? to_float(dy.base[row * dy.stride + col[u]]) : 0.0f;
                ex[u] = here && col[u] >= 0 ? to_float(x.base[row * x.stride + col[u]]) : 0.0f;
            }
    };
    load(row0);
    float4 *plane = reinterpret_cast<float4 *>(s_ring + kStages * 2 * NV * apart) + threadIdx.x;
    {
        F2 g[NV][kHalf];
        load_weights<VEC, NV, SHIFT>(g, gamma, pdt, 1.0f, c);
        put_weights<VEC, NV>(plane, apart, g);
    }
    if (MULTI) clear_sums<2>(&s_red[0][0][0][0], kMaxGroups);
    __syncthreads();
    const float inv = 1.0f / float(D);
    F2 dg[NV][kHalf], db[NV][kHalf];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < kHalf; ++i) dg[k][i] = db[k][i] = both(0.0f);
    int flip = 0, stage = 0;
    T *pdx = dx.base + row0 * dx.stride;
    const int64_t dxstep = step * dx.stride;
    const int64_t lead = MULTI ? row0 : row0 - ((threadIdx.x & 31) >> pl.shift);
    for (int64_t base = lead; base < n; base += step, pdx += dxstep) {
        const int64_t row = base + (row0 - lead);
        copies_wait<kStages - 2>();
        F2 a[NV][kHalf], h[NV][kHalf], s0 = both(0.0f), s1 = both(0.0f);
        const F2 neg = both(-mu), rr = both(r);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (c.lane + k * pl.lanes < c.vecs) {
                F2 g[kHalf];
                widen<T, VEC>(a[k], from_slot<T, VEC>(slot + (stage * 2 * NV + k) * apart));
                widen<T, VEC>(h[k], from_slot<T, VEC>(slot + ((stage * 2 + 1) * NV + k) * apart));
                weights_of<VEC>(g, plane, apart, k);
#pragma unroll
                for (int i = 0; i < kHalf; ++i) h[k][i] = mul2(add2(h[k][i], neg), rr);
#pragma unroll
                for (int i = 0; i < kHalf; ++i) {
                    dg[k][i] = fma2(a[k][i], h[k][i], dg[k][i]);
                    db[k][i] = add2(db[k][i], a[k][i]);
                    a[k][i] = mul2(a[k][i], g[i]);
                    s0 = add2(s0, a[k][i]);
                    s1 = fma2(a[k][i], h[k][i], s1);
                }
            }
        }
        float sum[2] = {sum_of(s0), sum_of(s1)}, ae[kX], he[kX];
        const float r0 = r;
        if (SHIFT)
#pragma unroll
            for (int u = 0; u < kX; ++u) {
                he[u] = col[u] >= 0 ? (ex[u] - mu) * r : 0.0f;
                dge[u] = fmaf(ed[u], he[u], dge[u]), dbe[u] += ed[u];
                ae[u] = ed[u] * ge[u];
                sum[0] += ae[u], sum[1] = fmaf(ae[u], he[u], sum[1]);
            }
        load(row + step);
        fetch(stage == 0 ? kStages - 1 : stage - 1, row + (kStages - 1) * step);   // the slots read one row ago
        stage = stage == kStages - 1 ? 0 : stage + 1;
        row_sum<2, MULTI>(sum, pl.lanes, group, c.lane, s_red[MULTI ? group : 0], flip);
        if (row >= n) continue;
        const F2 ma = both(-sum[0] * inv), mah = both(-sum[1] * inv);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int v = c.lane + k * pl.lanes;
            if (v >= c.vecs) continue;
#pragma unroll
            for (int i = 0; i < kHalf; ++i) a[k][i] = mul2(fma2(h[k][i], mah, add2(a[k][i], ma)), rr);
            store_row<T, VEC, SHIFT>(pdx, dx.same, v, c, a[k]);
        }
        if (SHIFT)
#pragma unroll
            for (int u = 0; u < kX; ++u)
                if (col[u] >= 0) pdx[col[u]] = from_float<T>(r0 * (ae[u] - sum[0] * inv - he[u] * (sum[1] * inv)));
    }
    start_dependents();
    if (!part) return;
    // The CTA's sum, in fixed order: the rows of a warp are joined by shuffles
    // first where they start alike (!MULTI, !SHIFT), then the warps or groups
    // in turn, in the ring's place.
    part += size_t(blockIdx.x) * 2 * D;
    const bool fold = !MULTI && !SHIFT;
    const int slots = fold ? kThreads / 32 : pl.groups;
    const int mine_at = fold ? threadIdx.x >> 5 : group;
    copies_wait<0>();
    __syncthreads();                       // the last rows' slots and gamma have been read
    float *s_sum = reinterpret_cast<float *>(s_ring);
    const bool direct = MULTI && !SHIFT && slots == 1;   // whole vectors, straight to their place
    float *mine = direct ? part : s_sum + size_t(mine_at) * 2 * D;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int v = c.lane + k * pl.lanes;
        float tg[VEC], tb[VEC];
#pragma unroll
        for (int i = 0; i < VEC; i += 2) {
            tg[i] = dg[k][i / 2].x, tg[i + 1] = dg[k][i / 2].y;
            tb[i] = db[k][i / 2].x, tb[i + 1] = db[k][i / 2].y;
        }
        if (fold)
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                for (int o = pl.lanes; o < 32; o <<= 1) {
                    tg[i] += __shfl_xor_sync(0xffffffffu, tg[i], o);
                    tb[i] += __shfl_xor_sync(0xffffffffu, tb[i], o);
                }
        if (fold && (threadIdx.x & 31) >= pl.lanes) continue;
        if (!SHIFT) {
            if (v < c.vecs) {
                store_floats<float, VEC>(mine + v * VEC, tg);
                store_floats<float, VEC>(mine + D + v * VEC, tb);
            }
        } else if (v < c.vecs) {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                mine[c.head + v * VEC + i] = tg[i], mine[D + c.head + v * VEC + i] = tb[i];
        }
    }
    if (SHIFT)
#pragma unroll
        for (int u = 0; u < kX; ++u)
            if (col[u] >= 0) mine[col[u]] = dge[u], mine[D + col[u]] = dbe[u];
    __syncthreads();
    if (direct && !dgamma) return;
    for (int j = threadIdx.x; j < 2 * D; j += blockDim.x) {
        float t = direct ? part[j] : 0.0f;
        if (!direct)
            for (int w = 0; w < slots; ++w) t += s_sum[size_t(w) * 2 * D + j];
        if (dgamma)
            store_param(j < D ? dgamma : dbeta, pdt, j < D ? j : j - D, t);
        else
            part[j] = t;
    }
}

// The CTAs' partial sums of 32 columns of [dgamma | dbeta].  Its launch begins while
// k_norm_bwd ends; bound by latency.
__global__ void __launch_bounds__(1024) k_norm_bwd_final(const float *part, int parts, int32_t D, void *dgamma,
                                                         void *dbeta, int pdt) {
    add_up_parts(part, parts, D, 2 * D, dgamma, dbeta, pdt);
}

// ------------------------------------------------------------------ rows wider than the registers

// A CTA a row, which is read three times (the second and third from L1 or L2),
// an element a thread: rows past too_wide() have work enough for
// their latency (2000 x 16,384 bfloat16: 70 us, 19 at copy bandwidth).  FAR: a row whose mean is far_off, as in k_norm_fwd.
template <typename T>
struct WideRow {
    const T *x;
    T *y;
    int32_t D;
    const void *gamma, *beta;
    int pdt;
    float eps, mu, off, v, r;      // v = var + eps
    template <bool FAR>
    __device__ __forceinline__ float centred(int j) const {
        const float c = to_float(x[j]) - mu;
        return FAR ? c - off : c;
    }
    template <bool FAR>
    __device__ __forceinline__ void statistics(float *s_red) {
        float s = 0.0f;
        for (int j = threadIdx.x; j < D; j += kThreads) {
            const float c = centred<FAR>(j);
            s += c * c;
        }
        v = block_sum(s, s_red) / float(D) + eps;
        r = __frsqrt_rn(v);
    }
    template <bool FAR>
    __device__ __forceinline__ void result() const {
        for (int j = threadIdx.x; j < D; j += kThreads) {
            const float g = gamma ? load_param(gamma, pdt, j) : 1.0f;
            const float b = beta ? load_param(beta, pdt, j) : 0.0f;
            y[j] = from_float<T>(centred<FAR>(j) * r * g + b);
        }
    }
};
template <typename T>
__device__ __noinline__ float2 far_row(WideRow<T> w, float *s_red) {   // its (mean, rstd)
    float s = 0.0f;
    for (int j = threadIdx.x; j < w.D; j += kThreads) s += w.template centred<false>(j);
    w.off = block_sum(s, s_red) / float(w.D);
    w.template statistics<true>(s_red);
    w.template result<true>();
    return make_float2(w.mu + w.off, w.r);
}
template <typename T>
__global__ void __launch_bounds__(kThreads, 8) k_norm_fwd_wide(const T *x, int64_t xs, int64_t n, int32_t D,
                                                       const void *gamma, const void *beta, int pdt, float eps, T *y,
                                                       int64_t ys, float *mean, float *rstd) {
    __shared__ float s_red[kThreads / 32];
    for (int64_t row = blockIdx.x; row < n; row += gridDim.x) {
        WideRow<T> w{x + row * xs, y + row * ys, D, gamma, beta, pdt, eps, 0.0f, 0.0f, 0.0f, 0.0f};
        float s = 0.0f;
        for (int j = threadIdx.x; j < D; j += kThreads) s += to_float(w.x[j]);
        w.mu = block_sum(s, s_red) / float(D);
        w.template statistics<false>(s_red);
        float2 m = make_float2(w.mu, w.r);
        if (far_off(w.mu, w.v))           // the same in every thread
            m = far_row(w, s_red);
        else
            w.template result<false>();
        if (threadIdx.x == 0) {
            if (mean) mean[row] = m.x;
            if (rstd) rstd[row] = m.y;
        }
    }
}

// The weights' partial sums: thread = column, CTA y = a slice of the rows.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_norm_bwd_weights_wide(const T *__restrict__ dy, int64_t dys,
                                                               const T *__restrict__ x, int64_t xs, int64_t n,
                                                               int32_t D, const float *mean, const float *rstd,
                                                               float *part) {
    const int j = blockIdx.x * kThreads + threadIdx.x;
    if (j >= D) return;
    float dg = 0.0f, db = 0.0f;
    for (int64_t row = blockIdx.y; row < n; row += gridDim.y) {
        const float d = to_float(dy[row * dys + j]);
        dg = fmaf(d, (to_float(x[row * xs + j]) - mean[row]) * rstd[row], dg);
        db += d;
    }
    part[size_t(blockIdx.y) * 2 * D + j] = dg;
    part[size_t(blockIdx.y) * 2 * D + D + j] = db;
}

// A CTA a row, as in the forward.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_norm_bwd_rows_wide(const T *dy, int64_t dys, const T *x, int64_t xs,
                                                            int64_t n, int32_t D, const void *gamma, int pdt,
                                                            const float *mean, const float *rstd, T *dx,
                                                            int64_t dxs) {
    __shared__ float s_red[kThreads / 32];
    for (int64_t row = blockIdx.x; row < n; row += gridDim.x) {
        const float mu = mean[row], r = rstd[row];
        float sa = 0.0f, sah = 0.0f;
        for (int j = threadIdx.x; j < D; j += kThreads) {
            const float a = to_float(dy[row * dys + j]) * (gamma ? load_param(gamma, pdt, j) : 1.0f);
            sa += a;
            sah = fmaf(a, (to_float(x[row * xs + j]) - mu) * r, sah);
        }
        const float ma = block_sum(sa, s_red) / float(D);
        const float mah = block_sum(sah, s_red) / float(D);
        for (int j = threadIdx.x; j < D; j += kThreads) {
            const float a = to_float(dy[row * dys + j]) * (gamma ? load_param(gamma, pdt, j) : 1.0f);
            const float h = (to_float(x[row * xs + j]) - mu) * r;
            dx[row * dxs + j] = from_float<T>(r * (a - ma - h * mah));
        }
    }
}

int pow2_at_least(int v) {
    int p = 1;
    while (p < v) p <<= 1;
    return p;
}

// Lanes of a row of D elements in vectors of `vec`: a power of two up to a
// warp while 16 elements a thread hold the row, else whole warps.  At least 4
// lanes, so that a load touches whole sectors.
// Several wide rows share a CTA of about `threads`.
Place place_of(int32_t D, int vec, int threads, bool *multi) {
    Place pl{};
    pl.vecs = D / vec;
    const int nv = kPerThread / vec;
    const int need = (pl.vecs + nv - 1) / nv;
    *multi = need > 32;
    if (*multi) {
        pl.lanes = (need + 31) / 32 * 32;
        pl.groups = pl.lanes < threads ? threads / pl.lanes : 1;
    } else {
        const int least = D < 4 ? pow2_at_least(D) : 4;
        pl.lanes = pow2_at_least(need);
        if (pl.lanes < least) pl.lanes = least;
        pl.groups = kThreads / pl.lanes;
    }
    while ((1 << pl.shift) < pl.lanes) ++pl.shift;
    return pl;
}

// Rows after which row starts repeat their distance from a 16-byte boundary.
int period_of(int64_t stride, int bytes) {
    const int r = int((stride * bytes) & 15);
    return r == 0 ? 1 : 16 / (r & -r);
}

template <typename Tag, typename K>
int grid_of(K kernel, int threads, size_t smem, int64_t n, int groups, int period, int waves, int most, int sms) {
    static std::atomic<unsigned long long> known{0};
    return ss::grid_of(&known, kernel, threads, smem, n, groups, period, waves, most, sms);
}

bool sizes_ok(int64_t n, int32_t D) { return n >= 0 && n < (int64_t(1) << 31) && D >= 1 && D <= kMaxD; }

ss_status check_rows(const char *who, const char *what, const void *p, int64_t stride, int32_t D, int dtype) {
    if (!p) return fail(SS_ERR_INVALID_ARG, "%s: %s is NULL", who, what);
    if (!aligned_to(p, dtype_bytes(dtype)))
        return fail(SS_ERR_INVALID_ARG, "%s: %s is not aligned to its type", who, what);
    if (stride < D || stride > (int64_t(1) << 31))
        return fail(SS_ERR_INVALID_ARG, "%s: %s stride %lld below D or above 2^31", who, what, (long long)stride);
    return SS_OK;
}

ss_status check_param(const char *who, const char *what, const void *p, int dtype) {
    if (p && !aligned_to(p, dtype_bytes(dtype)))
        return fail(SS_ERR_INVALID_ARG, "%s: %s is not aligned to its type", who, what);
    return SS_OK;
}

ss_status check_common(const char *who, int64_t n, int32_t D, int dtype, int pdt) {
    if (!sizes_ok(n, D))
        return fail(SS_ERR_UNSUPPORTED, "%s: %lld rows of %d outside 0..2^31-1 x 1..%d", who, (long long)n, D, kMaxD);
    if (!dtype_known(dtype)) return fail(SS_ERR_INVALID_ARG, "%s: unknown dtype %d", who, dtype);
    if (pdt != SS_F32 && pdt != dtype)
        return fail(SS_ERR_INVALID_ARG, "%s: param_dtype %d is neither SS_F32 nor the rows' type", who, pdt);
    return SS_OK;
}

struct FwdArgs {
    const void *x;
    int64_t xs, n;
    int32_t D;
    const void *gamma, *beta;
    int pdt;
    float eps;
    void *y;
    int64_t ys;
    float *mean, *rstd;
};

struct BwdArgs {
    const void *dy;
    int64_t dys;
    const void *x;
    int64_t xs, n;
    int32_t D;
    const void *gamma;
    int pdt;
    const float *mean, *rstd;
    void *dx;
    int64_t dxs;
    void *dgamma, *dbeta;
    float *part;
};

template <typename T>
bool same_start(const void *a, int64_t as, const void *b, int64_t bs) {
    return ((reinterpret_cast<uintptr_t>(a) ^ reinterpret_cast<uintptr_t>(b)) & 15) == 0 &&
           (((as - bs) * int64_t(sizeof(T))) & 15) == 0;
}

constexpr int kMaxSmem = 225 * 1024;   // 227 KB less 2 KB of static buffers

template <typename T, int VEC, int NV, bool MULTI, int X>
struct FwdTag {};
template <typename T, int VEC, int NV, bool MULTI, int X>
struct BwdTag {};

template <typename T, int VEC, int NV, bool MULTI, int X>
ss_status fwd_kernel(const FwdArgs &a, const Place &pl, int sms, cudaStream_t s) {
    const int threads = MULTI ? pl.lanes * pl.groups : kThreads;
    const size_t smem = size_t(stages_of(NV)) * NV * threads * 16;
    auto kernel = k_norm_fwd<T, VEC, NV, MULTI, X>;
    static std::atomic<unsigned long long> smem_ctx[kMaxDevices];   // see ensure_dyn_smem
    const void *fn = (const void *)kernel;
    const ss_status st = ensure_dyn_smem(smem_ctx, &fn, 1, kMaxSmem, "ss_layer_norm_fwd");
    if (st != SS_OK) return st;
    const int grid = grid_of<FwdTag<T, VEC, NV, MULTI, X>>(kernel, threads, smem, a.n, pl.groups,
                                                               period_of(a.xs, sizeof(T)), MULTI ? 1 : 8, 1 << 30, sms);
    const Rows<const T> x{static_cast<const T *>(a.x), a.xs, true};
    const Rows<T> y{static_cast<T *>(a.y), a.ys, same_start<T>(a.x, a.xs, a.y, a.ys)};
    SS_LAUNCH("k_norm_fwd", s,
              kernel<<<grid, threads, smem, s>>>(x, a.n, a.D, pl, a.gamma, a.beta, a.pdt, a.eps, y, a.mean, a.rstd));
    return SS_OK;
}

template <typename T, int VEC, int NV, bool MULTI, int X>
ss_status bwd_kernel(const BwdArgs &a, const Place &pl, int sms, cudaStream_t s) {
    const int threads = MULTI ? pl.lanes * pl.groups : kThreads;
    size_t smem = size_t(stages_of(2 * NV)) * 2 * NV * threads * 16 +
                  size_t(NV) * VEC * threads * sizeof(float);   // the ring and gamma
    constexpr bool SHIFT = X > 0;
    const int slots = MULTI || SHIFT ? pl.groups : kThreads / 32;
    const size_t sums = a.dgamma && !(MULTI && !SHIFT && slots == 1) ? size_t(slots) * 2 * a.D * sizeof(float) : 0;
    if (smem < sums) smem = sums;
    auto kernel = k_norm_bwd<T, VEC, NV, MULTI, X>;
    static std::atomic<unsigned long long> smem_ctx[kMaxDevices];
    const void *fn = (const void *)kernel;
    const ss_status st = ensure_dyn_smem(smem_ctx, &fn, 1, kMaxSmem, "ss_layer_norm_bwd");
    if (st != SS_OK) return st;
    // what one CTA takes at once needs no launch that adds up several CTAs' sums (four turns of one
    // CTA take longer than that launch: 4 x 8192, 16 us against 8)
    const bool alone = a.n <= pl.groups;
    const int grid = alone ? 1
                           : grid_of<BwdTag<T, VEC, NV, MULTI, X>>(kernel, threads, smem, a.n, pl.groups,
                                                                       period_of(a.xs, sizeof(T)), 1,
                                                                       kMaxParts - kMaxPeriod, sms);
    const Rows<const T> x{static_cast<const T *>(a.x), a.xs, true};
    const Rows<const T> dy{static_cast<const T *>(a.dy), a.dys, same_start<T>(a.x, a.xs, a.dy, a.dys)};
    const Rows<T> dx{static_cast<T *>(a.dx), a.dxs, same_start<T>(a.x, a.xs, a.dx, a.dxs)};
    SS_LAUNCH("k_norm_bwd", s,
              kernel<<<grid, threads, smem, s>>>(dy, x, a.n, a.D, pl, a.gamma, a.pdt, a.mean, a.rstd, dx,
                                                 a.dgamma ? a.part : nullptr, alone ? a.dgamma : nullptr,
                                                 alone ? a.dbeta : nullptr));
    if (a.dgamma && !alone)
        SS_LAUNCH("k_norm_bwd_final", s,
                  launch_after(k_norm_bwd_final, dim3((2 * a.D + 31) / 32), 1024, 0, s, a.part, grid, a.D, a.dgamma,
                               a.dbeta, a.pdt));
    return SS_OK;
}

// Picks the vectors a thread holds: all of them for wide rows, just enough
// for narrow ones.
template <typename T, bool SHIFT, typename Args>
ss_status pick_nv(const Args &a, int sms, cudaStream_t s) {
    constexpr int kVec = 16 / sizeof(T), kNv = kPerThread / kVec;
    bool multi;
    const Place pl = place_of(a.D, kVec, std::is_same<Args, FwdArgs>::value ? kThreads : kMaxRowThreads, &multi);
    const int nv = (pl.vecs + pl.lanes - 1) / pl.lanes;
    // elements outside the vectors, at most, and how many of them fall to a lane
    const int others = a.D < 2 * kVec - 2 ? a.D : 2 * kVec - 2, x = (others + pl.lanes - 1) / pl.lanes;
    auto go = [&](auto NV, auto MULTI, auto X) {
        if constexpr (std::is_same<Args, FwdArgs>::value)
            return fwd_kernel<T, kVec, decltype(NV)::value, decltype(MULTI)::value, decltype(X)::value>(a, pl, sms, s);
        else
            return bwd_kernel<T, kVec, decltype(NV)::value, decltype(MULTI)::value, decltype(X)::value>(a, pl, sms, s);
    };
    auto narrow = [&](auto NV) {
        if constexpr (!SHIFT) {
            return go(NV, std::false_type{}, std::integral_constant<int, 0>{});
        } else {
            if (x <= 1) return go(NV, std::false_type{}, std::integral_constant<int, 1>{});
            if constexpr (kVec == 8) {      // 14 on 4 lanes
                if (x > 2) return go(NV, std::false_type{}, std::integral_constant<int, 4>{});
            }
            return go(NV, std::false_type{}, std::integral_constant<int, 2>{});
        }
    };
    if (multi) return go(std::integral_constant<int, kNv>{}, std::true_type{}, std::integral_constant<int, SHIFT ? 1 : 0>{});
    if (nv <= 1) return narrow(std::integral_constant<int, 1>{});
    if constexpr (kNv == 4) {
        if (nv == 3) return narrow(std::integral_constant<int, 3>{});
        if (nv == 4) return narrow(std::integral_constant<int, 4>{});
    }
    return narrow(std::integral_constant<int, 2>{});
}

// Wider than 512 threads hold, whatever the row's start: from 8196 elements on in
// float32, from 8200 in 16 bits.
template <typename T>
bool too_wide(int32_t D) {
    constexpr int kVec = 16 / sizeof(T);
    return D / kVec > kMaxRowThreads * (kPerThread / kVec);
}

template <typename T>
ss_status launch_fwd(const FwdArgs &a, int sms, cudaStream_t s) {
    constexpr int kVec = 16 / sizeof(T);
    const bool shift = !(a.D % kVec == 0 && aligned_to(a.x, 16) && aligned_to(a.y, 16) && a.xs % kVec == 0 &&
                         a.ys % kVec == 0);
    if (!too_wide<T>(a.D)) return shift ? pick_nv<T, true>(a, sms, s) : pick_nv<T, false>(a, sms, s);
    SS_LAUNCH("k_norm_fwd_wide", s,
              k_norm_fwd_wide<T><<<wide_grid(a.n, sms), kThreads, 0, s>>>(
                  static_cast<const T *>(a.x), a.xs, a.n, a.D, a.gamma, a.beta, a.pdt, a.eps, static_cast<T *>(a.y),
                  a.ys, a.mean, a.rstd));
    return SS_OK;
}

template <typename T>
ss_status launch_bwd(const BwdArgs &a, int sms, cudaStream_t s) {
    constexpr int kVec = 16 / sizeof(T);
    const bool shift = !(a.D % kVec == 0 && aligned_to(a.dy, 16) && aligned_to(a.x, 16) && aligned_to(a.dx, 16) &&
                         a.dys % kVec == 0 && a.xs % kVec == 0 && a.dxs % kVec == 0);
    if (a.n > 0 && !too_wide<T>(a.D)) return shift ? pick_nv<T, true>(a, sms, s) : pick_nv<T, false>(a, sms, s);
    // the weights first: dx may overwrite dy or x
    if (a.dgamma) {
        const dim3 g((a.D + kThreads - 1) / kThreads, unsigned(a.n < 64 ? (a.n < 1 ? 1 : a.n) : 64));
        SS_LAUNCH("k_norm_bwd_weights_wide", s,
                  k_norm_bwd_weights_wide<T><<<g, kThreads, 0, s>>>(static_cast<const T *>(a.dy), a.dys,
                                                                    static_cast<const T *>(a.x), a.xs, a.n, a.D,
                                                                    a.mean, a.rstd, a.part));
        SS_LAUNCH("k_norm_bwd_final", s,
                  launch_after(k_norm_bwd_final, dim3((2 * a.D + 31) / 32), 1024, 0, s, a.part, int(g.y), a.D,
                               a.dgamma, a.dbeta, a.pdt));
    }
    if (a.n == 0) return SS_OK;
    SS_LAUNCH("k_norm_bwd_rows_wide", s,
              k_norm_bwd_rows_wide<T><<<wide_grid(a.n, sms), kThreads, 0, s>>>(
                  static_cast<const T *>(a.dy), a.dys, static_cast<const T *>(a.x), a.xs, a.n, a.D, a.gamma, a.pdt,
                  a.mean, a.rstd, static_cast<T *>(a.dx), a.dxs));
    return SS_OK;
}

}  // namespace
}  // namespace ss

using namespace ss;

extern "C" {

ss_status ss_layer_norm_fwd(const void *x, ss_dtype dtype, int64_t x_stride, int64_t n, int32_t D, const void *gamma,
                            const void *beta, ss_dtype param_dtype, float eps, void *y, int64_t y_stride, float *mean,
                            float *rstd, ss_stream_t stream) {
    clear_error();
    const char *who = "ss_layer_norm_fwd";
    ss_status st = check_common(who, n, D, dtype, param_dtype);
    if (st != SS_OK) return st;
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(SS_ERR_INVALID_ARG, "%s: eps negative or not finite", who);
    if (n == 0) return SS_OK;
    if ((st = check_rows(who, "x", x, x_stride, D, dtype)) != SS_OK) return st;
    if ((st = check_rows(who, "y", y, y_stride, D, dtype)) != SS_OK) return st;
    if ((st = check_param(who, "gamma", gamma, param_dtype)) != SS_OK) return st;
    if ((st = check_param(who, "beta", beta, param_dtype)) != SS_OK) return st;
    if ((st = check_param(who, "mean", mean, SS_F32)) != SS_OK) return st;
    if ((st = check_param(who, "rstd", rstd, SS_F32)) != SS_OK) return st;
    int dev = 0, sms = 0;
    if ((st = current_device(&dev, &sms, "ss_layer_norm_fwd: device query")) != SS_OK) return st;
    cudaStream_t s = (cudaStream_t)stream;
    const FwdArgs a{x, x_stride, n, D, gamma, beta, int(param_dtype), eps, y, y_stride, mean, rstd};
    if (dtype == SS_F32)
        st = launch_fwd<float>(a, sms, s);
    else if (dtype == SS_F16)
        st = launch_fwd<__half>(a, sms, s);
    else
        st = launch_fwd<__nv_bfloat16>(a, sms, s);
    if (st != SS_OK) return st;
    return check_launch(who);
}

size_t ss_layer_norm_workspace_bytes(int64_t n, int32_t D) {
    if (!sizes_ok(n, D)) return 0;
    return size_t(weight_parts(n)) * 2 * D * sizeof(float);
}

ss_status ss_layer_norm_bwd(const void *dy, int64_t dy_stride, const void *x, int64_t x_stride, ss_dtype dtype,
                            int64_t n, int32_t D, const void *gamma, ss_dtype param_dtype, const float *mean,
                            const float *rstd, void *dx, int64_t dx_stride, void *dgamma, void *dbeta,
                            void *workspace, size_t workspace_bytes, ss_stream_t stream) {
    clear_error();
    const char *who = "ss_layer_norm_bwd";
    ss_status st = check_common(who, n, D, dtype, param_dtype);
    if (st != SS_OK) return st;
    if (n > 0) {
        if ((st = check_rows(who, "dy", dy, dy_stride, D, dtype)) != SS_OK) return st;
        if ((st = check_rows(who, "x", x, x_stride, D, dtype)) != SS_OK) return st;
        if ((st = check_rows(who, "dx", dx, dx_stride, D, dtype)) != SS_OK) return st;
        if (!mean || !rstd) return fail(SS_ERR_INVALID_ARG, "%s: mean or rstd is NULL", who);
        if ((st = check_param(who, "mean", mean, SS_F32)) != SS_OK) return st;
        if ((st = check_param(who, "rstd", rstd, SS_F32)) != SS_OK) return st;
        if ((st = check_param(who, "gamma", gamma, param_dtype)) != SS_OK) return st;
    }
    if ((dgamma == nullptr) != (dbeta == nullptr))
        return fail(SS_ERR_INVALID_ARG, "%s: one of dgamma and dbeta is NULL", who);
    if ((st = check_param(who, "dgamma", dgamma, param_dtype)) != SS_OK) return st;
    if ((st = check_param(who, "dbeta", dbeta, param_dtype)) != SS_OK) return st;
    if (dgamma) {
        if (!workspace || !aligned_to(workspace, 256))
            return fail(SS_ERR_INVALID_ARG, "%s: workspace NULL or not 256-byte aligned", who);
        const size_t need = ss_layer_norm_workspace_bytes(n, D);
        if (workspace_bytes < need)
            return fail(SS_ERR_INVALID_ARG, "%s: workspace %zu bytes < %zu", who, workspace_bytes, need);
    }
    int dev = 0, sms = 0;
    if ((st = current_device(&dev, &sms, "ss_layer_norm_bwd: device query")) != SS_OK) return st;
    cudaStream_t s = (cudaStream_t)stream;
    const BwdArgs a{dy, dy_stride, x, x_stride, n, D, gamma, int(param_dtype), mean, rstd, dx, dx_stride, dgamma,
                    dbeta, static_cast<float *>(workspace)};
    if (dtype == SS_F32)
        st = launch_bwd<float>(a, sms, s);
    else if (dtype == SS_F16)
        st = launch_bwd<__half>(a, sms, s);
    else
        st = launch_bwd<__nv_bfloat16>(a, sms, s);
    if (st != SS_OK) return st;
    return check_launch(who);
}

}  // extern "C"
