// The norm of all gradients and their scaling by it (model: include/ss_clip.h).
//
// Bound by memory: every gradient has to be read for the norm and again to be
// scaled, and the scaled values written.  A sweep over the tensors' tiles,
// from the first to the last, adds squares; a second goes back from the last
// tile to the first, so that what the first read last is still in L2 (129 MB):
// tiles that it will not find there, and all that the second reads and writes,
// are marked to leave L2 first.  A few small tensors take one launch and never
// leave the registers of one cluster.  The list of tensors travels in the
// launches' parameters: nothing is copied to the device, and a captured graph
// keeps its own list.
//
// The five gradients of 2M splats, 472 MB: 204 us, of which 139 are one read and
// one write at copy bandwidth and 209 would be two reads from DRAM; the second
// sweep finds 65 MB in L2.  Three launches, each begun while the one before it
// ends, rather than one that waits on its whole grid: that one took 225 us (the
// tiles' registers spilled beside both sweeps).  300 tensors of mixed types, 115
// MB: 52 us (34; 51); the second sweep finds 60 MB, and both run at 4.8 TB/s of
// DRAM traffic, the first with 61 % of its issue slots (16-bit values widened,
// tiles that end inside).
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "ss_clip.h"
#include "ss_internal.h"
#include "ss_launch.cuh"
#include "ss_profile.h"
#include "ss_vec.cuh"

namespace ss {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 4;                          // 16-byte vectors of a tile in one thread
constexpr int kTile = kThreads * kPer * 16;      // bytes
constexpr int kMaxGrid = 2048;                   // partial sums of one launch
constexpr int kSmallList = 24, kLongList = 1000; // tensors in one launch's parameters
constexpr int32_t kMaxTensors = 65536;
// What of the first sweep's bytes the second is let find in L2: a part of its
// 129 MB, so that lines of the two memories' halves do not crowd one another out.
constexpr int64_t kKeep = 80 << 20;

template <int CAP>
struct Table {
    const void *in[CAP];
    void *out[CAP];
    int64_t numel[CAP];
    int32_t first[CAP + 1];      // first tile of each tensor
    uint8_t dtype[CAP];
    int32_t count, keep;         // tensors; tiles from `keep` on stay in L2
};

// The tensor of a tile (tensors without elements have no tile).
template <int CAP>
__device__ __forceinline__ int tensor_of(const Table<CAP> &t, int tile) {
    int a = 0, b = t.count;
    while (b - a > 1) {
        const int m = (a + b) >> 1;
        if (t.first[m] <= tile) a = m; else b = m;
    }
    return a;
}

template <typename T>
using Vector = Vec<T, 16 / int(sizeof(T))>;

template <typename T>
__device__ __forceinline__ float squares_of(const Vector<T> &x) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 16 / int(sizeof(T)); ++i) s = fmaf(x.get(i), x.get(i), s);
    return s;
}

template <typename T>
__device__ __forceinline__ float squares_of(const Vector<T> &x, float by) {   // of the values times `by`
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 16 / int(sizeof(T)); ++i) s = fmaf(x.get(i) * by, x.get(i) * by, s);
    return s;
}

// Whether there is a value other than 0 in it.
template <typename T>
__device__ __forceinline__ bool any_of(const Vector<T> &x) {
    return ((x.w[0] | x.w[1] | x.w[2] | x.w[3]) & (sizeof(T) == 4 ? 0x7fffffffu : 0x7fff7fffu)) != 0u;
}

// c x, rounded to T; by 1 the bits as they are (a product would change a NaN's).
template <typename T>
__device__ __forceinline__ Vector<T> scaled(Vector<T> x, float c) {
    if (c == 1.0f) return x;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x.w[i] = __float_as_uint(x.get(i) * c);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = pack2<T>(x.get(2 * i) * c, x.get(2 * i + 1) * c);
#pragma unroll
        for (int i = 0; i < 4; ++i) x.w[i] = w[i];
    }
    return x;
}

// One tensor.  Its 16-byte vectors lie on 16-byte boundaries; the first and
// the last may hold elements that are not its own, and go one by one.
template <typename E>
struct Flat {
    using T = E;
    static constexpr int kVec = 16 / sizeof(T);
    const T *in;
    T *out;
    int64_t numel;

    template <int CAP>
    __device__ __forceinline__ Flat(const Table<CAP> &t, int k)
        : in(static_cast<const T *>(t.in[k])), out(static_cast<T *>(t.out[k])), numel(t.numel[k]) {}
    // Elements before the first 16-byte boundary.
    __device__ __forceinline__ int head() const {
        const int h = int((16 - (reinterpret_cast<uintptr_t>(in) & 15)) & 15) / int(sizeof(T));
        return h < numel ? h : int(numel);
    }
    // The i-th of the elements before and after the body (past numel: none).
    __device__ __forceinline__ int64_t lone(int h, int64_t body, int i) const { return i < h ? i : i + body * kVec; }
    // Element at which vector v starts, counting from the boundary before the
    // tensor (negative: before the tensor).
    __device__ __forceinline__ int64_t start(int64_t v) const {
        return v * kVec - int((reinterpret_cast<uintptr_t>(in) & 15) / sizeof(T));
    }
    __device__ __forceinline__ bool whole(int64_t e) const { return e >= 0 && e + kVec <= numel; }
    __device__ __forceinline__ bool alike() const {
        return ((reinterpret_cast<uintptr_t>(in) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
    }
    // The vector at element e, zeros in the place of what is not the tensor's.
    __device__ __forceinline__ Vector<T> load(int64_t e) const {
        if (whole(e)) return load_vec<T, kVec>(in + e);
        Vector<T> x;
        x.clear();
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            if (e + i >= 0 && e + i < numel) x.set(i, in[e + i]);
        return x;
    }
    __device__ __forceinline__ void store(int64_t e, const Vector<T> &x) const {
        if (whole(e) && alike()) {
            *reinterpret_cast<uint4 *>(out + e) = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
        } else {
#pragma unroll
            for (int i = 0; i < kVec; ++i)
                if (e + i >= 0 && e + i < numel) out[e + i] = x.elem(i);
        }
    }
};

// A tensor's body, from its first 16-byte boundary on, is cut into tiles of
// vectors, kPer a thread and all in flight; the few elements before and after
// the body go with its first tile, one a thread.  lost: set where values other
// than 0 have squares that add up to 0.
template <int CAP, typename T>
__device__ __forceinline__ float tile_squares(const Table<CAP> &t, int k, int tile, bool *lost) {
    const Flat<T> a(t, k);
    constexpr int kVec = Flat<T>::kVec;
    const int head = a.head();
    const int64_t body = (a.numel - head) / kVec, v0 = int64_t(tile - t.first[k]) * (kThreads * kPer) + threadIdx.x;
    const T *p = a.in + head + v0 * kVec;
    constexpr int kStep = kThreads * kVec;
    Vector<T> x[kPer];
    if (v0 - threadIdx.x + kThreads * kPer <= body) {
#pragma unroll
        for (int u = 0; u < kPer; ++u)
            x[u] = tile < t.keep ? load_vec_cs<T, kVec>(p + u * kStep) : load_vec<T, kVec>(p + u * kStep);
    } else {
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            x[u].clear();
            if (v0 + u * kThreads < body) x[u] = load_vec<T, kVec>(p + u * kStep);
        }
    }
    float sum = 0.0f;
    const int64_t lone = a.lone(head, body, threadIdx.x);
    if (tile == t.first[k] && lone < a.numel) {
        const float f = to_float(a.in[lone]);
        sum = f * f;
    }
#pragma unroll
    for (int u = 0; u < kPer; ++u) sum += squares_of<T>(x[u]);
    if (!std::is_same<T, __half>::value && sum == 0.0f) {
        bool any = tile == t.first[k] && lone < a.numel && to_float(a.in[lone]) != 0.0f;
#pragma unroll
        for (int u = 0; u < kPer; ++u) any = any || any_of<T>(x[u]);
        *lost = *lost || any;
    }
    return sum;
}

// The same of the values times `by`, a vector at a time: few sums need it, and
// the others are not to hold registers for it.
template <int CAP, typename T>
__device__ __forceinline__ float tile_squares(const Table<CAP> &t, int k, int tile, float by) {
    const Flat<T> a(t, k);
    constexpr int kVec = Flat<T>::kVec;
    const int head = a.head();
    const int64_t body = (a.numel - head) / kVec, v0 = int64_t(tile - t.first[k]) * (kThreads * kPer);
    const int64_t end = v0 + kThreads * kPer < body ? v0 + kThreads * kPer : body;
    const int64_t lone = a.lone(head, body, threadIdx.x);
    const float f = tile == t.first[k] && lone < a.numel ? to_float(a.in[lone]) * by : 0.0f;
    float sum = f * f;
#pragma unroll 1
    for (int64_t v = v0 + threadIdx.x; v < end; v += kThreads)
        sum += squares_of<T>(load_vec<T, kVec>(a.in + head + v * kVec), by);
    return sum;
}

template <int CAP, typename T>
__device__ __forceinline__ void tile_scale(const Table<CAP> &t, int k, int tile, float c) {
    const Flat<T> a(t, k);
    constexpr int kVec = Flat<T>::kVec;
    const int head = a.head();
    const int64_t body = (a.numel - head) / kVec, v0 = int64_t(tile - t.first[k]) * (kThreads * kPer) + threadIdx.x;
    const int64_t lone = a.lone(head, body, threadIdx.x);
    if (tile == t.first[k] && lone < a.numel)
        a.out[lone] = c == 1.0f ? a.in[lone] : from_float<T>(to_float(a.in[lone]) * c);
    const T *p = a.in + head + v0 * kVec;
    T *o = a.out + head + v0 * kVec;
    constexpr int kStep = kThreads * kVec;
    if (a.alike()) {
        Vector<T> x[kPer];
        if (v0 - threadIdx.x + kThreads * kPer <= body) {
#pragma unroll
            for (int u = 0; u < kPer; ++u) x[u] = load_vec_cs<T, kVec>(p + u * kStep);
#pragma unroll
            for (int u = 0; u < kPer; ++u) store_vec_cs<T, kVec>(o + u * kStep, scaled<T>(x[u], c));
        } else {
#pragma unroll
            for (int u = 0; u < kPer; ++u)
                if (v0 + u * kThreads < body) x[u] = load_vec<T, kVec>(p + u * kStep);
#pragma unroll
            for (int u = 0; u < kPer; ++u)
                if (v0 + u * kThreads < body) store_vec_cs<T, kVec>(o + u * kStep, scaled<T>(x[u], c));
        }
    } else {                             // the results lie otherwise: element by element
        const T *q = a.in + head;
        T *r = a.out + head;
        int64_t i = (v0 - threadIdx.x) * kVec + threadIdx.x, end = (v0 - threadIdx.x + kThreads * kPer) * kVec;
        if (end > body * kVec) end = body * kVec;
#pragma unroll 4
        for (; i < end; i += kThreads) r[i] = c == 1.0f ? q[i] : from_float<T>(to_float(q[i]) * c);
    }
}

// A sum of float32 values with the rounding errors of its additions beside
// it: about 46 bits, at float32's rate (float64 additions of every thread
// would take longer than a small list's memory traffic).  An infinity or a
// NaN stays in `hi`.
struct Sum {
    float hi, lo;
};
__device__ __forceinline__ Sum plus(Sum a, Sum b) {
    const float s = a.hi + b.hi, v = s - a.hi;
    return Sum{s, a.lo + b.lo + ((a.hi - (s - v)) + (b.hi - v))};
}
__device__ __forceinline__ Sum plus(Sum a, float b) { return plus(a, Sum{b, 0.0f}); }
__device__ __forceinline__ float value_of(Sum a) { return isfinite(a.hi) ? a.hi + a.lo : a.hi; }
template <int FROM>
__device__ __forceinline__ Sum warp_sum(Sum v) {
#pragma unroll
    for (int o = FROM; o > 0; o >>= 1)
        v = plus(v, Sum{__shfl_xor_sync(0xffffffffu, v.hi, o), __shfl_xor_sync(0xffffffffu, v.lo, o)});
    return v;
}

// Sum over the CTA, the same value in every thread (fixed order).
constexpr int kWarps = kThreads / 32;
template <int WARPS = kWarps>
__device__ __forceinline__ Sum block_sum(Sum v, Sum *s_red) {
    v = warp_sum<16>(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sum<WARPS / 2>(s_red[threadIdx.x & (WARPS - 1)]);
}

// This CTA's squares: plain float32 over a thread's vectors of a tile (at
// most 33 elements), with the errors from there on.  how: `lost` or `by`.
template <int CAP, typename How>
__device__ __forceinline__ Sum sweep_squares(const Table<CAP> &t, Sum *s_red, How how) {
    Sum sum{0.0f, 0.0f};
    const int tiles = t.first[t.count];
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int k = tensor_of(t, tile);
        if (t.dtype[k] == SS_F32)
            sum = plus(sum, tile_squares<CAP, float>(t, k, tile, how));
        else if (t.dtype[k] == SS_F16)
            sum = plus(sum, tile_squares<CAP, __half>(t, k, tile, how));
        else
            sum = plus(sum, tile_squares<CAP, __nv_bfloat16>(t, k, tile, how));
    }
    return block_sum(sum, s_red);
}

// Squares of float32 and bfloat16 values may leave float32's range where their
// root does not.  A CTA's sum from kLeast to kMost has lost nothing to underflow
// that its rounding does not (2^30 values lose 2^-119 at most), and those of all
// CTAs add up to no infinity; nor has one of zeros.  Any other is taken again, of
// the values times 2^96 or 2^-96: its kind is kLow or kHigh.
constexpr float kLeast = 0x1p-90f, kMost = 0x1p100f, kUp = 0x1p96f, kDown = 0x1p-96f;
enum Kind { kLow = -1, kMiddle = 0, kHigh = 1 };

// The root of all squares, of each kind; what is not of the largest scarcely counts.
__device__ __forceinline__ float root_of(Sum low, Sum middle, Sum high) {
    const float h = value_of(high), m = value_of(middle);
    if (h != 0.0f) return sqrtf(h + m * kDown * kDown) * kUp;
    if (m != 0.0f) return sqrtf(m + value_of(low) * kDown * kDown);
    return sqrtf(value_of(low)) * kDown;
}

// (norm, coefficient).
__device__ __forceinline__ float2 result_of(float norm, float max_norm, float eps, bool clip) {
    const float coef = !isfinite(norm) ? 0.0f : (clip ? fminf(1.0f, max_norm / (norm + eps)) : 1.0f);
    return make_float2(norm, coef);
}
// part: (hi, lo, kind) of each CTA.
__device__ __forceinline__ float root_of_parts(const float4 *part, int parts, Sum *s_red) {
    Sum low{0.0f, 0.0f}, middle = low, high = low;
    bool some = false;                   // of other kinds
    for (int i = threadIdx.x; i < parts; i += kThreads) {
        const float4 q = __ldcg(part + i);
        const bool here = q.z == kMiddle;
        middle = plus(middle, Sum{here ? q.x : 0.0f, here ? q.y : 0.0f});
        some = some || !here;
    }
    middle = block_sum(middle, s_red);
    if (__syncthreads_or(some)) {
        for (int i = threadIdx.x; i < parts; i += kThreads) {
            const float4 q = __ldcg(part + i);
            if (q.z == kLow) low = plus(low, Sum{q.x, q.y});
            if (q.z == kHigh) high = plus(high, Sum{q.x, q.y});
        }
        low = block_sum(low, s_red), high = block_sum(high, s_red);
    }
    return root_of(low, middle, high);
}

template <int CAP>
__device__ __forceinline__ void scale_tile(const Table<CAP> &t, int tile, float c) {
    const int k = tensor_of(t, tile);
    if (c == 1.0f && t.in[k] == t.out[k]) return;
    if (t.dtype[k] == SS_F32)
        tile_scale<CAP, float>(t, k, tile, c);
    else if (t.dtype[k] == SS_F16)
        tile_scale<CAP, __half>(t, k, tile, c);
    else
        tile_scale<CAP, __nv_bfloat16>(t, k, tile, c);
}

// Gradients of up to 256 KB: one cluster of CTAs holds them in
// registers between the norm and the scaling, so they are read once and the
// CTAs meet at the cluster's barrier, which costs a fraction of a grid's.
// Tiles here are 4 KB, a vector in each thread of a team, and all of a CTA's
// tiles are on their way at once (in teams of one, with eight tiles after one
// another, 236 KB took 7.8 us).  Bound by latency, a trip to memory and one
// over the CTAs' shared memories: 60 KB 3.7 us, 236 KB 5.1; the three launches
// of larger lists take 4.7, but a call of theirs from Python 7.7, and of this
// one 6.2.
constexpr int kCluster = 8, kTeams = 4, kHeld = 2;
constexpr int kMostHeld = kCluster * kTeams * kHeld;      // tiles
__global__ void __launch_bounds__(kTeams *kThreads) __cluster_dims__(kCluster, 1, 1)
    k_clip_small(const __grid_constant__ Table<kSmallList> t, float max_norm, float eps, float *result) {
    __shared__ Sum s_red[kTeams * kWarps], s_part[2][kCluster];
    namespace cg = cooperative_groups;
    const cg::cluster_group cluster = cg::this_cluster();
    const int tiles = t.first[t.count], rank = int(cluster.block_rank()), team = threadIdx.x / kThreads;
    auto all_here = cluster.barrier_arrive();       // waited for before a CTA writes into another
    uint4 held[kHeld];
    auto at = [&](int u, auto f) {       // f on this thread's vector of its team's u-th tile
        const int tile = (u * kTeams + team) * kCluster + rank;
        if (tile >= tiles) return;
        const int k = tensor_of(t, tile);
        const int64_t v = int64_t(tile - t.first[k]) * kThreads + threadIdx.x % kThreads;
        if (t.dtype[k] == SS_F32)
            f(Flat<float>(t, k), v);
        else if (t.dtype[k] == SS_F16)
            f(Flat<__half>(t, k), v);
        else
            f(Flat<__nv_bfloat16>(t, k), v);
    };
    auto vector_of = [&](auto a, int u) {
        Vector<typename decltype(a)::T> x;
        x.w[0] = held[u].x, x.w[1] = held[u].y, x.w[2] = held[u].z, x.w[3] = held[u].w;
        return x;
    };
#pragma unroll
    for (int u = 0; u < kHeld; ++u)
        at(u, [&](auto a, int64_t v) {
            const auto x = a.load(a.start(v));
            held[u] = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
        });
    Sum sum{0.0f, 0.0f};
#pragma unroll
    for (int u = 0; u < kHeld; ++u)
        at(u, [&](auto a, int64_t) { sum = plus(sum, squares_of<typename decltype(a)::T>(vector_of(a, u))); });
    cluster.barrier_wait(static_cast<decltype(all_here) &&>(all_here));
    auto over_cluster = [&](Sum v, Sum *s_to) {      // the same in every thread
        v = block_sum<kTeams * kWarps>(v, s_red);
        if (threadIdx.x < kCluster) *cluster.map_shared_rank(&s_to[rank], threadIdx.x) = v;
        cluster.sync();
        v = s_to[0];
#pragma unroll
        for (int q = 1; q < kCluster; ++q) v = plus(v, s_to[q]);
        return v;
    };
    sum = over_cluster(sum, s_part[0]);
    float norm = sqrtf(value_of(sum));
    if (!(value_of(sum) >= kLeast && value_of(sum) <= kMost)) {      // scaled, as in k_clip_squares
        const float by = norm < 1.0f ? kUp : kDown;
        sum = Sum{0.0f, 0.0f};
#pragma unroll
        for (int u = 0; u < kHeld; ++u)
            at(u, [&](auto a, int64_t) { sum = plus(sum, squares_of<typename decltype(a)::T>(vector_of(a, u), by)); });
        norm = sqrtf(value_of(over_cluster(sum, s_part[1]))) * (norm < 1.0f ? kDown : kUp);
    }
    const float2 r = result_of(norm, max_norm, eps, true);
    if (rank == 0 && threadIdx.x == 0) result[0] = r.x, result[1] = r.y;
    const float c = isfinite(r.x) ? r.y : 1.0f;      // nothing is scaled by a norm that is not finite
#pragma unroll
    for (int u = 0; u < kHeld; ++u)
        at(u, [&](auto a, int64_t v) {
            if (c == 1.0f && static_cast<const void *>(a.in) == a.out) return;
            a.store(a.start(v), scaled<typename decltype(a)::T>(vector_of(a, u), c));
        });
}

// CTAs that stay on the device and share the tiles out: 6.3 TB/s, the copy's
// bandwidth within a tenth (239 MB, 38 us).
template <int CAP>
__global__ void __launch_bounds__(kThreads, 8) k_clip_squares(const __grid_constant__ Table<CAP> t, float4 *part) {
    __shared__ Sum s_red[kWarps];
    start_dependents();
    bool lost = false;
    Sum sum = sweep_squares(t, s_red, &lost);
    int kind = kMiddle;
    const float v = value_of(sum);                   // the same in every thread
    if (!(v >= kLeast && v <= kMost) && (v != 0.0f || __syncthreads_or(lost))) {
        kind = v < kLeast ? kLow : kHigh;
        sum = sweep_squares(t, s_red, kind == kLow ? kUp : kDown);
    }
    if (threadIdx.x == 0) part[blockIdx.x] = make_float4(sum.hi, sum.lo, float(kind), 0.0f);
}

__global__ void __launch_bounds__(kThreads) k_clip_result(const float4 *part, int parts, float max_norm, float eps,
                                                          bool clip, float *result) {
    __shared__ Sum s_red[kWarps];
    start_dependents();
    wait_for_previous();
    const float2 r = result_of(root_of_parts(part, parts, s_red), max_norm, eps, clip);
    if (threadIdx.x == 0) result[0] = r.x, result[1] = r.y;
}

// A CTA for each tile, the last tiles first: the device hands them out as
// CTAs finish, which keeps the two memories' halves evenly busy (472 MB, both
// sweeps: 204 us; CTAs that stay and draw their tiles by a counter, 230).
template <int CAP>
__global__ void __launch_bounds__(kThreads, 4) k_clip_scale(const __grid_constant__ Table<CAP> t, const float *result) {
    wait_for_previous();
    const float norm = result[0], coef = result[1];
    scale_tile(t, t.first[t.count] - 1 - int(blockIdx.x), isfinite(norm) ? coef : 1.0f);
}

// ------------------------------------------------------------------ host

// Tiles of a tensor with elements, counting from the boundary before it: at
// least as many as its body takes.
int64_t tiles_of(const ss_tensor &t, int tile) {
    const int64_t bytes = t.numel * int64_t(dtype_bytes(t.dtype)) + int64_t(reinterpret_cast<uintptr_t>(t.in) & 15);
    return (bytes + tile - 1) / tile;
}

// Tensors [from, to) that have elements into a launch's table.
template <int CAP>
void fill(Table<CAP> *t, const ss_tensor *h, int32_t from, int32_t to, int tile = kTile) {
    t->count = 0;
    t->first[0] = 0;
    for (int32_t i = from; i < to; ++i) {
        if (h[i].numel == 0) continue;
        const int k = t->count++;
        t->in[k] = h[i].in, t->out[k] = h[i].out, t->numel[k] = h[i].numel, t->dtype[k] = uint8_t(h[i].dtype);
        t->first[k + 1] = t->first[k] + int32_t(tiles_of(h[i], tile));
    }
    const int64_t keep = t->first[t->count] - kKeep / tile;
    t->keep = keep > 0 ? int32_t(keep) : 0;
}

// CTAs that are on the device together.
template <typename K>
int resident(K kernel, int sms) {
    static std::atomic<int> known{0};
    int per_sm = known.load(std::memory_order_relaxed);
    if (per_sm == 0) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kThreads, 0) != cudaSuccess || per_sm < 1)
            per_sm = 1;
        known.store(per_sm, std::memory_order_relaxed);
    }
    return sms * per_sm < kMaxGrid ? sms * per_sm : kMaxGrid;
}

// Squares of the table's tensors; parts: how many partial sums there are.
template <int CAP>
void launch_squares(const Table<CAP> &t, float4 *part, int *parts, int sms, cudaStream_t s) {
    auto kernel = k_clip_squares<CAP>;
    const int most = resident(kernel, sms), tiles = t.first[t.count], grid = tiles < 1 ? 1 : (tiles < most ? tiles : most);
    SS_LAUNCH("k_clip_squares", s, kernel<<<grid, kThreads, 0, s>>>(t, part + *parts));
    *parts += grid;
}

void launch_result(const float4 *part, int parts, float max_norm, float eps, bool clip, float *result, cudaStream_t s) {
    SS_LAUNCH("k_clip_result", s,
              launch_after(k_clip_result, dim3(1), kThreads, 0, s, part, parts, max_norm, eps, clip, result));
}

template <int CAP>
void launch_scale(const Table<CAP> &t, const float *result, cudaStream_t s) {
    if (t.first[t.count] > 0)
        SS_LAUNCH("k_clip_scale", s, launch_after(k_clip_scale<CAP>, dim3(t.first[t.count]), kThreads, 0, s, t, result));
}

// A list that fits one launch's parameters.
template <int CAP>
void clip_list(const ss_tensor *h, int32_t n, bool clip, float max_norm, float eps, float *result, float4 *part, int sms,
               cudaStream_t s) {
    Table<CAP> t;
    int parts = 0;
    fill(&t, h, 0, n);
    launch_squares(t, part, &parts, sms, s);
    launch_result(part, parts, max_norm, eps, clip, result, s);
    if (clip) launch_scale(t, result, s);
}

ss_status run(const char *who, const ss_tensor *h, int32_t n, bool clip, float max_norm, float eps, float *result,
              void *workspace, size_t bytes, cudaStream_t s) {
    clear_error();
    if (n < 0 || n > kMaxTensors)
        return fail(SS_ERR_UNSUPPORTED, "%s: %d tensors outside 0..%d", who, n, kMaxTensors);
    if (n > 0 && !h) return fail(SS_ERR_INVALID_ARG, "%s: the tensor list is NULL", who);
    if (!result || !aligned_to(result, 4)) return fail(SS_ERR_INVALID_ARG, "%s: result NULL or misaligned", who);
    if (clip && (!(max_norm >= 0.0f) || !(eps >= 0.0f)))
        return fail(SS_ERR_INVALID_ARG, "%s: max_norm or eps negative or NaN", who);
    int64_t total = 0;
    for (int32_t i = 0; i < n; ++i) {
        const ss_tensor &t = h[i];
        if (!dtype_known(t.dtype) || t.reserved != 0)
            return fail(SS_ERR_INVALID_ARG, "%s: tensor %d: unknown dtype or reserved not 0", who, i);
        if (t.numel < 0) return fail(SS_ERR_INVALID_ARG, "%s: tensor %d: numel < 0", who, i);
        if (t.numel == 0) continue;
        const size_t a = dtype_bytes(t.dtype);
        if (!t.in || !aligned_to(t.in, a) || (clip && (!t.out || !aligned_to(t.out, a))))
            return fail(SS_ERR_INVALID_ARG, "%s: tensor %d: a pointer is NULL or misaligned", who, i);
        if (t.numel >= (int64_t(1) << 40) || (total += t.numel) >= (int64_t(1) << 40))
            return fail(SS_ERR_UNSUPPORTED, "%s: 2^40 elements or more", who);
    }
    if (!workspace || !aligned_to(workspace, 256))
        return fail(SS_ERR_INVALID_ARG, "%s: workspace NULL or not 256-byte aligned", who);
    const size_t need = ss_clip_workspace_bytes(n);
    if (bytes < need) return fail(SS_ERR_INVALID_ARG, "%s: workspace %zu bytes < %zu", who, bytes, need);
    int dev = 0, sms = 0;
    ss_status st = current_device(&dev, &sms, who);
    if (st != SS_OK) return st;
    float4 *part = static_cast<float4 *>(workspace);
    if (clip && n <= kSmallList && total <= kMostHeld * (kThreads * 8)) {   // 16 bytes hold 8 at most
        Table<kSmallList> t;
        fill(&t, h, 0, n, kThreads * 16);
        if (t.first[t.count] <= kMostHeld) {
            SS_LAUNCH("k_clip_small", s,
                      k_clip_small<<<kCluster, kTeams * kThreads, 0, s>>>(t, max_norm, eps, result));
            return check_launch(who);
        }
    }
    if (n <= kSmallList) {
        clip_list<kSmallList>(h, n, clip, max_norm, eps, result, part, sms, s);
    } else if (n <= kLongList) {
        clip_list<kLongList>(h, n, clip, max_norm, eps, result, part, sms, s);
    } else {                             // a launch for each part of the list
        Table<kLongList> t;
        int parts = 0;
        for (int32_t from = 0; from < n; from += kLongList) {
            fill(&t, h, from, from + kLongList < n ? from + kLongList : n);
            launch_squares(t, part, &parts, sms, s);
        }
        launch_result(part, parts, max_norm, eps, clip, result, s);
        for (int32_t from = 0; clip && from < n; from += kLongList) {
            fill(&t, h, from, from + kLongList < n ? from + kLongList : n);
            launch_scale(t, result, s);
        }
    }
    return check_launch(who);
}

}  // namespace
}  // namespace ss

using namespace ss;

extern "C" {

size_t ss_clip_workspace_bytes(int32_t n_tensors) {
    if (n_tensors < 0 || n_tensors > kMaxTensors) return 0;
    return size_t(n_tensors < 1 ? 1 : (n_tensors + kLongList - 1) / kLongList) * kMaxGrid * sizeof(float4);
}

ss_status ss_grad_clip(const ss_tensor *h_tensors, int32_t n_tensors, float max_norm, float eps, float *result,
                       void *workspace, size_t workspace_bytes, ss_stream_t stream) {
    return run("ss_grad_clip", h_tensors, n_tensors, true, max_norm, eps, result, workspace, workspace_bytes,
               (cudaStream_t)stream);
}

ss_status ss_grad_norm(const ss_tensor *h_tensors, int32_t n_tensors, float *result, void *workspace,
                       size_t workspace_bytes, ss_stream_t stream) {
    return run("ss_grad_norm", h_tensors, n_tensors, false, 0.0f, 0.0f, result, workspace, workspace_bytes,
               (cudaStream_t)stream);
}

}  // extern "C"
