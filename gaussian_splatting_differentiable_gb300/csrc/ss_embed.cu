// Rows of a learned table looked up by id, and the table's gradient (model:
// include/ss_embed.h).
//
// Backward.  k_embed_hist counts the ids' digits and clears dtable;
// k_embed_pass is one stable onesweep pass over an 8-bit digit of the id
// (words id << 32 | position; an id outside [0, V) becomes V and sorts past
// every row); k_embed_sum walks fixed chunks of the sorted words and adds
// dout rows: an id whose words lie inside one chunk is finished there, one
// that crosses chunks leaves a partial sum at each end of each chunk that
// k_embed_join adds in chunk order.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "ss_embed.h"
#include "ss_internal.h"
#include "ss_profile.h"
#include "ss_vec.cuh"

namespace ss {
namespace {

constexpr int kThreads = 256;
constexpr int32_t kMaxD = 65536;
constexpr int kPart = 4096;              // words of one sort partition
constexpr int kKpt = kPart / kThreads;
constexpr int kMaxPasses = 4;
constexpr uint32_t kFlagAgg = 1u << 30, kFlagInc = 2u << 30, kValMask = kFlagAgg - 1;
constexpr uint32_t kSpinLimit = 1u << 22;

// ------------------------------------------------------------------ forward

template <typename T, typename I>
__global__ void __launch_bounds__(kThreads) k_embed_fwd(const T *__restrict__ table, int64_t ts, int64_t V, int32_t D,
                                                        const I *__restrict__ ids, int64_t n, float scale, T *out,
                                                        int64_t os) {
    const int64_t total = n * D, stride = int64_t(gridDim.x) * kThreads;
    for (int64_t e = int64_t(blockIdx.x) * kThreads + threadIdx.x; e < total; e += stride) {
        const int64_t i = e / D;
        const int j = int(e - i * D);
        const int64_t id = int64_t(ids[i]);
        const float v = id >= 0 && id < V ? to_float(table[id * ts + j]) * scale : 0.0f;
        out[i * os + j] = from_float<T>(v);
    }
}

// ------------------------------------------------------------------ sort

template <typename I>
__device__ __forceinline__ uint32_t id_key(const I *ids, int64_t i, uint32_t V) {
    const int64_t id = int64_t(ids[i]);
    return id >= 0 && id < int64_t(V) ? uint32_t(id) : V;
}

__device__ __forceinline__ uint32_t excl_scan256(uint32_t v, uint32_t *s_warp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    uint32_t base = 0;
    for (int w = 0; w < warp; ++w) base += s_warp[w];
    return base + x - v;
}

struct SortState {
    uint32_t status;                       // kDevErrTimeout
    uint32_t done;                         // histogram CTAs done
    uint32_t ticket[kMaxPasses];
    uint32_t hist[kMaxPasses][256];
    uint32_t start[kMaxPasses][256];       // exclusive digit starts
};

template <typename I, typename G>
__global__ void __launch_bounds__(kThreads) k_embed_hist(const I *__restrict__ ids, int64_t n, uint32_t V, int passes,
                                                         SortState *st, G *dtable, int64_t ds, int32_t D) {
    __shared__ uint32_t s_h[kMaxPasses][256];
    __shared__ uint32_t s_warp[8], s_last;
    for (int k = threadIdx.x; k < kMaxPasses * 256; k += kThreads) (&s_h[0][0])[k] = 0;
    __syncthreads();
    const int64_t stride = int64_t(gridDim.x) * kThreads;
    const int64_t first = int64_t(blockIdx.x) * kThreads + threadIdx.x;
    for (int64_t i = first; i < n; i += stride) {
        const uint32_t key = id_key(ids, i, V);
        for (int d = 0; d < passes; ++d) atomicAdd(&s_h[d][(key >> (8 * d)) & 255u], 1u);
    }
    __syncthreads();
    for (int k = threadIdx.x; k < passes * 256; k += kThreads) {
        const uint32_t v = (&s_h[0][0])[k];
        if (v) atomicAdd(&st->hist[0][0] + k, v);
    }
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) s_last = atomicAdd(&st->done, 1u) == gridDim.x - 1;
    __syncthreads();
    if (s_last) {
        __threadfence();
        for (int d = 0; d < passes; ++d)
            st->start[d][threadIdx.x] = excl_scan256(__ldcg(&st->hist[d][threadIdx.x]), s_warp);
    }
    const int64_t total = int64_t(V) * D;
    for (int64_t e = first; e < total; e += stride) {
        const int64_t v = e / D;
        dtable[v * ds + (e - v * D)] = from_float<G>(0.0f);
    }
}

__device__ __forceinline__ uint32_t ld_relaxed(const uint32_t *p) {
    uint32_t v;
    asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void st_relaxed(uint32_t *p, uint32_t v) {
    asm volatile("st.relaxed.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// One stable pass over digit d.  Partitions are taken by ticket, so every
// partition that one waits on has been started; a wait that runs out sets
// the status and goes on with the counts that it has (every write stays
// inside the n words).
template <typename I>
__global__ void __launch_bounds__(kThreads) k_embed_pass(const I *__restrict__ ids, const uint64_t *__restrict__ win,
                                                         uint64_t *__restrict__ wout, int64_t n, uint32_t V, int d,
                                                         SortState *st, uint32_t *lookback) {
    __shared__ uint32_t s_whist[8][256];
    __shared__ uint32_t s_lstart[256], s_gbase[256], s_warp[8], s_part;
    __shared__ uint64_t s_words[kPart];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) s_part = atomicAdd(&st->ticket[d], 1u);
    for (int k = tid; k < 8 * 256; k += kThreads) (&s_whist[0][0])[k] = 0;
    __syncthreads();
    const int64_t part = s_part, base = part * kPart, wbase = base + warp * (kKpt * 32);
    const int shift = 32 + 8 * d;
    uint64_t word[kKpt];
    uint32_t rank[kKpt];
#pragma unroll
    for (int j = 0; j < kKpt; ++j) {
        const int64_t i = wbase + j * 32 + lane;
        word[j] = ~0ull;
        if (i < n) word[j] = d == 0 ? uint64_t(id_key(ids, i, V)) << 32 | uint32_t(i) : win[i];
    }
    uint32_t lt;
    asm("mov.u32 %0, %%lanemask_lt;" : "=r"(lt));
#pragma unroll
    for (int j = 0; j < kKpt; ++j) {
        const bool ok = wbase + j * 32 + lane < n;
        const uint32_t dig = ok ? uint32_t(word[j] >> shift) & 255u : 256u + lane;
        const uint32_t peers = __match_any_sync(0xffffffffu, dig);
        const uint32_t before = __popc(peers & lt);
        const uint32_t cur = ok ? s_whist[warp][dig] : 0u;
        rank[j] = cur + before;
        __syncwarp();
        if (ok && before == 0) s_whist[warp][dig] = cur + __popc(peers);
        __syncwarp();
    }
    __syncthreads();
    uint32_t total = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        const uint32_t c = s_whist[w][tid];
        s_whist[w][tid] = total;
        total += c;
    }
    uint32_t *my = lookback + part * 256 + tid;
    st_relaxed(my, (part == 0 ? kFlagInc : kFlagAgg) | total);
    s_lstart[tid] = excl_scan256(total, s_warp);
    uint32_t excl = 0;
    if (part > 0) {
        uint32_t spins = 0;
        for (int64_t q = part - 1;;) {
            const uint32_t w = ld_relaxed(lookback + q * 256 + tid);
            if (w < kFlagAgg) {
                if (++spins > kSpinLimit) {
                    atomicOr(&st->status, kDevErrTimeout);
                    break;
                }
                continue;
            }
            excl += w & kValMask;
            if (w >= kFlagInc || q == 0) break;
            --q;
            spins = 0;
        }
        st_relaxed(my, kFlagInc | (excl + total));
    }
    s_gbase[tid] = st->start[d][tid] + excl;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kKpt; ++j) {
        if (wbase + j * 32 + lane < n) {
            const uint32_t dig = uint32_t(word[j] >> shift) & 255u;
            s_words[s_lstart[dig] + s_whist[warp][dig] + rank[j]] = word[j];
        }
    }
    __syncthreads();
    const int cnt = int(n - base < kPart ? n - base : kPart);
    for (int i = tid; i < cnt; i += kThreads) {
        const uint64_t w = s_words[i];
        const uint32_t dig = uint32_t(w >> shift) & 255u;
        const uint32_t g = s_gbase[dig] + uint32_t(i) - s_lstart[dig];
        if (int64_t(g) < n) wout[g] = w;
    }
}

// ------------------------------------------------------------------ sums

struct SumParams {
    const uint64_t *words;   // sorted id << 32 | position
    int64_t n, chunk;        // words of a CTA = groups * walk
    uint32_t V;
    int32_t D;
    int walk;                // words of one thread group
    int groups, cols;        // blockDim = groups * cols, a thread owns one vector of columns
    int vecs;                // vectors of a row
    int64_t in_stride, out_stride;
    float scale;
    float *head, *tail;      // [chunks][D] partial sums of ids that cross a chunk's ends
};

__device__ __forceinline__ uint32_t key_at(const SumParams &p, int64_t i) {
    return uint32_t(__ldg(p.words + i) >> 32);
}

// Chunk [lo, hi) as seen from its ends: `in` its first id began before it,
// `on` its last id goes on after it, `whole` one id fills it and does both.
struct Ends {
    bool in, on, whole;
};
__device__ __forceinline__ Ends ends_of(const SumParams &p, int64_t lo, int64_t hi) {
    Ends e;
    const uint32_t a = key_at(p, lo), b = key_at(p, hi - 1);
    e.in = lo > 0 && key_at(p, lo - 1) == a;
    e.on = hi < p.n && key_at(p, hi) == b;
    e.whole = e.in && e.on && a == b;
    return e;
}

template <typename G, int N>
__device__ __forceinline__ void finish_row(const SumParams &p, G *dtable, uint32_t key, int col, const float (&acc)[N]) {
    if (key >= p.V) return;
    float f[N];
#pragma unroll
    for (int k = 0; k < N; ++k) f[k] = acc[k] * p.scale;
    store_floats<G, N>(dtable + int64_t(key) * p.out_stride + int64_t(col) * N, f);
}

template <typename T, typename G, int N>
__global__ void __launch_bounds__(kThreads) k_embed_sum(SumParams p, const T *__restrict__ dout, G *dtable) {
    extern __shared__ float s_part[];      // head then tail: [groups][cols][N]
    constexpr int kBatch = 8;
    const int g = threadIdx.x / p.cols, c = threadIdx.x - g * p.cols;
    const int col = blockIdx.y * p.cols + c;
    const bool live = col < p.vecs;
    const int64_t cbase = int64_t(blockIdx.x) * p.chunk;
    const int64_t lo = cbase + int64_t(g) * p.walk;
    const int64_t hi = lo + p.walk < p.n ? lo + p.walk : p.n;
    float *head = s_part + size_t(threadIdx.x) * N;
    float *tail = head + size_t(p.groups) * p.cols * N;
    Ends e{false, false, false};
    float acc[N];
    if (live && lo < hi) {
        e = ends_of(p, lo, hi);
        uint32_t cur = key_at(p, lo);
        bool open = e.in;                 // the current id began before this walk
#pragma unroll
        for (int k = 0; k < N; ++k) acc[k] = 0.0f;
        for (int64_t i = lo; i < hi; i += kBatch) {
            uint64_t w[kBatch];
            Vec<T, N> x[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) w[u] = i + u < hi ? __ldg(p.words + i + u) : ~0ull;
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                x[u].clear();
                const uint32_t pos = uint32_t(w[u]);
                if (uint32_t(w[u] >> 32) < p.V && int64_t(pos) < p.n)
                    x[u] = load_vec<T, N>(dout + int64_t(pos) * p.in_stride + int64_t(col) * N);
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                if (i + u >= hi) break;
                const uint32_t key = uint32_t(w[u] >> 32);
                if (key != cur) {
                    if (open) {
#pragma unroll
                        for (int k = 0; k < N; ++k) head[k] = acc[k];
                    } else {
                        finish_row<G, N>(p, dtable, cur, col, acc);
                    }
                    open = false;
                    cur = key;
#pragma unroll
                    for (int k = 0; k < N; ++k) acc[k] = 0.0f;
                }
#pragma unroll
                for (int k = 0; k < N; ++k) acc[k] += x[u].get(k);
            }
        }
        if (open) {
#pragma unroll
            for (int k = 0; k < N; ++k) head[k] = acc[k];
        } else if (!e.on) {
            finish_row<G, N>(p, dtable, cur, col, acc);
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k) tail[k] = acc[k];
        }
    }
    __syncthreads();
    if (!live || lo >= hi) return;
    // Joins the groups of this chunk.  The thread of the group where an id
    // begins (or of group 0 for the id that the chunk before began) adds the
    // groups that follow, in order.
    const int64_t chi = cbase + p.chunk < p.n ? cbase + p.chunk : p.n;
    for (int pass = 0; pass < 2; ++pass) {
        const bool incoming = pass == 0;
        if (incoming ? !(g == 0 && e.in) : !(e.on && !e.whole)) continue;
        float *own = incoming ? head : tail;
#pragma unroll
        for (int k = 0; k < N; ++k) acc[k] = own[k];
        bool on = incoming ? e.whole : true;
        const uint32_t key = incoming ? key_at(p, lo) : key_at(p, hi - 1);
        int64_t q = hi;                    // first word of the next group
        int h = 1;
        while (on && q < chi) {
            const int64_t qe = q + p.walk < chi ? q + p.walk : chi;
#pragma unroll
            for (int k = 0; k < N; ++k) acc[k] += head[size_t(h) * p.cols * N + k];
            on = key_at(p, qe - 1) == key && qe < p.n && key_at(p, qe) == key;
            q = qe;
            ++h;
        }
        if (incoming || on) {
            float *dst = (incoming ? p.head : p.tail) + size_t(blockIdx.x) * p.D + size_t(col) * N;
#pragma unroll
            for (int k = 0; k < N; ++k) dst[k] = acc[k];
        } else {
            finish_row<G, N>(p, dtable, key, col, acc);
        }
    }
}

// One CTA per chunk (and slice of columns): if an id begins in the chunk and
// goes on after it, adds its partial sums, groups of threads taking every
// groups-th chunk and then joining in order.
template <typename G>
__global__ void __launch_bounds__(kThreads) k_embed_join(SumParams p, G *dtable) {
    __shared__ float s_acc[kThreads];
    const int64_t lo = int64_t(blockIdx.x) * p.chunk, hi = lo + p.chunk;
    if (hi >= p.n) return;                 // the last chunk: nothing follows
    const Ends e = ends_of(p, lo, hi);
    const uint32_t key = key_at(p, hi - 1);
    if (!e.on || e.whole || key >= p.V) return;
    // the id's last chunk: the chunk of its last word
    int64_t a = hi, b = p.n;               // words[a] has the id, words[b] (if any) has not
    while (b - a > 1) {
        const int64_t m = a + (b - a) / 2;
        if (key_at(p, m) == key) a = m; else b = m;
    }
    const int64_t last = a / p.chunk;
    const int cols = p.D < kThreads ? p.D : kThreads, groups = kThreads / cols;
    const int g = threadIdx.x / cols, c = threadIdx.x - g * cols;
    for (int col0 = blockIdx.y * cols; col0 < p.D; col0 += gridDim.y * cols) {
        const int col = col0 + c;
        float acc = 0.0f;
        if (g < groups && col < p.D) {
            if (g == 0) acc = p.tail[size_t(blockIdx.x) * p.D + col];
            for (int64_t q = blockIdx.x + 1 + g; q <= last; q += groups) acc += p.head[size_t(q) * p.D + col];
        }
        __syncthreads();
        s_acc[threadIdx.x] = acc;
        __syncthreads();
        if (g == 0 && col < p.D) {
            for (int h = 1; h < groups; ++h) acc += s_acc[h * cols + c];
            dtable[int64_t(key) * p.out_stride + col] = from_float<G>(acc * p.scale);
        }
    }
}

// ------------------------------------------------------------------ host

bool sizes_ok(int64_t n, int64_t V, int32_t D) {
    return n >= 0 && n < (int64_t(1) << 30) && V >= 1 && V < (int64_t(1) << 31) && D >= 1 && D <= kMaxD;
}

int sort_passes(int64_t V) {               // keys 0..V
    int b = 1;
    while (b < 32 && (int64_t(1) << b) <= V) ++b;
    return (b + 7) / 8;
}

struct SumShape {
    int vecs, cols, groups, slices, walk;
    int64_t chunk, chunks;
};

// Columns over threads: a row's vectors side by side, as many rows as fit in
// a CTA.  The walk (words added by one thread in turn) is as long as leaves
// about eight CTAs an SM.
SumShape sum_shape(int64_t n, int32_t D, int vec) {
    SumShape s;
    s.vecs = D / vec;
    s.slices = (s.vecs + kThreads - 1) / kThreads;
    s.cols = (s.vecs + s.slices - 1) / s.slices;
    s.groups = kThreads / s.cols;
    int64_t w = n * s.slices / (int64_t(s.groups) * 152 * 8);
    s.walk = int(w < 8 ? 8 : (w > 64 ? 64 : (w + 7) / 8 * 8));
    s.chunk = int64_t(s.groups) * s.walk;
    s.chunks = (n + s.chunk - 1) / s.chunk;
    return s;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct BwdLayout {
    size_t lookback, zero_end, words, head, tail, total;
    int64_t parts;
    int passes;
};

BwdLayout bwd_layout(int64_t n, int64_t V, int32_t D) {
    BwdLayout L;
    L.parts = (n + kPart - 1) / kPart;
    L.passes = sort_passes(V);
    L.lookback = align256(sizeof(SortState));
    L.zero_end = align256(L.lookback + size_t(L.passes) * L.parts * 256 * 4);
    L.words = L.zero_end;
    L.head = align256(L.words + size_t(n) * 16);
    int64_t chunks = 0;                    // of whichever vector width the pointers allow
    for (int vec : {1, 4, 8})
        if (D % vec == 0) {
            const SumShape s = sum_shape(n, D, vec);
            if (s.chunks > chunks) chunks = s.chunks;
        }
    L.tail = align256(L.head + size_t(chunks) * D * 4);
    L.total = align256(L.tail + size_t(chunks) * D * 4);
    return L;
}

ss_status check_rows(const char *who, const char *what, const void *p, int64_t stride, int32_t D, int dtype) {
    if (!p) return fail(SS_ERR_INVALID_ARG, "%s: %s is NULL", who, what);
    if (!aligned_to(p, dtype_bytes(dtype)))
        return fail(SS_ERR_INVALID_ARG, "%s: %s is not aligned to its type", who, what);
    if (stride < D || stride > (int64_t(1) << 31))
        return fail(SS_ERR_INVALID_ARG, "%s: %s stride %lld below D or above 2^31", who, what, (long long)stride);
    return SS_OK;
}

ss_status check_common(const char *who, int64_t n, int64_t V, int32_t D, int dtype, const void *ids, int id_bytes) {
    if (!sizes_ok(n, V, D))
        return fail(SS_ERR_UNSUPPORTED, "%s: %lld ids, a table of %lld x %d outside 0..2^30-1, 1..2^31-1 x 1..%d", who,
                    (long long)n, (long long)V, D, kMaxD);
    if (!dtype_known(dtype)) return fail(SS_ERR_INVALID_ARG, "%s: unknown dtype %d", who, dtype);
    if (id_bytes != 4 && id_bytes != 8) return fail(SS_ERR_INVALID_ARG, "%s: id_bytes is neither 4 nor 8", who);
    if (n > 0 && (!ids || !aligned_to(ids, id_bytes)))
        return fail(SS_ERR_INVALID_ARG, "%s: ids NULL or misaligned", who);
    return SS_OK;
}

template <typename T, typename I>
void launch_fwd(const void *table, int64_t ts, int64_t V, int32_t D, const void *ids, int64_t n, float scale,
                void *out, int64_t os, int sms, cudaStream_t s) {
    const int64_t want = (n * D + kThreads - 1) / kThreads;
    const int grid = int(want < int64_t(sms) * 32 ? want : int64_t(sms) * 32);
    SS_LAUNCH("k_embed_fwd", s,
              k_embed_fwd<T, I><<<grid, kThreads, 0, s>>>(static_cast<const T *>(table), ts, V, D,
                                                          static_cast<const I *>(ids), n, scale,
                                                          static_cast<T *>(out), os));
}

template <typename T, typename G, int N>
void launch_sums(const SumParams &p, const SumShape &sh, const T *dout, G *dtable, cudaStream_t s) {
    const dim3 grid(unsigned(sh.chunks), unsigned(sh.slices));
    const int threads = sh.groups * sh.cols;
    SS_LAUNCH("k_embed_sum", s,
              k_embed_sum<T, G, N><<<grid, threads, size_t(threads) * N * 8, s>>>(p, dout, dtable));
    if (sh.chunks > 1)
        SS_LAUNCH("k_embed_join", s, k_embed_join<G><<<dim3(unsigned(sh.chunks)), kThreads, 0, s>>>(p, dtable));
}

template <typename T, typename G, typename I>
ss_status launch_bwd(const void *dout, int64_t in_stride, const void *ids, int64_t n, int64_t V, int32_t D, float scale,
                     void *dtable, int64_t out_stride, char *ws, int sms, cudaStream_t s) {
    const BwdLayout L = bwd_layout(n, V, D);
    SortState *st = reinterpret_cast<SortState *>(ws);
    ss_status e = check_cuda(cudaMemsetAsync(ws, 0, L.zero_end, s), "ss_embed_bwd: memset");
    if (e != SS_OK) return e;
    const I *id = static_cast<const I *>(ids);
    G *dt = static_cast<G *>(dtable);
    SS_LAUNCH("k_embed_hist", s,
              k_embed_hist<I, G><<<sms * 4, kThreads, 0, s>>>(id, n, uint32_t(V), L.passes, st, dt, out_stride, D));
    if (n == 0) return SS_OK;
    uint64_t *w[2] = {reinterpret_cast<uint64_t *>(ws + L.words), reinterpret_cast<uint64_t *>(ws + L.words) + n};
    for (int d = 0; d < L.passes; ++d)
        SS_LAUNCH("k_embed_pass", s,
                  k_embed_pass<I><<<unsigned(L.parts), kThreads, 0, s>>>(
                      id, w[(d + 1) & 1], w[d & 1], n, uint32_t(V), d, st,
                      reinterpret_cast<uint32_t *>(ws + L.lookback) + size_t(d) * L.parts * 256));
    constexpr int kVec = 16 / sizeof(T);
    const bool vec = D % kVec == 0 && aligned_to(dout, 16) && in_stride % kVec == 0 &&
                     aligned_to(dtable, 16) && (out_stride * sizeof(G)) % 16 == 0;
    const SumShape sh = sum_shape(n, D, vec ? kVec : 1);
    SumParams p{};
    p.words = w[(L.passes - 1) & 1];
    p.n = n, p.chunk = sh.chunk, p.V = uint32_t(V), p.D = D, p.walk = sh.walk, p.groups = sh.groups, p.cols = sh.cols;
    p.vecs = sh.vecs, p.in_stride = in_stride, p.out_stride = out_stride, p.scale = scale;
    p.head = reinterpret_cast<float *>(ws + L.head), p.tail = reinterpret_cast<float *>(ws + L.tail);
    if (vec)
        launch_sums<T, G, kVec>(p, sh, static_cast<const T *>(dout), dt, s);
    else
        launch_sums<T, G, 1>(p, sh, static_cast<const T *>(dout), dt, s);
    return SS_OK;
}

template <typename T, typename G>
ss_status launch_bwd_ids(const void *dout, int64_t in_stride, const void *ids, int id_bytes, int64_t n, int64_t V,
                         int32_t D, float scale, void *dtable, int64_t out_stride, char *ws, int sms, cudaStream_t s) {
    return id_bytes == 4 ? launch_bwd<T, G, int32_t>(dout, in_stride, ids, n, V, D, scale, dtable, out_stride, ws, sms, s)
                         : launch_bwd<T, G, int64_t>(dout, in_stride, ids, n, V, D, scale, dtable, out_stride, ws, sms, s);
}

}  // namespace
}  // namespace ss

using namespace ss;

extern "C" {

ss_status ss_embed_fwd(const void *table, ss_dtype dtype, int64_t V, int32_t D, int64_t table_stride, const void *ids,
                       int32_t id_bytes, int64_t n, float scale, void *out, int64_t out_stride, ss_stream_t stream) {
    clear_error();
    const char *who = "ss_embed_fwd";
    ss_status st = check_common(who, n, V, D, dtype, ids, id_bytes);
    if (st != SS_OK || n == 0) return st;
    if ((st = check_rows(who, "table", table, table_stride, D, dtype)) != SS_OK) return st;
    if ((st = check_rows(who, "out", out, out_stride, D, dtype)) != SS_OK) return st;
    int dev = 0, sms = 0;
    if ((st = current_device(&dev, &sms, "ss_embed_fwd: device query")) != SS_OK) return st;
    cudaStream_t s = (cudaStream_t)stream;
#define SS_FWD(T)                                                                                             \
    (id_bytes == 4 ? launch_fwd<T, int32_t>(table, table_stride, V, D, ids, n, scale, out, out_stride, sms, s) \
                   : launch_fwd<T, int64_t>(table, table_stride, V, D, ids, n, scale, out, out_stride, sms, s))
    if (dtype == SS_F32) SS_FWD(float);
    else if (dtype == SS_F16) SS_FWD(__half);
    else SS_FWD(__nv_bfloat16);
#undef SS_FWD
    return check_launch(who);
}

size_t ss_embed_workspace_bytes(int64_t n, int64_t V, int32_t D) {
    return sizes_ok(n, V, D) ? bwd_layout(n, V, D).total : 0;
}

ss_status ss_embed_bwd(const void *dout, ss_dtype dtype, int64_t dout_stride, const void *ids, int32_t id_bytes,
                       int64_t n, int64_t V, int32_t D, float scale, void *dtable, ss_dtype grad_dtype,
                       int64_t dtable_stride, void *workspace, size_t workspace_bytes, ss_stream_t stream) {
    clear_error();
    const char *who = "ss_embed_bwd";
    ss_status st = check_common(who, n, V, D, dtype, ids, id_bytes);
    if (st != SS_OK) return st;
    if (grad_dtype != dtype && grad_dtype != SS_F32)
        return fail(SS_ERR_INVALID_ARG, "%s: grad_dtype %d is neither SS_F32 nor dout's type", who, int(grad_dtype));
    if (n > 0 && (st = check_rows(who, "dout", dout, dout_stride, D, dtype)) != SS_OK) return st;
    if ((st = check_rows(who, "dtable", dtable, dtable_stride, D, grad_dtype)) != SS_OK) return st;
    if (!workspace || !aligned_to(workspace, 256))
        return fail(SS_ERR_INVALID_ARG, "%s: workspace NULL or not 256-byte aligned", who);
    const size_t need = ss_embed_workspace_bytes(n, V, D);
    if (workspace_bytes < need)
        return fail(SS_ERR_INVALID_ARG, "%s: workspace %zu bytes < %zu", who, workspace_bytes, need);
    int dev = 0, sms = 0;
    if ((st = current_device(&dev, &sms, "ss_embed_bwd: device query")) != SS_OK) return st;
    cudaStream_t s = (cudaStream_t)stream;
    char *ws = static_cast<char *>(workspace);
#define SS_BWD(T, G) \
    launch_bwd_ids<T, G>(dout, dout_stride, ids, id_bytes, n, V, D, scale, dtable, dtable_stride, ws, sms, s)
    if (dtype == SS_F32) st = SS_BWD(float, float);
    else if (dtype == SS_F16) st = grad_dtype == SS_F32 ? SS_BWD(__half, float) : SS_BWD(__half, __half);
    else st = grad_dtype == SS_F32 ? SS_BWD(__nv_bfloat16, float) : SS_BWD(__nv_bfloat16, __nv_bfloat16);
#undef SS_BWD
    return st != SS_OK ? st : check_launch(who);
}

ss_status ss_embed_status(const void *workspace, ss_stream_t stream) {
    clear_error();
    if (!workspace) return fail(SS_ERR_INVALID_ARG, "ss_embed_status: workspace is NULL");
    uint32_t word = 0;
    ss_status st = check_cuda(cudaMemcpyAsync(&word, workspace, 4, cudaMemcpyDeviceToHost, (cudaStream_t)stream),
                              "ss_embed_status: cudaMemcpyAsync");
    if (st != SS_OK) return st;
    st = check_cuda(cudaStreamSynchronize((cudaStream_t)stream), "ss_embed_status: synchronize");
    if (st != SS_OK) return st;
    if (word & kDevErrTimeout)
        return fail(SS_ERR_TIMEOUT, "ss_embed_bwd: a look-back wait gave up (status 0x%x)", word);
    return SS_OK;
}

}  // extern "C"
