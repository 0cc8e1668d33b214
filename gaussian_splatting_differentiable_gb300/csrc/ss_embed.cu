// Rows of a learned table looked up by id, and the table's gradient (model:
// include/ss_embed.h).
//
// Backward.  (id, position) words are sorted by id: a few in k_embed_sum
// itself, more in k_embed_sort_small, else by k_embed_count / k_embed_scan /
// k_embed_move for each digit, while CTAs beside the sort's clear dtable.
// k_embed_sum walks fixed chunks of the sorted words and adds dout rows, and
// k_embed_join adds up the ids that cross chunks.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "ss_embed.h"
#include "ss_internal.h"
#include "ss_launch.cuh"
#include "ss_profile.h"
#include "ss_vec.cuh"

namespace ss {
namespace {

constexpr int kThreads = 256;
constexpr int32_t kMaxD = 65536;
constexpr int64_t kManyBytes = 64 << 20;   // of output, half of L2

// ------------------------------------------------------------------ forward

// `lanes` threads take a row, NV vectors each (N elements a vector: as many as
// every row's start and end are aligned to), and ROWS rows at a time so that
// the ids' loads, and then the rows', wait together.  Bound by the writes of
// out (and the table's reads where it does not stay in L2): 2M x 48 float32
// out of 65,536 rows (412 MB) 67 us, 61 at copy bandwidth.
//
// Where rows allow only narrow vectors the instructions bound it: a row's
// pointers and limits are made once, and WARP (a row to a warp) leaves the
// vectors' distances to the instructions (700,000 x 87 bfloat16: 107 us with
// all of that worked out for each value, 58 so; in pairs on 4-byte boundaries
// 80, for the registers and instructions that the rows' ends take).
template <typename T, typename I, int N, int NV, int ROWS, bool WARP>
__global__ void __launch_bounds__(kThreads)
    k_embed_fwd(const T *__restrict__ table, int64_t ts, int64_t V, const I *__restrict__ ids, int64_t n, float scale,
                T *out, int64_t os, int shift, int vecs, bool leave) {
    const int lanes = WARP ? 32 : 1 << shift, lane = threadIdx.x & (lanes - 1);
    const int rstep = WARP ? kThreads / 32 : kThreads >> shift;
    const int64_t row0 = int64_t(blockIdx.x) * (rstep * ROWS) + threadIdx.x / lanes;
    int64_t id[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) id[r] = row0 + r * rstep < n ? int64_t(ids[row0 + r * rstep]) : -1;
    const T *from[ROWS];
    T *const to = out + row0 * os + lane * N;
    const int64_t apart = rstep * os;
    int named[ROWS];                       // vectors to read of the row: none where the id names no row,
    float s[ROWS];                         // and zeros times 0, not times the scale
    const int mine = vecs - lane, left = n - row0 < ROWS * rstep ? int(n - row0) : ROWS * rstep;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const bool here = id[r] >= 0 && id[r] < V;
        from[r] = table + (here ? id[r] : 0) * ts + lane * N;
        named[r] = here ? mine : 0;
        s[r] = here ? scale : 0.0f;
    }
#pragma unroll 1                           // most rows take one turn (unrolled, 45 registers: 2M x 48, 80 us for 67)
    for (int v0 = 0; v0 < mine; v0 += lanes * NV) {
        Vec<T, N> x[ROWS][NV];
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                x[r][k].clear();
                if (v0 + k * lanes < named[r]) x[r][k] = load_vec<T, N>(from[r] + (v0 + k * lanes) * N);
            }
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            if (r * rstep >= left) break;
            T *row = to + r * apart;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                float f[N];
#pragma unroll
                for (int i = 0; i < N; ++i) f[i] = x[r][k].get(i) * s[r];
                if (v0 + k * lanes >= mine) continue;
                if (N * sizeof(T) == 16 && leave)
                    store_floats_cs<T, N>(row + (v0 + k * lanes) * N, f);
                else
                    store_floats<T, N>(row + (v0 + k * lanes) * N, f);
            }
        }
    }
}

// ------------------------------------------------------------------ sort

constexpr int kPart = 2048;              // ids of one sort partition
constexpr int kKpt = kPart / kThreads;
constexpr int kMaxBits = 8;              // of a digit: at most 256 bins
constexpr int kFewParts = 32;            // partitions whose counts the move adds up itself
constexpr int kSmallThreads = 1024;      // of the one CTA that sorts a small batch
constexpr int kSmallN = 4 * kSmallThreads;         // ids up to which it does,
constexpr int kSmallMost = 8 * kSmallThreads;      // and up to which it does beside a long clearing
constexpr int64_t kLongClearing = 32 << 20;        // bytes

struct SortState {
    int64_t count;                       // ids that name a row
    uint32_t joins;                      // ids that cross chunks of the sorted words
};

// The id as a key, V where it names no row.
template <typename I>
__device__ __forceinline__ uint32_t id_key(const I *ids, int64_t i, uint32_t V) {
    const int64_t id = int64_t(ids[i]);
    return id >= 0 && id < int64_t(V) ? uint32_t(id) : V;
}

// Exclusive scan of one value a thread over the CTA; s_warp: a word a warp.
__device__ __forceinline__ uint32_t warp_scan(uint32_t x) {   // inclusive
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}
__device__ __forceinline__ uint32_t excl_scan(uint32_t v, uint32_t *s_warp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const uint32_t x = warp_scan(v);
    __syncthreads();
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    const uint32_t sums = warp_scan(lane < warps ? s_warp[lane] : 0u);
    const uint32_t before = __shfl_sync(0xffffffffu, sums, (warp + 31) & 31);
    return (warp > 0 ? before : 0u) + x - v;
}

// The lanes whose digit of BITS bits is this lane's (of those with `ok`): a
// vote for each bit.  (A match instruction takes several times as long: the
// gradient of 2M ids of 12 bits became 23 us longer with it.)
template <int BITS>
__device__ __forceinline__ uint32_t same_digit(uint32_t dig, bool ok) {
    uint32_t peers = __ballot_sync(0xffffffffu, ok);
#pragma unroll
    for (int b = 0; b < BITS; ++b) {
        const bool one = (dig >> b) & 1u;
        const uint32_t v = __ballot_sync(0xffffffffu, one);
        peers &= one ? v : ~v;
    }
    return peers;
}

__device__ __forceinline__ uint32_t lanes_below() {
    uint32_t m;
    asm("mov.u32 %0, %%lanemask_lt;" : "=r"(m));
    return m;
}

// The table's gradient, cleared by the CTAs that a sort kernel has beside its
// own: the sort waits on latency, not on bandwidth, and the clearing, the
// larger part of the work for a large vocabulary, goes on meanwhile.  Each
// launch of the sort clears its share.
template <typename G>
struct Clearing {
    G *p;
    int64_t rows, stride;
    int32_t D;
    int share, shares;                   // this launch's
};
template <typename G>
__device__ __forceinline__ void clear_share(const Clearing<G> &c, int cta, int ctas) {
    const int64_t part = int64_t(c.share) * ctas + cta, parts = int64_t(c.shares) * ctas;
    if (c.stride == c.D) {               // one run of values, 16 bytes at a time
        const int64_t total = c.rows * c.D;
        int64_t head = int64_t((16 - (reinterpret_cast<uintptr_t>(c.p) & 15)) & 15) / int64_t(sizeof(G));
        if (head > total) head = total;
        constexpr int kVec = 16 / sizeof(G);
        const int64_t body = (total - head) / kVec, each = (body + parts - 1) / parts;
        const int64_t lo = part * each, hi = lo + each < body ? lo + each : body;
        uint4 *q = reinterpret_cast<uint4 *>(c.p + head);
#pragma unroll 4
        for (int64_t v = lo + threadIdx.x; v < hi; v += blockDim.x) q[v] = make_uint4(0, 0, 0, 0);
        if (part == 0) {
            for (int64_t e = threadIdx.x; e < head; e += blockDim.x) c.p[e] = from_float<G>(0.0f);
            for (int64_t e = head + body * kVec + threadIdx.x; e < total; e += blockDim.x) c.p[e] = from_float<G>(0.0f);
        }
        return;
    }
    // rows apart from one another: whole rows to a CTA, their elements to its threads in turn
    const int64_t each = (c.rows + parts - 1) / parts;
    const int64_t lo = part * each, hi = lo + each < c.rows ? lo + each : c.rows;
    if (lo >= hi) return;
    const int dr = int(blockDim.x) / c.D, dj = int(blockDim.x) - dr * c.D;   // a step of blockDim.x elements
    int64_t r = lo + int(threadIdx.x) / c.D;
    int j = int(threadIdx.x) % c.D;
    while (r < hi) {
        c.p[r * c.stride + j] = from_float<G>(0.0f);
        r += dr, j += dj;
        if (j >= c.D) j -= c.D, ++r;
    }
}

// One CTA sorts up to KPT ids a thread in its shared memory, 8 bits a pass,
// the others clear.  The sort waits on its barriers and on shared memory, the
// clearing on the stores' bandwidth: 8191 ids and 131 MB together 25 us.
template <typename I, typename G, int KPT>
__global__ void __launch_bounds__(kSmallThreads) k_embed_sort_small(const I *__restrict__ ids, int n, uint32_t V,
                                                                    int passes, uint64_t *words, SortState *st,
                                                                    Clearing<G> clear) {
    constexpr int kWarps = kSmallThreads / 32;
    extern __shared__ uint32_t s_small[];
    uint32_t *s_key = s_small;                                            // [KPT * kSmallThreads]
    uint16_t *s_pos = reinterpret_cast<uint16_t *>(s_key + KPT * kSmallThreads);      // [KPT * kSmallThreads]
    uint16_t (*s_hist)[256] = reinterpret_cast<uint16_t (*)[256]>(s_pos + KPT * kSmallThreads);   // [kWarps][256]
    __shared__ uint32_t s_warp[kWarps], s_start[256], s_count;
    start_dependents();
    if (blockIdx.x > 0) {
        clear_share(clear, blockIdx.x - 1, gridDim.x - 1);
        return;
    }
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) s_count = 0;
    const uint32_t lt = lanes_below();
    // every warp has as many ids in turn, and no more than there are: a few
    // hundred take one step of eight
    const int per = (n + kSmallThreads - 1) / kSmallThreads * 32, used = per > 0 ? (n + per - 1) / per : 0;
    uint32_t key[KPT], pos[KPT];
    uint32_t named = 0;
#pragma unroll
    for (int j = 0; j < KPT; ++j) {
        const int i = j * 32 < per ? warp * per + j * 32 + lane : n;
        key[j] = i < n ? id_key(ids, i, V) : 0u;
        pos[j] = uint32_t(i);
        named += i < n && key[j] < V;
    }
    __syncthreads();
    named = __reduce_add_sync(0xffffffffu, named);
    if (lane == 0 && named) atomicAdd(&s_count, named);
    for (int d = 0; d < passes; ++d) {
        for (int e = tid; e < used * 128; e += kSmallThreads) reinterpret_cast<uint32_t *>(&s_hist[0][0])[e] = 0u;
        __syncthreads();
        uint32_t rank[KPT];
#pragma unroll
        for (int j = 0; j < KPT; ++j) {
            if (j * 32 >= per || warp >= used) break;
            const bool ok = warp * per + j * 32 + lane < n;
            const uint32_t dig = (key[j] >> (8 * d)) & 255u;
            const uint32_t peers = same_digit<8>(dig, ok);
            const uint32_t before = __popc(peers & lt);
            const uint32_t cur = ok ? s_hist[warp][dig] : 0u;
            rank[j] = cur + before;
            __syncwarp();
            if (ok && before == 0) s_hist[warp][dig] = uint16_t(cur + __popc(peers));
            __syncwarp();
        }
        __syncthreads();
        uint32_t total = 0;
        if (tid < 256) {
            uint32_t c[kWarps];            // all of a bin's counts at once, not one behind the other
#pragma unroll
            for (int w = 0; w < kWarps; ++w) c[w] = w < used ? s_hist[w][tid] : 0u;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                if (w < used) s_hist[w][tid] = uint16_t(total);
                total += c[w];
            }
        }
        const uint32_t start = excl_scan(total, s_warp);
        if (tid < 256) s_start[tid] = start;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < KPT; ++j)
            if (j * 32 < per && warp * per + j * 32 + lane < n) {
                const uint32_t dig = (key[j] >> (8 * d)) & 255u;
                const uint32_t to = s_start[dig] + s_hist[warp][dig] + rank[j];
                s_key[to] = key[j];
                s_pos[to] = uint16_t(pos[j]);
            }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < KPT; ++j) {
            const int i = j * 32 < per ? warp * per + j * 32 + lane : n;
            if (i < n) key[j] = s_key[i], pos[j] = s_pos[i];
        }
        __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < KPT; ++j) {
        const int i = j * 32 < per ? warp * per + j * 32 + lane : n;
        if (i < n) words[i] = uint64_t(key[j]) << 32 | pos[j];
    }
    if (tid == 0) st->count = int64_t(s_count), st->joins = 0;
}

// More ids: stable passes over digits of the key, least significant first,
// each a count of every partition's digits, a scan of the counts over the
// partitions, and a move.  Partitions do not wait on one another: a look-back
// from each to the ones before it is a chain of L2 round trips, and a pass
// over 2M ids took 41 us with it, 25 in the three launches.  Ids that name no
// row are not moved by the first pass.  2M ids of 12 bits: 35 us in all (two
// passes; the words stay in L2, and the launches' latencies and the votes for
// the ranks are what is left).
struct PassParams {
    const uint64_t *in;
    uint64_t *out;
    int64_t n;               // ids
    uint32_t V;
    int shift, bits;         // the digit
    int parts;
    bool first;
    uint32_t *counts;        // [bins][parts, to a multiple of 4]: of the digit in each partition; where there
                             // are more than kFewParts, k_embed_scan makes them exclusive sums
    int row;                 // of counts
    uint32_t *totals;        // [bins]
    SortState *st;
};

// Words of a pass: the ids themselves in the first, else what the first moved.
__device__ __forceinline__ int64_t pass_size(const PassParams &p) { return p.first ? p.n : p.st->count; }

template <typename I>
__device__ __forceinline__ uint64_t word_at(const PassParams &p, const I *ids, int64_t i) {
    return p.first ? uint64_t(id_key(ids, i, p.V)) << 32 | uint32_t(i) : p.in[i];
}

template <typename I, typename G>
__global__ void __launch_bounds__(kThreads) k_embed_count(const I *__restrict__ ids, PassParams p, Clearing<G> clear) {
    __shared__ uint32_t s_hist[1 << kMaxBits];
    start_dependents();
    if (int(blockIdx.x) >= p.parts) {
        wait_for_previous();
        clear_share(clear, blockIdx.x - p.parts, gridDim.x - p.parts);
        return;
    }
    const int bins = 1 << p.bits;
    for (int k = threadIdx.x; k < bins; k += kThreads) s_hist[k] = 0u;
    wait_for_previous();
    __syncthreads();
    const int64_t n = pass_size(p), base = int64_t(blockIdx.x) * kPart;
    uint32_t key[kKpt];
#pragma unroll
    for (int j = 0; j < kKpt; ++j) {
        const int64_t i = base + j * kThreads + threadIdx.x;
        key[j] = i < n ? uint32_t(word_at(p, ids, i) >> 32) : p.V;
    }
#pragma unroll
    for (int j = 0; j < kKpt; ++j)
        if (key[j] < p.V) atomicAdd(&s_hist[(key[j] >> p.shift) & uint32_t(bins - 1)], 1u);
    __syncthreads();
    for (int k = threadIdx.x; k < bins; k += kThreads) p.counts[int64_t(k) * p.row + blockIdx.x] = s_hist[k];
}

// A CTA for each bin: exclusive sums of its counts over the partitions.
template <typename G>
__global__ void __launch_bounds__(kThreads) k_embed_scan(PassParams p, Clearing<G> clear) {
    __shared__ uint32_t s_warp[kThreads / 32];
    const int bins = 1 << p.bits;
    start_dependents();
    wait_for_previous();
    if (int(blockIdx.x) >= bins) {
        clear_share(clear, blockIdx.x - bins, gridDim.x - bins);
        return;
    }
    uint32_t *c = p.counts + int64_t(blockIdx.x) * p.row;
    uint32_t run = 0;
    for (int q0 = 0; q0 < p.parts; q0 += kThreads * 4) {
        uint32_t v[4], mine = 0;           // four neighbours a thread
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int q = q0 + threadIdx.x * 4 + u;
            v[u] = q < p.parts ? c[q] : 0u;
            mine += v[u];
        }
        const uint32_t before = excl_scan(mine, s_warp);
        uint32_t at = run + before;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int q = q0 + threadIdx.x * 4 + u;
            if (q < p.parts) c[q] = at;
            at += v[u];
        }
        __syncthreads();
        if (threadIdx.x == kThreads - 1) s_warp[0] = before + mine;
        __syncthreads();
        run += s_warp[0];
    }
    if (threadIdx.x == 0) p.totals[blockIdx.x] = run;
}

template <typename I, typename G, int BITS>
__global__ void __launch_bounds__(kThreads) k_embed_move(const I *__restrict__ ids, PassParams p, Clearing<G> clear) {
    extern __shared__ uint64_t s_words[];                                        // [kPart]
    uint16_t *s_hist = reinterpret_cast<uint16_t *>(s_words + kPart);            // [8 warps][bins]
    constexpr int bins = 1 << BITS;
    uint32_t *s_lstart = reinterpret_cast<uint32_t *>(s_hist + 8 * bins);        // [bins] starts in this partition
    uint32_t *s_gbase = s_lstart + bins;                                         // [bins] destinations less starts
    __shared__ uint32_t s_warp[8];
    start_dependents();
    if (int(blockIdx.x) >= p.parts) {
        wait_for_previous();
        clear_share(clear, blockIdx.x - p.parts, gridDim.x - p.parts);
        return;
    }
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int k = tid; k < 4 * bins; k += kThreads) reinterpret_cast<uint32_t *>(s_hist)[k] = 0u;
    wait_for_previous();
    __syncthreads();
    const int64_t n = pass_size(p), base = int64_t(blockIdx.x) * kPart, wbase = base + warp * (kKpt * 32);
    const int shift = 32 + p.shift;
    constexpr uint32_t mask = uint32_t(bins - 1);
    uint64_t word[kKpt];
#pragma unroll
    for (int j = 0; j < kKpt; ++j) {
        const int64_t i = wbase + j * 32 + lane;
        word[j] = i < n ? word_at(p, ids, i) : ~0ull;
    }
    const uint32_t lt = lanes_below();
    uint16_t *mine = s_hist + warp * bins;
    uint32_t rank[kKpt];
#pragma unroll
    for (int j = 0; j < kKpt; ++j) {
        const bool ok = uint32_t(word[j] >> 32) < p.V;
        const uint32_t dig = uint32_t(word[j] >> shift) & mask;
        const uint32_t peers = same_digit<BITS>(dig, ok);
        const uint32_t before = __popc(peers & lt);
        const uint32_t cur = ok ? mine[dig] : 0u;
        rank[j] = cur + before;
        __syncwarp();
        if (ok && before == 0) mine[dig] = uint16_t(cur + __popc(peers));
        __syncwarp();
    }
    __syncthreads();
    // a thread a bin: the warps' starts in it, the partition's start, the destination
    uint32_t total = 0, all = 0, earlier = 0;
    if (tid < bins) {
        const uint32_t *c = p.counts + int64_t(tid) * p.row;
        if (p.parts <= kFewParts) {
            uint4 v[kFewParts / 4];
#pragma unroll
            for (int q = 0; q < kFewParts; q += 4)
                v[q / 4] = q < p.parts ? *reinterpret_cast<const uint4 *>(c + q) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int q = 0; q < kFewParts; ++q) {
                const uint4 f = v[q / 4];
                const uint32_t x = q % 4 == 0 ? f.x : (q % 4 == 1 ? f.y : (q % 4 == 2 ? f.z : f.w));
                if (q < p.parts) all += x;
                if (q < int(blockIdx.x)) earlier += x;
            }
        } else {
            all = p.totals[tid];
            earlier = c[blockIdx.x];
        }
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            const uint32_t m = s_hist[w * bins + tid];
            s_hist[w * bins + tid] = uint16_t(total);
            total += m;
        }
    }
    const uint32_t ls = excl_scan(total, s_warp), gs = excl_scan(all, s_warp);
    if (tid < bins) s_lstart[tid] = ls, s_gbase[tid] = gs + earlier - ls;
    __syncthreads();
    if (tid == kThreads - 1) s_warp[0] = ls + total, s_warp[1] = gs + all;   // the sums of all bins
    __syncthreads();
    const uint32_t local = s_warp[0], global = s_warp[1];
    if (p.first && blockIdx.x == 0 && tid == 0) p.st->count = int64_t(global), p.st->joins = 0;
#pragma unroll
    for (int j = 0; j < kKpt; ++j)
        if (uint32_t(word[j] >> 32) < p.V) {
            const uint32_t dig = uint32_t(word[j] >> shift) & mask;
            s_words[s_lstart[dig] + mine[dig] + rank[j]] = word[j];
        }
    __syncthreads();
    for (int i = tid; i < int(local); i += kThreads) {
        const uint64_t w = s_words[i];
        p.out[s_gbase[uint32_t(w >> shift) & mask] + uint32_t(i)] = w;
    }
}

// ------------------------------------------------------------------ sums

// Chunks of the sorted words, one a CTA: `groups` walks side by side, each by
// `cols` threads that own a vector of columns.  An id that lies inside one
// walk is finished there.  One that goes on over walks leaves a sum in shared
// memory at the end of each, which the thread of the walk where it begins
// adds in order; one that goes on over chunks leaves them in `head` and
// `tail`, for k_embed_join.  Every row of dout is read once, in the order of
// the ids: 2M rows of 192 bytes (384 MB) in about 70 us, 5.5 TB/s.
// Flags of a walk or chunk: its first id began before it, its last goes on
// after it, one id fills it and does both; of every kBlock-th walk: one id
// fills it and the walks up to the next of those.
enum : uint32_t { kIn = 1u, kOn = 2u, kWhole = 4u, kFilled = 8u };
constexpr int kBlock = 16;
struct SumParams {
    const uint64_t *words;   // sorted id << 32 | position
    SortState *st;
    int64_t n, chunk;        // ids; words of a CTA = groups * walk
    uint32_t V;
    int32_t D;
    int walk, groups, cols;
    int vecs;                // vectors of a row; a thread owns every cols-th of its CTA's slice
    int64_t in_stride, out_stride;
    float scale;
    float *head, *tail;      // [chunks][D]
    uint32_t *flags;         // [chunks]
    uint32_t *list;          // chunks whose last id goes on after them and began in them
    const void *ids;         // a tiny batch's, sorted by the sum's own CTAs (else NULL)
    int id_bytes;
};

__device__ __forceinline__ uint32_t key_of(const uint64_t *words, int64_t i) { return uint32_t(words[i] >> 32); }

// A vector of a row that is read once and whose neighbours are not: no line
// in L1, and no more of its L2 line than the 64 bytes it lies in (by default
// the rest of the line comes too, 489 MB for the 384 of 2M rows of 192 bytes:
// 118 us for the whole gradient, 109 so).
template <typename T, int N>
__device__ __forceinline__ Vec<T, N> load_once(const T *p) {
    if constexpr (N * sizeof(T) == 16) {
        Vec<T, N> x;
        asm volatile("ld.global.nc.L1::no_allocate.L2::64B.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(x.w[0]), "=r"(x.w[1]), "=r"(x.w[2]), "=r"(x.w[3])
                     : "l"(p));
        return x;
    } else {
        return load_vec<T, N>(p);
    }
}

// Vector k of a thread: column col0 + k * cols (in vectors).
template <typename G, int N, int K>
__device__ __forceinline__ void finish_row(const SumParams &p, G *dtable, uint32_t key, int col0, const float (&acc)[K][N]) {
    if (key >= p.V) return;
    G *row = dtable + int64_t(key) * p.out_stride;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (col0 + k * p.cols >= p.vecs) continue;
        float f[N];
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = acc[k][i] * p.scale;
        store_floats<G, N>(row + (col0 + k * p.cols) * N, f);
    }
}

// A tiny batch, one id a thread at most: every CTA of the sum (a slice of the
// columns) puts the words in order by itself, each word's place being the
// number of smaller ones, and clears its columns of dtable; the sort's launch
// and its end are spared (256 x 48 float32 into 1000 rows: 8.3 us with a sort,
// 6.5 so; 200 x 700 into 1000 rows: 9.8 and 6.1).  The slices are narrow, for
// short walks and little to clear, but no narrower than a sector.
constexpr int kTinyN = kThreads;
constexpr int64_t kTinyClearing = 16 << 10;    // bytes of a slice, if it can be that narrow,
constexpr int64_t kTinyMost = 64 << 10;        // and at most (128 KB: 10.3 us a call against 9.7; 192 KB: 13 against 8)
template <typename G, int N, int K>
__device__ __forceinline__ int tiny_sort(const SumParams &p, uint64_t *s_sorted, G *dtable, int g, int col0) {
    __shared__ uint64_t s_raw[kTinyN];
    const int t = threadIdx.x, n = int(p.n);
    uint32_t mine = 0;
    for (int i = t; i < kTinyN; i += blockDim.x) {      // the CTA may have fewer threads
        uint64_t w = ~0ull;
        if (i < n) {
            const uint32_t key = p.id_bytes == 4 ? id_key(static_cast<const int32_t *>(p.ids), i, p.V)
                                                 : id_key(static_cast<const int64_t *>(p.ids), i, p.V);
            w = uint64_t(key) << 32 | uint32_t(i);
            mine += key < p.V;
        }
        s_raw[i] = w;
    }
    for (int64_t r = g; r < int64_t(p.V); r += p.groups)
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (col0 + k * p.cols < p.vecs) {
                const float zero[N] = {};
                store_floats<G, N>(dtable + r * p.out_stride + (col0 + k * p.cols) * N, zero);
            }
    __syncthreads();                       // the words are there, and the rows cleared before any is summed
    for (int i = t; i < n; i += blockDim.x) {
        const uint64_t w = s_raw[i];
        int place = 0;
#pragma unroll 16
        for (int j = 0; j < n; ++j) place += s_raw[j] < w;
        s_sorted[place] = w;
    }
    __shared__ int s_count;
    if (t == 0) s_count = 0;
    __syncthreads();
    if (mine) atomicAdd(&s_count, int(mine));
    __syncthreads();
    return s_count;
}

template <typename T, typename G, int N, int K>
__global__ void __launch_bounds__(kThreads, 2) k_embed_sum(SumParams p, const T *__restrict__ dout, G *dtable) {
    extern __shared__ float s_part[];      // head then tail: [K * N][threads], blocks [K * N][blocks * cols], flags [groups]
    constexpr int kBatch = 8;
    const int g = threadIdx.x / p.cols, c = threadIdx.x - g * p.cols;
    const int col0 = blockIdx.y * p.cols * K + c, threads = blockDim.x;
    // where a thread's several vectors are read: one past the row's end reads another in its place, and
    // what it adds up is never stored (with a test for each load 20,000 x 2503 bfloat16 took 88 us, 81 so)
    const int first = col0 < p.vecs ? col0 * N : 0;
    int ahead[K];
#pragma unroll
    for (int k = 0; k < K; ++k) ahead[k] = col0 + k * p.cols < p.vecs ? k * p.cols * N : 0;
    float *head = s_part + threadIdx.x;
    float *tail = head + size_t(threads) * K * N;
    const int blocks = (p.groups + kBlock - 1) / kBlock, across = blocks * p.cols;
    float *s_block = s_part + size_t(threads) * K * N * 2;
    uint32_t *s_flags = reinterpret_cast<uint32_t *>(s_block + size_t(across) * K * N);
    auto put = [&](float *to, const float (&v)[K][N]) {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < N; ++i) to[(k * N + i) * threads] = v[k][i];
    };
    __shared__ uint64_t s_sorted[kTinyN];
    const uint64_t *words = p.words;
    int64_t n;
    if (p.ids) {
        n = tiny_sort<G, N, K>(p, s_sorted, dtable, g, col0);
        words = s_sorted;
    } else {
        start_dependents();
        wait_for_previous();
        n = p.st->count < p.n ? p.st->count : p.n;
    }
    const int64_t lo = int64_t(blockIdx.x) * p.chunk + int64_t(g) * p.walk;
    const int64_t hi = lo + p.walk < n ? lo + p.walk : n;
    uint32_t flags = 0, cur = 0;
    float acc[K][N];
    auto clear = [&] {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < N; ++i) acc[k][i] = 0.0f;
    };
    clear();
    if (lo < hi) {
        uint64_t w[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) w[u] = lo + u < hi ? words[lo + u] : ~0ull;
        cur = uint32_t(w[0] >> 32);
        bool open = lo > 0 && key_of(words, lo - 1) == cur;   // the current id began before this walk
        const uint32_t after = hi < n ? key_of(words, hi) : p.V;
        flags = open ? kIn : 0u;
        for (int64_t i = lo; i < hi; i += kBatch) {
            Vec<T, N> x[kBatch][K];
            uint32_t key[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const uint32_t pos = uint32_t(w[u]);
                key[u] = uint32_t(w[u] >> 32);
                const T *row = dout + int64_t(pos) * p.in_stride + (K == 1 ? col0 * N : first);
                const bool here = key[u] < p.V && int64_t(pos) < p.n;
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    x[u][k].clear();
                    if constexpr (K == 1) {
                        if (here && col0 < p.vecs) x[u][0] = load_once<T, N>(row);
                    } else {
                        if (here) x[u][k] = load_once<T, N>(row + ahead[k]);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u)              // the next words, while the rows arrive
                w[u] = i + kBatch + u < hi ? words[i + kBatch + u] : ~0ull;
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                if (i + u >= hi) break;
                if (key[u] != cur) {
                    if (open)
                        put(head, acc);
                    else
                        finish_row<G, N, K>(p, dtable, cur, col0, acc);
                    open = false;
                    cur = key[u];
                    clear();
                }
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int e = 0; e < N; ++e) acc[k][e] += x[u][k].get(e);
            }
        }
        const bool on = hi < n && after == cur;
        flags |= (on ? kOn : 0u) | (open && on ? kWhole : 0u);
        if (open)
            put(head, acc);
        else if (on)
            put(tail, acc);
        else
            finish_row<G, N, K>(p, dtable, cur, col0, acc);
    }
    if (c == 0) s_flags[g] = flags;
    __syncthreads();
    if (p.groups > kBlock) {               // sums of the blocks of walks that one id fills
        if (g % kBlock == 0 && g + kBlock <= p.groups) {
            bool whole = true;
            clear();
            for (int h = 0; h < kBlock; ++h) {
                whole = whole && (s_flags[g + h] & kWhole);
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int e = 0; e < N; ++e) acc[k][e] += head[(k * N + e) * threads + h * p.cols];
            }
            float *to = s_block + g / kBlock * p.cols + c;
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int e = 0; e < N; ++e) to[(k * N + e) * across] = acc[k][e];
            if (whole) flags |= kFilled;
        }
        __syncthreads();
        if (c == 0 && (flags & kFilled)) s_flags[g] = flags;
        __syncthreads();
    }
    if (lo >= hi) return;
    for (int pass = 0; pass < 2; ++pass) {
        const bool incoming = pass == 0;   // the id that the chunk before began: walk 0's threads
        if (incoming ? !(g == 0 && (flags & kIn)) : (flags & (kOn | kWhole)) != kOn) continue;
        const float *own = incoming ? head : tail;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < N; ++e) acc[k][e] = own[(k * N + e) * threads];
        bool on = incoming ? (flags & kWhole) != 0 : true;
        for (int h = g + 1; on && h < p.groups;) {
            const uint32_t f = s_flags[h];
            const bool all = (f & kFilled) != 0;         // a block at a time
            const float *from = all ? s_block + h / kBlock * p.cols + c : s_part + h * p.cols + c;
            const int apart = all ? across : threads;
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int e = 0; e < N; ++e) acc[k][e] += from[(k * N + e) * apart];
            on = (f & kWhole) != 0;
            h += all ? kBlock : 1;
        }
        if (incoming || on) {
            float *to = (incoming ? p.head : p.tail) + size_t(blockIdx.x) * p.D;
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (col0 + k * p.cols < p.vecs) store_floats<float, N>(to + (col0 + k * p.cols) * N, acc[k]);
            if (!incoming && c == 0 && blockIdx.y == 0) p.list[atomicAdd(&p.st->joins, 1u)] = blockIdx.x;
        } else {
            finish_row<G, N, K>(p, dtable, cur, col0, acc);
        }
    }
    if (c == 0 && blockIdx.y == 0 && !p.ids && (hi == n || g == p.groups - 1)) {
        // the chunk's last walk: one id fills the chunk if every walk is whole
        bool whole = true;
        for (int h = 0; h <= g; ++h) whole = whole && (s_flags[h] & kWhole);
        p.flags[blockIdx.x] = (s_flags[0] & kIn) | (flags & kOn) | (whole ? kWhole : 0u);
    }
}

// The ids that cross chunks (in whatever order the sums found them: each is
// its own task, and so is each slice of its columns).  A task's walks of
// threads take every groups-th chunk and then join in order.  (Four columns a
// thread spill 8 bytes.)
template <typename G, int N>
__global__ void __launch_bounds__(kThreads) k_embed_join(SumParams p, int chunks, int cols, int slices, G *dtable) {
    __shared__ float s_acc[N][kThreads];
    __shared__ int s_first;
    wait_for_previous();
    const int64_t tasks = int64_t(p.st->joins) * slices;
    const int vecs = p.D / N, groups = kThreads / cols;
    const int g = threadIdx.x / cols, c = threadIdx.x - g * cols;
    for (int64_t task = blockIdx.x; task < tasks; task += gridDim.x) {
        const int chunk = int(p.list[task / slices]), col = int(task % slices) * cols + c;
        const uint32_t key = key_of(p.words, (int64_t(chunk) + 1) * p.chunk - 1);
        int last = chunk + 1;              // the first of the chunks after this one that the id does not fill
        for (;; last += kThreads) {
            const int q = last + int(threadIdx.x);
            const bool ends = q >= chunks || !(p.flags[q] & kWhole);
            if (threadIdx.x == 0) s_first = kThreads;
            __syncthreads();
            if (ends) atomicMin(&s_first, int(threadIdx.x));
            __syncthreads();
            const int first = s_first;
            __syncthreads();
            if (first < kThreads) {
                last += first;
                break;
            }
        }
        if (last >= chunks) last = chunks - 1;
        const bool live = g < groups && col < vecs;
        float acc[N];
#pragma unroll
        for (int k = 0; k < N; ++k) acc[k] = 0.0f;
        if (live) {
            if (g == 0) {
                const Vec<float, N> x = load_vec<float, N>(p.tail + size_t(chunk) * p.D + col * N);
#pragma unroll
                for (int k = 0; k < N; ++k) acc[k] = x.get(k);
            }
#pragma unroll 8
            for (int q = chunk + 1 + g; q <= last; q += groups) {
                const Vec<float, N> x = load_vec<float, N>(p.head + size_t(q) * p.D + col * N);
#pragma unroll
                for (int k = 0; k < N; ++k) acc[k] += x.get(k);
            }
        }
#pragma unroll
        for (int k = 0; k < N; ++k) s_acc[k][threadIdx.x] = acc[k];
        __syncthreads();
        if (live && g == 0) {
            for (int h = 1; h < groups; ++h)
#pragma unroll
                for (int k = 0; k < N; ++k) acc[k] += s_acc[k][h * cols + c];
#pragma unroll
            for (int k = 0; k < N; ++k)
                dtable[int64_t(key) * p.out_stride + col * N + k] = from_float<G>(acc[k] * p.scale);
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------ host

bool sizes_ok(int64_t n, int64_t V, int32_t D) {
    return n >= 0 && n < (int64_t(1) << 30) && V >= 1 && V < (int64_t(1) << 31) && D >= 1 && D <= kMaxD;
}

int bits_of(int64_t v) {                   // of the numbers below v
    int b = 0;
    while (b < 32 && (int64_t(1) << b) < v) ++b;
    return b;
}

// Passes over `bits` bits of the key, and the bits of each.
int passes_of(int bits) { return bits < 1 ? 1 : (bits + kMaxBits - 1) / kMaxBits; }
int digit_of(int bits) {                   // 6 or 8 (10 would spare a pass of 17 to 20 bits, and takes
    const int p = passes_of(bits);         // twice the time in each: 2M ids, 27 us against 14)
    return (bits + p - 1) / p <= 6 ? 6 : 8;
}

struct SumShape {
    int vecs, cols, groups, slices, walk;
    int64_t chunk, chunks;
};

// Columns over threads: a row's vectors side by side, as many walks as fit in
// a CTA.  A walk is as long as gives every SM its two CTAs once (2M x 48: with
// walks of a quarter, several CTAs after one another, the gradient took 7 us
// more), or a little longer where that spares the join.
// Vectors of a row in one thread, so that what each word costs beside its
// values (its key, its place) is spread over a few of them.
constexpr int vectors_of(int vec, int bytes) {
    return vec >= 4 ? 1 : (vec == 2 && bytes == 4 ? 2 : 4);
}

SumShape sum_shape(int64_t n, int32_t D, int vec, int bytes, int slices = 1) {
    SumShape s;
    s.vecs = D / vec;
    const int own = vectors_of(vec, bytes), most = kThreads * own;
    s.slices = (s.vecs + most - 1) / most;
    if (s.slices < slices) s.slices = slices;
    s.cols = ((s.vecs + s.slices - 1) / s.slices + own - 1) / own;
    s.groups = kThreads / s.cols;
    const int64_t w = n * s.slices / (int64_t(s.groups) * 152 * 2);
    s.walk = int(w < 8 ? 8 : (w > 512 ? 512 : (w + 7) / 8 * 8));
    if (n <= int64_t(s.groups) * 32) s.walk = int((n + s.groups * 8 - 1) / (s.groups * 8)) * 8;   // one chunk: no join
    if (s.walk < 8) s.walk = 8;
    s.chunk = int64_t(s.groups) * s.walk;
    s.chunks = (n + s.chunk - 1) / s.chunk;
    return s;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct BwdLayout {
    size_t totals, counts, words, flags, list, head, tail, total;
    int parts;
};

BwdLayout bwd_layout(int64_t n, int64_t V, int32_t D) {
    BwdLayout L;
    const size_t bins = size_t(1) << digit_of(bits_of(V));
    L.parts = int((n + kPart - 1) / kPart);
    L.totals = align256(sizeof(SortState));
    L.counts = align256(L.totals + bins * 4);
    L.words = align256(L.counts + (n > kSmallN ? bins * ((L.parts + 3) / 4 * 4) * 4 : 0));
    L.flags = align256(L.words + size_t(n) * 16);
    int64_t chunks = 0;                    // of whichever type and vector width the call has
    for (int vec = 1; vec <= 8; vec *= 2)
        for (int bytes = 2; bytes <= 4; bytes += 2)
            if (D % vec == 0 && vec * bytes <= 16) {
                const SumShape s = sum_shape(n, D, vec, bytes);
                if (s.chunks > chunks) chunks = s.chunks;
            }
    L.list = align256(L.flags + size_t(chunks) * 4);
    L.head = align256(L.list + size_t(chunks) * 4);
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

// The most elements that one access may take: every row of both tensors
// starts and ends on such a boundary.
int access_bytes(const void *a, int64_t a_row, const void *b, int64_t b_row, int64_t row) {
    const uint64_t all = reinterpret_cast<uintptr_t>(a) | uint64_t(a_row) | reinterpret_cast<uintptr_t>(b) |
                         uint64_t(b_row) | uint64_t(row);
    return all % 16 == 0 ? 16 : (all % 8 == 0 ? 8 : (all % 4 == 0 ? 4 : 2));
}

template <typename T, typename I, int N>
void launch_fwd_n(const void *table, int64_t ts, int64_t V, int32_t D, const void *ids, int64_t n, float scale,
                  void *out, int64_t os, cudaStream_t s) {
    const int vecs = D / N;
    int shift = 0;                         // up to four vectors a lane, at least 4 lanes, at most a warp
    while ((1 << shift) < 32 && (1 << shift) * 4 < vecs) ++shift;
    while (shift < 2 && (1 << shift) < vecs) ++shift;
    // too few rows to fill the device so: more lanes, and a row at a time
    const bool few = (n << shift) < int64_t(kThreads) * 152 * 4;
    while (few && (1 << shift) < kThreads && (1 << shift) < vecs) ++shift;
    const int nv = (vecs + (1 << shift) - 1) >> shift;
    // what L2 could not keep anyway leaves room in it for the table (2M x 48 float32: 66 us, 72 without)
    const bool leave = n * D * int64_t(sizeof(T)) > kManyBytes;
    auto go = [&](auto NV, auto ROWS) {
        constexpr int kNv = decltype(NV)::value, kRows = decltype(ROWS)::value;
        const int64_t per = int64_t(kThreads >> shift) * kRows;
        // (a row of a warp that has few of them has three or four vectors a lane)
        auto kernel = kNv >= 3 && shift == 5 ? k_embed_fwd<T, I, N, kNv, kRows, (kNv >= 3)>
                                             : k_embed_fwd<T, I, N, kNv, kRows, false>;
        SS_LAUNCH("k_embed_fwd", s,
                  kernel<<<unsigned((n + per - 1) / per), kThreads, 0, s>>>(
                      static_cast<const T *>(table), ts, V, static_cast<const I *>(ids), n, scale,
                      static_cast<T *>(out), os, shift, vecs, leave));
    };
    // several rows at a time where one brings a thread little to wait for (1M x 33 float16: 53 us with
    // two; with four, and more registers, 67)
    auto rows = [&](auto NV) {
        constexpr int kBytes = decltype(NV)::value * N * int(sizeof(T));
        if (few) return go(NV, std::integral_constant<int, 1>{});
        go(NV, std::integral_constant<int, (kBytes >= 24 ? 1 : (kBytes >= 12 ? 2 : 4))>{});
    };
    if (nv == 1) rows(std::integral_constant<int, 1>{});
    else if (nv == 2) rows(std::integral_constant<int, 2>{});
    else if (nv == 3) rows(std::integral_constant<int, 3>{});
    else rows(std::integral_constant<int, 4>{});
}

template <typename T, typename I>
void launch_fwd(const void *table, int64_t ts, int64_t V, int32_t D, const void *ids, int64_t n, float scale,
                void *out, int64_t os, cudaStream_t s) {
    const int b = access_bytes(table, ts * sizeof(T), out, os * sizeof(T), int64_t(D) * sizeof(T));
    constexpr int E = sizeof(T);
    if (b == 16) launch_fwd_n<T, I, 16 / E>(table, ts, V, D, ids, n, scale, out, os, s);
    else if (b == 8) launch_fwd_n<T, I, 8 / E>(table, ts, V, D, ids, n, scale, out, os, s);
    else if (b == 4) launch_fwd_n<T, I, 4 / E>(table, ts, V, D, ids, n, scale, out, os, s);
    else launch_fwd_n<T, I, 1>(table, ts, V, D, ids, n, scale, out, os, s);
}

template <typename T, typename G, int N>
void launch_sums(const SumParams &p, const SumShape &sh, const T *dout, G *dtable, int sms, cudaStream_t s) {
    const dim3 grid(unsigned(sh.chunks), unsigned(sh.slices));
    const int threads = sh.groups * sh.cols;
    constexpr int kOwn = vectors_of(N, sizeof(T));
    const size_t smem = (size_t(threads) * 2 + size_t((sh.groups + kBlock - 1) / kBlock) * sh.cols) * N * kOwn * 4 +
                        sh.groups * 4;
    if (p.ids) {                           // waits for all that is before it: it has no sort to overlap
        SS_LAUNCH("k_embed_sum", s, k_embed_sum<T, G, N, kOwn><<<grid, threads, smem, s>>>(p, dout, dtable));
        return;
    }
    SS_LAUNCH("k_embed_sum", s,
              launch_after(k_embed_sum<T, G, N, kOwn>, grid, threads, smem, s,
                           p, dout, dtable));
    if (sh.chunks > 1) {
        // slices of half a kilobyte: a long chain of sums is spread over eight walks at least
        constexpr int kJoin = N < 4 ? N : 4;
        const int vecs = p.D / kJoin, cols = vecs < 32 ? vecs : 32, slices = (vecs + cols - 1) / cols;
        const int64_t most = sh.chunks * slices;
        SS_LAUNCH("k_embed_join", s,
                  launch_after(k_embed_join<G, kJoin>, dim3(unsigned(most < sms * 8 ? most : sms * 8)), kThreads, 0, s, p,
                               int(sh.chunks), cols, slices, dtable));
    }
}

template <typename T, typename G, typename I>
ss_status launch_bwd(const void *dout, int64_t in_stride, const void *ids, int64_t n, int64_t V, int32_t D, float scale,
                     void *dtable, int64_t out_stride, char *ws, int sms, cudaStream_t s) {
    const BwdLayout L = bwd_layout(n, V, D);
    SortState *st = reinterpret_cast<SortState *>(ws);
    const I *id = static_cast<const I *>(ids);
    G *dt = static_cast<G *>(dtable);
    uint64_t *w[2] = {reinterpret_cast<uint64_t *>(ws + L.words), reinterpret_cast<uint64_t *>(ws + L.words) + n};
    Clearing<G> clear{dt, V, out_stride, D, 0, 1};
    // the gradient's rows are written in the vectors that dout's are read in (of 32 bytes in two halves)
    constexpr int E = sizeof(T);
    int b = access_bytes(dout, in_stride * E, dout, in_stride * E, int64_t(D) * E);
    for (; b > E; b /= 2) {
        const int64_t a = int64_t(b) / E * int64_t(sizeof(G)) < 16 ? int64_t(b) / E * int64_t(sizeof(G)) : 16;
        if (aligned_to(dtable, size_t(a)) && (out_stride * int64_t(sizeof(G))) % a == 0) break;
    }
    auto with_vector = [&](auto f) {
        if (b == 16) return f(std::integral_constant<int, 16 / E>{});
        if (b == 8) return f(std::integral_constant<int, 8 / E>{});
        if (b == 4 && E == 2) return f(std::integral_constant<int, E == 2 ? 2 : 1>{});
        return f(std::integral_constant<int, 1>{});
    };
    auto sums = [&](const uint64_t *sorted, int tiny) {
        return with_vector([&](auto NE) {
            constexpr int kN = decltype(NE)::value;
            const SumShape sh = sum_shape(n, D, kN, E, tiny);
            SumParams p{};
            p.words = sorted, p.st = st;
            p.n = n, p.chunk = sh.chunk, p.V = uint32_t(V), p.D = D, p.walk = sh.walk, p.groups = sh.groups;
            p.cols = sh.cols, p.vecs = sh.vecs, p.in_stride = in_stride, p.out_stride = out_stride, p.scale = scale;
            p.head = reinterpret_cast<float *>(ws + L.head), p.tail = reinterpret_cast<float *>(ws + L.tail);
            p.flags = reinterpret_cast<uint32_t *>(ws + L.flags), p.list = reinterpret_cast<uint32_t *>(ws + L.list);
            p.ids = tiny ? ids : nullptr, p.id_bytes = sizeof(I);
            launch_sums<T, G, kN>(p, sh, static_cast<const T *>(dout), dt, sms, s);
            return SS_OK;
        });
    };
    if (n > 0 && n <= kTinyN) {
        // slices of the columns, or 0 where a CTA would have too much to clear
        const int slices = with_vector([&](auto NE) {
            constexpr int kN = decltype(NE)::value, kOwn = vectors_of(kN, E);
            constexpr int64_t kBytes = kN * int64_t(sizeof(G)), kLeast = (32 + kBytes - 1) / kBytes;
            const int64_t vecs = D / kN;
            int64_t own = kTinyClearing / (V * kBytes);    // vectors of a slice that its CTA clears,
            if (own > 2048 / n * kOwn) own = 2048 / n * kOwn;      // and that leave a walk of eight ids
            if (own < (vecs + sms - 1) / sms) own = (vecs + sms - 1) / sms;
            if (own < kLeast) own = kLeast;
            own = (own + kOwn - 1) / kOwn * kOwn;
            if (own > vecs) own = vecs;
            const int slices = int((vecs + own - 1) / own);
            return V * own * kBytes <= kTinyMost && sum_shape(n, D, kN, E, slices).chunks == 1 ? slices : 0;
        });
        if (slices > 0) return sums(nullptr, slices);
    }
    // CTAs that clear: enough to draw on the whole bandwidth where there is much to clear
    const int64_t row_bytes = int64_t(D) * sizeof(G), bytes = V * (out_stride == D || row_bytes > 64 ? row_bytes : 64);
    const uint64_t *sorted = w[0];
    if (n <= kSmallN || (n <= kSmallMost && bytes >= kLongClearing)) {
        // (the whole gradient, one CTA against several launches: 8000 ids, 24.6 us and 20.3 beside 2 MB of
        // clearing, 25.5 and 23.8 beside 16, 25.9 and 27.2 beside 25, 34 and 38 beside 131; 4200 ids, 18.8 and
        // 18.3 beside 2 MB, 18.9 and 21.8 beside 16, so that fewer ids would gain from 8 MB on)
        const int want = int(bytes / (64 * 1024)) + 1, ctas = want < sms * 2 ? want : sms * 2;
        auto go = [&](auto KPT) {
            constexpr int kKpts = decltype(KPT)::value, kSmem = kKpts * kSmallThreads * 6 + kSmallThreads / 32 * 512;
            auto kernel = k_embed_sort_small<I, G, kKpts>;
            static std::atomic<unsigned long long> smem_ctx[kMaxDevices];   // see ensure_dyn_smem
            const void *fn = (const void *)kernel;
            const ss_status e = ensure_dyn_smem(smem_ctx, &fn, 1, kSmem, "ss_embed_bwd");
            if (e != SS_OK) return e;
            SS_LAUNCH("k_embed_sort_small", s,
                      kernel<<<1 + ctas, kSmallThreads, kSmem, s>>>(id, int(n), uint32_t(V), (bits_of(V + 1) + 7) / 8,
                                                                    w[0], st, clear));
            return SS_OK;
        };
        const ss_status e = n <= kSmallThreads ? go(std::integral_constant<int, 1>{})
                                               : (n <= kSmallN ? go(std::integral_constant<int, kSmallN / kSmallThreads>{})
                                                               : go(std::integral_constant<int, kSmallMost / kSmallThreads>{}));
        if (e != SS_OK) return e;
    } else {
        const int bits = bits_of(V), passes = passes_of(bits);
        PassParams p{};
        p.n = n, p.V = uint32_t(V), p.bits = digit_of(bits), p.parts = L.parts, p.row = (L.parts + 3) / 4 * 4;
        p.counts = reinterpret_cast<uint32_t *>(ws + L.counts), p.totals = reinterpret_cast<uint32_t *>(ws + L.totals);
        p.st = st;
        const bool scan = p.parts > kFewParts;
        clear.shares = (scan ? 3 : 2) * passes;
        const int64_t share = bytes / clear.shares;
        const int want = int(share / (32 * 1024) < 1 << 20 ? share / (32 * 1024) : 1 << 20) + 1;
        const int ctas = want < sms * 4 ? want : sms * 4;
        const size_t smem = size_t(kPart) * 8 + (size_t(8) << p.bits) * 2 + (size_t(2) << p.bits) * 4;
        auto move = p.bits == 6 ? k_embed_move<I, G, 6> : k_embed_move<I, G, 8>;
        static std::atomic<unsigned long long> smem_ctx[kMaxDevices];
        const void *fns[] = {(const void *)k_embed_move<I, G, 6>, (const void *)k_embed_move<I, G, 8>};
        const ss_status e = ensure_dyn_smem(smem_ctx, fns, 2, kPart * 8 + (8 << kMaxBits) * 2 + (2 << kMaxBits) * 4,
                                            "ss_embed_bwd");
        if (e != SS_OK) return e;
        for (int d = 0; d < passes; ++d) {
            p.first = d == 0, p.shift = d * p.bits, p.in = w[(d + 1) & 1], p.out = w[d & 1];
            if (d == 0)
                SS_LAUNCH("k_embed_count", s,
                          k_embed_count<I, G><<<p.parts + ctas, kThreads, 0, s>>>(id, p, clear));
            else
                SS_LAUNCH("k_embed_count", s,
                          launch_after(k_embed_count<I, G>, dim3(p.parts + ctas), kThreads, 0, s, id, p, clear));
            ++clear.share;
            if (scan) {
                SS_LAUNCH("k_embed_scan", s,
                          launch_after(k_embed_scan<G>, dim3((1 << p.bits) + ctas), kThreads, 0, s, p, clear));
                ++clear.share;
            }
            SS_LAUNCH("k_embed_move", s,
                      launch_after(move, dim3(p.parts + ctas), kThreads, smem, s, id, p, clear));
            ++clear.share;
        }
        sorted = w[(passes - 1) & 1];
    }
    if (n == 0) return SS_OK;
    return sums(sorted, 0);
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
    cudaStream_t s = (cudaStream_t)stream;
#define SS_FWD(T)                                                                                             \
    (id_bytes == 4 ? launch_fwd<T, int32_t>(table, table_stride, V, D, ids, n, scale, out, out_stride, s) \
                   : launch_fwd<T, int64_t>(table, table_stride, V, D, ids, n, scale, out, out_stride, s))
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

}  // extern "C"
