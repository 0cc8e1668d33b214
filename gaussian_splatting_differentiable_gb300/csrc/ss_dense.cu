// The weight gradient of a dense layer from its input kept in 8 bits (model:
// include/ss_dense.h; the method: ss_dense.cuh): weights of one tile or a few, and the
// joining of partial sums.
#include <cuda_runtime.h>

#include <atomic>
#include <climits>
#include <cstdint>
#include <type_traits>

#include "ss_dense.cuh"
#include "ss_dense.h"
#include "ss_internal.h"
#include "ss_profile.h"
#include "ss_rows8.cuh"
#include "ss_tensor.cuh"
#include "ss_unit.cuh"

namespace ss {
namespace {

// A weight of one tile, up to 128 x 128: rows come in faster than they are worked on, so all of
// dy and x pass once, and are converted on the way.  A CTA has a range of rows, stages of
// which go through a ring in shared memory.  Where dy and x lie on 16-byte boundaries (FAST), a thread
// has the copy engine bring them: a bfloat16 dy, which needs no change, to its place, all
// else to a ring of its own, out of which the loader warps convert it (other rows pass through
// their registers).  One thread of another
// warp issues the products; at the end the loaders read the sums out of the tensor memory.  A range is one
// chain.
//
// 2M x 48 x 48 (484 MB float32, 292 bfloat16): 135 us and 92 by ncu, at 3.7 and 3.3 TB/s.  In chains of 2816 rows 134
// and 84; there, through registers 145 and 86, without the conversions 95 and 77: what bounds it is the way of a stage
// through copies, barriers and products, of which shared memory has room for four at a time on an SM, and then the
// conversions.  (Stages of 32 rows: 156 us and more; three or four of them of raw rows ahead, or 128, 384 or 512
// loaders: nothing gained.)
//
// TI = 64 (N up to 64): two parts of dy side by side are the 128 rows of one product, so
// a float32 takes two products and not three; the parts' sums are joined through shared memory.
template <typename T, int TI, int TJ, int ROWS>
struct Config {
    static constexpr int kParts = parts_of<T>();
    static constexpr bool kStacked = TI == 64;
    static constexpr int kLoaders = 256;
    static constexpr int kThreads = kLoaders + 64;                  // and the warps of the products and of the copies
    static constexpr int kRows = ROWS;                              // of a stage
    static constexpr int kBlock = kRows * 128;                      // bytes of 64 columns of a stage
    static constexpr int kABlocks = kStacked ? (kParts + 1) / 2 * 2 : 2 * kParts;
    static constexpr int kPart = TI / 64 * kBlock;                  // bytes from one part to the next
    static constexpr int kABytes = kABlocks * kBlock, kBBytes = TJ / 64 * kBlock;
    static constexpr int kStageBytes = kABytes + kBBytes;
    static constexpr int kProducts = kABlocks / 2;                  // of 128 rows each, a step
    static constexpr int kSums = kStacked ? kProducts : (kParts > 1 ? 2 : 1);
    static constexpr int kStages = 2;
    static constexpr int kRawStages = 2;
    static constexpr int kTurnsA = kRows * (TI / kUnit) / kLoaders < 1 ? 1 : kRows * (TI / kUnit) / kLoaders;
    static constexpr int kTurnsB = kRows * (TJ / kWide) / kLoaders < 1 ? 1 : kRows * (TJ / kWide) / kLoaders;
    static constexpr int kColumns = kSums * TJ <= 64 ? 64 : (kSums * TJ <= 128 ? 128 : 256);   // of tensor memory
    static constexpr int kMinCtas = 2;
};

// Where a thread's pieces of W columns of a stage lie: `valid` of them a row, the threads
// one after the other along them, rows after rows; turn k's are k * rows rows on.  A
// thread without a piece has row ROWS.
template <int ROWS, int W>
struct Turns {
    int piece, row, rows;     // rows: of a turn
    __device__ __forceinline__ Turns(int thread, int threads, int valid) {
        rows = threads / valid;
        row = thread / valid, piece = thread - row * valid;
        if (row >= rows) piece = 0, row = ROWS;
    }
    // Of turn k's piece in an operand: 64 columns of a row, swizzled by 16 bytes.
    __device__ __forceinline__ uint32_t place(int k) const {
        const int r = row + k * rows, u = piece * (W / kUnit);
        return (u >> 3) * (ROWS * 128) + r * 128 + (((u ^ r) & 7) << 4);
    }
    __device__ __forceinline__ bool has(int k, int of) const { return row + k * rows < of; }
};

// A unit of dy as bfloat16s, a part APART bytes from the one before.
template <typename T, int APART>
__device__ __noinline__ void store_parts_special(uint32_t at, Raw<T> r) {
    uint32_t w[parts_of<T>()][4];
    cut_parts_special(w, r);
#pragma unroll
    for (int p = 0; p < parts_of<T>(); ++p) store16(at + p * APART, w[p]);
}
template <typename T, int APART>
__device__ __forceinline__ void store_parts(uint32_t at, const Raw<T> &r) {
    if constexpr (parts_of<T>() == 1) {
        store16(at, r.w);
    } else {
        F2 f[4];
        floats_of(f, r);
        if (any_special(f)) {
            store_parts_special<T, APART>(at, r);
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
}

// A stage of the ring of what is to be converted: rows of dy (in several parts), then of x.
struct RawStage {
    int dy_pitch, x_pitch, bytes;
};

template <typename T, int TI, int TJ, int ROWS, int FMT, bool FAST>
__global__ void __launch_bounds__(Config<T, TI, TJ, ROWS>::kThreads, Config<T, TI, TJ, ROWS>::kMinCtas)
    k_dense(DenseArgs a, int64_t rows, RawStage raw, const __grid_constant__ CUtensorMap dy_map,
            const __grid_constant__ CUtensorMap x_map) {
    using C = Config<T, TI, TJ, ROWS>;
    constexpr bool kCopies = FAST && C::kParts == 1;
    extern __shared__ uint8_t s_raw[];
    __shared__ uint64_t s_full[C::kStages], s_copied[C::kStages], s_empty[C::kStages], s_done;
    __shared__ uint64_t s_raw_full[C::kRawStages], s_raw_empty[C::kRawStages];
    __shared__ uint32_t s_tensor, s_failed;
    const uint32_t ring = (smem_of(s_raw) + 1023u) & ~1023u;
    uint8_t *ring_ptr = s_raw + (ring - smem_of(s_raw));
    const uint8_t *raw_ring = ring_ptr + C::kStages * C::kStageBytes;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ni = a.N, nj = a.D;
    const int64_t first = int64_t(blockIdx.x) * rows;
    const int64_t last = first + rows < a.n ? first + rows : a.n;
    const int stages = last > first ? int((last - first + C::kRows - 1) / C::kRows) : 0;
    const bool bias = a.db;

    if (threadIdx.x == 0) {
        s_failed = 0;
        for (int k = 0; k < C::kStages; ++k) {
            barrier_init(&s_full[k], C::kLoaders / 32);
            barrier_init(&s_copied[k], 1);
            barrier_init(&s_empty[k], 1);
        }
        for (int k = 0; k < C::kRawStages; ++k) barrier_init(&s_raw_full[k], 1), barrier_init(&s_raw_empty[k], C::kLoaders / 32);
        barrier_init(&s_done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == C::kLoaders / 32) {
        tensor_take<C::kColumns>(&s_tensor);
    }
    // (columns past the matrices hold anything: they make columns and rows of dW that nobody reads)
    tensor_fence_before();
    __syncthreads();
    tensor_fence_after();
    const uint32_t tensor = s_tensor;

    F2 sums[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[i] = both(0.0f);
    const Turns<C::kRows, kUnit> ta(threadIdx.x, C::kLoaders, (ni + kUnit - 1) / kUnit);
    // x from the other end of the threads: neither of the two takes all of them
    const Turns<C::kRows, kWide> tb(C::kLoaders - 1 - int(threadIdx.x), C::kLoaders, (nj + kWide - 1) / kWide);

    // The sums out of the tensor memory, to where they go.  A warp reads the 32 lanes
    // (rows of dW) of its quarter, the warps of a quarter 8 columns in turn.
    auto drain = [&] {
        const int quarter = warp & 3;
        const bool failed = *static_cast<volatile uint32_t *>(&s_failed) != 0;
        auto checked = [&](uint32_t (&v)[8]) {
            if (stages == 0 || failed)      // a wait that ran out leaves NaN
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = failed ? 0x7fffffffu : 0u;
        };
        if constexpr (C::kStacked && C::kParts > 1) {
            // parts [p][64 rows][32 columns] through the ring, 32 columns at a time
            constexpr int kPitch = 36;
            float *s = reinterpret_cast<float *>(ring_ptr);
            for (int c0 = 0; c0 < nj; c0 += 32) {
                asm volatile("bar.sync 1, %0;" ::"n"(C::kLoaders) : "memory");   // the ring's operands, or the columns before, are read
#pragma unroll 1
                for (int t = 0; t < C::kProducts; ++t) {
                    const int p = 2 * t + (quarter >> 1);
#pragma unroll 1
                    for (int c = (warp >> 2) * 8; c < 32; c += 16) {
                        uint32_t v[8];
                        __syncwarp();
                        tensor_load8(v, tensor + (uint32_t(quarter * 32) << 16) + t * TJ + c0 + c);
                        if (p >= C::kParts) continue;
                        checked(v);
                        float *to = s + (p * 64 + (quarter & 1) * 32 + lane) * kPitch + c;
                        *reinterpret_cast<uint4 *>(to) = make_uint4(v[0], v[1], v[2], v[3]);
                        *reinterpret_cast<uint4 *>(to + 4) = make_uint4(v[4], v[5], v[6], v[7]);
                    }
                }
                asm volatile("bar.sync 1, %0;" ::"n"(C::kLoaders) : "memory");
                const int i = threadIdx.x >> 2, c = (threadIdx.x & 3) * 8;
                if (i < ni && c0 + c < nj) {
                    uint32_t v[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        float t = s[i * kPitch + c + k];
#pragma unroll
                        for (int p = 1; p < C::kParts; ++p) t = joined(t, s[(p * 64 + i) * kPitch + c + k]);
                        v[k] = __float_as_uint(t);
                    }
                    put(a, blockIdx.x, i, c0 + c, nj - c0 - c < 8 ? nj - c0 - c : 8, v, true, true);
                }
            }
        } else {
            const int i = quarter * 32 + lane;
#pragma unroll 1
            for (int c = (warp >> 2) * 8; c < nj; c += C::kLoaders / 128 * 8) {
                uint32_t v[8];
                __syncwarp();
                tensor_load8(v, tensor + (uint32_t(quarter * 32) << 16) + c);
                if (C::kSums > 1) {
                    uint32_t w[8];
                    tensor_load8(w, tensor + (uint32_t(quarter * 32) << 16) + TJ + c);
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] = __float_as_uint(joined(__uint_as_float(v[k]), __uint_as_float(w[k])));
                }
                checked(v);
                if (i < ni) put(a, blockIdx.x, i, c, nj - c < 8 ? nj - c : 8, v, true, true);
            }
        }
    };
    if (warp < C::kLoaders / 32) {
        Raw<T> ra[C::kTurnsA];
        Wide rb[C::kTurnsB];
        const int ca = ni - ta.piece * kUnit < kUnit ? ni - ta.piece * kUnit : kUnit;
        const bool all = nj - tb.piece * kWide > kUnit;
        // the next stage to load: its pieces (FAST: x's scales), and how many of its rows there are
        const T *pa = static_cast<const T *>(a.dy) + (first + ta.row) * a.dys + ta.piece * kUnit;
        const uint8_t *pq = a.x.q + (first + tb.row) * a.x.stride + tb.piece * kWide;
        const uint8_t *ps = a.x.scales + (first + tb.row) * a.x.scale_stride + tb.piece / (kGroup / kWide);
        int64_t left = last - first;
        auto load = [&] {
            const int there = left < C::kRows ? int(left) : C::kRows;
            if (!FAST)
#pragma unroll
                for (int k = 0; k < C::kTurnsA; ++k)
                    if (ta.has(k, there))
                        ra[k] = load_unit<T, false>(pa + k * ta.rows * a.dys, ca);
                    else
                        ra[k].clear();
#pragma unroll
            for (int k = 0; k < C::kTurnsB; ++k) {
                if (FAST)
                    rb[k].e = tb.has(k, there) ? ps[k * tb.rows * a.x.scale_stride] : 127u;
                else if (tb.has(k, there))
                    rb[k].template load<false>(pq + k * tb.rows * a.x.stride, ps + k * tb.rows * a.x.scale_stride, all);
                else
                    rb[k] = Wide{{0u, 0u, 0u, 0u}, 127u};
            }
            pa += C::kRows * a.dys, pq += C::kRows * a.x.stride, ps += C::kRows * a.x.scale_stride;
            left -= C::kRows;
        };
        load();
        auto add_bias = [&](const Raw<T> &r) {
            F2 f[4];
            floats_of(f, r);
#pragma unroll
            for (int i = 0; i < 4; ++i) sums[i] = add2(sums[i], f[i]);
        };
        int slot = 0, raw_slot = 0;
        uint32_t parity = 1, raw_parity = 0;
        bool ok = true;
        for (int stage = 0; stage < stages; ++stage) {
            if (FAST) {
                ok &= barrier_wait(&s_raw_full[raw_slot], raw_parity, a.tries);
                const uint8_t *from = raw_ring + raw_slot * raw.bytes;
                if (!kCopies) {
#pragma unroll
                    for (int k = 0; k < C::kTurnsA; ++k)
                        if (ta.has(k, C::kRows)) {
                            const uint8_t *at = from + (ta.row + k * ta.rows) * raw.dy_pitch + ta.piece * int(kUnit * sizeof(T));
#pragma unroll
                            for (int v = 0; v < Raw<T>::kWords / 4; ++v) {
                                const uint4 u = reinterpret_cast<const uint4 *>(at)[v];
                                ra[k].w[4 * v] = u.x, ra[k].w[4 * v + 1] = u.y, ra[k].w[4 * v + 2] = u.z, ra[k].w[4 * v + 3] = u.w;
                            }
                        }
                    from += C::kRows * raw.dy_pitch;
                }
#pragma unroll
                for (int k = 0; k < C::kTurnsB; ++k)
                    if (tb.has(k, C::kRows)) load_words(rb[k].w, from + (tb.row + k * tb.rows) * raw.x_pitch + tb.piece * kWide);
            }
            // a warp's lanes go on together, or leave
            ok &= barrier_wait(&s_empty[slot], parity, a.tries);
            if (!__all_sync(0xffffffffu, ok)) {
                ok = false;
                break;
            }
            const uint32_t at = ring + slot * C::kStageBytes;
            if (!kCopies)
#pragma unroll
                for (int k = 0; k < C::kTurnsA; ++k) {
                    if (!ta.has(k, C::kRows)) continue;
                    store_parts<T, C::kPart>(at + ta.place(k), ra[k]);
                    if (bias) add_bias(ra[k]);
                }
#pragma unroll
            for (int k = 0; k < C::kTurnsB; ++k)
                if (tb.has(k, C::kRows)) {
                    uint32_t w[8];
                    convert<FMT>(w, rb[k]);
                    const uint32_t to = at + C::kABytes + tb.place(k);
                    store16(to, {w[0], w[1], w[2], w[3]});
                    store16(to ^ 16u, {w[4], w[5], w[6], w[7]});
                }
            if constexpr (kCopies)
                if (bias) {       // the copy engine's rows, before the slot may be filled again
                    if (!barrier_wait(&s_copied[slot], parity ^ 1, a.tries)) {
                        ok = false;
                        s_failed = 1;
                    }
#pragma unroll
                    for (int k = 0; k < C::kTurnsA; ++k)
                        if (ta.has(k, C::kRows)) {
                            load_words(ra[k].w, ring_ptr + slot * C::kStageBytes + ta.place(k));
                            add_bias(ra[k]);
                        }
                }
            writes_to_async();
            __syncwarp();
            if (lane == 0) {
                barrier_arrive(&s_full[slot]);
                if (FAST) barrier_arrive(&s_raw_empty[raw_slot]);
            }
            load();
            if (++slot == C::kStages) slot = 0, parity ^= 1;
            if (++raw_slot == C::kRawStages) raw_slot = 0, raw_parity ^= 1;
        }
        if (!barrier_wait(&s_done, 0, a.tries) || !ok) s_failed = 1;
        __syncwarp();
        tensor_fence_after();
        drain();
        tensor_fence_before();
    } else if (warp == C::kLoaders / 32) {
        if (lane == 0) {
            const uint32_t what = product_of((nj + 15) / 16 * 16);
            int slot = 0;
            uint32_t parity = 0;
            for (int stage = 0; stage < stages; ++stage) {
                if (!barrier_wait(&s_full[slot], parity, a.tries) || (kCopies && !barrier_wait(&s_copied[slot], parity, a.tries))) {
                    s_failed = 1;
                    __threadfence_block();      // before those that wait for s_done look at it
                    break;
                }
                tensor_fence_after();
                const uint32_t at = ring + slot * C::kStageBytes, bt = at + C::kABytes;
#pragma unroll
                for (int k = 0; k < C::kRows / kStep; ++k)
#pragma unroll
                    for (int p = 0; p < C::kProducts; ++p) {
                        const int set = C::kStacked ? p : (p > 0 ? 1 : 0);
                        product(tensor + set * TJ, operand_at<C::kBlock>(at + p * 2 * C::kBlock + k * kStep * 128),
                                operand_at<C::kBlock>(bt + k * kStep * 128), what,
                                stage > 0 || k > 0 || (!C::kStacked && p > 1));
                    }
                products_arrive(&s_empty[slot]);
                if (++slot == C::kStages) slot = 0, parity ^= 1;
            }
            products_arrive(&s_done);
            if (!barrier_wait(&s_done, 0, a.tries)) s_failed = 1;    // the tensor memory is freed after them
        }
        __syncwarp();
    } else {
        if (FAST && lane == 0) {
            const int boxes = (ni + 63) / 64;
            const uint32_t raw_at = ring + C::kStages * C::kStageBytes;
            int slot = 0, raw_slot = 0, stage = 0, copied = 0;
            uint32_t parity = 1, raw_parity = 1;
            for (; stage < stages && stage < a.sent; ++stage) {
                const int row = int(first + int64_t(stage) * C::kRows);
                if (!barrier_wait(&s_raw_empty[raw_slot], raw_parity, a.tries)) {
                    s_failed = 1;
                    break;
                }
                uint32_t to = raw_at + raw_slot * raw.bytes;
                barrier_expect(&s_raw_full[raw_slot], raw.bytes);
                if (!kCopies) {
                    copy_box(to, &dy_map, 0, row, &s_raw_full[raw_slot]);
                    to += C::kRows * raw.dy_pitch;
                }
                copy_box(to, &x_map, 0, row, &s_raw_full[raw_slot]);
                if (++raw_slot == C::kRawStages) raw_slot = 0, raw_parity ^= 1;
                if (kCopies) {
                    if (!barrier_wait(&s_empty[slot], parity, a.tries)) {
                        s_failed = 1;
                        ++stage;
                        break;
                    }
                    barrier_expect(&s_copied[slot], boxes * C::kBlock);
                    for (int k = 0; k < boxes; ++k)
                        copy_box(ring + slot * C::kStageBytes + k * C::kBlock, &dy_map, 64 * k, row, &s_copied[slot]);
                    ++copied;
                    if (++slot == C::kStages) slot = 0, parity ^= 1;
                }
            }
            // every copy has come before the block ends
            for (int k = copied < C::kStages ? copied : C::kStages; k > 0; --k)
                if (!barrier_wait(&s_copied[(copied - k) % C::kStages], (copied - k) / C::kStages & 1, a.tries)) s_failed = 1;
            for (int k = stage < C::kRawStages ? stage : C::kRawStages; k > 0; --k)
                if (!barrier_wait(&s_raw_full[(stage - k) % C::kRawStages], (stage - k) / C::kRawStages & 1, a.tries)) s_failed = 1;
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
            if (s_failed) t = __uint_as_float(0x7fffffffu);
            if (a.splits > 1)
                a.part_bias[size_t(blockIdx.x) * a.N + j] = t;
            else
                store_param(a.db, a.gdt, j, t);
        }
    }
    tensor_fence_before();
    __syncthreads();
    if (warp == C::kLoaders / 32)
        tensor_free<C::kColumns>(tensor);
}

// The partial sums' totals.  SLICES warps of a CTA take the partial sums s, s + SLICES, ... of the
// same 32 V values side by side, and the slices are added in order: many slices of few values, or 4
// values a lane where there are enough to fill the device.  The first w_ctas CTAs have dW, the others the bias.
template <int SLICES, int V>
__global__ void __launch_bounds__(SLICES * 32) k_dense_join(DenseArgs a, int w_ctas) {
    __shared__ float s_t[SLICES][32 * V + 1];
    const bool weight = int(blockIdx.x) < w_ctas;
    const int64_t all = weight ? int64_t(a.N) * a.D : a.N;
    const int64_t first = int64_t(weight ? blockIdx.x : blockIdx.x - w_ctas) * (32 * V);
    const int count = weight ? a.splits : a.bias_splits, lane = threadIdx.x & 31, q = threadIdx.x >> 5;
    const float *p = (weight ? a.part : a.part_bias) + first + lane;
    float t[V] = {};
#pragma unroll 4
    for (int v = q; v < count; v += SLICES)
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (first + lane + 32 * k < all) t[k] += p[v * all + 32 * k];
#pragma unroll
    for (int k = 0; k < V; ++k) s_t[q][lane + 32 * k] = t[k];
    __syncthreads();
    for (int j = threadIdx.x; j < 32 * V; j += SLICES * 32) {
        const int64_t e = first + j;
        if (e >= all) break;
        float u = 0.0f;
#pragma unroll
        for (int v = 0; v < SLICES; ++v) u += s_t[v][j];
        if (weight)
            store_param(a.dw, a.gdt, e / a.D * a.dws + e % a.D, u);
        else
            store_param(a.db, a.gdt, e, u);
    }
}

// Ranges of rows with sums of their own: as many as fill the device, in as many rounds as it takes
// for none to be longer than a chain; of kLeastRows at least, and one where that is as fast as ranges and
// the launch that joins them. (One range of 256 rows and two, in us a call: 48 x 48 bfloat16 8.3 and 10.4, 128 x 128
// float32 14.5 and 16.5, 100 x 64 float16 14.4 and 14.4; of 384 rows 8.3 and 10.4, 16.9 and 16.5, 18.5 and 14.4.
// Ranges of at least 64, 128 and 256 rows, both kernels: 8191 rows of 128 x 128 float32 21.0, 22.8 and 25.6, 20,000
// 29.2, 28.3 and 28.0; of 48 x 48 bfloat16 15.3, 16.7 and 17.8, then 18.1, 16.6 and 18.7.)
constexpr int kMostSmem = 113 * 1024, kTwoSmem = 112 * 1024 + 512;     // two CTAs of an SM
constexpr int kLeastRows = 128, kOneRange = 256;
int splits_of(int64_t n, int gdt) {
    const int64_t once = kSms * 2, chain = gdt == SS_F32 ? kChain32 : kChain16;
    const int64_t most = (n + kLeastRows - 1) / kLeastRows, rounds = (n + once * chain - 1) / (once * chain);
    const int64_t s = once * rounds;
    return n <= kOneRange ? 1 : int(s < most ? s : most);
}

template <typename T, int TI, int TJ, int ROWS, int FMT>
ss_status launch(DenseArgs a, const RawStage &raw, bool fast, size_t smem, cudaStream_t s, const char *who) {
    using C = Config<T, TI, TJ, ROWS>;
    const int64_t each = (a.n + a.splits - 1) / a.splits, rows = (each + C::kRows - 1) / C::kRows * C::kRows;
    static std::atomic<unsigned long long> smem_ctx[kMaxDevices];   // see ensure_dyn_smem
    const void *fn[2] = {(const void *)k_dense<T, TI, TJ, ROWS, FMT, true>, (const void *)k_dense<T, TI, TJ, ROWS, FMT, false>};
    ss_status st = ensure_dyn_smem(smem_ctx, fn, 2, kMostSmem, who);
    if (st != SS_OK) return st;
    CUtensorMap dy_map = {}, x_map = {};
    if (fast) {
        constexpr int kSize = int(sizeof(T));
        st = C::kParts == 1 ? map_of(&dy_map, a.dy, a.n, a.N, a.dys, C::kRows, who)
                            : map_of(&dy_map, kSize == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, a.dy, a.n,
                                     a.N, a.dys * kSize, raw.dy_pitch / kSize, C::kRows, false, who);
        if (st != SS_OK) return st;
        st = map_of(&x_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.x.q, a.n, units_of(a.D) * kUnit, a.x.stride, raw.x_pitch, C::kRows, false,
                    who);
        if (st != SS_OK) return st;
    }
    auto kernel = fast ? k_dense<T, TI, TJ, ROWS, FMT, true> : k_dense<T, TI, TJ, ROWS, FMT, false>;
    SS_LAUNCH("k_dense", s, kernel<<<a.splits, C::kThreads, smem, s>>>(a, rows, raw, dy_map, x_map));
    return SS_OK;
}

// Stages of 64 rows where two CTAs of an SM have room for them, else of 32.
template <typename T, int TI, int TJ, int FMT>
ss_status launch(const DenseArgs &a, cudaStream_t s, const char *who) {
    const bool fast = a.n > 0 && aligned_to(a.dy, 16) && a.dys * int64_t(sizeof(T)) % 16 == 0 && aligned_to(a.x.q, 16) &&
                      a.x.stride % 16 == 0;
    RawStage raw{parts_of<T>() == 1 ? 0 : (a.N * int(sizeof(T)) + 15) / 16 * 16, (a.D + 15) / 16 * 16, 0};
    raw.bytes = raw.dy_pitch + raw.x_pitch;       // of a row
    using C64 = Config<T, TI, TJ, 64>;
    using C32 = Config<T, TI, TJ, 32>;
    // what the widest rows take; float32 of up to 64 x 64 goes by its own
    constexpr int kWidest = C64::kStages * C64::kStageBytes + C64::kRawStages * 64 * (TI * (parts_of<T>() == 1 ? 0 : int(sizeof(T))) + TJ);
    constexpr bool kBoth = parts_of<T>() == 3 && TI == 64 && TJ == 64;
    if constexpr (kBoth || kWidest <= kTwoSmem) {
        const size_t smem = C64::kStages * C64::kStageBytes + (fast ? C64::kRawStages * 64 * raw.bytes : 0) + 1280;
        if (!kBoth || smem <= kTwoSmem) {
            raw.bytes *= 64;
            return launch<T, TI, TJ, 64, FMT>(a, raw, fast, smem, s, who);
        }
    }
    if constexpr (kBoth || kWidest > kTwoSmem) {
        const size_t smem = C32::kStages * C32::kStageBytes + (fast ? C32::kRawStages * 32 * raw.bytes : 0) + 1280;
        raw.bytes *= 32;
        return launch<T, TI, TJ, 32, FMT>(a, raw, fast, smem, s, who);
    }
    return SS_OK;
}

template <typename T, int FMT>
ss_status tile(const DenseArgs &a, cudaStream_t s, const char *who) {
    if (a.N <= 64 && a.D <= 64) return launch<T, 64, 64, FMT>(a, s, who);
    if (a.N <= 64) return launch<T, 64, 128, FMT>(a, s, who);
    if (a.D <= 64) return launch<T, 128, 64, FMT>(a, s, who);
    return launch<T, 128, 128, FMT>(a, s, who);
}

// A weight past one tile goes to the kernel of large ones, but for one of up to eight tiles in a row or a
// column and many rows of dy in float32 or float16: that kernel writes dy's parts to memory and
// reads them back, here dy is read once, and a tile's two launches cost 20 us (200,000 x 256 x 128 float32: 104 us
// for 227, 400,000 x 48 x 256 float16: 88 for 252; 16384 rows of 512 x 48 float32: 60 for 45, of 256 x 128
// float16: 37 for 35).  bfloat16 needs no parts (131,072 x 1024 x 32: 172 for 90), and 2 x 2 tiles read both twice.
constexpr int32_t kSide = 128, kMostTiles = 8;
constexpr int64_t kTileRows = 32768;
bool dense_is_big(int64_t n, int32_t N, int32_t D, int dtype) {
    const int64_t tiles = int64_t((N + kSide - 1) / kSide) * ((D + kSide - 1) / kSide);
    if (tiles == 1) return false;
    return dtype == SS_BF16 || (N > kSide && D > kSide) || tiles > kMostTiles || n < tiles * kTileRows;
}

// A tile's partial sums, the bias's behind them.
size_t tile_workspace(int splits, int32_t N, int32_t D) {
    const size_t rows = N < kSide ? N : kSide, columns = D < kSide ? D : kSide;
    return splits > 1 ? size_t(splits) * rows * (columns + 1) * sizeof(float) : 256;
}

bool dense_sizes_ok(int64_t n, int32_t N, int32_t D) { return row_sizes_ok(n, D) && N >= 1 && N <= kMaxWidth; }

}  // namespace

void dense_join(const DenseArgs &a, bool weight, cudaStream_t s, int sms) {
    int64_t values = weight ? int64_t(a.N) * a.D : 0, biases = a.db ? a.N : 0;
    const bool wide = values >= int64_t(sms) * 256;
    if (wide && biases && a.bias_splits > 64) {      // too many for few slices
        dense_join(a, false, s, sms);
        biases = 0;
    }
    const int each = wide ? 128 : 32;
    const int64_t w = (values + each - 1) / each, ctas = w + (biases + each - 1) / each;
    if (ctas == 0) return;
    if (wide && a.splits < 16)
        SS_LAUNCH("k_dense_join", s, k_dense_join<4, 4><<<unsigned(ctas), 128, 0, s>>>(a, int(w)));
    else if (wide)
        SS_LAUNCH("k_dense_join", s, k_dense_join<8, 4><<<unsigned(ctas), 256, 0, s>>>(a, int(w)));
    else
        SS_LAUNCH("k_dense_join", s, k_dense_join<32, 1><<<unsigned(ctas), 1024, 0, s>>>(a, int(w)));
}

}  // namespace ss

using namespace ss;

static ss_status dense_grad8(const char *who, const void *dy, ss_dtype dtype, int64_t dy_stride, const ss_rows8 *x, int64_t n,
                             int32_t N, int32_t D, void *dweight, int64_t dweight_stride, void *dbias, ss_dtype grad_dtype,
                             void *workspace, size_t workspace_bytes, uint32_t tries, int sent, ss_stream_t stream) {
    clear_error();
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
    if ((st = current_device(&dev, &sms, who)) != SS_OK) return st;
    cudaStream_t s = (cudaStream_t)stream;
    DenseArgs a{dy, dy_stride, rows8_of(x), n, N, D, 1, 1, 0, nullptr, nullptr, dweight, dweight_stride, dbias,
                int(grad_dtype), tries, sent};
    const int format = x ? x->format : SS_INT8;
    if (dense_is_big(n, N, D, dtype)) {
        st = dense_big(who, a, dtype, format, workspace, s, sms);
        return st != SS_OK ? st : check_launch(who);
    }
    // tile after tile, all in the same workspace
    a.splits = a.bias_splits = splits_of(n, grad_dtype);
    a.part = static_cast<float *>(workspace);
    const size_t size = dtype_bytes(dtype), out_size = dtype_bytes(grad_dtype);
    for (int32_t i = 0; i < N; i += kSide)
        for (int32_t j = 0; j < D; j += kSide) {
            DenseArgs t = a;
            t.N = N - i < kSide ? N - i : kSide, t.D = D - j < kSide ? D - j : kSide;
            t.dy = static_cast<const char *>(dy) + i * size;
            t.x.q += j, t.x.scales += j / kGroup;
            t.dw = static_cast<char *>(dweight) + (i * dweight_stride + j) * out_size;
            t.db = dbias && j == 0 ? static_cast<char *>(dbias) + i * out_size : nullptr;
            t.part_bias = t.part + size_t(t.splits) * t.N * t.D;
            with_type(dtype, [&](auto v) {
                with_format(format, [&](auto F) { st = tile<decltype(v), decltype(F)::value>(t, s, who); });
            });
            if (st != SS_OK) return st;
            if (t.splits > 1) dense_join(t, true, s, sms);
        }
    return check_launch(who);
}

extern "C" {

size_t ss_dense_grad8_workspace_bytes(int64_t n, int32_t N, int32_t D, ss_dtype dtype, ss_dtype grad_dtype) {
    if (!dense_sizes_ok(n, N, D) || !dtype_known(dtype) || (grad_dtype != SS_F32 && grad_dtype != dtype)) return 0;
    if (dense_is_big(n, N, D, dtype)) return dense_big_workspace(n, N, D, dtype, grad_dtype);
    return tile_workspace(splits_of(n, grad_dtype), N, D);
}

ss_status ss_dense_grad8(const void *dy, ss_dtype dtype, int64_t dy_stride, const ss_rows8 *x, int64_t n, int32_t N,
                         int32_t D, void *dweight, int64_t dweight_stride, void *dbias, ss_dtype grad_dtype,
                         void *workspace, size_t workspace_bytes, ss_stream_t stream) {
    return dense_grad8("ss_dense_grad8", dy, dtype, dy_stride, x, n, N, D, dweight, dweight_stride, dbias, grad_dtype,
                       workspace, workspace_bytes, kWaitTries, INT_MAX, stream);
}

// A test's: nothing else differs from ss_dense_grad8.  Each wait ends after 4096 tries; the copies that have
// been issued are waited for and the tensor memory is given back as ever.
ss_status ss_test_dense_wait_timeout(const void *dy, ss_dtype dtype, int64_t dy_stride, const ss_rows8 *x, int64_t n,
                                     int32_t N, int32_t D, void *dweight, int64_t dweight_stride, void *dbias,
                                     ss_dtype grad_dtype, void *workspace, size_t workspace_bytes, ss_stream_t stream) {
    return dense_grad8("ss_test_dense_wait_timeout", dy, dtype, dy_stride, x, n, N, D, dweight, dweight_stride, dbias,
                       grad_dtype, workspace, workspace_bytes, 4096, 1, stream);
}

}  // extern "C"
