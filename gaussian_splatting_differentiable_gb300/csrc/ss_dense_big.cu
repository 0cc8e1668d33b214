// The weight gradient of a dense layer from its input kept in 8 bits, for weights past one
// tile (model: include/ss_dense.h; the method: ss_dense.cuh).
//
// Here every value of dy and x goes into many products, and converting it for each tile
// anew would take longer than the products (8191 x 4096 x 4096 in tiles of 256 x 256: 285
// us, of which the products 140).  So x, and dy where it is not bfloat16 on 16-byte boundaries, are
// converted once, a chunk of rows at a time, into the workspace, and the products' kernel
// has the copy engine bring both.  8191 x 4096 x 4096 bfloat16: 21 us and 158 by ncu; the products' tiles come at 62
// bytes a clock and SM (of 64 KB a stage, for 1024 clocks of products), the tensor cores are busy 74 % of
// the time (304 tiles of 256 x 224, two to an SM).  Into float32 223: the products wait while a chain leaves the tensor
// memory.
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <type_traits>

#include "ss_dense.cuh"
#include "ss_internal.h"
#include "ss_profile.h"
#include "ss_rows8.cuh"
#include "ss_tensor.cuh"
#include "ss_unit.cuh"

namespace ss {
namespace {

// ------------------------------------------------------------------ conversion

constexpr int kThreads = 256;
constexpr int kSlab = 64;              // rows of a CTA
constexpr int kDyColumns = 256;

struct ConvertArgs {
    int64_t first, rows, padded;   // the chunk: its first row, its rows, and with rows of zeros a multiple of kRows
    __nv_bfloat16 *x;              // [padded][x_stride]
    int64_t x_stride;
    __nv_bfloat16 *dy;             // [parts][padded][dy_stride], NULL: dy is used where it is
    int64_t dy_stride;
    int x_ctas, dy_blocks;
    float *bias;                   // [slab][N] of this chunk, NULL: not wanted
};

// The first x_ctas CTAs turn x into bfloat16, pieces of 16 columns one after the other along their threads,
// four in flight; the others, by slabs of rows and blocks of columns, dy into its parts, with
// the slab's sum of each column.  Bound by memory.
template <typename T, int FMT, bool FAST>
__global__ void __launch_bounds__(kThreads) k_dense_convert(DenseArgs a, ConvertArgs c) {
    constexpr int kParts = parts_of<T>(), kAhead = 4;
    __shared__ float s_sum[kThreads / 32][kDyColumns];
    if (int(blockIdx.x) < c.x_ctas) {
        const int per_row = (a.D + kWide - 1) / kWide;
        const int64_t step = int64_t(c.x_ctas) * kThreads, rows = step / per_row;
        const int more = int(step - rows * per_row);
        int64_t r = (int64_t(blockIdx.x) * kThreads + threadIdx.x) / per_row;
        int u = int(int64_t(blockIdx.x) * kThreads + threadIdx.x - r * per_row);
        while (r < c.padded) {
            Wide h[kAhead];
            __nv_bfloat16 *to[kAhead];
            bool all[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int j = u * kWide;
                to[k] = r < c.padded ? c.x + r * c.x_stride + j : nullptr, all[k] = a.D - j > kUnit;
                h[k] = Wide{{0u, 0u, 0u, 0u}, 127u};
                if (r < c.rows)
                    h[k].template load<FAST>(a.x.q + (c.first + r) * a.x.stride + j,
                                             a.x.scales + (c.first + r) * a.x.scale_stride + j / kGroup, all[k]);
                r += rows, u += more;
                if (u >= per_row) u -= per_row, ++r;
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (!to[k]) continue;
                uint32_t w[8];
                convert<FMT>(w, h[k]);
                uint4 *p = reinterpret_cast<uint4 *>(to[k]);
                p[0] = make_uint4(w[0], w[1], w[2], w[3]);
                if (all[k]) p[1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
        }
        return;
    }
    const int slab = (int(blockIdx.x) - c.x_ctas) / c.dy_blocks, block = (int(blockIdx.x) - c.x_ctas) % c.dy_blocks;
    const int64_t r0 = int64_t(slab) * kSlab, r1 = r0 + kSlab < c.padded ? r0 + kSlab : c.padded;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int i0 = block * kDyColumns, i = i0 + lane * kUnit;
    const int count = a.N - i < kUnit ? a.N - i : kUnit;
    F2 sums[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) sums[k] = both(0.0f);
    if (count > 0)
#pragma unroll 4
        for (int64_t r = r0 + warp; r < r1; r += kThreads / 32) {
            const Raw<T> v = load_unit<T, FAST>(static_cast<const T *>(a.dy) + (c.first + r) * a.dys + i, r < c.rows ? count : 0);
            F2 f[4];
            floats_of(f, v);
#pragma unroll
            for (int k = 0; k < 4; ++k) sums[k] = add2(sums[k], f[k]);
            if (!c.dy) continue;
            uint32_t w[kParts][4];
            cut_parts(w, v);
#pragma unroll
            for (int p = 0; p < kParts; ++p)
                *reinterpret_cast<uint4 *>(c.dy + (p * c.padded + r) * c.dy_stride + i) =
                    make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]);
        }
    if (!c.bias) return;
#pragma unroll
    for (int k = 0; k < 4; ++k) reinterpret_cast<float2 *>(&s_sum[warp][lane * kUnit])[k] = sums[k];
    __syncthreads();
    const int j = i0 + threadIdx.x;
    if (j >= a.N) return;
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) t += s_sum[w][threadIdx.x];
    c.bias[size_t(slab) * a.N + j] = t;
}

// ------------------------------------------------------------------ products

// Tiles of 256 rows of dW for one part of dy, 128 for several (which have two sets of sums), and
// up to 256 columns; 512 columns of tensor memory either way.
template <int PARTS>
struct Big {
    static constexpr int kTI = PARTS == 1 ? 256 : 128, kTJ = 256;
    static constexpr int kRows = 64;                                // of a stage, and of a copy (32: 272 us for 161)
    static constexpr int kBlock = kRows * 128;                      // bytes of 64 columns of a stage
    static constexpr int kABytes = kTI / 64 * kBlock, kBBytes = kTJ / 64 * kBlock;
    static constexpr int kStageBytes = PARTS * kABytes + kBBytes;
    static constexpr int kStages = 200 * 1024 / kStageBytes;
    static constexpr int kSmem = kStages * kStageBytes + 1024;
    static constexpr int kDrainers = 256;
    static constexpr int kThreads = kDrainers + 64;
};

struct BigArgs {
    int64_t rows, split_rows;      // of the chunk; of a range of it, a multiple of kRows
    int64_t dy_row, dy_part;       // where the chunk begins in dy's map, and how far one part is from the next
    int width;                     // columns of a tile
    bool first, last;              // chunk
    int bias;                      // the bias' sums: 0 not from here, 1 to part_bias from row bias_row on, 2 to db
    int bias_row;
};

// CTA (range of the rows, tile of D, tile of N).  Warps 0 to 7 read the sums, one thread
// of warp 8 issues the products, one of warp 9 the copies.  Where dy is used as it lies, the CTAs of the
// first columns of x have warps 0 to 7 add up its columns out of shared memory on the way.
template <int PARTS>
__global__ void __launch_bounds__(Big<PARTS>::kThreads, 1)
    k_dense_big(DenseArgs a, BigArgs b, const __grid_constant__ CUtensorMap dy_map, const __grid_constant__ CUtensorMap x_map) {
    using C = Big<PARTS>;
    extern __shared__ uint8_t s_raw[];
    __shared__ uint64_t s_full[C::kStages], s_empty[C::kStages], s_done, s_drained;
    __shared__ uint32_t s_tensor, s_failed;
    const uint32_t ring = (smem_of(s_raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int i0 = blockIdx.z * C::kTI, j0 = blockIdx.y * b.width;
    const int ni = a.N - i0 < C::kTI ? a.N - i0 : C::kTI, nj = a.D - j0 < b.width ? a.D - j0 : b.width;
    const int64_t first = int64_t(blockIdx.x) * b.split_rows;
    const int64_t last = first + b.split_rows < b.rows ? first + b.split_rows : b.rows;
    const int stages = last > first ? int((last - first + C::kRows - 1) / C::kRows) : 0;
    const bool bias = PARTS == 1 && b.bias && blockIdx.y == 0;
    const uint8_t *ring_ptr = s_raw + (ring - smem_of(s_raw));

    if (threadIdx.x == 0) {
        s_failed = 0;
        for (int k = 0; k < C::kStages; ++k) barrier_init(&s_full[k], 1), barrier_init(&s_empty[k], bias ? 9 : 1);
        barrier_init(&s_done, 1);
        barrier_init(&s_drained, C::kDrainers / 32);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 8) tensor_take<512>(&s_tensor);
    tensor_fence_before();
    __syncthreads();
    tensor_fence_after();
    const uint32_t tensor = s_tensor;

    F2 sums[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) sums[k] = both(0.0f);
    if (warp < 8) {
        int slot = 0;
        uint32_t parity = 0;
        const int chains = stages ? (stages + a.chain - 1) / a.chain : 1;
        for (int chain = 0; chain < chains; ++chain) {
            if (bias) {
                // warp w rows w, w + 8, ... of a stage, lane l columns 8 l to 8 l + 7
                const int stop = (chain + 1) * a.chain < stages ? (chain + 1) * a.chain : stages;
                for (int stage = chain * a.chain; stage < stop; ++stage) {
                    if (!warp_wait(&s_full[slot], parity, a.tries)) {
                        s_failed = 1;
                        break;
                    }
                    const uint8_t *at = ring_ptr + slot * C::kStageBytes + (lane >> 3) * C::kBlock;
                    if (lane * kUnit < ni)
#pragma unroll
                        for (int r = warp; r < C::kRows; r += 8) {
                            Raw<__nv_bfloat16> v;
                            load_words(v.w, at + r * 128 + (((lane ^ r) & 7) << 4));
                            F2 f[4];
                            floats_of(f, v);
#pragma unroll
                            for (int k = 0; k < 4; ++k) sums[k] = add2(sums[k], f[k]);
                        }
                    __syncwarp();
                    if (lane == 0) barrier_arrive(&s_empty[slot]);
                    if (++slot == C::kStages) slot = 0, parity ^= 1;
                }
            }
            if (!barrier_wait(&s_done, chain & 1, a.tries)) s_failed = 1;
            tensor_fence_after();
            // a wait that ran out leaves NaN, and no other chain is waited for
            const bool failed = __any_sync(0xffffffffu, *static_cast<volatile uint32_t *>(&s_failed) != 0);
            const bool begins = b.first && chain == 0, ends = b.last && (failed || chain == chains - 1);
            // a warp reads the 32 lanes (rows of dW) of its quarter, the two warps of a quarter 8
            // columns in turn
            const int quarter = warp & 3;
            if (stages > 0 || begins || ends)
#pragma unroll 1
                for (int h = 0; h < C::kTI / 128 && h * 128 < ni; ++h) {
                    const int i = i0 + h * 128 + quarter * 32 + lane;
#pragma unroll 2
                    for (int c = (warp >> 2) * 8; c < nj; c += 16) {
                        uint32_t v[8];
                        const uint32_t at = tensor + (uint32_t(quarter * 32) << 16) + h * C::kTJ + c;
                        __syncwarp();
                        tensor_load8(v, at);
                        if (PARTS > 1) {
                            uint32_t w[8];
                            tensor_load8(w, at + C::kTJ);
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                v[k] = __float_as_uint(joined(__uint_as_float(v[k]), __uint_as_float(w[k])));
                        }
                        if (stages == 0 || failed)
#pragma unroll
                            for (int k = 0; k < 8; ++k) v[k] = failed ? 0x7fffffffu : 0u;
                        if (i < a.N) put(a, blockIdx.x, i, j0 + c, nj - c < 8 ? nj - c : 8, v, begins, ends);
                    }
                }
            tensor_fence_before();
            __syncwarp();
            if (lane == 0) barrier_arrive(&s_drained);
            if (failed) break;
        }
    } else if (warp == 8) {
        if (lane == 0) {
            const uint32_t what = product_of((nj + 15) / 16 * 16);
            int slot = 0, chains = 0, link = 0;
            uint32_t parity = 0;
            bool told = false;         // s_done of this chain
            for (int stage = 0; stage < stages; ++stage) {
                if (!barrier_wait(&s_full[slot], parity, a.tries)) {
                    s_failed = 1;
                    __threadfence_block();      // before those that wait for s_done look at it
                    break;
                }
                tensor_fence_after();
                const uint32_t at = ring + slot * C::kStageBytes, bt = at + PARTS * C::kABytes;
#pragma unroll
                for (int k = 0; k < C::kRows / kStep; ++k)
#pragma unroll
                    for (int p = 0; p < PARTS; ++p)
#pragma unroll
                        for (int h = 0; h < C::kTI / 128; ++h)
                            if (h * 128 < ni)
                                product(tensor + (p > 0 ? C::kTJ : 0) + h * C::kTJ,
                                        operand_at<C::kBlock>(at + p * C::kABytes + h * 2 * C::kBlock + k * kStep * 128),
                                        operand_at<C::kBlock>(bt + k * kStep * 128), what, link > 0 || k > 0 || p > 1);
                products_arrive(&s_empty[slot]);
                if (++slot == C::kStages) slot = 0, parity ^= 1;
                if (++link == a.chain && stage + 1 < stages) {
                    products_arrive(&s_done);
                    if (!barrier_wait(&s_drained, chains & 1, a.tries)) {
                        s_failed = 1;
                        told = true;
                        break;
                    }
                    link = 0, ++chains;
                    tensor_fence_after();
                }
            }
            if (!told) products_arrive(&s_done);
            if (!barrier_wait(&s_done, chains & 1, a.tries)) s_failed = 1;    // the tensor memory is freed after them
        }
        __syncwarp();
    } else {
        if (lane == 0) {
            const int a_boxes = (ni + 63) / 64, b_boxes = (nj + 63) / 64;
            int slot = 0, stage = 0;
            uint32_t parity = 1;
            for (; stage < stages && stage < a.sent; ++stage) {
                if (!barrier_wait(&s_empty[slot], parity, a.tries)) {
                    s_failed = 1;
                    break;
                }
                const uint32_t at = ring + slot * C::kStageBytes;
                const int64_t row = first + int64_t(stage) * C::kRows;
                barrier_expect(&s_full[slot], (a_boxes * PARTS + b_boxes) * C::kBlock);
                for (int p = 0; p < PARTS; ++p)
                    for (int k = 0; k < a_boxes; ++k)
                        copy_box(at + p * C::kABytes + k * C::kBlock, &dy_map, i0 + 64 * k, int(b.dy_row + p * b.dy_part + row),
                                 &s_full[slot]);
                for (int k = 0; k < b_boxes; ++k)
                    copy_box(at + PARTS * C::kABytes + k * C::kBlock, &x_map, j0 + 64 * k, int(row), &s_full[slot]);
                if (++slot == C::kStages) slot = 0, parity ^= 1;
            }
            // every copy has come before the block ends
            for (int k = stage < C::kStages ? stage : C::kStages; k > 0; --k)
                if (!barrier_wait(&s_full[(stage - k) % C::kStages], (stage - k) / C::kStages & 1, a.tries)) s_failed = 1;
        }
        __syncwarp();
    }
    tensor_fence_before();
    __syncthreads();
    if (warp == 8) tensor_free<512>(tensor);
    if (!bias) return;
    float *s = reinterpret_cast<float *>(s_raw + (ring - smem_of(s_raw)));     // [8][256]
    if (warp < 8)
#pragma unroll
        for (int k = 0; k < 4; ++k) reinterpret_cast<float2 *>(s + warp * 256 + lane * kUnit)[k] = sums[k];
    __syncthreads();
    for (int i = threadIdx.x; i < ni; i += C::kThreads) {
        float t = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) t += s[w * 256 + i];
        if (s_failed) t = __uint_as_float(0x7fffffffu);
        if (b.bias == 2)
            store_param(a.db, a.gdt, i0 + i, t);
        else
            a.part_bias[size_t(b.bias_row + blockIdx.x) * a.N + i0 + i] = t;
    }
}

// ------------------------------------------------------------------ shares

int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// How the work is shared out: the width of a tile, how many ranges of rows have sums of their own, and
// the rows of a chunk.
struct Plan {
    int width, splits;
    int64_t chunk;
    bool part;
    int64_t x_stride, dy_stride;
    size_t bias_at, x_at, dy_at, bytes;
};
constexpr size_t kConverted = size_t(192) << 20;    // bytes of a chunk's converted rows
constexpr int kLeastChunk = 1024, kLeastRange = 256;

// A tile's products take half a clock a column and step; a tile has about 6000 clocks beside them;
// an SM moves 16 to 20 bytes a clock of partial sums.  The least of the waves' times.
Plan plan_of(int64_t n, int32_t N, int32_t D, int dtype, int gdt) {
    const int parts = dtype == SS_F32 ? 3 : (dtype == SS_F16 ? 2 : 1), ti = parts == 1 ? 256 : 128;
    Plan p{};
    p.x_stride = round_up(D, kUnit), p.dy_stride = round_up(N, kUnit);
    const int64_t each = 2 * (p.x_stride + parts * p.dy_stride);
    p.chunk = int64_t(kConverted) / each / 64 * 64;      // whole stages
    if (p.chunk < kLeastChunk) p.chunk = kLeastChunk;
    if (p.chunk > n) p.chunk = n < 1 ? 1 : n;
    const int64_t tiles_i = (N + ti - 1) / ti;
    const double steps = double(p.chunk) / kStep * parts * (N < ti ? (N + 127) / 128 : ti / 128);
    double best = 0;
    for (int width = 256; width >= 128; width -= 32) {
        if (width < 256 && D <= width / 2) break;
        const int64_t tiles = tiles_i * ((D + width - 1) / width);
        for (int s = 1; s <= 128; s += s < 8 ? 1 : s / 4) {
            if (s > 1 && (p.chunk / s < kLeastRange || tiles * (s - 1) >= 4 * kSms)) break;
            const int64_t waves = (tiles * s + kSms - 1) / kSms;
            const int columns = D < width ? (D + 15) / 16 * 16 : width;
            double t = double(waves) * (steps / s * columns / 2 + 6000);
            if (s > 1) t += (2.0 * s + 1) * N * double(D) * 4 / (18.0 * kSms) + 4000;
            if (best == 0 || t < best) best = t, p.width = width, p.splits = s;
        }
    }
    const int chain = gdt == SS_F32 ? kChain32 : kChain16;
    p.part = p.splits > 1 || (gdt != SS_F32 && n > (p.chunk < chain ? p.chunk : chain));
    const size_t sums = p.part ? size_t(p.splits) * N * D * sizeof(float) : 0;
    const int64_t chunks = (n + p.chunk - 1) / p.chunk, slabs = chunks * (round_up(p.chunk, 64) / kSlab + 1 + p.splits);
    const int64_t padded = round_up(p.chunk, 64);
    p.bias_at = round_up(sums, 256);
    p.x_at = p.bias_at + round_up(size_t(slabs) * N * sizeof(float), 256);
    p.dy_at = p.x_at + round_up(size_t(padded) * p.x_stride * 2, 256);
    p.bytes = p.dy_at + size_t(parts) * padded * p.dy_stride * 2;
    return p;
}

template <typename T, int FMT>
ss_status run(const char *who, DenseArgs a, const Plan &p, uint8_t *ws, cudaStream_t s, int sms) {
    constexpr int kParts = parts_of<T>();
    using C = Big<kParts>;
    const bool aligned = units_aligned<T>(a.dy, a.dys), q16 = aligned_to(a.x.q, 16) && a.x.stride % 16 == 0;
    const bool direct = kParts == 1 && aligned;
    a.splits = p.splits;
    a.part = reinterpret_cast<float *>(ws);
    a.part_bias = reinterpret_cast<float *>(ws + p.bias_at);
    a.chain = (a.gdt == SS_F32 ? kChain32 : kChain16) / C::kRows;
    static std::atomic<unsigned long long> smem_ctx[kMaxDevices];   // see ensure_dyn_smem
    const void *fn = (const void *)k_dense_big<kParts>;
    ss_status st = ensure_dyn_smem(smem_ctx, &fn, 1, C::kSmem, who);
    if (st != SS_OK) return st;
    a.bias_splits = 0;
    bool bias_left = false;        // to be added up yet
    __nv_bfloat16 *xw = reinterpret_cast<__nv_bfloat16 *>(ws + p.x_at), *dyw = reinterpret_cast<__nv_bfloat16 *>(ws + p.dy_at);
    for (int64_t first = 0; first < a.n || first == 0; first += p.chunk) {
        const int64_t rows = a.n - first < p.chunk ? a.n - first : p.chunk, padded = round_up(rows, 64);
        const int64_t pieces = (padded * ((a.D + kWide - 1) / kWide) + 4 * kThreads - 1) / (4 * kThreads);
        const int x_ctas = int(pieces < sms * 8 ? pieces : sms * 8), dy_blocks = (a.N + kDyColumns - 1) / kDyColumns;
        ConvertArgs c{first, rows, padded, xw, p.x_stride, direct ? nullptr : dyw, p.dy_stride, x_ctas, dy_blocks,
                      a.db && !direct ? a.part_bias + size_t(a.bias_splits) * a.N : nullptr};
        const int slabs = int((padded + kSlab - 1) / kSlab);
        CUtensorMap x_map = {}, dy_map = {};
        if (rows > 0) {
            const int64_t grid = x_ctas + (direct ? 0 : int64_t(slabs) * dy_blocks);
            auto kernel = aligned && q16 ? k_dense_convert<T, FMT, true> : k_dense_convert<T, FMT, false>;
            SS_LAUNCH("k_dense_convert", s, kernel<<<unsigned(grid), kThreads, 0, s>>>(a, c));
            if ((st = map_of(&x_map, xw, padded, a.D, p.x_stride, C::kRows, who)) != SS_OK) return st;
            st = direct ? map_of(&dy_map, a.dy, a.n, a.N, a.dys, C::kRows, who)
                        : map_of(&dy_map, dyw, kParts * padded, a.N, p.dy_stride, C::kRows, who);
            if (st != SS_OK) return st;
            if (!direct) a.bias_splits += slabs;
        }
        const int bias = !a.db || !direct ? 0 : (p.splits == 1 && a.n <= p.chunk ? 2 : 1);
        bias_left |= a.db && bias != 2;
        const BigArgs b{rows, round_up((rows + p.splits - 1) / p.splits, C::kRows), direct ? first : 0, padded, p.width,
                        first == 0, first + p.chunk >= a.n, bias, a.bias_splits};
        if (direct) a.bias_splits += p.splits;
        const dim3 grid(p.splits, (a.D + p.width - 1) / p.width, (a.N + C::kTI - 1) / C::kTI);
        SS_LAUNCH("k_dense_big", s, k_dense_big<kParts><<<grid, C::kThreads, C::kSmem, s>>>(a, b, dy_map, x_map));
    }
    if (!bias_left) a.db = nullptr;
    if (a.splits > 1 || bias_left) dense_join(a, a.splits > 1, s, sms);
    return SS_OK;
}

}  // namespace

size_t dense_big_workspace(int64_t n, int32_t N, int32_t D, int dtype, int gdt) {
    return plan_of(n, N, D, dtype, gdt).bytes;
}

ss_status dense_big(const char *who, DenseArgs a, int dtype, int format, void *workspace, cudaStream_t s, int sms) {
    const Plan p = plan_of(a.n, a.N, a.D, dtype, a.gdt);
    ss_status st = SS_OK;
    with_type(dtype, [&](auto t) {
        with_format(format, [&](auto F) {
            st = run<decltype(t), decltype(F)::value>(who, a, p, static_cast<uint8_t *>(workspace), s, sms);
        });
    });
    return st;
}

}  // namespace ss
