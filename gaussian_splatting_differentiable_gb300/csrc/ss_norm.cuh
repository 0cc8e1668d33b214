// What both norms' kernels share: sums over a row's threads, the adding up of the weights' partial
// sums, and how many CTAs take the rows.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstddef>
#include <cstdint>

#include "ss_launch.cuh"
#include "ss_vec.cuh"

namespace ss {

constexpr int kNormThreads = 256;
constexpr int kMaxRowThreads = 512;    // of a row held in registers
constexpr int kRowWarps = kMaxRowThreads / 32;

// 16 bytes into shared memory, asynchronously.
__device__ __forceinline__ void copy16(void *smem, const void *p) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(uint32_t(__cvta_generic_to_shared(smem))), "l"(p)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Sums K values over the `lanes` threads of a row; every one gets the same sums (one
// fixed order).  MULTI: whole warps, through shared memory, alternating two buffers, so one barrier a
// sum is enough; their slots past the row's warps hold zeros.
template <int K, bool MULTI>
__device__ __forceinline__ void row_sum(float (&v)[K], int lanes, int group, int lane, float (*s_red)[K][kRowWarps],
                                        int &flip) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        if (MULTI || o < lanes)
#pragma unroll
            for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if (!MULTI) return;
    if ((lane & 31) == 0)
#pragma unroll
        for (int k = 0; k < K; ++k) s_red[flip][k][lane >> 5] = v[k];
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(lanes) : "memory");
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const float4 *q = reinterpret_cast<const float4 *>(s_red[flip][k]);
        v[k] = 0.0f;
        for (int w = 0; w < lanes; w += 128) {
            const float4 t = q[w >> 7];
            v[k] += (t.x + t.y) + (t.z + t.w);
        }
    }
    flip ^= 1;
}

// Sum over a CTA of kNormThreads, the same value in every thread (fixed order).
__device__ __forceinline__ float block_sum(float v, float *s_red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.0f;
    for (int w = 0; w < kNormThreads / 32; ++w) t += s_red[w];
    return t;
}

// A CTA of 1024 adds up the partial sums of 32 of `cols` columns, dgamma's D and behind them dbeta's: 32
// slices of them side by side, then the slices in order.
__device__ __forceinline__ void add_up_parts(const float *part, int parts, int32_t D, int cols, void *dgamma, void *dbeta,
                                             int pdt) {
    __shared__ float s_t[32][33];
    wait_for_previous();
    const int c = threadIdx.x & 31, q = threadIdx.x >> 5;
    const int j = blockIdx.x * 32 + c;
    float t = 0.0f;
    if (j < cols)
#pragma unroll 4
        for (int p = q; p < parts; p += 32) t += part[size_t(p) * cols + j];
    s_t[q][c] = t;
    __syncthreads();
    t = s_t[c][q];                         // column q of the 32, slice c
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    const int col = blockIdx.x * 32 + q;
    if (c == 0 && col < cols) store_param(col < D ? dgamma : dbeta, pdt, col < D ? col : col - D, t);
}

// Partial sums of the weights' gradients that the workspace has room for: at
// most one for each row, and up to kMaxPeriod - 1 more where the grid is rounded up
// to a multiple of the period of the rows' starts.
constexpr int kMaxPeriod = 8, kMaxParts = 1024;
inline int64_t weight_parts(int64_t n) { return n + kMaxPeriod < kMaxParts ? n + kMaxPeriod : kMaxParts; }

// CTAs of the kernels for wide rows.
inline int wide_grid(int64_t n, int sms) { return int(n < int64_t(sms) * 8 ? n : int64_t(sms) * 8); }

// As many CTAs as fit the device at once, and no more than share the rows
// evenly; a multiple of the period where rows start differently.  `waves`
// times as many where each would have many rows of few values: the device
// hands out the later ones as the first end, which evens out what the
// memory's two halves take (2M x 48 float32: 115 us, 131 in one wave).
// `known`: a kernel's last answer, by what it depends on (one architecture).
template <typename K>
int grid_of(std::atomic<unsigned long long> *known, K kernel, int threads, size_t smem, int64_t n, int groups, int period,
            int waves, int most, int sms) {
    const unsigned long long key = (unsigned long long)(threads) << 40 | (unsigned long long)(smem) << 8;
    const unsigned long long k = known->load(std::memory_order_relaxed);
    int per_sm = int(k & 255);
    if ((k ^ key) >> 8) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem) != cudaSuccess || per_sm < 1)
            per_sm = 1;
        known->store(key | per_sm, std::memory_order_relaxed);
    }
    int64_t fit = int64_t(sms) * per_sm;
    if (n >= fit * groups * 48) fit *= waves;
    if (fit > most) fit = most;
    const int64_t turns = (n + fit * groups - 1) / (fit * groups);
    int64_t grid = (n + turns * groups - 1) / (turns * groups);
    const int p = groups % period == 0 ? 1 : period;
    grid = (grid + p - 1) / p * p;
    return int(grid < 1 ? 1 : grid);
}

}  // namespace ss
