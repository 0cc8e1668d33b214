// Layer normalisation of rows and its gradient (model: include/ss_norm.h).
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "ss_internal.h"
#include "ss_norm.h"
#include "ss_profile.h"
#include "ss_vec.cuh"

namespace ss {
namespace {

constexpr int kThreads = 256;
constexpr int32_t kMaxD = 65536;

// A row's place in the threads: `lanes` threads share it, thread l of them
// holding vectors l, l + lanes, ... (NV of VEC elements) in registers, so the
// row is read once for the mean, the centred squares and the result.  Narrow
// rows (MULTI false) take a power of two of lanes inside a warp and reduce by
// shuffles; wide ones take a CTA and reduce through shared memory.  The next
// row's loads are issued before this row's reduction waits.
constexpr int kPerThread = 16;       // elements of a row in one thread
constexpr int kMaxRowThreads = 512;  // x 16 = the widest row held in registers
constexpr int32_t kMaxRegD = kPerThread * kMaxRowThreads;

struct Place {
    int lanes, shift;   // lanes = 1 << shift where !MULTI
    int vecs;           // vectors of a row
};

// Sums K values over the row's lanes; every lane gets the same sums (one
// fixed order).  MULTI alternates two buffers, so one barrier a sum is enough.
template <int K, bool MULTI>
__device__ __forceinline__ void row_sum(float (&v)[K], const Place &pl, float (*s_red)[K][16], int &flip) {
    const int top = MULTI ? 16 : pl.lanes >> 1;
    for (int o = top; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if (!MULTI) return;
    const int warps = pl.lanes >> 5, warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int k = 0; k < K; ++k) s_red[flip][k][warp] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
        v[k] = 0.0f;
        for (int w = 0; w < warps; ++w) v[k] += s_red[flip][k][w];
    }
    flip ^= 1;
}

template <typename T, int VEC, int NV>
__device__ __forceinline__ void load_row(Vec<T, VEC> (&r)[NV], const T *p, int lane, const Place &pl) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
        if (lane + k * pl.lanes < pl.vecs) r[k] = load_vec<T, VEC>(p + size_t(lane + k * pl.lanes) * VEC);
}

template <typename T, int VEC, int NV, bool MULTI>
__global__ void __launch_bounds__(MULTI ? kMaxRowThreads : kThreads)
    k_norm_fwd(const T *x, int64_t xs, int64_t n, int32_t D, Place pl, const void *gamma, const void *beta, int pdt,
               float eps, T *y, int64_t ys, float *mean, float *rstd) {
    __shared__ float s_red[2][1][16];
    const int lane = MULTI ? threadIdx.x : threadIdx.x & (pl.lanes - 1);
    const int rows = MULTI ? 1 : 32 >> pl.shift;                    // of a warp (or CTA)
    const int64_t step = MULTI ? int64_t(gridDim.x) : int64_t(gridDim.x) * (kThreads / 32) * rows;
    const int sub = MULTI ? 0 : (threadIdx.x & 31) >> pl.shift;
    const int64_t row0 = MULTI ? int64_t(blockIdx.x)
                               : (int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5)) * rows;
    const float inv = 1.0f / float(D);
    float g[NV][VEC], b[NV][VEC];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int v = lane + k * pl.lanes;
            g[k][i] = gamma && v < pl.vecs ? load_param(gamma, pdt, int64_t(v) * VEC + i) : 1.0f;
            b[k][i] = beta && v < pl.vecs ? load_param(beta, pdt, int64_t(v) * VEC + i) : 0.0f;
        }
    Vec<T, VEC> next[NV];
    if (row0 + sub < n) load_row<T, VEC, NV>(next, x + (row0 + sub) * xs, lane, pl);
    int flip = 0;
    for (int64_t base = row0; base < n; base += step) {
        const int64_t row = base + sub;
        float f[NV][VEC], sum[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                f[k][i] = row < n && lane + k * pl.lanes < pl.vecs ? next[k].get(i) : 0.0f;
                sum[0] += f[k][i];
            }
        if (row + step < n) load_row<T, VEC, NV>(next, x + (row + step) * xs, lane, pl);
        row_sum<1, MULTI>(sum, pl, s_red, flip);
        const float mu = sum[0] * inv;
        sum[0] = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (lane + k * pl.lanes < pl.vecs)
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    f[k][i] -= mu;
                    sum[0] = fmaf(f[k][i], f[k][i], sum[0]);
                }
        row_sum<1, MULTI>(sum, pl, s_red, flip);
        const float r = 1.0f / sqrtf(fmaf(sum[0], inv, eps));
        if (row >= n) continue;
        T *out = y + row * ys;
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (lane + k * pl.lanes < pl.vecs) {
                float o[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) o[i] = fmaf(f[k][i] * r, g[k][i], b[k][i]);
                store_floats<T, VEC>(out + size_t(lane + k * pl.lanes) * VEC, o);
            }
        if (lane == 0) {
            if (mean) mean[row] = mu;
            if (rstd) rstd[row] = r;
        }
    }
}

// As the forward, with dy and x of a row in registers; the weights' sums stay
// in the threads' registers over all of a CTA's rows and leave one partial
// sum a CTA in `part` [CTAs][2][D] (none where part is NULL).
template <typename T, int VEC, int NV, bool MULTI>
__global__ void __launch_bounds__(MULTI ? kMaxRowThreads : kThreads, MULTI || NV * VEC > 12 ? 1 : 2)
    k_norm_bwd(const T *dy, int64_t dys, const T *x, int64_t xs, int64_t n, int32_t D, Place pl, const void *gamma,
               int pdt, const float *mean, const float *rstd, T *dx, int64_t dxs, float *part) {
    extern __shared__ float s_dyn[];     // !MULTI: [8 warps][2][D]
    __shared__ float s_red[2][2][16];
    const int lane = MULTI ? threadIdx.x : threadIdx.x & (pl.lanes - 1);
    const int rows = MULTI ? 1 : 32 >> pl.shift;
    const int64_t step = MULTI ? int64_t(gridDim.x) : int64_t(gridDim.x) * (kThreads / 32) * rows;
    const int sub = MULTI ? 0 : (threadIdx.x & 31) >> pl.shift;
    const int64_t row0 = MULTI ? int64_t(blockIdx.x)
                               : (int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5)) * rows;
    const float inv = 1.0f / float(D);
    float g[NV][VEC], dg[NV][VEC], db[NV][VEC];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int v = lane + k * pl.lanes;
            g[k][i] = gamma && v < pl.vecs ? load_param(gamma, pdt, int64_t(v) * VEC + i) : 1.0f;
            dg[k][i] = db[k][i] = 0.0f;
        }
    Vec<T, VEC> nx[NV], nd[NV];
    float mu = 0.0f, r = 0.0f;
    if (row0 + sub < n) {
        load_row<T, VEC, NV>(nd, dy + (row0 + sub) * dys, lane, pl);
        load_row<T, VEC, NV>(nx, x + (row0 + sub) * xs, lane, pl);
        mu = mean[row0 + sub], r = rstd[row0 + sub];
    }
    int flip = 0;
    for (int64_t base = row0; base < n; base += step) {
        const int64_t row = base + sub;
        float a[NV][VEC], h[NV][VEC], sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const bool ok = row < n && lane + k * pl.lanes < pl.vecs;
                const float d = ok ? nd[k].get(i) : 0.0f;
                h[k][i] = ok ? (nx[k].get(i) - mu) * r : 0.0f;
                a[k][i] = d * g[k][i];
                dg[k][i] = fmaf(d, h[k][i], dg[k][i]);
                db[k][i] += d;
                sum[0] += a[k][i];
                sum[1] = fmaf(a[k][i], h[k][i], sum[1]);
            }
        const float rr = r;
        if (row + step < n) {
            load_row<T, VEC, NV>(nd, dy + (row + step) * dys, lane, pl);
            load_row<T, VEC, NV>(nx, x + (row + step) * xs, lane, pl);
            mu = mean[row + step], r = rstd[row + step];
        }
        row_sum<2, MULTI>(sum, pl, s_red, flip);
        if (row >= n) continue;
        const float ma = sum[0] * inv, mah = sum[1] * inv;
        T *out = dx + row * dxs;
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (lane + k * pl.lanes < pl.vecs) {
                float o[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) o[i] = rr * (a[k][i] - ma - h[k][i] * mah);
                store_floats<T, VEC>(out + size_t(lane + k * pl.lanes) * VEC, o);
            }
    }
    if (!part) return;
    part += size_t(blockIdx.x) * 2 * D;
    if (MULTI) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (lane + k * pl.lanes < pl.vecs) {
                store_floats<float, VEC>(part + size_t(lane + k * pl.lanes) * VEC, dg[k]);
                store_floats<float, VEC>(part + D + size_t(lane + k * pl.lanes) * VEC, db[k]);
            }
        return;
    }
    // the warp's rows, then the CTA's warps, in fixed order
    float *mine = s_dyn + size_t(threadIdx.x >> 5) * 2 * D;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            for (int o = pl.lanes; o < 32; o <<= 1) {
                dg[k][i] += __shfl_xor_sync(0xffffffffu, dg[k][i], o);
                db[k][i] += __shfl_xor_sync(0xffffffffu, db[k][i], o);
            }
            const int v = lane + k * pl.lanes;
            if (sub == 0 && v < pl.vecs) {
                mine[v * VEC + i] = dg[k][i];
                mine[D + v * VEC + i] = db[k][i];
            }
        }
    __syncthreads();
    for (int j = threadIdx.x; j < 2 * D; j += kThreads) {
        float t = 0.0f;
        for (int w = 0; w < kThreads / 32; ++w) t += s_dyn[size_t(w) * 2 * D + j];
        part[j] = t;
    }
}

// The CTAs' partial sums of 32 columns of [dgamma | dbeta]: 32 slices of the
// CTAs side by side, then the slices in order.
__global__ void __launch_bounds__(1024) k_norm_bwd_final(const float *part, int parts, int32_t D, void *dgamma,
                                                         void *dbeta, int pdt) {
    __shared__ float s_t[32][33];
    const int c = threadIdx.x & 31, q = threadIdx.x >> 5;
    const int j = blockIdx.x * 32 + c;
    float t = 0.0f;
    if (j < 2 * D)
#pragma unroll 4
        for (int p = q; p < parts; p += 32) t += part[size_t(p) * 2 * D + j];
    s_t[q][c] = t;
    __syncthreads();
    t = s_t[c][q];                         // column q of the 32, slice c
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    const int col = blockIdx.x * 32 + q;
    if (c == 0 && col < 2 * D) store_param(col < D ? dgamma : dbeta, pdt, col < D ? col : col - D, t);
}

// ------------------------------------------------------------------ rows wider than the registers

// Sum over the CTA, the same value in every thread (fixed order).
__device__ __forceinline__ float block_sum(float v, float *s_red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.0f;
    for (int w = 0; w < kThreads / 32; ++w) t += s_red[w];
    return t;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_norm_fwd_wide(const T *__restrict__ x, int64_t xs, int64_t n, int32_t D,
                                                       const void *gamma, const void *beta, int pdt, float eps, T *y,
                                                       int64_t ys, float *mean, float *rstd) {
    __shared__ float s_red[kThreads / 32];
    for (int64_t row = blockIdx.x; row < n; row += gridDim.x) {
        const T *xr = x + row * xs;
        float s = 0.0f;
        for (int j = threadIdx.x; j < D; j += kThreads) s += to_float(xr[j]);
        const float mu = block_sum(s, s_red) / float(D);
        s = 0.0f;
        for (int j = threadIdx.x; j < D; j += kThreads) {
            const float c = to_float(xr[j]) - mu;
            s += c * c;
        }
        const float r = 1.0f / sqrtf(block_sum(s, s_red) / float(D) + eps);
        for (int j = threadIdx.x; j < D; j += kThreads) {
            const float g = gamma ? load_param(gamma, pdt, j) : 1.0f;
            const float b = beta ? load_param(beta, pdt, j) : 0.0f;
            y[row * ys + j] = from_float<T>((to_float(xr[j]) - mu) * r * g + b);
        }
        if (threadIdx.x == 0) {
            if (mean) mean[row] = mu;
            if (rstd) rstd[row] = r;
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

// CTAs of a launch over n rows, so many rows at a time in each.
int grid_of(int64_t n, int rows, int per_sm, int sms) {
    const int64_t want = (n + rows - 1) / rows, most = int64_t(sms) * per_sm;
    return int(want < 1 ? 1 : (want < most ? want : most));
}

constexpr int kMaxParts = 1024;      // partial sums of the weights' gradients
int64_t weight_parts(int64_t n) { return n < 1 ? 1 : (n < kMaxParts ? n : kMaxParts); }

int pow2_at_least(int v) {
    int p = 1;
    while (p < v) p <<= 1;
    return p;
}

// Lanes of a row of `vecs` vectors of `vec` elements: a power of two up to a
// warp while 16 elements a thread hold the row, else whole warps.  At least
// 4 lanes of 16-byte vectors (16 of single elements), so that a load touches
// whole sectors.
Place place_of(int32_t D, int vec, bool *multi) {
    Place pl{};
    pl.vecs = D / vec;
    const int nv = kPerThread / vec;
    const int need = (pl.vecs + nv - 1) / nv;
    *multi = need > 32;
    if (*multi) {
        pl.lanes = (need + 31) / 32 * 32;
    } else {
        const int least = vec > 1 ? 4 : 16, most = pow2_at_least(pl.vecs);
        pl.lanes = pow2_at_least(need);
        if (pl.lanes < least) pl.lanes = least;
        if (pl.lanes > most) pl.lanes = most;
        if (pl.lanes > 32) pl.lanes = 32;
    }
    while ((1 << pl.shift) < pl.lanes) ++pl.shift;
    return pl;
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

template <typename T, int VEC, int NV, bool MULTI>
void fwd_kernel(const FwdArgs &a, const Place &pl, int sms, cudaStream_t s) {
    const int rows = MULTI ? 1 : kThreads / pl.lanes, threads = MULTI ? pl.lanes : kThreads;
    const int grid = grid_of(a.n, rows, MULTI ? 2048 / threads : 8, sms);
    SS_LAUNCH("k_norm_fwd", s,
              k_norm_fwd<T, VEC, NV, MULTI><<<grid, threads, 0, s>>>(static_cast<const T *>(a.x), a.xs, a.n, a.D, pl,
                                                                     a.gamma, a.beta, a.pdt, a.eps,
                                                                     static_cast<T *>(a.y), a.ys, a.mean, a.rstd));
}

template <typename T, int VEC, int NV, bool MULTI>
void bwd_kernel(const BwdArgs &a, const Place &pl, int sms, cudaStream_t s) {
    const int rows = MULTI ? 1 : kThreads / pl.lanes, threads = MULTI ? pl.lanes : kThreads;
    int per_sm = MULTI ? 512 / threads : 2;
    if (per_sm > 6) per_sm = 6;      // kMaxParts / SMs
    int grid = grid_of(a.n, rows, per_sm, sms);
    if (grid > kMaxParts) grid = kMaxParts;
    const size_t smem = MULTI || !a.dgamma ? 0 : size_t(kThreads / 32) * 2 * a.D * sizeof(float);
    SS_LAUNCH("k_norm_bwd", s,
              k_norm_bwd<T, VEC, NV, MULTI><<<grid, threads, smem, s>>>(
                  static_cast<const T *>(a.dy), a.dys, static_cast<const T *>(a.x), a.xs, a.n, a.D, pl, a.gamma,
                  a.pdt, a.mean, a.rstd, static_cast<T *>(a.dx), a.dxs, a.dgamma ? a.part : nullptr));
    if (a.dgamma)
        SS_LAUNCH("k_norm_bwd_final", s,
                  k_norm_bwd_final<<<(2 * a.D + 31) / 32, 1024, 0, s>>>(a.part, grid, a.D, a.dgamma, a.dbeta, a.pdt));
}

// Picks the vectors a thread holds: all of them for wide rows, just enough
// for narrow ones.
template <typename T, int VEC, typename Args>
void pick_nv(const Args &a, int sms, cudaStream_t s) {
    constexpr int kNv = kPerThread / VEC;
    bool multi;
    const Place pl = place_of(a.D, VEC, &multi);
    const int nv = (pl.vecs + pl.lanes - 1) / pl.lanes;
    auto go = [&](auto NV, auto MULTI) {
        if constexpr (std::is_same<Args, FwdArgs>::value)
            fwd_kernel<T, VEC, decltype(NV)::value, decltype(MULTI)::value>(a, pl, sms, s);
        else
            bwd_kernel<T, VEC, decltype(NV)::value, decltype(MULTI)::value>(a, pl, sms, s);
    };
    if (multi) return go(std::integral_constant<int, kNv>{}, std::true_type{});
    if (nv <= 1) return go(std::integral_constant<int, 1>{}, std::false_type{});
    if (nv <= 2) return go(std::integral_constant<int, 2>{}, std::false_type{});
    if constexpr (kNv == 4) {
        if (nv == 3) return go(std::integral_constant<int, 3>{}, std::false_type{});
    }
    if constexpr (kNv >= 4) {
        if (nv <= 4) return go(std::integral_constant<int, 4>{}, std::false_type{});
    }
    if constexpr (kNv == 16) {
        if (nv <= 8) return go(std::integral_constant<int, 8>{}, std::false_type{});
        go(std::integral_constant<int, 16>{}, std::false_type{});
    }
}

template <typename T>
void launch_fwd(const FwdArgs &a, int sms, cudaStream_t s) {
    constexpr int kVec = 16 / sizeof(T);
    if (a.D > kMaxRegD) {
        const int grid = grid_of(a.n, 1, 8, sms);
        SS_LAUNCH("k_norm_fwd_wide", s,
                  k_norm_fwd_wide<T><<<grid, kThreads, 0, s>>>(static_cast<const T *>(a.x), a.xs, a.n, a.D, a.gamma,
                                                               a.beta, a.pdt, a.eps, static_cast<T *>(a.y), a.ys,
                                                               a.mean, a.rstd));
    } else if (a.D % kVec == 0 && aligned_to(a.x, 16) && aligned_to(a.y, 16) && a.xs % kVec == 0 && a.ys % kVec == 0) {
        pick_nv<T, kVec>(a, sms, s);
    } else {
        pick_nv<T, 1>(a, sms, s);
    }
}

template <typename T>
void launch_bwd(const BwdArgs &a, int sms, cudaStream_t s) {
    constexpr int kVec = 16 / sizeof(T);
    if (a.D > kMaxRegD || a.n == 0) {
        // the weights first: dx may overwrite dy or x
        if (a.dgamma) {
            const dim3 g((a.D + kThreads - 1) / kThreads, unsigned(a.n < 64 ? (a.n < 1 ? 1 : a.n) : 64));
            SS_LAUNCH("k_norm_bwd_weights_wide", s,
                      k_norm_bwd_weights_wide<T><<<g, kThreads, 0, s>>>(static_cast<const T *>(a.dy), a.dys,
                                                                        static_cast<const T *>(a.x), a.xs, a.n, a.D,
                                                                        a.mean, a.rstd, a.part));
            SS_LAUNCH("k_norm_bwd_final", s,
                      k_norm_bwd_final<<<(2 * a.D + 31) / 32, 1024, 0, s>>>(a.part, int(g.y), a.D, a.dgamma, a.dbeta,
                                                                            a.pdt));
        }
        if (a.n == 0) return;
        SS_LAUNCH("k_norm_bwd_rows_wide", s,
                  k_norm_bwd_rows_wide<T><<<grid_of(a.n, 1, 8, sms), kThreads, 0, s>>>(
                      static_cast<const T *>(a.dy), a.dys, static_cast<const T *>(a.x), a.xs, a.n, a.D, a.gamma, a.pdt,
                      a.mean, a.rstd, static_cast<T *>(a.dx), a.dxs));
    } else if (a.D % kVec == 0 && aligned_to(a.dy, 16) && aligned_to(a.x, 16) && aligned_to(a.dx, 16) &&
               a.dys % kVec == 0 && a.xs % kVec == 0 && a.dxs % kVec == 0) {
        pick_nv<T, kVec>(a, sms, s);
    } else {
        pick_nv<T, 1>(a, sms, s);
    }
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
        launch_fwd<float>(a, sms, s);
    else if (dtype == SS_F16)
        launch_fwd<__half>(a, sms, s);
    else
        launch_fwd<__nv_bfloat16>(a, sms, s);
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
        launch_bwd<float>(a, sms, s);
    else if (dtype == SS_F16)
        launch_bwd<__half>(a, sms, s);
    else
        launch_bwd<__nv_bfloat16>(a, sms, s);
    return check_launch(who);
}

}  // extern "C"
