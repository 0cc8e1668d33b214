// Rows packed into 8 bits and unpacked (model: include/ss_rows8.h).
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "ss_internal.h"
#include "ss_profile.h"
#include "ss_rows8.cuh"
#include "ss_unit.cuh"

namespace ss {
namespace {

constexpr int kThreads = 256;

// A thread a unit at a time.  A row takes whole groups of four lanes (its last lanes may
// have no unit), so that a group's maximum is two shuffles.  The units of all rows lie
// one after the other along the threads of the grid; a thread's next unit is a grid's
// threads on, and its row and column follow by additions.
struct Walk {
    int64_t n, row, rows;       // rows: whole rows in a grid's threads
    int per_row, u, more;       // more: and units beyond them
    __device__ __forceinline__ Walk(int64_t n_, int32_t D) : n(n_) {
        per_row = groups_of(D) * (kGroup / kUnit);
        const int64_t k = int64_t(blockIdx.x) * kThreads + threadIdx.x, step = int64_t(gridDim.x) * kThreads;
        row = k / per_row, u = int(k - row * per_row);
        rows = step / per_row, more = int(step - rows * per_row);
    }
    __device__ __forceinline__ void next() {
        row += rows, u += more;
        if (u >= per_row) u -= per_row, ++row;
    }
    // Elements of this unit that are a row's.
    __device__ __forceinline__ int count(int32_t D) const {
        const int c = D - u * kUnit;
        return row >= n || c <= 0 ? 0 : (c < kUnit ? c : kUnit);
    }
};

// Bound by memory.  A unit at a time and many warps (2M x 48 float32: 79 us by ncu; a call 82, with
// two units' loads in flight 87, four 92, with the registers that they take).
template <typename T, int FMT, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) k_rows8_pack(const T *x, int64_t xs, int64_t n, int32_t D, Rows8 out) {
    for (Walk w(n, D); __any_sync(0xffffffffu, w.row < n); w.next()) {
        const int count = w.count(D);
        F2 f[4];
        floats_of(f, load_unit<T, ALIGNED>(x + w.row * xs + w.u * kUnit, count));
        const uint32_t e = group_exponent<FMT>(f);
        if (count > 0) put_unit<FMT>(out, w.row, w.u, e, f);
    }
}

template <typename T>
__device__ __forceinline__ F2 held_to(F2 v) { return v; }
// Finite values stay finite.
template <>
__device__ __forceinline__ F2 held_to<__half>(F2 v) {
    return make_float2(isnan(v.x) ? v.x : fminf(fmaxf(v.x, -65504.0f), 65504.0f),
                       isnan(v.y) ? v.y : fminf(fmaxf(v.y, -65504.0f), 65504.0f));
}

// 2M x 48 to float32 (484 MB, four fifths of it stores): 75 us by ncu.  Where x's rows start off their blocks' boundaries,
// units lie on them all the same, and take what is held from two units (one more of them a row then).
template <typename T, int FMT, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) k_rows8_unpack(Rows8 in, int64_t n, int32_t D, T *x, int64_t xs) {
    for (Walk w(n, ALIGNED ? D : D + kUnit - 1); w.row < n; w.next()) {
        T *at = x + w.row * xs;
        const int head = ALIGNED ? 0 : head_of<T>(at), column = w.u * kUnit - head;
        if (column >= D) continue;
        F2 f[4];
        if constexpr (ALIGNED) {
            Held h;
            h.load(in, w.row, w.u, true);
            h.values<FMT>(f);
        } else {
            HeldAcross h;
            h.load(in, w.row, column, D, true);
            h.values<FMT>(f, column);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = held_to<T>(f[i]);
        store_block(at + column, raw_of<T>(f), w.u == 0 ? head : 0, D - column < kUnit ? D - column : kUnit);
    }
}

int grid_for(int64_t n, int32_t D, int sms, int per_sm) {
    const int64_t ctas = (n * groups_of(D) * (kGroup / kUnit) + kThreads - 1) / kThreads;
    return int(ctas < int64_t(sms) * per_sm ? ctas : int64_t(sms) * per_sm);
}

}  // namespace
}  // namespace ss

using namespace ss;

extern "C" {

ss_status ss_rows8_pack(const void *x, ss_dtype dtype, int64_t x_stride, int64_t n, int32_t D, const ss_rows8 *out,
                        ss_stream_t stream) {
    clear_error();
    const char *who = "ss_rows8_pack";
    ss_status st = check_row_sizes(who, n, D);
    if (st != SS_OK) return st;
    if ((st = check_row_types(who, dtype, SS_F32)) != SS_OK) return st;
    if (n == 0) return SS_OK;
    if ((st = check_row_tensor(who, "x", x, x_stride, D, dtype)) != SS_OK) return st;
    if ((st = check_rows8(who, "out", out, D)) != SS_OK) return st;
    int dev = 0, sms = 0;
    if ((st = current_device(&dev, &sms, "ss_rows8_pack: device query")) != SS_OK) return st;
    cudaStream_t s = (cudaStream_t)stream;
    const Rows8 o = rows8_of(out);
    with_type(dtype, [&](auto t) {
        using T = decltype(t);
        const T *p = static_cast<const T *>(x);
        const int grid = grid_for(n, D, sms, 16);
        const bool aligned = units_aligned<T>(x, x_stride);
        with_format(out->format, [&](auto F) {
            constexpr int FMT = decltype(F)::value;
            if (aligned)
                SS_LAUNCH("k_rows8_pack", s, k_rows8_pack<T, FMT, true><<<grid, kThreads, 0, s>>>(p, x_stride, n, D, o));
            else
                SS_LAUNCH("k_rows8_pack", s, k_rows8_pack<T, FMT, false><<<grid, kThreads, 0, s>>>(p, x_stride, n, D, o));
        });
    });
    return check_launch(who);
}

ss_status ss_rows8_unpack(const ss_rows8 *in, int64_t n, int32_t D, void *x, ss_dtype dtype, int64_t x_stride,
                          ss_stream_t stream) {
    clear_error();
    const char *who = "ss_rows8_unpack";
    ss_status st = check_row_sizes(who, n, D);
    if (st != SS_OK) return st;
    if ((st = check_row_types(who, dtype, SS_F32)) != SS_OK) return st;
    if (n == 0) return SS_OK;
    if ((st = check_rows8(who, "in", in, D)) != SS_OK) return st;
    if ((st = check_row_tensor(who, "x", x, x_stride, D, dtype)) != SS_OK) return st;
    int dev = 0, sms = 0;
    if ((st = current_device(&dev, &sms, "ss_rows8_unpack: device query")) != SS_OK) return st;
    cudaStream_t s = (cudaStream_t)stream;
    const Rows8 r = rows8_of(in);
    with_type(dtype, [&](auto t) {
        using T = decltype(t);
        T *p = static_cast<T *>(x);
        const int grid = grid_for(n, D, sms, 16);
        const bool aligned = units_aligned<T>(x, x_stride);
        with_format(in->format, [&](auto F) {
            constexpr int FMT = decltype(F)::value;
            if (aligned)
                SS_LAUNCH("k_rows8_unpack", s, k_rows8_unpack<T, FMT, true><<<grid, kThreads, 0, s>>>(r, n, D, p, x_stride));
            else
                SS_LAUNCH("k_rows8_unpack", s, k_rows8_unpack<T, FMT, false><<<grid, kThreads, 0, s>>>(r, n, D, p, x_stride));
        });
    });
    return check_launch(who);
}

}  // extern "C"
