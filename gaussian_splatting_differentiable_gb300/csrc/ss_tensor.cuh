// Wrappers of the instructions that the matrix products are made of: barriers in shared
// memory, the copy engine, the tensor cores and their memory.  Every wait has an end.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "ss_internal.h"

namespace ss {

__device__ __forceinline__ uint32_t smem_of(const void *p) { return uint32_t(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void barrier_init(uint64_t *b, uint32_t count) {
    asm volatile("mbarrier.init.shared.b64 [%0], %1;" ::"r"(smem_of(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void barrier_arrive(uint64_t *b) {
    asm volatile("mbarrier.arrive.shared.b64 _, [%0];" ::"r"(smem_of(b)) : "memory");
}
// Waits for the phase of that parity to end; false after so many tries, each of which may
// itself wait: something has gone wrong then.
constexpr uint32_t kWaitTries = 1u << 20;
__device__ __forceinline__ bool barrier_try(uint64_t *b, uint32_t parity) {
    uint32_t done;
    asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
                 : "=r"(done) : "r"(smem_of(b)), "r"(parity) : "memory");
    return done;
}
__device__ __forceinline__ bool barrier_wait(uint64_t *b, uint32_t parity, uint32_t tries) {
    while (!barrier_try(b, parity))
        if (--tries == 0) return false;
    return true;
}
// The same by a whole warp, with one answer for all of its lanes: they go on together.
__device__ __forceinline__ bool warp_wait(uint64_t *b, uint32_t parity, uint32_t tries) {
    return __all_sync(0xffffffffu, barrier_wait(b, parity, tries));
}
__device__ __forceinline__ void writes_to_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// A map's box at (column, row), zeros outside the matrix.
__device__ __forceinline__ void copy_box(uint32_t smem, const CUtensorMap *map, int column, int row, uint64_t *b) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
                 ::"r"(smem), "l"(map), "r"(column), "r"(row), "r"(smem_of(b)) : "memory");
}
__device__ __forceinline__ void barrier_expect(uint64_t *b, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared.b64 _, [%0], %1;" ::"r"(smem_of(b)), "r"(bytes) : "memory");
}

// 64 columns of 128 bytes a row, swizzled, columns side by side: blocks of 64
// columns BLOCK apart, groups of 8 rows 1 KB apart.
template <int BLOCK>
__device__ __forceinline__ uint64_t operand_at(uint32_t smem) {
    return uint64_t((smem & 0x3ffff) >> 4) | uint64_t(BLOCK >> 4) << 16 | uint64_t(1024 >> 4) << 32 | uint64_t(1) << 46 |
           uint64_t(2) << 61;
}
// bfloat16 x bfloat16 into float32, both operands MN-major, 128 x n.
__device__ __forceinline__ uint32_t product_of(int n) {
    return 1u << 4 | 1u << 7 | 1u << 10 | 1u << 15 | 1u << 16 | uint32_t(n >> 3) << 17 | uint32_t(128 >> 4) << 24;
}
__device__ __forceinline__ void product(uint32_t d, uint64_t a, uint64_t b, uint32_t what, bool add) {
    asm volatile("{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\n"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d), "l"(a), "l"(b), "r"(what),
                 "r"(uint32_t(add)) : "memory");
}
__device__ __forceinline__ void products_arrive(uint64_t *b) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_of(b)) : "memory");
}
__device__ __forceinline__ void tensor_load8(uint32_t (&v)[8], uint32_t at) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(at));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tensor_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tensor_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Tensor memory, by one whole warp.
template <int COLUMNS>
__device__ __forceinline__ void tensor_take(uint32_t *at) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_of(at)), "n"(COLUMNS) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
template <int COLUMNS>
__device__ __forceinline__ void tensor_free(uint32_t tensor) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tensor), "n"(COLUMNS));
}

// The driver's function that describes a matrix to the copy engine.
using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                              const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline ss_status encoder(EncodeFn *fn, const char *who) {
    static std::atomic<EncodeFn> known{nullptr};
    *fn = known.load(std::memory_order_acquire);
    if (*fn) return SS_OK;
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    const ss_status st =
        check_cuda(cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q), who);
    if (st != SS_OK) return st;
    if (q != cudaDriverEntryPointSuccess || !p) return fail(SS_ERR_CUDA, "%s: the driver has no cuTensorMapEncodeTiled", who);
    *fn = reinterpret_cast<EncodeFn>(p);
    known.store(*fn, std::memory_order_release);
    return SS_OK;
}

// A matrix (rows of `columns`, `stride` bytes apart) in boxes of box_columns x box_rows, side by side
// as they lie, or (64 columns of bfloat16) swizzled as the products read them.
inline ss_status map_of(CUtensorMap *map, CUtensorMapDataType type, const void *p, int64_t rows, int64_t columns, int64_t stride,
                        int box_columns, int box_rows, bool swizzled, const char *who) {
    EncodeFn encode;
    const ss_status st = encoder(&encode, who);
    if (st != SS_OK) return st;
    const cuuint64_t dims[2] = {cuuint64_t(columns), cuuint64_t(rows)}, strides[1] = {cuuint64_t(stride)};
    const cuuint32_t box[2] = {cuuint32_t(box_columns), cuuint32_t(box_rows)}, each[2] = {1, 1};
    const CUresult r = encode(map, type, 2, const_cast<void *>(p), dims, strides, box, each, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              swizzled ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? SS_OK : fail(SS_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed (%d)", who, int(r));
}
inline ss_status map_of(CUtensorMap *map, const void *p, int64_t rows, int64_t columns, int64_t stride, int box_rows,
                        const char *who) {
    return map_of(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p, rows, columns, stride * 2, 64, box_rows, true, who);
}

}  // namespace ss
