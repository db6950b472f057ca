// pa_tmap.h -- tensor maps of packed rows and of the paged pool (host side,
// internal to the library).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime_api.h>

#include <atomic>

#include "paged_gqa.h"

namespace pa {

inline PFN_cuTensorMapEncodeTiled_v12000 tmap_encode_fn() {
    static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> known{nullptr};  // the driver's, the same for every thread
    PFN_cuTensorMapEncodeTiled_v12000 fn = known.load(std::memory_order_relaxed);
    if (!fn) {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess) {
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
            known.store(fn, std::memory_order_relaxed);
        }
    }
    return fn;
}

// 16-bit types, 128-byte swizzle, zeros outside.
inline bool tmap_encode(CUtensorMap* m, pa_dtype dt, int rank, const void* ptr, const cuuint64_t* dims,
                        const cuuint64_t* strides, const cuuint32_t* box) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tmap_encode_fn();
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return enc && enc(m, dt == PA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank,
                      const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Packed rows as (head_dim, head, row); the box is 64 dims x heads x rows.
inline bool tmap_rows(CUtensorMap* m, pa_dtype dt, const void* ptr, int D, int heads, int rows, int64_t stride,
                      int box_heads, int box_rows) {
    const cuuint64_t dims[3] = {cuuint64_t(D), cuuint64_t(heads), cuuint64_t(rows)};
    const cuuint64_t strides[2] = {cuuint64_t(D) * 2, cuuint64_t(stride) * 2};
    const cuuint32_t box[3] = {64, cuuint32_t(box_heads), cuuint32_t(box_rows)};
    return tmap_encode(m, dt, 3, ptr, dims, strides, box);
}

// The pool as (head_dim, kv head, slot, page), the middle two in stride order
// (head_first: the head's stride is not the larger); the box is one page of one
// kv head, 64 dims at a time.
inline bool tmap_pages(CUtensorMap* m, pa_dtype dt, const void* ptr, int D, int heads, int page_size, int pages,
                       int64_t head_stride, int64_t token_stride, int64_t page_stride, bool head_first) {
    const cuuint64_t hs = cuuint64_t(head_stride) * 2, ts = cuuint64_t(token_stride) * 2;
    const cuuint64_t nh = cuuint64_t(heads), P = cuuint64_t(page_size);
    const cuuint64_t dims[4] = {cuuint64_t(D), head_first ? nh : P, head_first ? P : nh, cuuint64_t(pages)};
    const cuuint64_t strides[3] = {head_first ? hs : ts, head_first ? ts : hs, cuuint64_t(page_stride) * 2};
    const cuuint32_t box[4] = {64, head_first ? 1u : cuuint32_t(P), head_first ? cuuint32_t(P) : 1u, 1};
    return tmap_encode(m, dt, 4, ptr, dims, strides, box);
}

}  // namespace pa
