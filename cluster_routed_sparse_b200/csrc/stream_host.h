// stream_host.h -- tensor maps of strided [B, H, L, d] views.
#pragma once

#include "stream_internal.h"

namespace ac {

// dims[0] = d, the others with strides in elements; boxes of 64 columns, 128-byte
// swizzle.  The strides of dimensions of one entry are never used: any valid
// value does.
inline cudaError_t map_view(CUtensorMap *tm, const void *base, int rank, const int64_t *dims, const int64_t *strides,
                            const int *box) {
    typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                      const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                      CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static std::atomic<void *> cached{nullptr};
    void *fn = cached.load(std::memory_order_relaxed);
    if (!fn) {
        cudaDriverEntryPointQueryResult q;
        const cudaError_t e = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q);
        if (e != cudaSuccess) return e;
        if (q != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
        cached.store(fn, std::memory_order_relaxed);
    }
    cuuint64_t d[5], st[4];
    cuuint32_t bx[5], es[5];
    for (int i = 0; i < rank; ++i) {
        d[i] = (cuuint64_t)dims[i];
        bx[i] = (cuuint32_t)box[i];
        es[i] = 1;
        if (i > 0) st[i - 1] = dims[i] > 1 ? (cuuint64_t)strides[i] * 2 : (cuuint64_t)dims[0] * 2;
    }
    const CUresult r = reinterpret_cast<EncodeTiledFn>(fn)(
        tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(base), d, st, bx, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Rows of one head: coordinates (column, row, head, sequence), boxes of box_rows rows.
inline cudaError_t map_rows(CUtensorMap *tm, const View &v, int B, int H, int L, int d, int box_rows) {
    const int64_t dims[4] = {d, L, H, B}, st[4] = {1, v.l, v.h, v.b};
    const int box[4] = {64, box_rows, 1, 1};
    return map_view(tm, v.p, 4, dims, st, box);
}

// Rows of the G query heads of a key head, token by token: coordinates (column,
// head within the group, token, key head, sequence), boxes of G heads x TT tokens.
inline cudaError_t map_rows_packed(CUtensorMap *tm, const View &v, int B, int Hk, int G, int L, int d, int TT) {
    const int64_t dims[5] = {d, G, L, Hk, B}, st[5] = {1, v.h, v.l, v.h * G, v.b};
    const int box[5] = {64, G, TT, 1, 1};
    return map_view(tm, v.p, 5, dims, st, box);
}

}  // namespace ac
