// Tiled tensor maps of the pools (host).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime_api.h>
#include <stdint.h>

#include <mutex>

namespace pkv {

// The driver's tiled tensor-map encoder (a host computation), looked up once.
inline PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// A pool [num_blocks][H][B][D] seen as rows of D 16-bit elements; boxes of
// 64 columns x box_rows rows, 128-byte swizzle.
inline bool pool_map(CUtensorMap* m, bool bf16, const void* pool, int64_t rows, int D, int box_rows) {
    const PFN_cuTensorMapEncodeTiled_v12000 fn = map_encoder();
    if (!fn || rows >= (1LL << 31)) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)D * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
              const_cast<void*>(pool), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same pool as rows of D / 64 lines of 64 elements; boxes of box_rows whole
// rows, 128-byte swizzle over the lines in row order.
inline bool row_map(CUtensorMap* m, bool bf16, const void* pool, int64_t rows, int D, int box_rows) {
    const PFN_cuTensorMapEncodeTiled_v12000 fn = map_encoder();
    if (!fn || rows >= (1LL << 31)) return false;
    const cuuint64_t dims[3] = {64, (cuuint64_t)(D / 64), (cuuint64_t)rows};
    const cuuint64_t strides[2] = {128, (cuuint64_t)D * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)(D / 64), (cuuint32_t)box_rows};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
              const_cast<void*>(pool), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace pkv
