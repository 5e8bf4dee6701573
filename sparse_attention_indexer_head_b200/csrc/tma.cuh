// TMA tensor maps (host) and 2-D tiled TMA loads (device).
//
// The encoder, cuTensorMapEncodeTiled, is a driver-API entry point; it is
// fetched once through cudaGetDriverEntryPoint so the library needs no link
// against libcuda. Only the CUtensorMap type and enums come from <cuda.h>.
#pragma once

#include <cuda.h>

#include "common.cuh"

namespace dsa {

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_tiled() {
    static EncodeTiledFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return (EncodeTiledFn) nullptr;
        return reinterpret_cast<EncodeTiledFn>(p);
    }();
    return fn;
}

// Row-major bf16 matrix [rows, cols] (row stride in bytes), boxes of
// box_cols x box_rows elements landing in shared memory with the 128-byte
// swizzle. Rows outside [0, rows) read as zero.
inline bool make_map_bf16_2d(CUtensorMap *m, const void *base, uint64_t rows, uint64_t cols,
                             uint64_t row_stride_bytes, uint32_t box_cols, uint32_t box_rows) {
    const EncodeTiledFn fn = encode_tiled();
    if (!fn || rows == 0) return false;
    cuuint64_t dims[2] = {cols, rows};
    cuuint64_t strides[1] = {row_stride_bytes};
    cuuint32_t box[2] = {box_cols, box_rows};
    cuuint32_t elem[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box,
              elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Row-major bf16 matrix [rows, 64 * atoms] seen as [atoms][rows][64]: a box is
// box_atoms columns of 64 channels (128 bytes) by box_rows rows, each column of
// the box landing as box_rows 128-byte rows with the 128-byte swizzle.
inline bool make_map_bf16_atoms(CUtensorMap *m, const void *base, uint64_t rows, uint32_t atoms,
                                uint32_t box_rows, uint32_t box_atoms) {
    const EncodeTiledFn fn = encode_tiled();
    if (!fn || rows == 0) return false;
    cuuint64_t dims[3] = {64, rows, atoms};
    cuuint64_t strides[2] = {(cuuint64_t)atoms * 128, 128};
    cuuint32_t box[3] = {64, box_rows, box_atoms};
    cuuint32_t elem[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box,
              elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tiled 2-D load of the box at element coordinates (x = column, y = row) into
// shared memory at dst, completing on bar through the transaction count. x is
// a multiple of 64 elements (128 bytes) at every call site.
DSA_DEVINL void tma_load_2d(uint32_t dst, const CUtensorMap *map, int x, int y, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar))
        : "memory");
}

// The same for a 3-D map: the box at (x = column, y = row, z = plane).
DSA_DEVINL void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

}  // namespace dsa
