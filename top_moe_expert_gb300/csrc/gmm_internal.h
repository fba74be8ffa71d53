// gmm_internal.h -- pieces shared by the ragged grouped products.
#pragma once

#include <cuda.h>
#include <stdint.h>

namespace moe {

// Tensor map of rank 2 ([d1][d0]) or 3 ([d2][d1][d0]), densely packed, box b0 x
// b1 (x 1), swizzled over b0 elements (128 or 64 bytes).
// Reads past d0 or d1 give zeros.
bool tmap_tile(CUtensorMap *m, int rank, CUtensorMapDataType t, int elem_bytes, const void *base, uint64_t d0, uint64_t d1,
             uint64_t d2, uint32_t b0, uint32_t b1,
               CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B);

// The map that drain_rows stores through: 32 columns x 32 rows of [rows][cols].
inline bool tmap_rows_out(CUtensorMap *m, CUtensorMapDataType t, int elem_bytes, const void *base, uint64_t cols,
                          uint64_t rows)
{
    return tmap_tile(m, 2, t, elem_bytes, base, cols, rows, 1, 32, 32,
                     elem_bytes == 4 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

}  // namespace moe
