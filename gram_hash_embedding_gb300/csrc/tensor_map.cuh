// The driver's encoding of a 2-D tiled tensor map (proj.cu), for the kernels that move tiles by TMA.
#pragma once

#include <cuda.h>

#include <cstdint>

namespace engram {

// [rows][cols] elements of `type`, rows `row_bytes` apart, moved in boxes of box_rows x box_cols; reads past the matrix
// are filled with zeros, writes past it dropped. False where the driver refuses it.
bool tensor_map_2d(CUtensorMap* m, CUtensorMapDataType type, const void* ptr, uint64_t rows, uint64_t cols,
                   uint64_t row_bytes, uint32_t box_rows, uint32_t box_cols, CUtensorMapSwizzle swz);

}  // namespace engram
