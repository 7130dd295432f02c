// tilemap.h -- TMA maps of the 8-bit matrices.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace moe {

// The map of a row-major [rows][k] matrix of bytes whose tiles are box_rows
// rows of 128 bytes, swizzled as the tensor cores read them; rows outside
// the matrix read as zeros.  Valid for one call's launch: nothing is kept.
cudaError_t tile_map(CUtensorMap *map, const void *base, int64_t rows, int k, int box_rows);

}  // namespace moe
