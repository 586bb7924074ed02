// Tensor maps for tiled TMA copies (host side).
#pragma once

#include <cuda.h>
#include <stdint.h>

namespace kda {

// 2-D map over `rows` rows of `cols` elements, `row_bytes` apart (a multiple of 16), read in boxes of
// box_rows x box_cols (box_cols elements = 128 bytes) with the 128-byte swizzle; reads past the edges
// give zeros.  The base must be 16-byte aligned.
bool tensor_map_2d(CUtensorMap* map, const void* base, CUtensorMapDataType type, uint64_t rows, uint64_t cols,
                   uint64_t row_bytes, uint32_t box_rows, uint32_t box_cols);

}  // namespace kda
