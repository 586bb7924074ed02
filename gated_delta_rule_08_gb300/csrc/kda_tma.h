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

// 4-D map over a paged cache [blocks, tokens of a block, heads, d] of bf16 whose strides are in elements (multiples of
// 8), read in boxes of box_tokens tokens of one head x 64 values, with the 128-byte swizzle: coordinates
// {value, token, head, block}.  Blocks past the end read as zeros.
bool tensor_map_cache(CUtensorMap* map, const void* base, uint64_t blocks, uint64_t tokens, uint64_t heads, uint64_t d,
                      uint64_t block_stride, uint64_t token_stride, uint64_t head_stride, uint32_t box_tokens);

// 3-D map over token rows [tokens, heads, d] of bf16, tokens token_stride elements apart (a multiple of 8), read in
// boxes of box_tokens x box_heads x 64 values, with the 128-byte swizzle: coordinates {value, head, token}.
bool tensor_map_rows(CUtensorMap* map, const void* base, uint64_t tokens, uint64_t heads, uint64_t d,
                     uint64_t token_stride, uint32_t box_tokens, uint32_t box_heads);

}  // namespace kda
