// tensor_map.h -- TMA descriptors of token rows (host side; internal to libretnet.so).
#pragma once

#include <cuda.h>
#include <stdint.h>

namespace retnet {

// Rows of bf16 elements `stride` elements apart, `cols` of them (a multiple of 64) contiguous in each, as
// a map of (column of 64, row, block of 64 columns): a box is box_blocks blocks of box_rows rows of 128
// bytes, each block in the 128-byte swizzle.  Rows past the last read as zeros.  base 16-byte aligned,
// stride a multiple of 8.  False without the driver's entry point.
bool encode_token_rows(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int64_t stride, int box_rows,
                       int box_blocks);

}  // namespace retnet
