// tensor_map.h -- TMA descriptors of token rows (host side; internal to libretnet.so).
#pragma once

#include <cuda.h>
#include <stdint.h>

namespace retnet {

// Rows of bf16 elements `stride` elements apart, `cols` of them contiguous in each, as a tensor map
// whose box is 64 columns x `box_rows` rows in the 128-byte swizzle; rows past the last read as zeros.
// base 16-byte aligned, stride and cols multiples of 8.  False without the driver's entry point.
bool encode_token_rows(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int64_t stride, int box_rows);

}  // namespace retnet
