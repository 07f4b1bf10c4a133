// Which bytes of an operand the int8 products may load. Plain C++, constexpr,
// so that the kernels (gemm_i8.hip) and a test on the host take the same
// functions.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace moe {

// Byte offset, from a tile's first row on, of K byte `at` of the tile's row r;
// rows past the operand's last one (`last`, counted from the tile's first) are
// that one again.
constexpr uint32_t row_offset(int r, int last, int K, int at) { return (uint32_t)(r < last ? r : last) * (uint32_t)K + (uint32_t)at; }

// Record count of an operand of n bytes from a tile's first row on. (2^31 - 16
// at most: 256 rows of the longest K end far below that.)
constexpr int records(size_t n) { return n > 0x7FFFFFF0u ? 0x7FFFFFF0 : (int)n; }

// The records that are left from K position k0 >= 0 on. Lane offsets below this
// are loaded, the rest is dropped; offsets, positions and operands are
// multiples of 16 bytes, so a 16-byte access lies on one side. From NOWHERE on
// no operand has any.
constexpr int NOWHERE = 0x7FFFFFF0;
constexpr int records_from(int all, int k0) { return all - k0 > 0 ? all - k0 : 0; }

}  // namespace moe
