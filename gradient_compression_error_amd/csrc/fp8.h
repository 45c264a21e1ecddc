// The layout of an 8-bit matrix: E4M3 codes with one E8M0 scale for each block of 128 columns by 1 or 128 rows.
#pragma once

#include "mxfp4.h"

namespace gc {

// A row is held in groups of 128 columns, a byte a code.  A row of blocks has one scale
// byte a group, and zeros up to a multiple of four bytes.
inline int64_t f8_code_bytes(int64_t rows, int64_t cols) { return rows * mx_groups(cols) * 128; }
inline int64_t f8_scale_pitch(int64_t cols) { return (mx_groups(cols) + 3) / 4 * 4; }
inline int64_t f8_scale_rows(int64_t rows, int block_rows) { return block_rows == 1 ? rows : (rows + 127) / 128; }
inline int64_t f8_scale_bytes(int64_t rows, int64_t cols, int block_rows) {
    return f8_scale_rows(rows, block_rows) * f8_scale_pitch(cols);
}
inline bool f8_block_ok(int block_rows) { return block_rows == 1 || block_rows == 128; }
inline int f8_shift(int block_rows) { return block_rows == 1 ? 0 : 7; }   // a row's place among the rows of blocks

}  // namespace gc
