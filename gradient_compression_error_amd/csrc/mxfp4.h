// What the MXFP4 sources share: the layout of a matrix and its scales.
#pragma once

#include "gc_common.h"

namespace gc {

constexpr int64_t MX_MAX_ENTRIES = int64_t(1) << 34;   // entries of one matrix, padded columns included

// A row is held in groups of 128 columns: 64 bytes of codes, 4 scale bytes.
inline int64_t mx_groups(int64_t cols) { return (cols + 127) / 128; }
inline int64_t mx_code_bytes(int64_t rows, int64_t cols) { return rows * mx_groups(cols) * 64; }
inline int64_t mx_scale_bytes(int64_t rows, int64_t cols) { return rows * mx_groups(cols) * 4; }
inline bool mx_shape_ok(int64_t rows, int64_t cols) {
    return rows >= 1 && cols >= 1 && cols <= MX_MAX_ENTRIES && rows <= MX_MAX_ENTRIES / (mx_groups(cols) * 128);
}

constexpr int64_t MX_MAX_DIM = int64_t(1) << 30;       // rows or columns of a product
constexpr int64_t MX_MAX_K = int64_t(1) << 24;         // its depth: 256 rows of codes stay within 32-bit offsets

constexpr int MX_MAX_MESSAGES = 1 << 20;               // of a decode; with strides of up to 2^40 bytes
constexpr int64_t MX_MAX_SPAN = int64_t(1) << 40;      // entries between a pitched matrix's first and last row

int mx_check_matrix(const char* fn, const char* name, const void* codes, const void* scales);

typedef float f32x2 __attribute__((ext_vector_type(2)));

// Rows may start anywhere: vector accesses that need the alignment of an entry only.
typedef unsigned u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef unsigned u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Two float32 as packed bf16 (round to nearest even), the first in the low half.
__device__ __forceinline__ unsigned pack_bf16(float a, float b) {
    const bf16x2 r = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
    return __builtin_bit_cast(unsigned, r);
}

// Workgroups b, b + 8, ... run on one XCD: gives XCD x the x-th stretch of the work
// in order, so that its L2 serves what neighbours share.
__device__ __forceinline__ unsigned xcd_place(unsigned b, unsigned count) {
    const unsigned per = count / 8, more = count % 8, x = b % 8;
    return x * per + min(x, more) + b / 8;
}

}  // namespace gc
