// What the kernels over the entries of low-precision matrices share: loads, stores and launches.
#pragma once

#include <algorithm>

#include "mxfp4.h"

namespace gc {
namespace {

constexpr int MX_THREADS = 256;
constexpr int MX_MAXGRID = 1 << 20;   // workgroups of a launch; more work loops

unsigned grid_of(long long work) { return static_cast<unsigned>(std::min<long long>(work, MX_MAXGRID)); }

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ unsigned max_u16(unsigned a, unsigned b) {        // of either half
    return __builtin_bit_cast(unsigned, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}

// Eight neighbouring entries of a row as they are held: bf16 pairs, or float32.
template <bool BF16>
struct Entries8;
template <>
struct Entries8<true> {
    unsigned w[4];
    __device__ __forceinline__ void load(const void* p, long long i) {
        const u32x4_any v = *reinterpret_cast<const u32x4_any*>(reinterpret_cast<const unsigned short*>(p) + i);
        w[0] = v[0]; w[1] = v[1]; w[2] = v[2]; w[3] = v[3];
    }
    __device__ __forceinline__ void load(const void* p, long long i, int count) {   // the first `count` of them, zeros behind
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const unsigned short* q = reinterpret_cast<const unsigned short*>(p) + i + 2 * c;
            w[c] = (2 * c < count ? q[0] : 0u) | (2 * c + 1 < count ? static_cast<unsigned>(q[1]) << 16 : 0u);
        }
    }
};
template <>
struct Entries8<false> {
    float v[8];
    __device__ __forceinline__ void load(const void* p, long long i) {
        const f32x4_any* q = reinterpret_cast<const f32x4_any*>(reinterpret_cast<const float*>(p) + i);
        const f32x4_any a = q[0], b = q[1];
        v[0] = a[0]; v[1] = a[1]; v[2] = a[2]; v[3] = a[3];
        v[4] = b[0]; v[5] = b[1]; v[6] = b[2]; v[7] = b[3];
    }
    __device__ __forceinline__ void load(const void* p, long long i, int count) {
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = c < count ? reinterpret_cast<const float*>(p)[i + c] : 0.0f;
    }
};

// N entries of out from `at` on, sixteen bytes at a time.
template <bool BF16, int N>
__device__ __forceinline__ void load_out(const void* p, long long at, float (&v)[N]) {
    constexpr int M = BF16 ? 8 : 4;
    static_assert(N % M == 0, "whole accesses");
    const u32x4_any* from = reinterpret_cast<const u32x4_any*>(reinterpret_cast<const char*>(p) + at * (BF16 ? 2 : 4));
#pragma unroll
    for (int o = 0; o < N; o += M) {
        const u32x4_any w = __builtin_nontemporal_load(from + o / M);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if constexpr (BF16) {
                v[o + 2 * q] = __uint_as_float(w[q] << 16);
                v[o + 2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
            } else {
                v[o + q] = __uint_as_float(w[q]);
            }
        }
    }
}
template <bool BF16, int N>
__device__ __forceinline__ void store_out(void* p, long long at, const float (&v)[N]) {
    constexpr int M = BF16 ? 8 : 4;
    static_assert(N % M == 0, "whole accesses");
    u32x4_any* to = reinterpret_cast<u32x4_any*>(reinterpret_cast<char*>(p) + at * (BF16 ? 2 : 4));
#pragma unroll
    for (int o = 0; o < N; o += M) {
        u32x4_any w;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if constexpr (BF16) w[q] = pack_bf16(v[o + 2 * q], v[o + 2 * q + 1]);
            else w[q] = __float_as_uint(v[o + q]);
        }
        __builtin_nontemporal_store(w, to + o / M);
    }
}

template <bool BF16>
__device__ __forceinline__ void store1(void* p, long long i, float v) {
    if constexpr (BF16) reinterpret_cast<unsigned short*>(p)[i] = static_cast<unsigned short>(pack_bf16(v, 0.0f));
    else reinterpret_cast<float*>(p)[i] = v;
}

// Unit `u` of a matrix of `per_row` units a row, found from the
// workgroup's first unit by one uniform 64-bit division and a 32-bit one.
struct Unit {
    long long row;
    int unit;
};
__device__ __forceinline__ Unit unit_of(long long base, unsigned per_row) {
    const long long row0 = base / per_row;
    const unsigned r = static_cast<unsigned>(base - row0 * per_row) + threadIdx.x;
    return {row0 + r / per_row, static_cast<int>(r % per_row)};
}

}  // namespace
}  // namespace gc
