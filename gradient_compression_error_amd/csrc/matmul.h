// What the matrix products share: copies from memory into LDS and their waits, rows of out, the join of parts of k.
#pragma once

#include "mxfp4.h"

namespace gc {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

enum { OUT_F32, OUT_F32_ADD, OUT_BF16, OUT_BF16_ADD, OUT_PART };

constexpr int MAX_SPLITS = 8;   // parts of k

// Sixteen bytes of a row of out, past the caches' replacement order: a tile is
// written (and, when adding, read) once, and what the L2 holds of the operands is
// worth more (8192^3 to bf16: 278 us with plain stores, 261 us with these).
template <bool BF16>
__device__ __forceinline__ u32x4_any load16(const void* out, long long at) {
    return __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(reinterpret_cast<const char*>(out) + at * (BF16 ? 2 : 4)));
}
template <bool BF16, int N>
__device__ __forceinline__ void add16(float (&v)[N], u32x4_any old) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if constexpr (BF16) {
            v[2 * q] += __uint_as_float(old[q] << 16);
            v[2 * q + 1] += __uint_as_float(old[q] & 0xFFFF0000u);
        } else {
            v[q] += __uint_as_float(old[q]);
        }
    }
}
template <bool BF16, bool STREAM = true, int N>
__device__ __forceinline__ void store16(void* out, long long at, const float (&v)[N]) {
    u32x4_any w;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if constexpr (BF16) w[q] = pack_bf16(v[2 * q], v[2 * q + 1]);
        else w[q] = __float_as_uint(v[q]);
    }
    u32x4_any* const to = reinterpret_cast<u32x4_any*>(reinterpret_cast<char*>(out) + at * (BF16 ? 2 : 4));
    if constexpr (STREAM) __builtin_nontemporal_store(w, to);
    else *to = w;                                           // a part that is read again at once
}

// Writes (or adds) up to N neighbours of a row of out, `left` of them inside it; N entries are 16 bytes.
template <bool BF16, bool ADD, int N>
__device__ __forceinline__ void put(void* out, long long at, float (&v)[N], int left) {
    if (left >= N) {
        if constexpr (ADD) add16<BF16>(v, load16<BF16>(out, at));
        store16<BF16>(out, at, v);
    } else {
#pragma unroll
        for (int q = 0; q < N; ++q) {
            if (q < left) {
                float w = v[q];
                if constexpr (ADD) w += load_grad1<BF16>(out, at + q);
                if constexpr (BF16) reinterpret_cast<unsigned short*>(out)[at + q] = static_cast<unsigned short>(pack_bf16(w, 0.0f));
                else reinterpret_cast<float*>(out)[at + q] = w;
            }
        }
    }
}

// Writes (or adds) up to four neighbours of a row of out, `left` of them inside it.
template <bool BF16>
__device__ __forceinline__ void put4(void* out, long long at, f32x4 v, int left, bool add) {
    if (left >= 4) {
        if constexpr (BF16) {
            u32x2_any* to = reinterpret_cast<u32x2_any*>(reinterpret_cast<unsigned short*>(out) + at);
            if (add) {
                const u32x2_any o = *to;
                v += f32x4{__uint_as_float(o[0] << 16), __uint_as_float(o[0] & 0xFFFF0000u), __uint_as_float(o[1] << 16),
                           __uint_as_float(o[1] & 0xFFFF0000u)};
            }
            *to = u32x2_any{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
        } else {
            f32x4_any* to = reinterpret_cast<f32x4_any*>(reinterpret_cast<float*>(out) + at);
            if (add) v += *to;
            *to = v;
        }
    } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (q < left) {
                float w = v[q];
                if (add) w += load_grad1<BF16>(out, at + q);
                if constexpr (BF16) reinterpret_cast<unsigned short*>(out)[at + q] = static_cast<unsigned short>(pack_bf16(w, 0.0f));
                else reinterpret_cast<float*>(out)[at + q] = w;
            }
        }
    }
}

// Copies 16 (or 4) bytes a lane from memory straight into LDS: the wave's lanes
// land one after the other from LDS address `to`.  Written as assembly since the
// compiler otherwise waits for every outstanding copy before any LDS read; the
// kernel counts them itself (wait_for).  No register is written, so nothing can
// be reused under a copy in flight.
__device__ __forceinline__ void copy16(const unsigned char* base, unsigned offset, unsigned to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to), "v"(offset), "s"(base) : "memory", "m0");
}
__device__ __forceinline__ void copy4(const unsigned char* base, unsigned offset, unsigned to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(to), "v"(offset), "s"(base) : "memory", "m0");
}

// Waits until at most VM of this wave's copies are outstanding.
template <int VM>
__device__ __forceinline__ void wait_for() {
    static_assert(VM >= 0 && VM < 64, "vmcnt has six bits");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(VM) : "memory");
}

// All waves of the workgroup; no memory access is moved over it by the compiler.
__device__ __forceinline__ void meet() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Waits until all of this wave's LDS reads are back.
__device__ __forceinline__ void wait_reads() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// Uses a value that was read from LDS, so that the compiler waits for that read here,
// counting the ones issued since by itself.
template <typename T>
__device__ __forceinline__ void arrived(const T& v) { asm volatile("" ::"v"(v) : "memory"); }

// Joins the parts of k: out = [out +] the sum of `splits` float32 matrices m x n
// (rows ldp entries apart), added in order, so that every run gives the same bits.
template <bool BF16>
__device__ __forceinline__ void join_parts(const float* parts, int splits, long long split_floats, int m, int n, int ldp, void* out,
                                           long long ldo, bool add) {
    const unsigned quads = ldp / 4;
    for (long long q = blockIdx.x * 256ll + threadIdx.x; q < static_cast<long long>(m) * quads; q += gridDim.x * 256ll) {
        const int row = static_cast<int>(q / quads), col = static_cast<int>(q % quads) * 4;
        f32x4 part[MAX_SPLITS];                              // loaded together, then added in order
#pragma unroll
        for (int s = 0; s < MAX_SPLITS; ++s)
            if (s < splits) part[s] = *reinterpret_cast<const f32x4*>(parts + s * split_floats + q * 4);
        f32x4 v = part[0];
#pragma unroll
        for (int s = 1; s < MAX_SPLITS; ++s)
            if (s < splits) v += part[s];
        put4<BF16>(out, row * ldo + col, v, n - col, add);
    }
}

int64_t tiles_of(int64_t m, int64_t n, int64_t tm, int64_t tn) { return ((m + tm - 1) / tm) * ((n + tn - 1) / tn); }

}  // namespace
}  // namespace gc
