// Product of two MXFP4 matrices: out[i, j] = [out +] sum_k A[i, k] * B[j, k].
//
// v_mfma_scale_f32_16x16x128_f8f6f4 multiplies 16 x 128 by 128 x 16 E2M1 codes
// with one E8M0 scale per 32 codes and adds in float32.  A lane holds 32
// consecutive codes (16 bytes) of one row, which is one block, and the block's
// scale byte: row lane % 16, block lane / 16 of the step's four.  B goes in as
// the first operand, so that a lane's four results are neighbours in a row of
// out: row lane % 16, columns 4 * (lane / 16) + 0..3.
#include <algorithm>
#include <type_traits>

#include "mxfp4.h"

namespace gc {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int E2M1 = 4;   // operand format of the f8f6f4 matrix instructions

__device__ __forceinline__ f32x4 mfma16(i32x4 a, i32x4 b, f32x4 c, int sa, int sb) {
    const i32x8 x = {a[0], a[1], a[2], a[3], 0, 0, 0, 0}, y = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, E2M1, E2M1, 0, sa, 0, sb);
}

// One wave per 16 x 16 tile of out, operands straight from memory.
template <bool BF16, bool ADD>
__global__ __launch_bounds__(256) void mxfp4_mm(const unsigned char* ac, const unsigned char* as,
                                                const unsigned char* bc, const unsigned char* bs, int m, int n,
                                                int groups, void* out, long long ldo) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const long long tiles_n = (n + 15) / 16, tiles = tiles_n * ((m + 15) / 16);
    for (long long t = static_cast<long long>(blockIdx.x) * 4 + wave; t < tiles; t += static_cast<long long>(gridDim.x) * 4) {
        const int i0 = static_cast<int>(t / tiles_n) * 16, j0 = static_cast<int>(t % tiles_n) * 16;
        const long long ra = min(i0 + (lane & 15), m - 1), rb = min(j0 + (lane & 15), n - 1);
        const int blk = lane >> 4;
        f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int g = 0; g < groups; ++g) {
            const i32x4 a = *reinterpret_cast<const i32x4*>(ac + (ra * groups + g) * 64 + blk * 16);
            const i32x4 b = *reinterpret_cast<const i32x4*>(bc + (rb * groups + g) * 64 + blk * 16);
            acc = mfma16(b, a, acc, bs[(rb * groups + g) * 4 + blk], as[(ra * groups + g) * 4 + blk]);
        }
        const int i = i0 + (lane & 15), j = j0 + 4 * blk;
        if (i >= m) continue;
        for (int q = 0; q < 4; ++q) {
            if (j + q >= n) break;
            const long long at = i * ldo + j + q;
            float v = acc[q];
            if constexpr (ADD) v += load_grad1<BF16>(out, at);
            if constexpr (BF16) reinterpret_cast<unsigned short*>(out)[at] = static_cast<unsigned short>(pack_bf16(v, 0.0f));
            else reinterpret_cast<float*>(out)[at] = v;
        }
    }
}


// Writes (or adds) up to eight neighbours of a row of out, `left` of them inside it.
template <bool BF16, bool ADD>
__device__ __forceinline__ void put8(void* out, long long at, const float (&v)[8], int left, bool wide) {
    if (wide && left >= 8) {
        float w[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) w[q] = v[q];
        if constexpr (ADD) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const float4 o = load_grad4<BF16>(out, at / 4 + q);
                w[4 * q] += o.x; w[4 * q + 1] += o.y; w[4 * q + 2] += o.z; w[4 * q + 3] += o.w;
            }
        }
        if constexpr (BF16) {
            reinterpret_cast<uint4*>(out)[at / 8] = make_uint4(pack_bf16(w[0], w[1]), pack_bf16(w[2], w[3]),
                                                                 pack_bf16(w[4], w[5]), pack_bf16(w[6], w[7]));
        } else {
            reinterpret_cast<float4*>(out)[at / 4] = make_float4(w[0], w[1], w[2], w[3]);
            reinterpret_cast<float4*>(out)[at / 4 + 1] = make_float4(w[4], w[5], w[6], w[7]);
        }
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            if (q < left) {
                float w = v[q];
                if constexpr (ADD) w += load_grad1<BF16>(out, at + q);
                if constexpr (BF16) reinterpret_cast<unsigned short*>(out)[at + q] = static_cast<unsigned short>(pack_bf16(w, 0.0f));
                else reinterpret_cast<float*>(out)[at + q] = w;
            }
        }
    }
}

// ---------------------------------------------------------------- tiled kernel

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

struct Operand {
    const unsigned char* codes;
    const unsigned char* scales;
    int rows;
};

// Workgroup tile BM x BN of out over all of k, waves WM x WN.  Stages of 128
// columns of k (one group) go from memory to LDS, up to four in flight; a wave
// reads the fragments of the next stage while its matrix instructions work on
// the present one.
//
// LDS holds a row's 64 bytes of a group together, its four 16-byte blocks
// permuted so that the 16 rows of a fragment read in one instruction lie in
// different banks: block b of row r at b ^ (r >> 2 & 3) (A), b ^ (r >> 3 & 3) (B).
// Scale bytes come in chunks of four groups (16 bytes of a row, so that a line
// is touched once for four stages), a quarter of a chunk each stage.
template <int BM, int BN, int WM, int WN, bool BF16, bool ADD>
__global__ __launch_bounds__(WM* WN * 64) void mxfp4_tile(const Operand A, const Operand B, int groups, void* out,
                                                        long long ldo) {
    constexpr int S = 4, NW = WM * WN, ROWS = BM + BN;
    constexpr int MI = BM / WM / 16, NI = BN / WN / 16;      // fragments of a wave
    constexpr int CP = ROWS / 16 / NW;                      // 16-row copies of codes a wave makes each stage
    constexpr int PC = ROWS / 64 / NW;                      // 16-row copies of scales a wave makes each stage
    static_assert(CP * 16 * NW == ROWS && PC * 64 * NW == ROWS && NI % 2 == 0 && BM % (16 * NW) == 0, "tile and waves must fit");
    constexpr int STAGE = ROWS * 64, CHUNK = ROWS * 16;
    __shared__ __attribute__((aligned(1024))) unsigned char lds[S * STAGE + 3 * CHUNK];
    unsigned char* const scale_lds = lds + S * STAGE;
    const unsigned lds_at = static_cast<unsigned>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) unsigned char*)lds));

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int i0, j0;
    {
        // workgroups b, b + 8, ... run on one XCD: give it neighbouring tiles, in
        // bands of eight tile rows, so that its L2 serves each operand row many times
        const int tiles_m = (A.rows + BM - 1) / BM, tiles_n = (B.rows + BN - 1) / BN;
        const int tiles = tiles_m * tiles_n, b = blockIdx.x;
        const int per = tiles / 8, more = tiles % 8, x = b % 8;
        const int t = x * per + min(x, more) + b / 8;
        const int band = t / (8 * tiles_n), first = band * 8, height = min(8, tiles_m - first);
        const int in = t - band * 8 * tiles_n;
        i0 = (first + in % height) * BM;
        j0 = in / height * BN;
    }

    // Where this wave's copies come from: a uniform base per operand and a lane's
    // offset (below 2^32: a tile's rows are at most 256 times 2^23 bytes).  Rows
    // past the operand are its last row again; their results are not written.
    const long long pitch = static_cast<long long>(groups) * 64;
    const unsigned char* const base_a = A.codes + i0 * pitch;
    const unsigned char* const base_b = B.codes + j0 * pitch;
    const unsigned char* const sbase_a = A.scales + i0 * (pitch / 16);
    const unsigned char* const sbase_b = B.scales + j0 * (pitch / 16);
    const unsigned left_a = A.rows - 1 - i0, left_b = B.rows - 1 - j0;
    unsigned off[CP], soff[4 * PC];
#pragma unroll
    for (int c = 0; c < CP; ++c) {
        const bool a = c * 16 * NW < BM;
        const unsigned r = (c * NW + wave) * 16 + (lane >> 2) - (a ? 0 : BM);
        const unsigned swz = a ? (r >> 2) & 3 : (r >> 3) & 3;
        off[c] = min(r, a ? left_a : left_b) * static_cast<unsigned>(pitch) + ((lane & 3) ^ swz) * 16;
    }
#pragma unroll
    for (int c = 0; c < 4 * PC; ++c) {
        const bool a = c * 16 * NW < BM;
        const unsigned r = (c * NW + wave) * 16 + (lane >> 2) - (a ? 0 : BM);
        soff[c] = min(r, a ? left_a : left_b) * static_cast<unsigned>(pitch / 16);
    }
    auto copy_codes = [&](int g, int buf) {
        const long long at = static_cast<long long>(min(g, groups - 1)) * 64;
#pragma unroll
        for (int c = 0; c < CP; ++c)
            copy16((c * 16 * NW < BM ? base_a : base_b) + at, off[c], lds_at + buf * STAGE + (c * NW + wave) * 1024);
    };
    auto copy_scales = [&](int chunk, int quarter, int ring) {
        const unsigned gg = min(chunk * 4 + (lane & 3), groups - 1) * 4;
#pragma unroll
        for (int p = 0; p < PC; ++p) {
            const int c = quarter * PC + p;
            copy4(c * 16 * NW < BM ? sbase_a : sbase_b, soff[c] + gg, lds_at + S * STAGE + ring * CHUNK + (c * NW + wave) * 256);
        }
    };

    // Where this wave's fragments lie.  Rows of a pair of B fragments are mixed so
    // that a lane's results are eight neighbours of out.
    const int wm = wave / WN, wn = wave % WN, blk = lane >> 4, i = lane & 15;
    const int ra = wm * (BM / WM) + i, rb = wn * (BN / WN) + 8 * (i >> 2) + (i & 3);
    const int a_at = ra * 64 + ((blk ^ (ra >> 2)) & 3) * 16, as_at = ra * 16 + blk;
    const int b_at = (BM + rb) * 64 + ((blk ^ (rb >> 3)) & 3) * 16, bs_at = (BM + rb) * 16 + blk;

    // buf, ring, quarter: where the stage lies
    auto read_a = [&](i32x4 (&a)[MI], int (&sa)[MI], int x, int buf, int ring, int quarter) {
        a[x] = *reinterpret_cast<const i32x4*>(lds + buf * STAGE + a_at + x * 1024);
        sa[x] = scale_lds[ring * CHUNK + quarter * 4 + as_at + x * 256];
    };
    auto read_b = [&](i32x4 (&b)[NI], int (&sb)[NI], int buf, int ring, int quarter) {
#pragma unroll
        for (int y = 0; y < NI; ++y) {
            const int r = (y >> 1) * 32 + 4 * (y & 1);
            b[y] = *reinterpret_cast<const i32x4*>(lds + buf * STAGE + b_at + r * 64);
            sb[y] = scale_lds[ring * CHUNK + quarter * 4 + bs_at + r * 16];
        }
    };

    f32x4 acc[MI][NI];
#pragma unroll
    for (int x = 0; x < MI; ++x)
#pragma unroll
        for (int y = 0; y < NI; ++y) acc[x][y] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    // Stage g is copied at step g - 3, its fragments read during step g - 1 and
    // used at step g.  The copies of step g go where stage g - 1 was: its last
    // reads came back before the matrix instructions of step g - 1 could start,
    // so a barrier needs no wait for reads.  Scale chunk c is copied over steps
    // 4 (c - 2) .. 4 (c - 2) + 3, where chunk c - 3 was.  Before the first step
    // every stage past 0 comes with at least as many scale copies as a step
    // makes, so that the steps' wait counts hold from the start.
#pragma unroll
    for (int q = 0; q < 4; ++q) copy_scales(0, q, 0);
    copy_codes(0, 0);
    copy_scales(1, 0, 1);
    copy_scales(1, 1, 1);
    copy_codes(1, 1);
    copy_scales(1, 2, 1);
    copy_scales(1, 3, 1);
    copy_codes(2, 2);
    wait_for<2 * CP + 4 * PC>();
    __builtin_amdgcn_s_barrier();
    i32x4 fa[MI], fb0[NI], fb1[NI];
    int sa[MI], sb0[NI], sb1[NI];
    read_b(fb0, sb0, 0, 0, 0);
#pragma unroll
    for (int x = 0; x < MI; ++x) read_a(fa, sa, x, 0, 0, 0);

    int chunk = 0, ring = 0, ring1 = 1, ring2 = 2;          // LDS places of chunks c, c + 1, c + 2
    auto step = [&](auto quarter, const i32x4 (&fb)[NI], const int (&sb)[NI], i32x4 (&fbn)[NI], int (&sbn)[NI]) {
        constexpr int Q = decltype(quarter)::value;
        wait_for<CP + PC>();                                // stage g + 1 has landed
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        copy_scales(chunk + 2, Q, ring2);
        copy_codes(chunk * 4 + Q + 3, (Q + 3) & 3);
        const int r1 = Q == 3 ? ring1 : ring;
        read_b(fbn, sbn, (Q + 1) & 3, r1, (Q + 1) & 3);
        __builtin_amdgcn_sched_barrier(0);
        // a fragment of A gives way to the next stage's as soon as it is used
#pragma unroll
        for (int x = 0; x < MI; ++x) {
#pragma unroll
            for (int y = 0; y < NI; ++y) acc[x][y] = mfma16(fb[y], fa[x], acc[x][y], sb[y], sa[x]);
            read_a(fa, sa, x, (Q + 1) & 3, r1, (Q + 1) & 3);
        }
    };
    using std::integral_constant;
    for (; chunk < groups / 4; ++chunk) {
        step(integral_constant<int, 0>{}, fb0, sb0, fb1, sb1);
        step(integral_constant<int, 1>{}, fb1, sb1, fb0, sb0);
        step(integral_constant<int, 2>{}, fb0, sb0, fb1, sb1);
        step(integral_constant<int, 3>{}, fb1, sb1, fb0, sb0);
        const int t = ring;
        ring = ring1;
        ring1 = ring2;
        ring2 = t;
    }
    const int rest = groups & 3;
    if (rest > 0) step(integral_constant<int, 0>{}, fb0, sb0, fb1, sb1);
    if (rest > 1) step(integral_constant<int, 1>{}, fb1, sb1, fb0, sb0);
    if (rest > 2) step(integral_constant<int, 2>{}, fb0, sb0, fb1, sb1);
    wait_for<0>();                                          // no copy outlives the workgroup's LDS

    // a lane's results: row i of fragment x, eight columns from each pair of fragments
    const bool wide = ldo % 8 == 0;
#pragma unroll
    for (int x = 0; x < MI; ++x) {
        const int row = i0 + wm * (BM / WM) + x * 16 + i;
        if (row >= A.rows) continue;
#pragma unroll
        for (int y = 0; y < NI; y += 2) {
            const int col = j0 + wn * (BN / WN) + y * 16 + 8 * blk;
            const float v[8] = {acc[x][y][0], acc[x][y][1], acc[x][y][2], acc[x][y][3],
                                acc[x][y + 1][0], acc[x][y + 1][1], acc[x][y + 1][2], acc[x][y + 1][3]};
            put8<BF16, ADD>(out, row * ldo + col, v, B.rows - col, wide);
        }
    }
}
}  // namespace
}  // namespace gc

using namespace gc;

extern "C" {

size_t gc_mxfp4_matmul_workspace_bytes(int64_t m, int64_t n, int64_t k) {
    (void)m; (void)n; (void)k;
    return 0;
}

int gc_mxfp4_matmul(const uint8_t* a_codes, const uint8_t* a_scales, const uint8_t* b_codes, const uint8_t* b_scales,
                    int64_t m, int64_t n, int64_t k, void* out, int64_t ldo, int out_dtype, int accumulate, void* ws,
                    size_t ws_bytes, void* stream) {
    const char* fn = "gc_mxfp4_matmul";
    int rc = mx_check_matrix(fn, "A", a_codes, a_scales);
    if (rc == GC_OK) rc = mx_check_matrix(fn, "B", b_codes, b_scales);
    if (rc != GC_OK) return rc;
    if (!out || !aligned16(out)) return fail(GC_ERR_ARG, "gc_mxfp4_matmul: out is null or not 16-byte aligned");
    if (out_dtype != GC_F32 && out_dtype != GC_BF16)
        return fail(GC_ERR_DTYPE, "gc_mxfp4_matmul: out_dtype must be GC_F32 or GC_BF16");
    if (m > MX_MAX_DIM || n > MX_MAX_DIM || k > MX_MAX_K || !mx_shape_ok(m, k) || !mx_shape_ok(n, k) || !mx_shape_ok(m, n))
        return fail(GC_ERR_ARG, "gc_mxfp4_matmul: m, n or k out of range");
    if (ldo < n || ldo > MX_MAX_ENTRIES) return fail(GC_ERR_ARG, "gc_mxfp4_matmul: ldo must be in [n, 2^34]");
    const size_t ob = static_cast<size_t>((m - 1) * ldo + n) * (out_dtype == GC_BF16 ? 2 : 4);
    if (overlaps(out, ob, a_codes, mx_code_bytes(m, k)) || overlaps(out, ob, a_scales, mx_scale_bytes(m, k)) ||
        overlaps(out, ob, b_codes, mx_code_bytes(n, k)) || overlaps(out, ob, b_scales, mx_scale_bytes(n, k)))
        return fail(GC_ERR_ARG, "gc_mxfp4_matmul: out overlaps an operand");
    const long long tiles = ((n + 15) / 16) * ((m + 15) / 16);
    const unsigned grid = static_cast<unsigned>(std::min<long long>((tiles + 3) / 4, 1 << 20));
    const int groups = static_cast<int>(mx_groups(k)), mi = static_cast<int>(m), ni = static_cast<int>(n);
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (m > 16) {
        const Operand A = {a_codes, a_scales, mi}, B = {b_codes, b_scales, ni};
        const unsigned tiles256 = static_cast<unsigned>(((m + 255) / 256) * ((n + 255) / 256));
        const unsigned tiles128 = static_cast<unsigned>(((m + 127) / 128) * ((n + 127) / 128));
        TimedLaunch tl("mxfp4_tile", s);
#define GO(BF, AD)                                                                                              \
        if (tiles256 >= 200) mxfp4_tile<256, 256, 2, 4, BF, AD><<<tiles256, 512, 0, s>>>(A, B, groups, out, ldo);   \
        else mxfp4_tile<128, 128, 2, 2, BF, AD><<<tiles128, 256, 0, s>>>(A, B, groups, out, ldo)
        if (out_dtype == GC_BF16) {
            if (accumulate) { GO(true, true); } else { GO(true, false); }
        } else {
            if (accumulate) { GO(false, true); } else { GO(false, false); }
        }
        return check_launch(fn);
    }
    TimedLaunch tl("mxfp4_mm", s);
    if (out_dtype == GC_BF16) {
        if (accumulate) mxfp4_mm<true, true><<<grid, 256, 0, s>>>(a_codes, a_scales, b_codes, b_scales, mi, ni, groups, out, ldo);
        else mxfp4_mm<true, false><<<grid, 256, 0, s>>>(a_codes, a_scales, b_codes, b_scales, mi, ni, groups, out, ldo);
    } else {
        if (accumulate) mxfp4_mm<false, true><<<grid, 256, 0, s>>>(a_codes, a_scales, b_codes, b_scales, mi, ni, groups, out, ldo);
        else mxfp4_mm<false, false><<<grid, 256, 0, s>>>(a_codes, a_scales, b_codes, b_scales, mi, ni, groups, out, ldo);
    }
    return check_launch(fn);
}

}  // extern "C"
