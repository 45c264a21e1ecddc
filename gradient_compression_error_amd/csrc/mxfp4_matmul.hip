// Product of two MXFP4 matrices: out[i, j] = [out +] sum_k A[i, k] * B[j, k].
//
// v_mfma_scale_f32_16x16x128_f8f6f4 multiplies 16 x 128 by 128 x 16 E2M1 codes
// with one E8M0 scale per 32 codes and adds in float32.  A lane holds 32
// consecutive codes (16 bytes) of one row, which is one block, and the block's
// scale byte: row lane % 16, block lane / 16 of the step's four.  B goes in as
// the first operand, so that a lane's four results are neighbours in a row of
// out: row lane % 16, columns 4 * (lane / 16) + 0..3.
#include <algorithm>

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
    if (m > MX_MAX_DIM || n > MX_MAX_DIM || k > MX_MAX_DIM || !mx_shape_ok(m, k) || !mx_shape_ok(n, k) || !mx_shape_ok(m, n))
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
