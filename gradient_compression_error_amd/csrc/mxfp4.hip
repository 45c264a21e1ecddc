// MXFP4: error-feedback encode, decode of gathered messages, quantisation of matrices.
//
// An MXFP4 matrix holds blocks of 32 E2M1 values along its rows, each block
// with one E8M0 scale byte s (the scale 2^(s - 127)).  Block quantiser:
//     s = max(E(max |x|) - 2, 0)      E: biased float32 exponent
//     code = RNE_E2M1(x * 2^(127 - s)), saturating at 6
// so the largest entry lands in [4, 8) and the step is 2^(s - 127) times 0.5,
// 1 or 2 by binade.  x * 2^(127 - s) is exact where it matters: it can only
// lose bits below 2^-126, far under the first rounding border at 0.25.
// A block with an entry that is not finite gets s = 255 (NaN) and zero codes.
//
// All kernels here are bound by HBM traffic: about 10 operations per entry
// against 2.5 to 12.5 bytes.
#include <algorithm>

#include "mxfp4.h"

namespace gc {
namespace {

constexpr int MX_THREADS = 256;
constexpr int MX_MAXGRID = 1 << 20;   // workgroups of a launch; more work loops

// Scale byte of a block from the key (sign-stripped bits) of its largest entry.
__device__ __forceinline__ unsigned scale_byte(unsigned key) {
    const unsigned e = key >> 23;
    return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}
// 2^(127 - s); 0 for s = 255 (the codes of such a block are zeroed anyway)
__device__ __forceinline__ float scale_inverse(unsigned s) {
    return s == 255u ? 0.0f : __uint_as_float((254u - s) << 23);
}

// Eight entries -> eight codes (entry 0 in the low nibble); the conversion
// rounds to nearest even and saturates.
__device__ __forceinline__ unsigned codes8(const float (&x)[8], unsigned s) {
    const float inv = scale_inverse(s);
    unsigned c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[0] * inv, x[1] * inv, 1.0f, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[2] * inv, x[3] * inv, 1.0f, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[4] * inv, x[5] * inv, 1.0f, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[6] * inv, x[7] * inv, 1.0f, 3);
    return s == 255u ? 0u : c;
}

// Eight codes -> eight float32 values (exact, subnormal scales included).
__device__ __forceinline__ void values8(unsigned c, unsigned s, float (&v)[8]) {
    const float scale = scale_value(s);
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0);
    const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1);
    const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2);
    const f32x2 e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3);
    v[0] = a.x * scale; v[1] = a.y * scale; v[2] = b.x * scale; v[3] = b.y * scale;
    v[4] = d.x * scale; v[5] = d.y * scale; v[6] = e.x * scale; v[7] = e.y * scale;
}

// Largest key of the 32-entry block that four neighbouring lanes hold.
__device__ __forceinline__ unsigned block_key(const float (&x)[8]) {
    unsigned k = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) k = max(k, key_of(x[j]));
    k = max(k, dpp_u32<DPP_XOR1>(k));
    return max(k, dpp_u32<DPP_XOR2>(k));
}

// The four scale bytes of a 16-lane row (one per quad of lanes) as one word.
__device__ __forceinline__ unsigned scales_of_row(unsigned s) {
    unsigned w = s << (8 * ((threadIdx.x >> 2) & 3));
    w |= dpp_u32<DPP_ROR4>(w);
    return w | dpp_u32<DPP_ROR8>(w);
}

template <bool BF16>
__device__ __forceinline__ void load8(const void* p, long long i, float (&x)[8]) {
    if constexpr (BF16) {
        const uint4 v = *reinterpret_cast<const uint4*>(reinterpret_cast<const unsigned short*>(p) + i);
        x[0] = __uint_as_float(v.x << 16); x[1] = __uint_as_float(v.x & 0xFFFF0000u);
        x[2] = __uint_as_float(v.y << 16); x[3] = __uint_as_float(v.y & 0xFFFF0000u);
        x[4] = __uint_as_float(v.z << 16); x[5] = __uint_as_float(v.z & 0xFFFF0000u);
        x[6] = __uint_as_float(v.w << 16); x[7] = __uint_as_float(v.w & 0xFFFF0000u);
    } else {
        const float4 a = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + i);
        const float4 b = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + i + 4);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
}

template <bool BF16>
__device__ __forceinline__ void store8(void* p, long long i, const float (&v)[8]) {
    if constexpr (BF16) {
        *reinterpret_cast<uint4*>(reinterpret_cast<unsigned short*>(p) + i) =
            make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    } else {
        float* f = reinterpret_cast<float*>(p) + i;
        *reinterpret_cast<float4*>(f) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(f + 4) = make_float4(v[4], v[5], v[6], v[7]);
    }
}

template <bool BF16>
__device__ __forceinline__ void store1(void* p, long long i, float v) {
    if constexpr (BF16) reinterpret_cast<unsigned short*>(p)[i] = static_cast<unsigned short>(pack_bf16(v, 0.0f));
    else reinterpret_cast<float*>(p)[i] = v;
}

// Unit `u` (eight columns) of a matrix of `per_row` units a row, found from the
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

// Quantisation along the rows.  A thread takes eight columns, four lanes a
// block.  EF: x is the gradient, acc = fl32(mem + fl32(eta * x)) is quantised
// and mem becomes acc minus the values the codes stand for (one row only).
template <bool BF16, bool EF, bool VEC>
__global__ __launch_bounds__(MX_THREADS) void mxfp4_rows(const void* x, long long ld, float* mem, float eta,
                                                         long long units, unsigned per_row, long long cols,
                                                         unsigned* codes, unsigned* scales) {
    for (long long base = static_cast<long long>(blockIdx.x) * MX_THREADS; base < units;
         base += static_cast<long long>(gridDim.x) * MX_THREADS) {
        // units is a multiple of 16: a 16-lane row is active or idle as a whole
        const bool on = base + threadIdx.x < units;
        long long row, col;
        if constexpr (EF) {
            row = 0;
            col = (base + threadIdx.x) * 8;
        } else {
            const Unit u = unit_of(base, per_row);
            row = u.row;
            col = static_cast<long long>(u.unit) * 8;
        }
        const long long at = row * ld + col;
        float v[8] = {}, m[8] = {};
        const bool full = on && col + 8 <= cols;
        if (VEC && full) {
            load8<BF16>(x, at, v);
            if constexpr (EF) load8<false>(mem, at, m);
        } else if (on) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (col + j < cols) {
                    v[j] = load_grad1<BF16>(x, at + j);
                    if constexpr (EF) m[j] = mem[at + j];
                }
            }
        }
        if constexpr (EF) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = ef_acc(m[j], eta, v[j]);
        }
        const unsigned s = scale_byte(block_key(v));
        const unsigned c = codes8(v, s);
        const unsigned sw = scales_of_row(s);
        if (!on) continue;
        const long long u = base + threadIdx.x;
        codes[u] = c;
        if ((threadIdx.x & 15) == 0) scales[u >> 4] = sw;
        if constexpr (EF) {
            float q[8];
            values8(c, s, q);
#pragma unroll
            for (int j = 0; j < 8; ++j) q[j] = v[j] - q[j];
            if (VEC && full) {
                store8<false>(mem, at, q);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (col + j < cols) mem[at + j] = q[j];
            }
        }
    }
}

// Quantisation along the columns: the codes of the transposed matrix.  A
// thread takes one column of a 32-row block.
template <bool BF16>
__global__ __launch_bounds__(MX_THREADS) void mxfp4_cols(const void* x, long long ld, long long rows, long long cols,
                                                         long long groups, uint4* codes, unsigned char* scales) {
    const long long strips = (cols + MX_THREADS - 1) / MX_THREADS, blocks = groups * 4;
    for (long long w = blockIdx.x; w < strips * blocks; w += gridDim.x) {
        const long long blk = w / strips, col = (w - blk * strips) * MX_THREADS + threadIdx.x;
        if (col >= cols) continue;
        unsigned key = 0;
        float v[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const long long r = blk * 32 + j;
            v[j] = r < rows ? load_grad1<BF16>(x, r * ld + col) : 0.0f;
            key = max(key, key_of(v[j]));
        }
        const unsigned s = scale_byte(key);
        unsigned c[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float part[8] = {v[8 * q], v[8 * q + 1], v[8 * q + 2], v[8 * q + 3],
                                   v[8 * q + 4], v[8 * q + 5], v[8 * q + 6], v[8 * q + 7]};
            c[q] = codes8(part, s);
        }
        codes[col * blocks + blk] = make_uint4(c[0], c[1], c[2], c[3]);
        scales[col * blocks + blk] = static_cast<unsigned char>(s);
    }
}

// out = [out +] weight * sum over the messages of their values, added in
// message order in float32 and rounded once to the output type.
template <bool BF16, bool ADD, bool VEC>
__global__ __launch_bounds__(MX_THREADS) void mxfp4_decode(const unsigned char* codes, const unsigned char* scales,
                                                           int nmsg, long long code_stride, long long scale_stride,
                                                           long long units, unsigned per_row, long long cols,
                                                           float weight, void* out) {
    for (long long base = static_cast<long long>(blockIdx.x) * MX_THREADS; base < units;
         base += static_cast<long long>(gridDim.x) * MX_THREADS) {
        const long long u = base + threadIdx.x;
        if (u >= units) continue;
        const Unit p = unit_of(base, per_row);
        const long long col = static_cast<long long>(p.unit) * 8;
        if (col >= cols) continue;
        float sum[8];
        values8(reinterpret_cast<const unsigned*>(codes)[u], scales[u >> 2], sum);
        for (int i = 1; i < nmsg; ++i) {
            float v[8];
            values8(reinterpret_cast<const unsigned*>(codes + i * code_stride)[u], scales[i * scale_stride + (u >> 2)], v);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[j] += v[j];
        }
        const long long at = p.row * cols + col;
        const bool full = VEC && col + 8 <= cols;
        float old[8] = {};
        if constexpr (ADD) {
            if (full) {
                load8<BF16>(out, at, old);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (col + j < cols) old[j] = load_grad1<BF16>(out, at + j);
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            sum[j] *= weight;
            if constexpr (ADD) sum[j] += old[j];
        }
        if (full) {
            store8<BF16>(out, at, sum);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (col + j < cols) store1<BF16>(out, at + j, sum[j]);
        }
    }
}

unsigned grid_of(long long work) { return static_cast<unsigned>(std::min<long long>(work, MX_MAXGRID)); }

template <bool BF16, bool EF>
void launch_rows(const void* x, long long ld, float* mem, float eta, long long rows, long long cols, uint8_t* codes,
                 uint8_t* scales, bool vec, hipStream_t s) {
    const long long per_row = mx_groups(cols) * 16, units = rows * per_row;
    const unsigned grid = grid_of((units + MX_THREADS - 1) / MX_THREADS);
    unsigned* c = reinterpret_cast<unsigned*>(codes);
    unsigned* sc = reinterpret_cast<unsigned*>(scales);
    TimedLaunch tl("mxfp4_rows", s);
    if (vec)
        mxfp4_rows<BF16, EF, true><<<grid, MX_THREADS, 0, s>>>(x, ld, mem, eta, units, static_cast<unsigned>(per_row),
                                                               cols, c, sc);
    else
        mxfp4_rows<BF16, EF, false><<<grid, MX_THREADS, 0, s>>>(x, ld, mem, eta, units, static_cast<unsigned>(per_row),
                                                                cols, c, sc);
}

template <bool BF16, bool ADD>
void launch_decode(const uint8_t* codes, const uint8_t* scales, int nmsg, long long cstride, long long sstride,
                   long long rows, long long cols, float weight, void* out, hipStream_t s) {
    const long long per_row = mx_groups(cols) * 16, units = rows * per_row;
    const unsigned grid = grid_of((units + MX_THREADS - 1) / MX_THREADS);
    TimedLaunch tl("mxfp4_decode", s);
    if (rows == 1 || cols % 8 == 0)
        mxfp4_decode<BF16, ADD, true><<<grid, MX_THREADS, 0, s>>>(codes, scales, nmsg, cstride, sstride, units,
                                                                  static_cast<unsigned>(per_row), cols, weight, out);
    else
        mxfp4_decode<BF16, ADD, false><<<grid, MX_THREADS, 0, s>>>(codes, scales, nmsg, cstride, sstride, units,
                                                                   static_cast<unsigned>(per_row), cols, weight, out);
}

}  // namespace

int mx_check_matrix(const char* fn, const char* name, const void* codes, const void* scales) {
    if (!codes || !scales) return fail(GC_ERR_ARG, std::string(fn) + ": null " + name + " codes or scales");
    if (!aligned16(codes) || !aligned16(scales))
        return fail(GC_ERR_ARG, std::string(fn) + ": device pointers must be 16-byte aligned");
    return GC_OK;
}

}  // namespace gc

using namespace gc;

extern "C" {

size_t gc_mxfp4_code_bytes(int64_t rows, int64_t cols) {
    return mx_shape_ok(rows, cols) ? static_cast<size_t>(mx_code_bytes(rows, cols)) : 0;
}

size_t gc_mxfp4_scale_bytes(int64_t rows, int64_t cols) {
    return mx_shape_ok(rows, cols) ? static_cast<size_t>(mx_scale_bytes(rows, cols)) : 0;
}

int gc_mxfp4_ef_encode(const void* grad, int grad_dtype, float* mem, int64_t d, float eta, uint8_t* codes,
                       uint8_t* scales, void* stream) {
    const char* fn = "gc_mxfp4_ef_encode";
    if (!grad || !mem) return fail(GC_ERR_ARG, "gc_mxfp4_ef_encode: null grad or mem");
    if (grad_dtype != GC_F32 && grad_dtype != GC_BF16)
        return fail(GC_ERR_DTYPE, "gc_mxfp4_ef_encode: grad_dtype must be GC_F32 or GC_BF16");
    if (!mx_shape_ok(1, d)) return fail(GC_ERR_ARG, "gc_mxfp4_ef_encode: d must be in [1, 2^34]");
    const int rc = mx_check_matrix(fn, "message", codes, scales);
    if (rc != GC_OK) return rc;
    if (!aligned16(grad) || !aligned16(mem))
        return fail(GC_ERR_ARG, "gc_mxfp4_ef_encode: device pointers must be 16-byte aligned");
    const size_t cb = mx_code_bytes(1, d), sb = mx_scale_bytes(1, d), gb = static_cast<size_t>(d) * (grad_dtype == GC_BF16 ? 2 : 4);
    const size_t mb = static_cast<size_t>(d) * 4;
    if (overlaps(mem, mb, grad, gb) || overlaps(codes, cb, grad, gb) || overlaps(scales, sb, grad, gb) ||
        overlaps(codes, cb, mem, mb) || overlaps(scales, sb, mem, mb) || overlaps(codes, cb, scales, sb))
        return fail(GC_ERR_ARG, "gc_mxfp4_ef_encode: buffers overlap");
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (grad_dtype == GC_BF16) launch_rows<true, true>(grad, 0, mem, eta, 1, d, codes, scales, true, s);
    else launch_rows<false, true>(grad, 0, mem, eta, 1, d, codes, scales, true, s);
    return check_launch(fn);
}

int gc_mxfp4_decode(const uint8_t* codes, const uint8_t* scales, int nmsg, int64_t code_stride, int64_t scale_stride,
                    int64_t rows, int64_t cols, float weight, void* out, int out_dtype, int accumulate, void* stream) {
    const char* fn = "gc_mxfp4_decode";
    const int rc = mx_check_matrix(fn, "message", codes, scales);
    if (rc != GC_OK) return rc;
    if (!out || !aligned16(out)) return fail(GC_ERR_ARG, "gc_mxfp4_decode: out is null or not 16-byte aligned");
    if (out_dtype != GC_F32 && out_dtype != GC_BF16)
        return fail(GC_ERR_DTYPE, "gc_mxfp4_decode: out_dtype must be GC_F32 or GC_BF16");
    if (!mx_shape_ok(rows, cols)) return fail(GC_ERR_ARG, "gc_mxfp4_decode: rows or cols out of range");
    if (nmsg < 1) return fail(GC_ERR_ARG, "gc_mxfp4_decode: nmsg must be at least 1");
    const int64_t cb = mx_code_bytes(rows, cols), sb = mx_scale_bytes(rows, cols);
    if (nmsg > 1) {
        if (code_stride < cb || code_stride % 16 != 0 || code_stride > (int64_t(1) << 40))
            return fail(GC_ERR_ARG, "gc_mxfp4_decode: code_stride must be a multiple of 16 and hold a message");
        if (scale_stride < sb || scale_stride % 4 != 0 || scale_stride > (int64_t(1) << 40))
            return fail(GC_ERR_ARG, "gc_mxfp4_decode: scale_stride must be a multiple of 4 and hold a message");
    }
    const size_t ob = static_cast<size_t>(rows * cols) * (out_dtype == GC_BF16 ? 2 : 4);
    if (overlaps(out, ob, codes, static_cast<size_t>(nmsg - 1) * code_stride + cb) ||
        overlaps(out, ob, scales, static_cast<size_t>(nmsg - 1) * scale_stride + sb))
        return fail(GC_ERR_ARG, "gc_mxfp4_decode: out overlaps a message");
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (out_dtype == GC_BF16) {
        if (accumulate) launch_decode<true, true>(codes, scales, nmsg, code_stride, scale_stride, rows, cols, weight, out, s);
        else launch_decode<true, false>(codes, scales, nmsg, code_stride, scale_stride, rows, cols, weight, out, s);
    } else {
        if (accumulate) launch_decode<false, true>(codes, scales, nmsg, code_stride, scale_stride, rows, cols, weight, out, s);
        else launch_decode<false, false>(codes, scales, nmsg, code_stride, scale_stride, rows, cols, weight, out, s);
    }
    return check_launch(fn);
}

int gc_mxfp4_quantize(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes,
                      uint8_t* scales, uint8_t* codes_t, uint8_t* scales_t, void* stream) {
    const char* fn = "gc_mxfp4_quantize";
    if (!x || !aligned16(x)) return fail(GC_ERR_ARG, "gc_mxfp4_quantize: x is null or not 16-byte aligned");
    if (dtype != GC_F32 && dtype != GC_BF16)
        return fail(GC_ERR_DTYPE, "gc_mxfp4_quantize: dtype must be GC_F32 or GC_BF16");
    const bool by_rows = codes || scales, by_cols = codes_t || scales_t;
    if (!by_rows && !by_cols) return fail(GC_ERR_ARG, "gc_mxfp4_quantize: no output given");
    if (!mx_shape_ok(rows, cols) || (by_cols && !mx_shape_ok(cols, rows)))
        return fail(GC_ERR_ARG, "gc_mxfp4_quantize: rows or cols out of range");
    if (ld < cols || ld > MX_MAX_ENTRIES) return fail(GC_ERR_ARG, "gc_mxfp4_quantize: ld must be in [cols, 2^34]");
    int rc;
    if (by_rows && (rc = mx_check_matrix(fn, "row", codes, scales)) != GC_OK) return rc;
    if (by_cols && (rc = mx_check_matrix(fn, "column", codes_t, scales_t)) != GC_OK) return rc;
    struct { const void* p; size_t n; } b[5] = {
        {x, static_cast<size_t>((rows - 1) * ld + cols) * (dtype == GC_BF16 ? 2 : 4)},
        {codes, by_rows ? static_cast<size_t>(mx_code_bytes(rows, cols)) : 0},
        {scales, by_rows ? static_cast<size_t>(mx_scale_bytes(rows, cols)) : 0},
        {codes_t, by_cols ? static_cast<size_t>(mx_code_bytes(cols, rows)) : 0},
        {scales_t, by_cols ? static_cast<size_t>(mx_scale_bytes(cols, rows)) : 0}};
    for (int i = 0; i < 5; ++i)
        for (int j = i + 1; j < 5; ++j)
            if (b[i].n && b[j].n && overlaps(b[i].p, b[i].n, b[j].p, b[j].n))
                return fail(GC_ERR_ARG, "gc_mxfp4_quantize: buffers overlap");
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (by_rows) {
        const bool vec = rows == 1 || ld % (dtype == GC_BF16 ? 8 : 4) == 0;
        if (dtype == GC_BF16) launch_rows<true, false>(x, ld, nullptr, 0.0f, rows, cols, codes, scales, vec, s);
        else launch_rows<false, false>(x, ld, nullptr, 0.0f, rows, cols, codes, scales, vec, s);
        if ((rc = check_launch(fn)) != GC_OK) return rc;
    }
    if (by_cols) {
        const long long groups = mx_groups(rows);
        const unsigned grid = grid_of((cols + MX_THREADS - 1) / MX_THREADS * groups * 4);
        TimedLaunch tl("mxfp4_cols", s);
        if (dtype == GC_BF16)
            mxfp4_cols<true><<<grid, MX_THREADS, 0, s>>>(x, ld, rows, cols, groups, reinterpret_cast<uint4*>(codes_t), scales_t);
        else
            mxfp4_cols<false><<<grid, MX_THREADS, 0, s>>>(x, ld, rows, cols, groups, reinterpret_cast<uint4*>(codes_t), scales_t);
        return check_launch(fn);
    }
    return GC_OK;
}

}  // extern "C"
