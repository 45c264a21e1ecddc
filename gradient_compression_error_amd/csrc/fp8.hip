// 8-bit floating point in blocks of 128: quantisation of matrices and the values of a held one.
//
// A matrix holds E4M3 codes (sign, four exponent bits, three mantissa bits, largest
// magnitude 448) in blocks of 128 columns of one row, or of 128 rows, each with one E8M0
// byte s (the scale 2^(s - 127)).  Block quantiser, E the biased float32 exponent of the
// largest magnitude and f its fraction in [1, 2):
//     s = max(E - 8 + (f > 1.75), 0)
//     code = RNE_E4M3(x * 2^(127 - s))
// so the largest entry lands in (224, 448] and nothing saturates, but for float32's last half
// step: what would round to 2^128 (256 at s = 247) becomes 240, so that finite entries stay finite.
// A power of two costs no bit of the codes' significands, and the matrix instructions take it as
// an operand.  A block with an entry that is not finite gets s = 255 (NaN) and zero codes.
//
// All of it is bound by HBM traffic (3 to 6 bytes an entry and form), small calls by the
// launch.
#include <type_traits>

#include "entries.h"
#include "fp8.h"

namespace gc {
namespace {

// Scale byte of a block from its largest magnitude's float32 bits.
__device__ __forceinline__ unsigned scale_byte(unsigned key) {
    const unsigned e = (key + 0x1FFFFFu) >> 23;              // one more where the fraction is above 1.75
    return key >= 0x7F800000u ? 255u : (e > 8u ? e - 8u : 0u);
}

// The scale operand of the conversions: they take its exponent field as E8M0
// (0 stands for 2^-127) and round to nearest even.
__device__ __forceinline__ float scale_operand(unsigned s) { return __uint_as_float(s == 255u ? 0x7FC00000u : s << 23); }

typedef short s16x2 __attribute__((ext_vector_type(2)));

template <bool BF16>
struct Eight;
template <>
struct Eight<true> : Entries8<true> {
    __device__ __forceinline__ unsigned key() const {        // of the largest
        unsigned k = max_u16(max_u16(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu), max_u16(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
        return max(k << 16, k & 0xFFFF0000u);
    }
    __device__ __forceinline__ unsigned four(int h, float scale) const {   // the codes of entries 4 h .. 4 h + 3
        s16x2 c = {0, 0};
        c = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(c, __builtin_bit_cast(bf16x2, w[2 * h]), scale, false);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(c, __builtin_bit_cast(bf16x2, w[2 * h + 1]), scale, true);
        return __builtin_bit_cast(unsigned, c);
    }
};
template <>
struct Eight<false> : Entries8<false> {
    __device__ __forceinline__ unsigned key() const {
        unsigned k = 0;
#pragma unroll
        for (int c = 0; c < 8; ++c) k = max(k, key_of(v[c]));
        return k;
    }
    __device__ __forceinline__ unsigned four(int h, float scale) const {
        s16x2 c = {0, 0};
        c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, v[4 * h], v[4 * h + 1], scale, false);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, v[4 * h + 2], v[4 * h + 3], scale, true);
        return __builtin_bit_cast(unsigned, c);
    }
};

// Four codes at s = 247, where 256 (magnitude 0x78, the largest that occurs) would be 2^128.
__device__ __forceinline__ unsigned below_2_128(unsigned c) { return c - ((c >> 3) & (c >> 4) & (c >> 5) & (c >> 6) & 0x01010101u); }

// Eight entries' codes; zeros where the block is not finite.
template <bool BF16>
__device__ __forceinline__ uint2 codes_of(const Eight<BF16>& e, unsigned s) {
    const float scale = scale_operand(s);
    unsigned a = e.four(0, scale), b = e.four(1, scale);
    if (s == 247u) a = below_2_128(a), b = below_2_128(b);
    return s == 255u ? make_uint2(0, 0) : make_uint2(a, b);
}

__device__ __forceinline__ unsigned row16_max(unsigned k) {  // over a row of 16 lanes
    k = max(k, dpp_u32<DPP_XOR1>(k));
    k = max(k, dpp_u32<DPP_XOR2>(k));
    k = max(k, dpp_u32<DPP_HALF_MIRROR>(k));
    return max(k, dpp_u32<DPP_MIRROR>(k));
}

// Where this thread's unit lies, of per_row units a row (0: all of them one row).
struct Place {
    long long row, unit;
};
__device__ __forceinline__ Place place_of(long long base, unsigned per_row) {
    if (per_row == 0) return {0, base + threadIdx.x};
    const Unit p = unit_of(base, per_row);
    return {p.row, p.unit};
}

// Quantisation along the rows in blocks of 1 x 128.  A thread takes eight columns, 16
// lanes a block, a wave the four groups of one scale word; F units a thread are read
// together.  Bound by HBM: 8192 x 4096 bf16 in 21 us (4.8 TB/s), float32 31 us (5.4).
template <bool BF16, int F>
__global__ __launch_bounds__(MX_THREADS) void fp8_rows(const void* x, long long ld, long long units, unsigned per_row,
                                                       long long cols, long long row_units, uint2* codes, unsigned* scales) {
    for (long long base = static_cast<long long>(blockIdx.x) * (F * MX_THREADS); base < units;
         base += static_cast<long long>(gridDim.x) * (F * MX_THREADS)) {
        Place p[F];
        Eight<BF16> e[F];
#pragma unroll
        for (int f = 0; f < F; ++f) {
            const long long first = base + f * MX_THREADS;
            if (first + threadIdx.x >= units) break;         // (whole waves: a row's units are a multiple of 64)
            p[f] = place_of(first, per_row);
            const long long col = p[f].unit * 8, left = cols - col;
            if (left >= 8) e[f].load(x, p[f].row * ld + col);
            else e[f].load(x, p[f].row * ld + col, static_cast<int>(left < 0 ? 0 : left));
        }
#pragma unroll
        for (int f = 0; f < F; ++f) {
            const long long u = base + f * MX_THREADS + threadIdx.x;
            if (u >= units) break;
            const unsigned s = scale_byte(row16_max(e[f].key()));
            if (p[f].unit < row_units) codes[p[f].row * row_units + p[f].unit] = codes_of(e[f], s);
            const unsigned word = readlane_any(s, 0) | readlane_any(s, 16) << 8 | readlane_any(s, 32) << 16 | readlane_any(s, 48) << 24;
            if ((threadIdx.x & 63) == 0) scales[u >> 6] = word;
        }
    }
}

// A block's scale byte, and zeros behind the last one of its row.
__device__ __forceinline__ void put_scale(unsigned char* scales, long long row, long long groups, long long g, unsigned s) {
    unsigned char* const to = scales + row * ((groups + 3) & ~3ll);
    to[g] = static_cast<unsigned char>(s);
    if (g == groups - 1) {
        for (long long p = groups; p & 3; ++p) to[p] = 0;
    }
}

// Quantisation by way of 128 x 128 entries a workgroup, one group of either form, from one
// read: along the rows, along the columns (the codes of the transposed matrix), or both;
// with TILE one scale for all of them, the same in both forms.  A wave takes 32 rows: lane
// l has columns 8 (l % 16) .. + 7 of the eight rows 8 (l / 16) .. + 7, so that a row's
// block is 16 neighbouring lanes, whose codes leave together, 128 bytes a row.  A
// column's eight codes of a lane go through LDS, at slots that keep the banks apart, and
// leave 128 bytes a column.  Tiles go down four and along on an XCD, since neighbours
// share lines of either form.  Bound by memory and by what registers leave of waves to wait
// for it: 8192 x 4096 both forms bf16 33.8 us from HBM (4.0 TB/s) and 25 where the input is
// in the last-level cache, float32 54 and 37 us; one form 24.5 and 43.6 us from HBM.
template <bool BF16, bool ROWS, bool COLS, bool TILE>
__global__ __launch_bounds__(MX_THREADS) void fp8_tiles(const void* x, long long ld, long long rows, long long cols, uint2* codes,
                                                        unsigned char* scales, uint2* codes_t, unsigned char* scales_t) {
    __shared__ unsigned col_keys[COLS && !TILE ? 4 : 1][128];
    __shared__ unsigned wave_keys[4];
    __shared__ uint2 col_codes[COLS ? 128 * 16 : 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, j = lane & 15, g = lane >> 4;
    const long long row_groups = (cols + 127) / 128, col_groups = (rows + 127) / 128, tiles = row_groups * col_groups;
    // whole: every entry of the tile is there
    auto tile = [&](auto whole, long long cg, long long rg) {
        constexpr bool WHOLE = decltype(whole)::value;
        const long long row0 = cg * 128 + wave * 32 + g * 8, col0 = rg * 128 + j * 8;
        const int left = WHOLE ? 8 : static_cast<int>(max(0ll, min(8ll, cols - col0)));
        const int down = WHOLE ? 8 : static_cast<int>(max(0ll, min(8ll, rows - row0)));
        Eight<BF16> e[8];
        {
            long long at = row0 * ld + col0;
#pragma unroll
            for (int p = 0; p < 8; ++p, at += ld) {
                if (WHOLE || (p < down && left == 8)) e[p].load(x, at);
                else e[p].load(x, at, p < down ? left : 0);
            }
        }
        unsigned s_tile = 0;
        if constexpr (TILE) {
            unsigned k = 0;
#pragma unroll
            for (int p = 0; p < 8; ++p) k = max(k, e[p].key());
            k = row16_max(k);
            k = max(max(readlane_any(k, 0), readlane_any(k, 16)), max(readlane_any(k, 32), readlane_any(k, 48)));
            if (lane == 0) wave_keys[wave] = k;
            __syncthreads();
            s_tile = scale_byte(max(max(wave_keys[0], wave_keys[1]), max(wave_keys[2], wave_keys[3])));
            if (threadIdx.x == 0) {
                if constexpr (ROWS) put_scale(scales, cg, row_groups, rg, s_tile);
                if constexpr (COLS) put_scale(scales_t, rg, col_groups, cg, s_tile);
            }
        }
        if constexpr (COLS && !TILE) {                       // the columns' largest magnitudes, from the four waves
            unsigned k[8];
            if constexpr (BF16) {
                unsigned pair[4];                            // of two columns each
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    pair[w] = 0;
#pragma unroll
                    for (int p = 0; p < 8; ++p) pair[w] = max_u16(pair[w], e[p].w[w] & 0x7FFF7FFFu);
                }
#pragma unroll
                for (int w = 0; w < 4; ++w) pair[w] = max_u16(pair[w], static_cast<unsigned>(__shfl_xor(static_cast<int>(pair[w]), 16, WAVE)));
#pragma unroll
                for (int w = 0; w < 4; ++w) pair[w] = max_u16(pair[w], static_cast<unsigned>(__shfl_xor(static_cast<int>(pair[w]), 32, WAVE)));
#pragma unroll
                for (int c = 0; c < 8; ++c) k[c] = c & 1 ? pair[c >> 1] & 0xFFFF0000u : pair[c >> 1] << 16;
            } else {
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    k[c] = 0;
#pragma unroll
                    for (int p = 0; p < 8; ++p) k[c] = max(k[c], key_of(e[p].v[c]));
                }
#pragma unroll
                for (int c = 0; c < 8; ++c) k[c] = max(k[c], static_cast<unsigned>(__shfl_xor(static_cast<int>(k[c]), 16, WAVE)));
#pragma unroll
                for (int c = 0; c < 8; ++c) k[c] = max(k[c], static_cast<unsigned>(__shfl_xor(static_cast<int>(k[c]), 32, WAVE)));
            }
            if (g == 0) {
#pragma unroll
                for (int c = 0; c < 8; c += 4) *reinterpret_cast<uint4*>(&col_keys[wave][j * 8 + c]) = make_uint4(k[c], k[c + 1], k[c + 2], k[c + 3]);
            }
        }
        if constexpr (ROWS) {
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                const unsigned s = TILE ? s_tile : scale_byte(row16_max(e[p].key()));
                const uint2 c = codes_of(e[p], s);
                if (WHOLE || p < down) {
                    codes[((row0 + p) * row_groups + rg) * 16 + j] = c;
                    if (!TILE && j == 0) put_scale(scales, row0 + p, row_groups, rg, s);
                }
            }
        }
        if constexpr (COLS) {
            if constexpr (!TILE) __syncthreads();
            unsigned s[8];
            if constexpr (!TILE) {
                unsigned k[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) k[c] = 0;
#pragma unroll
                for (int w = 0; w < 4; ++w)
#pragma unroll
                    for (int c = 0; c < 8; c += 4) {
                        const uint4 o = *reinterpret_cast<const uint4*>(&col_keys[w][j * 8 + c]);
                        k[c] = max(k[c], o.x); k[c + 1] = max(k[c + 1], o.y); k[c + 2] = max(k[c + 2], o.z); k[c + 3] = max(k[c + 3], o.w);
                    }
#pragma unroll
                for (int c = 0; c < 8; ++c) s[c] = scale_byte(k[c]);
                if (wave == 0 && g == 0) {
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        if (WHOLE || c < left) put_scale(scales_t, col0 + c, col_groups, cg, s[c]);
                }
            }
#pragma unroll
            for (int c = 0; c < 8; ++c) {                    // a column's eight rows
                Eight<BF16> turned;
                if constexpr (BF16) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        turned.w[q] = __builtin_amdgcn_perm(e[2 * q + 1].w[c >> 1], e[2 * q].w[c >> 1], c & 1 ? 0x07060302u : 0x05040100u);
                } else {
#pragma unroll
                    for (int p = 0; p < 8; ++p) turned.v[p] = e[p].v[c];
                }
                col_codes[(j * 8 + c) * 16 + ((wave * 4 + g) ^ j)] = codes_of(turned, TILE ? s_tile : s[c]);
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 4; ++i) {                    // eight lanes a column, 16 bytes each
                const int place = i * 256 + threadIdx.x, c = place >> 3, part = place & 7;
                const long long col = rg * 128 + c;
                if (WHOLE || col < cols) {
                    const uint2 a = col_codes[c * 16 + ((2 * part) ^ (c >> 3))], b = col_codes[c * 16 + ((2 * part + 1) ^ (c >> 3))];
                    reinterpret_cast<uint4*>(codes_t)[(col * col_groups + cg) * 8 + part] = make_uint4(a.x, a.y, b.x, b.y);
                }
            }
        }
        if constexpr (COLS || TILE) __syncthreads();
    };
    for (long long b = blockIdx.x; b < tiles; b += gridDim.x) {
        const long long t = tiles <= gridDim.x ? xcd_place(blockIdx.x, static_cast<unsigned>(tiles)) : b;
        const long long band = t / (4 * row_groups), height = min<long long>(4, col_groups - band * 4);
        const long long in = t - band * 4 * row_groups, cg = band * 4 + in % height, rg = in / height;
        if (cg * 128 + 128 <= rows && rg * 128 + 128 <= cols) tile(std::true_type{}, cg, rg);
        else tile(std::false_type{}, cg, rg);
    }
}

// The values of a held matrix, exact in float32, rounded once to bf16 (half a step of bf16,
// which is what was asked for).  A thread writes 16 bytes.  Bound by HBM: 8192 x 4096 to bf16 in
// 20.4 us (4.9 TB/s), to float32 in 35 us (4.8); 17 and 25 us where the codes are in the last-level cache.
template <bool BF16>
__global__ __launch_bounds__(MX_THREADS) void fp8_values(const unsigned char* codes, const unsigned char* scales, int shift,
                                                         long long scale_pitch, long long units, unsigned per_row, long long cols,
                                                         void* out, long long ldo) {
    constexpr int N = BF16 ? 8 : 4;                          // entries of a unit
    typedef std::conditional_t<BF16, uint2, unsigned> Word;
    for (long long base = static_cast<long long>(blockIdx.x) * MX_THREADS; base < units;
         base += static_cast<long long>(gridDim.x) * MX_THREADS) {
        const long long u = base + threadIdx.x;
        if (u >= units) continue;
        const Place p = place_of(base, per_row);
        const long long col = p.unit * N;
        if (col >= cols) continue;
        const Word w = reinterpret_cast<const Word*>(codes)[u];
        const float scale = scale_operand(scales[(p.row >> shift) * scale_pitch + p.unit / (128 / N)]);
        float v[N];
        if constexpr (BF16) {
            const unsigned h[2] = {w.x, w.y};
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(h[q], scale, false);
                const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(h[q], scale, true);
                v[4 * q] = a.x; v[4 * q + 1] = a.y; v[4 * q + 2] = b.x; v[4 * q + 3] = b.y;
            }
        } else {
            const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, scale, false);
            const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, scale, true);
            v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
        }
        const long long at = p.row * ldo + col;
        if (col + N <= cols) {
            store_out<BF16>(out, at, v);
        } else {
#pragma unroll
            for (int q = 0; q < N; ++q)
                if (col + q < cols) store1<BF16>(out, at + q, v[q]);
        }
    }
}

template <bool BF16>
void launch_rows(const void* x, long long ld, long long rows, long long cols, uint8_t* codes, uint8_t* scales, hipStream_t s) {
    if (ld == cols && cols % 512 == 0) {                     // whole scale words, no gaps: one long row
        cols *= rows;
        rows = 1;
    }
    const long long per_row = f8_scale_pitch(cols) * 16, units = rows * per_row;
    const unsigned pr = rows == 1 ? 0 : static_cast<unsigned>(per_row);
    TimedLaunch tl("fp8_rows", s);
    auto go = [&](auto flight) {
        constexpr int F = decltype(flight)::value;
        fp8_rows<BF16, F><<<grid_of((units + F * MX_THREADS - 1) / (F * MX_THREADS)), MX_THREADS, 0, s>>>(
            x, ld, units, pr, cols, mx_groups(cols) * 16, reinterpret_cast<uint2*>(codes), reinterpret_cast<unsigned*>(scales));
    };
    // Sixteen bytes a thread leave memory waiting once all waves are resident; below that a
    // wave's second unit only comes later: one and two units, bf16 8192 x 4096 22.9 and 20.6 us,
    // 4096 x 1024 4.3 and 4.1, 1024 x 1024 3.0 and 3.1; float32 (32 bytes) 31.1 and 31.9.
    if (BF16 && units >= 1 << 19) go(std::integral_constant<int, 2>{});
    else go(std::integral_constant<int, 1>{});
}

template <bool BF16>
void launch_tiles(const void* x, long long ld, long long rows, long long cols, int block_rows, uint8_t* codes, uint8_t* scales,
                  uint8_t* codes_t, uint8_t* scales_t, hipStream_t s) {
    const unsigned grid = grid_of(mx_groups(rows) * mx_groups(cols));
    uint2 *c = reinterpret_cast<uint2*>(codes), *ct = reinterpret_cast<uint2*>(codes_t);
    TimedLaunch tl("fp8_tiles", s);
    if (block_rows == 1) {
        if (c) fp8_tiles<BF16, true, true, false><<<grid, MX_THREADS, 0, s>>>(x, ld, rows, cols, c, scales, ct, scales_t);
        else fp8_tiles<BF16, false, true, false><<<grid, MX_THREADS, 0, s>>>(x, ld, rows, cols, c, scales, ct, scales_t);
    } else if (c && ct) {
        fp8_tiles<BF16, true, true, true><<<grid, MX_THREADS, 0, s>>>(x, ld, rows, cols, c, scales, ct, scales_t);
    } else if (c) {
        fp8_tiles<BF16, true, false, true><<<grid, MX_THREADS, 0, s>>>(x, ld, rows, cols, c, scales, ct, scales_t);
    } else {
        fp8_tiles<BF16, false, true, true><<<grid, MX_THREADS, 0, s>>>(x, ld, rows, cols, c, scales, ct, scales_t);
    }
}

}  // namespace
}  // namespace gc

using namespace gc;

extern "C" {

size_t gc_fp8_code_bytes(int64_t rows, int64_t cols) {
    return mx_shape_ok(rows, cols) ? static_cast<size_t>(f8_code_bytes(rows, cols)) : 0;
}

size_t gc_fp8_scale_bytes(int64_t rows, int64_t cols, int block_rows) {
    return mx_shape_ok(rows, cols) && f8_block_ok(block_rows) ? static_cast<size_t>(f8_scale_bytes(rows, cols, block_rows)) : 0;
}

int gc_fp8_quantize(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ld, int block_rows, uint8_t* codes,
                    uint8_t* scales, uint8_t* codes_t, uint8_t* scales_t, void* stream) {
    const char* fn = "gc_fp8_quantize";
    if (!x || !aligned16(x)) return fail(GC_ERR_ARG, "gc_fp8_quantize: x is null or not 16-byte aligned");
    if (dtype != GC_F32 && dtype != GC_BF16) return fail(GC_ERR_DTYPE, "gc_fp8_quantize: dtype must be GC_F32 or GC_BF16");
    if (!f8_block_ok(block_rows)) return fail(GC_ERR_ARG, "gc_fp8_quantize: block_rows must be 1 or 128");
    const bool by_rows = codes || scales, by_cols = codes_t || scales_t;
    if (!by_rows && !by_cols) return fail(GC_ERR_ARG, "gc_fp8_quantize: no output given");
    if (!mx_shape_ok(rows, cols) || (by_cols && !mx_shape_ok(cols, rows)))
        return fail(GC_ERR_ARG, "gc_fp8_quantize: rows or cols out of range");
    if (ld < cols || ld > MX_MAX_ENTRIES) return fail(GC_ERR_ARG, "gc_fp8_quantize: ld must be in [cols, 2^34]");
    if (rows - 1 > MX_MAX_SPAN / ld) return fail(GC_ERR_ARG, "gc_fp8_quantize: (rows - 1) * ld must be at most 2^40");
    int rc;
    if (by_rows && (rc = mx_check_matrix(fn, "row", codes, scales)) != GC_OK) return rc;
    if (by_cols && (rc = mx_check_matrix(fn, "column", codes_t, scales_t)) != GC_OK) return rc;
    struct { const void* p; size_t n; } b[5] = {
        {x, static_cast<size_t>((rows - 1) * ld + cols) * (dtype == GC_BF16 ? 2 : 4)},
        {codes, by_rows ? static_cast<size_t>(f8_code_bytes(rows, cols)) : 0},
        {scales, by_rows ? static_cast<size_t>(f8_scale_bytes(rows, cols, block_rows)) : 0},
        {codes_t, by_cols ? static_cast<size_t>(f8_code_bytes(cols, rows)) : 0},
        {scales_t, by_cols ? static_cast<size_t>(f8_scale_bytes(cols, rows, block_rows)) : 0}};
    for (int i = 0; i < 5; ++i)
        for (int j = i + 1; j < 5; ++j)
            if (b[i].n && b[j].n && overlaps(b[i].p, b[i].n, b[j].p, b[j].n))
                return fail(GC_ERR_ARG, "gc_fp8_quantize: buffers overlap");
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (!by_cols && block_rows == 1) {
        if (dtype == GC_BF16) launch_rows<true>(x, ld, rows, cols, codes, scales, s);
        else launch_rows<false>(x, ld, rows, cols, codes, scales, s);
    } else if (dtype == GC_BF16) {
        launch_tiles<true>(x, ld, rows, cols, block_rows, codes, scales, codes_t, scales_t, s);
    } else {
        launch_tiles<false>(x, ld, rows, cols, block_rows, codes, scales, codes_t, scales_t, s);
    }
    return check_launch(fn);
}

int gc_fp8_dequantize(const uint8_t* codes, const uint8_t* scales, int block_rows, int64_t rows, int64_t cols, void* out,
                      int64_t ldo, int out_dtype, void* stream) {
    const char* fn = "gc_fp8_dequantize";
    const int rc = mx_check_matrix(fn, "matrix", codes, scales);
    if (rc != GC_OK) return rc;
    if (!out || !aligned16(out)) return fail(GC_ERR_ARG, "gc_fp8_dequantize: out is null or not 16-byte aligned");
    if (out_dtype != GC_F32 && out_dtype != GC_BF16)
        return fail(GC_ERR_DTYPE, "gc_fp8_dequantize: out_dtype must be GC_F32 or GC_BF16");
    if (!f8_block_ok(block_rows)) return fail(GC_ERR_ARG, "gc_fp8_dequantize: block_rows must be 1 or 128");
    if (!mx_shape_ok(rows, cols)) return fail(GC_ERR_ARG, "gc_fp8_dequantize: rows or cols out of range");
    if (ldo < cols || ldo > MX_MAX_ENTRIES) return fail(GC_ERR_ARG, "gc_fp8_dequantize: ldo must be in [cols, 2^34]");
    if (rows - 1 > MX_MAX_SPAN / ldo) return fail(GC_ERR_ARG, "gc_fp8_dequantize: (rows - 1) * ldo must be at most 2^40");
    const size_t ob = static_cast<size_t>((rows - 1) * ldo + cols) * (out_dtype == GC_BF16 ? 2 : 4);
    if (overlaps(out, ob, codes, f8_code_bytes(rows, cols)) || overlaps(out, ob, scales, f8_scale_bytes(rows, cols, block_rows)))
        return fail(GC_ERR_ARG, "gc_fp8_dequantize: out overlaps the matrix");
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (ldo == cols && cols % 512 == 0 && block_rows == 1) { // whole scale words, no gaps: one long row
        cols *= rows;
        rows = ldo = 1;
    }
    const long long per_row = mx_groups(cols) * (out_dtype == GC_BF16 ? 16 : 32), units = rows * per_row;
    const unsigned grid = grid_of((units + MX_THREADS - 1) / MX_THREADS), pr = rows == 1 ? 0 : static_cast<unsigned>(per_row);
    const int shift = f8_shift(block_rows);
    TimedLaunch tl("fp8_values", s);
    if (out_dtype == GC_BF16) fp8_values<true><<<grid, MX_THREADS, 0, s>>>(codes, scales, shift, f8_scale_pitch(cols), units, pr, cols, out, ldo);
    else fp8_values<false><<<grid, MX_THREADS, 0, s>>>(codes, scales, shift, f8_scale_pitch(cols), units, pr, cols, out, ldo);
    return check_launch(fn);
}

}  // extern "C"
