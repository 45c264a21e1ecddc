// MXFP4: error-feedback encode, decode of gathered messages, quantisation of matrices.
//
// An MXFP4 matrix holds blocks of 32 E2M1 values along its rows, each block
// with one E8M0 scale byte s (the scale 2^(s - 127)).  Block quantiser:
//     s = max(E(max |x|) - 2, 0)      E: biased float32 exponent
//     code = RNE_E2M1(x * 2^(127 - s)), saturating at 6
// so the largest entry lands in [4, 8) and the step is 2^(s - 127) times 0.5,
// 1 or 2 by binade.  The conversion instructions take the scale as an operand and
// round once.  A block with an entry that is not finite gets s = 255 (NaN) and zero
// codes.
//
// Encode, decode and quantisation along one axis are bound by HBM traffic (2.5 to
// 12.5 bytes an entry), small calls by the launch.
#include <algorithm>
#include <type_traits>

#include "entries.h"
#include "mxfp4.h"

namespace gc {
namespace {

// Scale byte of a block from the biased exponent of its largest entry.
__device__ __forceinline__ unsigned scale_byte(unsigned e) { return e == 255u ? 255u : (e > 2u ? e - 2u : 0u); }

// The scale operand of the conversions: they take its exponent field as E8M0
// (0 stands for 2^-127), round to nearest even and saturate.
__device__ __forceinline__ float scale_operand(unsigned s) { return __uint_as_float(s == 255u ? 0x7FC00000u : s << 23); }

// A pair of entries into byte SEL of a word, the first in its low nibble.
template <int SEL>
__device__ __forceinline__ unsigned code_pair(unsigned word, float a, float b, float scale) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, a, b, scale, SEL);
}
template <int SEL>
__device__ __forceinline__ unsigned code_pair(unsigned word, unsigned bf16_pair, float scale) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(word, __builtin_bit_cast(bf16x2, bf16_pair), scale, SEL);
}
// A word whose bytes are all about to be written.
__device__ __forceinline__ unsigned any_word() {
    unsigned w;
    asm("" : "=v"(w));
    return w;
}

// Four (eight) codes -> float32 values, exact, subnormal scales included.
__device__ __forceinline__ void values(unsigned c, unsigned s, float (&v)[4]) {
    const float scale = scale_operand(s);
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 0);
    const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 1);
    v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
}
__device__ __forceinline__ void values(unsigned c, unsigned s, float (&v)[8]) {
    const float scale = scale_operand(s);
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 0);
    const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 1);
    const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 2);
    const f32x2 e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, 3);
    v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
    v[4] = d.x; v[5] = d.y; v[6] = e.x; v[7] = e.y;
}

// The four scale bytes of a 16-lane row (one per quad of lanes) as one word.
__device__ __forceinline__ unsigned scales_of_row(unsigned s) {
    unsigned w = s << (8 * ((threadIdx.x >> 2) & 3));
    w |= dpp_u32<DPP_ROR4>(w);
    return w | dpp_u32<DPP_ROR8>(w);
}

// Eight neighbouring entries with what the quantiser needs of them.
template <bool BF16>
struct Eight;
template <>
struct Eight<true> : Entries8<true> {
    // exponent of the largest of the 32 entries that four neighbouring lanes hold
    __device__ __forceinline__ unsigned exponent() const {
        unsigned k = max_u16(max_u16(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu), max_u16(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
        k = max(k & 0xFFFFu, k >> 16);
        k = max(k, dpp_u32<DPP_XOR1>(k));
        return max(k, dpp_u32<DPP_XOR2>(k)) >> 7;
    }
    template <int SEL>
    __device__ __forceinline__ unsigned pair(unsigned word, float scale) const { return code_pair<SEL>(word, w[SEL], scale); }
};
template <>
struct Eight<false> : Entries8<false> {
    __device__ __forceinline__ unsigned exponent() const {
        unsigned k = 0;
#pragma unroll
        for (int c = 0; c < 8; ++c) k = max(k, key_of(v[c]));
        k = max(k, dpp_u32<DPP_XOR1>(k));
        return max(k, dpp_u32<DPP_XOR2>(k)) >> 23;
    }
    template <int SEL>
    __device__ __forceinline__ unsigned pair(unsigned word, float scale) const { return code_pair<SEL>(word, v[2 * SEL], v[2 * SEL + 1], scale); }
};

// Codes of N times eight entries (entry 0 in the low nibble), zero where a block is not
// finite.  A conversion waits for the last one into its word, so N words take turns.
template <int N, typename E>
__device__ __forceinline__ void codes_of(const E (&e)[N], const unsigned (&s)[N], unsigned (&c)[N]) {
    float scale[N];
#pragma unroll
    for (int i = 0; i < N; ++i) scale[i] = scale_operand(s[i]), c[i] = any_word();
#pragma unroll
    for (int i = 0; i < N; ++i) c[i] = e[i].template pair<0>(c[i], scale[i]);
#pragma unroll
    for (int i = 0; i < N; ++i) c[i] = e[i].template pair<1>(c[i], scale[i]);
#pragma unroll
    for (int i = 0; i < N; ++i) c[i] = e[i].template pair<2>(c[i], scale[i]);
#pragma unroll
    for (int i = 0; i < N; ++i) c[i] = e[i].template pair<3>(c[i], scale[i]);
#pragma unroll
    for (int i = 0; i < N; ++i) c[i] = s[i] == 255u ? 0u : c[i];
}

// One step with memory: acc = fl32(mem + fl32(eta * grad)) is quantised and mem becomes
// acc minus the values the codes stand for.  A thread takes four entries, so that a
// wave's loads and stores are whole lines; eight lanes hold a block.  All of it goes
// past the caches' replacement order: nothing is read twice before far more than they
// hold has gone by.  25.6M float32 entries: 64 us with four units a thread, 57.8 with
// one, 52.3 with streaming accesses (6.1 TB/s); eight entries a thread 62.
template <bool BF16>
__global__ __launch_bounds__(MX_THREADS) void mxfp4_ef(const void* grad, float* mem, float eta, long long d, long long units,
                                                       unsigned short* codes, unsigned char* scales) {
    const long long whole = d / 4;                           // units with four entries
    for (long long base = static_cast<long long>(blockIdx.x) * MX_THREADS; base < units;
         base += static_cast<long long>(gridDim.x) * MX_THREADS) {
        const long long i = base + threadIdx.x;
        float4 g, m;
        if (i < whole) {
            g = load_grad4_stream<BF16>(grad, i);
            m = load_stream(reinterpret_cast<const float4*>(mem) + i);
        } else {
            float a[4], b[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const bool in = 4 * i + q < d;
                a[q] = in ? load_grad1<BF16>(grad, 4 * i + q) : 0.0f;
                b[q] = in ? mem[4 * i + q] : 0.0f;
            }
            g = make_float4(a[0], a[1], a[2], a[3]);
            m = make_float4(b[0], b[1], b[2], b[3]);
        }
        const float acc[4] = {ef_acc(m.x, eta, g.x), ef_acc(m.y, eta, g.y), ef_acc(m.z, eta, g.z), ef_acc(m.w, eta, g.w)};
        unsigned k = max(max(key_of(acc[0]), key_of(acc[1])), max(key_of(acc[2]), key_of(acc[3])));
        k = max(k, dpp_u32<DPP_XOR1>(k));
        k = max(k, dpp_u32<DPP_XOR2>(k));
        k = max(k, dpp_u32<DPP_HALF_MIRROR>(k));
        const unsigned s = scale_byte(k >> 23);
        const float scale = scale_operand(s);
        unsigned c = code_pair<1>(code_pair<0>(any_word(), acc[0], acc[1], scale), acc[2], acc[3], scale);
        if (s == 255u) c = 0;
        float v[4];
        values(c, s, v);
        if (i >= units) continue;                            // (whole blocks of lanes)
        codes[i] = static_cast<unsigned short>(c);
        if ((threadIdx.x & 7) == 0) scales[i >> 3] = static_cast<unsigned char>(s);
        if (i < whole) {
            store_stream(reinterpret_cast<float4*>(mem) + i, make_float4(acc[0] - v[0], acc[1] - v[1], acc[2] - v[2], acc[3] - v[3]));
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (4 * i + q < d) mem[4 * i + q] = acc[q] - v[q];
        }
    }
}

// Quantisation along the rows.  A thread takes eight columns, four lanes a block, so
// that a wave reads 1 KiB of bf16 together.  8192 x 4096 bf16: 14.2 us, 6.0 TB/s;
// float32, whose 32 bytes a thread are two loads that each pass over every other 16: 27.5 us,
// 5.5 TB/s.
template <bool BF16>
__global__ __launch_bounds__(MX_THREADS) void mxfp4_rows(const void* x, long long ld, long long units, unsigned per_row,
                                                         long long cols, unsigned* codes, unsigned* scales) {
    for (long long base = static_cast<long long>(blockIdx.x) * MX_THREADS; base < units;
         base += static_cast<long long>(gridDim.x) * MX_THREADS) {
        // units is a multiple of 16: a 16-lane row is active or idle as a whole
        const long long u = base + threadIdx.x;
        const Unit p = unit_of(base, per_row);
        const long long col = static_cast<long long>(p.unit) * 8, left = u < units ? cols - col : 0;
        Eight<BF16> e;
        if (left >= 8) e.load(x, p.row * ld + col);
        else e.load(x, p.row * ld + col, static_cast<int>(left < 0 ? 0 : left > 8 ? 8 : left));
        const unsigned s = scale_byte(e.exponent()), sw = scales_of_row(s);
        unsigned c[1];
        codes_of<1>({e}, {s}, c);
        if (u < units) {
            codes[u] = c[0];
            if ((threadIdx.x & 15) == 0) scales[u >> 4] = sw;
        }
    }
}

// Quantisation along the columns (the codes of the transposed matrix), and with
// ROWS along the rows too, from one read.  A workgroup takes 128 x 128 entries, one
// group of either form, a wave 32 rows of them: lane l has columns 8 (l % 16) .. + 7 of
// the eight rows 8 (l / 16) .. + 7, so that a row block is four neighbouring lanes, a
// column block lanes 16 apart, and a lane's eight codes of a column one word of its 16
// bytes.  The words meet in LDS, at places that keep the banks apart, and leave 16
// bytes a lane, 64 of a row or column together: stored word by word they took 11 of 29
// us (8192 x 4096 bf16, both forms).  Both take 25.7 us now, 4.0 TB/s (a kernel for
// each: 58), the columns alone 14.6.  float32: 42.5 us and 38.5, 4.0 TB/s.  For both forms
// of bf16 ten waves fit a compute unit and wait, for memory and each other, 58% of their
// time; LDS is busy for 11% of it.  Tiles go down four and along on an XCD, since
// neighbours share lines of either form's codes and scales.
template <bool BF16, bool ROWS>
__global__ __launch_bounds__(MX_THREADS) void mxfp4_cols(const void* x, long long ld, long long rows, long long cols,
                                                         unsigned* codes, unsigned* scales, unsigned* codes_t,
                                                         unsigned* scales_t) {
    __shared__ unsigned char col_scales[128][4];
    __shared__ uint4 col_codes[512], row_codes[ROWS ? 4 : 1][ROWS ? 128 : 1];
    __shared__ unsigned row_scales[4][32];
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
        if constexpr (ROWS) {
            unsigned s[8];
#pragma unroll
            for (int p = 0; p < 8; ++p) s[p] = scale_byte(e[p].exponent());
            unsigned c[8];
            codes_of(e, s, c);
#pragma unroll
            for (int p = 0; p < 8; ++p) reinterpret_cast<unsigned*>(row_codes[wave])[(p * 4 + g) * 16 + j] = c[p];
            unsigned word[8];
#pragma unroll
            for (int p = 0; p < 8; ++p) word[p] = scales_of_row(s[p]);
            if (j == 0) {
#pragma unroll
                for (int p = 0; p < 8; ++p) row_scales[wave][p * 4 + g] = word[p];
            }
        }
        Eight<BF16> turned[8];                               // a column's eight rows
        unsigned s[8];
        if constexpr (BF16) {
            unsigned k[4];                                   // of two columns each
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                k[w] = 0;
#pragma unroll
                for (int p = 0; p < 8; ++p) k[w] = max_u16(k[w], e[p].w[w] & 0x7FFF7FFFu);
            }
#pragma unroll
            for (int w = 0; w < 4; ++w) k[w] = max_u16(k[w], static_cast<unsigned>(__shfl_xor(static_cast<int>(k[w]), 16, WAVE)));
#pragma unroll
            for (int w = 0; w < 4; ++w) k[w] = max_u16(k[w], static_cast<unsigned>(__shfl_xor(static_cast<int>(k[w]), 32, WAVE)));
#pragma unroll
            for (int c = 0; c < 8; ++c) s[c] = scale_byte((c & 1 ? k[c >> 1] >> 16 : k[c >> 1] & 0xFFFFu) >> 7);
#pragma unroll
            for (int c = 0; c < 8; ++c)
#pragma unroll
                for (int q = 0; q < 4; ++q)                  // rows 2 q, 2 q + 1 of the column
                    turned[c].w[q] = __builtin_amdgcn_perm(e[2 * q + 1].w[c >> 1], e[2 * q].w[c >> 1], c & 1 ? 0x07060302u : 0x05040100u);
        } else {
            unsigned k[8];
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
#pragma unroll
            for (int c = 0; c < 8; ++c) {
#pragma unroll
                for (int p = 0; p < 8; ++p) turned[c].v[p] = e[p].v[c];
                s[c] = scale_byte(k[c] >> 23);
            }
        }
        unsigned c8[8];
        codes_of(turned, s, c8);
#pragma unroll
        for (int c = 0; c < 8; ++c)
            reinterpret_cast<unsigned*>(&col_codes[wave * 128 + c * 16 + ((j + 4 * wave) & 15)])[g] = c8[c];
        if (g == 0) {
#pragma unroll
            for (int c = 0; c < 8; ++c) col_scales[j * 8 + c][wave] = static_cast<unsigned char>(s[c]);
        }
        __syncthreads();
        const int part = lane & 3, of = lane >> 2;           // of four lanes together
#pragma unroll
        for (int c = 2 * wave; c < 2 * wave + 2; ++c) {
            const long long col = rg * 128 + of * 8 + c;
            if (WHOLE || col < cols)
                reinterpret_cast<uint4*>(codes_t)[(col * col_groups + cg) * 4 + part] =
                    col_codes[part * 128 + c * 16 + ((of + 4 * part) & 15)];
        }
        if (threadIdx.x < 128 && (WHOLE || rg * 128 + threadIdx.x < cols))
            scales_t[(rg * 128 + threadIdx.x) * col_groups + cg] = *reinterpret_cast<const unsigned*>(col_scales[threadIdx.x]);
        if constexpr (ROWS) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int place = i * 16 + of;               // row 8 (place % 4) + place / 4 of the wave's
                const long long row = cg * 128 + wave * 32 + 8 * (place & 3) + (place >> 2);
                if (WHOLE || row < rows)
                    reinterpret_cast<uint4*>(codes)[(row * row_groups + rg) * 4 + part] = row_codes[wave][i * 64 + lane];
            }
            if (lane < 32) {
                const long long row = cg * 128 + wave * 32 + 8 * (lane & 3) + (lane >> 2);
                if (WHOLE || row < rows) scales[row * row_groups + rg] = row_scales[wave][lane];
            }
        }
        __syncthreads();
    };
    for (long long b = blockIdx.x; b < tiles; b += gridDim.x) {
        const long long t = tiles <= gridDim.x ? xcd_place(blockIdx.x, static_cast<unsigned>(tiles)) : b;
        const long long band = t / (4 * row_groups), height = min<long long>(4, col_groups - band * 4);
        const long long in = t - band * 4 * row_groups, cg = band * 4 + in % height, rg = in / height;
        if (cg * 128 + 128 <= rows && rg * 128 + 128 <= cols) tile(std::true_type{}, cg, rg);
        else tile(std::false_type{}, cg, rg);
    }
}

// out = [out +] weight * sum over the messages of their values, added in message
// order in float32 and rounded once to the output type.  A thread writes 16 bytes (32
// to float32 from several messages); four messages' codes are in flight at a time.
// 25.6M float32 entries of one message: 17.5 us, 6.6 TB/s; added to what is there 33.9,
// 6.4 TB/s.
template <bool BF16, bool ADD, bool FLAT, int N>
__global__ __launch_bounds__(MX_THREADS) void mxfp4_decode(const unsigned char* codes, const unsigned char* scales,
                                                           int nmsg, long long code_stride, long long scale_stride,
                                                           long long units, unsigned per_row, long long cols,
                                                           float weight, void* out) {
    typedef std::conditional_t<N == 8, unsigned, unsigned short> Word;   // the codes of a unit of N entries
    for (long long base = static_cast<long long>(blockIdx.x) * MX_THREADS; base < units;
         base += static_cast<long long>(gridDim.x) * MX_THREADS) {
        const long long u = base + threadIdx.x;
        if (u >= units) continue;
        long long row = 0, col = u * N;
        if constexpr (!FLAT) {
            const Unit p = unit_of(base, per_row);
            row = p.row;
            col = static_cast<long long>(p.unit) * N;
        }
        if (col >= cols) continue;
        auto word = [&](int i) -> unsigned { return reinterpret_cast<const Word*>(codes + i * code_stride)[u]; };
        auto scale = [&](int i) -> unsigned { return scales[i * scale_stride + u / (32 / N)]; };
        const long long at = row * cols + col;
        const bool full = col + N <= cols;
        float sum[N], old[N];
        values(word(0), scale(0), sum);
        int i = 1;
        for (; i + 4 <= nmsg; i += 4) {
            unsigned c[4], s[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) c[q] = word(i + q), s[q] = scale(i + q);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float v[N];
                values(c[q], s[q], v);
#pragma unroll
                for (int j = 0; j < N; ++j) sum[j] += v[j];
            }
        }
        for (; i < nmsg; ++i) {
            float v[N];
            values(word(i), scale(i), v);
#pragma unroll
            for (int j = 0; j < N; ++j) sum[j] += v[j];
        }
        if constexpr (ADD) {
            if (full) {
                load_out<BF16>(out, at, old);
            } else {
#pragma unroll
                for (int j = 0; j < N; ++j) old[j] = col + j < cols ? load_grad1<BF16>(out, at + j) : 0.0f;
            }
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
            sum[j] *= weight;
            if constexpr (ADD) sum[j] += old[j];
        }
        if (full) {
            store_out<BF16>(out, at, sum);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (col + j < cols) store1<BF16>(out, at + j, sum[j]);
        }
    }
}

template <bool BF16>
void launch_rows(const void* x, long long ld, long long rows, long long cols, uint8_t* codes, uint8_t* scales,
                 hipStream_t s) {
    if (ld == cols && cols % 128 == 0) {                     // whole groups, no gaps: one long row
        cols *= rows;
        rows = 1;
    }
    const long long per_row = mx_groups(cols) * 16, units = rows * per_row;
    const unsigned grid = grid_of((units + MX_THREADS - 1) / MX_THREADS);
    unsigned* c = reinterpret_cast<unsigned*>(codes);
    unsigned* sc = reinterpret_cast<unsigned*>(scales);
    TimedLaunch tl("mxfp4_rows", s);
    mxfp4_rows<BF16><<<grid, MX_THREADS, 0, s>>>(x, ld, units, static_cast<unsigned>(per_row), cols, c, sc);
}

template <bool BF16>
void launch_cols(const void* x, long long ld, long long rows, long long cols, uint8_t* codes, uint8_t* scales,
                 uint8_t* codes_t, uint8_t* scales_t, hipStream_t s) {
    const unsigned grid = grid_of(mx_groups(rows) * mx_groups(cols));
    unsigned *c = reinterpret_cast<unsigned*>(codes), *sc = reinterpret_cast<unsigned*>(scales);
    unsigned *ct = reinterpret_cast<unsigned*>(codes_t), *st = reinterpret_cast<unsigned*>(scales_t);
    TimedLaunch tl("mxfp4_cols", s);
    if (c) mxfp4_cols<BF16, true><<<grid, MX_THREADS, 0, s>>>(x, ld, rows, cols, c, sc, ct, st);
    else mxfp4_cols<BF16, false><<<grid, MX_THREADS, 0, s>>>(x, ld, rows, cols, c, sc, ct, st);
}

template <bool BF16, bool ADD>
void launch_decode(const uint8_t* codes, const uint8_t* scales, int nmsg, long long cstride, long long sstride,
                   long long rows, long long cols, float weight, void* out, hipStream_t s) {
    if (cols % 128 == 0) {                                   // whole groups: one long row
        cols *= rows;
        rows = 1;
    }
    auto go = [&](auto entries) {
        constexpr int N = decltype(entries)::value;
        const long long per_row = mx_groups(cols) * (128 / N), units = rows * per_row;
        const unsigned grid = grid_of((units + MX_THREADS - 1) / MX_THREADS), pr = static_cast<unsigned>(per_row);
        TimedLaunch tl("mxfp4_decode", s);
        if (rows == 1)
            mxfp4_decode<BF16, ADD, true, N><<<grid, MX_THREADS, 0, s>>>(codes, scales, nmsg, cstride, sstride, units, pr, cols, weight, out);
        else
            mxfp4_decode<BF16, ADD, false, N><<<grid, MX_THREADS, 0, s>>>(codes, scales, nmsg, cstride, sstride, units, pr, cols, weight, out);
    };
    // One message to float32 is bound by its stores (whole lines with four entries a
    // thread: 17.5 against 28 us for 25.6M entries), several by their loads.
    if constexpr (!BF16) {
        if (nmsg == 1) return go(std::integral_constant<int, 4>{});
    }
    go(std::integral_constant<int, 8>{});
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
    const long long units = mx_groups(d) * 32;
    const unsigned grid = grid_of((units + MX_THREADS - 1) / MX_THREADS);
    TimedLaunch tl("mxfp4_ef", s);
    if (grad_dtype == GC_BF16) mxfp4_ef<true><<<grid, MX_THREADS, 0, s>>>(grad, mem, eta, d, units, reinterpret_cast<unsigned short*>(codes), scales);
    else mxfp4_ef<false><<<grid, MX_THREADS, 0, s>>>(grad, mem, eta, d, units, reinterpret_cast<unsigned short*>(codes), scales);
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
    if (nmsg < 1 || nmsg > MX_MAX_MESSAGES) return fail(GC_ERR_ARG, "gc_mxfp4_decode: nmsg must be in [1, 2^20]");
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
    if (rows - 1 > MX_MAX_SPAN / ld) return fail(GC_ERR_ARG, "gc_mxfp4_quantize: (rows - 1) * ld must be at most 2^40");
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
    if (!by_cols) {
        if (dtype == GC_BF16) launch_rows<true>(x, ld, rows, cols, codes, scales, s);
        else launch_rows<false>(x, ld, rows, cols, codes, scales, s);
    } else if (dtype == GC_BF16) {
        launch_cols<true>(x, ld, rows, cols, codes, scales, codes_t, scales_t, s);
    } else {
        launch_cols<false>(x, ld, rows, cols, codes, scales, codes_t, scales_t, s);
    }
    return check_launch(fn);
}

}  // extern "C"
