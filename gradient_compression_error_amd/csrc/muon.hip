// Orthogonalised updates: momentum, then Newton-Schulz steps on the matrix units.
//
//     mem = beta mem + grad;  u = grad + beta mem (nesterov) or mem
//     X = u / |u|_F, on the shorter side n of the matrix;  `steps` times
//         A = X X^T;  P = a I + b A + c A A;  X = P X
//     out = scale X
// X keeps its singular directions and every step maps a singular value s to
// a s + b s^3 + c s^5, which drives those above zero towards one.
//
// Numerics.  A step multiplies what it finds at small singular values by a (3.4), so a
// rounding of the first step is 140 times as large after the fifth: products of bf16 or f16
// operands alone are 0.003 to 0.15 off in the end.  So X, A and P are held as pairs of f16,
// hi = fl16(v 2^e), lo = fl16(v 2^e - hi), 22 to 24 bits together, and a product is three
// matrix instructions, hi hi + hi lo + lo hi, summed in float32: as good as float32
// products.  The powers of two (SX, SA, SP) keep hi below f16's largest value, which the
// caller's coefficients are checked for, and lo above its least for all but entries that
// do not matter; f16 subnormals are kept by the matrix instructions.
//
// Layout.  A held matrix has rows of groups of 32 columns, 128 bytes each: 32 hi, then
// 32 lo, zeros behind the last column.  X is held by rows (for A) and transposed (for P X), A
// and P are symmetric: tiles on and below the diagonal are computed and written twice.
#include <algorithm>
#include <cmath>
#include <memory>
#include <new>
#include <type_traits>

#include "entries.h"
#include "matmul.h"

namespace gc {
namespace {

constexpr int MU_MAX = 64;             // matrices of a launch
constexpr int MU_TILE = 16384;         // entries of a partial sum of squares
constexpr int64_t MU_MAX_SIDE = int64_t(1) << 22;
constexpr int MU_MAX_STEPS = 32;
constexpr int MU_MAX_PARTS = 64;
constexpr float SX = 4096.0f, SA = 2048.0f, SP = 2048.0f;

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// ---------------------------------------------------------------- a call's matrices

// Where a matrix's parts lie in the workspace, n <= m the oriented sides.
struct Shape {
    long long base;
    int n, m;
};
__host__ __device__ inline long long mu_groups(long long cols) { return (cols + 31) / 32; }
__host__ __device__ inline long long at_x(const Shape& s) { return s.base; }
__host__ __device__ inline long long at_xt(const Shape& s, int which) {
    return at_x(s) + s.n * mu_groups(s.m) * 128 + which * (s.m * mu_groups(s.n) * 128);
}
__host__ __device__ inline long long at_a(const Shape& s) { return at_xt(s, 2); }
__host__ __device__ inline long long at_p(const Shape& s) { return at_a(s) + s.n * mu_groups(s.n) * 128; }
__host__ __device__ inline long long at_parts(const Shape& s) { return at_p(s) + s.n * mu_groups(s.n) * 128; }

// One launch's work: workgroups begin[i] .. are matrix i's.
struct Batch {
    Shape s[MU_MAX];
    int begin[MU_MAX];
    int per[MU_MAX];                                         // groups of k of a part (A = X X^T)
    int count;
};
struct Ends {
    void* out[MU_MAX];
    float scale[MU_MAX];
    unsigned char turned[MU_MAX];                            // X is the transposed matrix
};
struct Sources {
    const void* grad[MU_MAX];
    float* mem[MU_MAX];
    int n[MU_MAX], m[MU_MAX];                                // as given
    int begin[MU_MAX];
    int partial[MU_MAX];                                     // the first of its partial sums
    long long base[MU_MAX];
    int count;
};

__device__ __forceinline__ f16x8 halves(const float (&v)[8], f16x8& lo) {
    f16x8 hi;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        hi[q] = static_cast<_Float16>(v[q]);
        lo[q] = static_cast<_Float16>(v[q] - static_cast<float>(hi[q]));
    }
    return hi;
}

// Writes eight columns of a held row, `col` a multiple of 8; columns from `cols` on are zeros.
__device__ __forceinline__ void put8(char* row, int col, int cols, float (&v)[8]) {
    if (col >= ((cols + 31) & ~31)) return;
#pragma unroll
    for (int q = 0; q < 8; ++q)
        if (col + q >= cols) v[q] = 0.0f;
    f16x8 lo;
    const f16x8 hi = halves(v, lo);
    char* const to = row + (col >> 5) * 128ll + (col & 31) * 2;
    *reinterpret_cast<f16x8*>(to) = hi;
    *reinterpret_cast<f16x8*>(to + 64) = lo;
}

// ---------------------------------------------------------------- momentum and norm

__device__ __forceinline__ float moved(float mem, float beta, float g) { return __fadd_rn(__fmul_rn(beta, mem), g); }
__device__ __forceinline__ float direction(float mem, float beta, float g, bool nesterov) {
    return nesterov ? __fadd_rn(g, __fmul_rn(beta, mem)) : mem;
}

// mem = beta mem + grad, and the sum of u^2 over MU_TILE entries in float64.
template <bool BF16>
__global__ __launch_bounds__(256) void muon_moment(const Sources src, float beta, int nesterov, double* partial) {
    __shared__ double sums[4];
    const int w = find_segment(src.begin, src.count, blockIdx.x), tile = blockIdx.x - src.begin[w];
    const void* const grad = src.grad[w];
    float* const mem = src.mem[w];
    const long long count = static_cast<long long>(src.n[w]) * src.m[w], first = static_cast<long long>(tile) * MU_TILE;
    const long long quads = min(count, first + MU_TILE) / 4;
    double sum = 0.0;
    for (long long q = first / 4 + threadIdx.x; q < quads; q += 256) {
        const float4 g = load_grad4<BF16>(grad, q);
        float4 u = g;
        if (mem) {
            float4 v = reinterpret_cast<const float4*>(mem)[q];
            v = make_float4(moved(v.x, beta, g.x), moved(v.y, beta, g.y), moved(v.z, beta, g.z), moved(v.w, beta, g.w));
            reinterpret_cast<float4*>(mem)[q] = v;
            u = make_float4(direction(v.x, beta, g.x, nesterov), direction(v.y, beta, g.y, nesterov),
                            direction(v.z, beta, g.z, nesterov), direction(v.w, beta, g.w, nesterov));
        }
        sum += (static_cast<double>(u.x) * u.x + static_cast<double>(u.y) * u.y) +
               (static_cast<double>(u.z) * u.z + static_cast<double>(u.w) * u.w);
    }
    const long long i = quads * 4 + threadIdx.x;             // up to three entries behind the last four
    if (quads * 4 < first + MU_TILE && i < count) {
        const float g = load_grad1<BF16>(grad, i);
        float u = g;
        if (mem) {
            const float v = moved(mem[i], beta, g);
            mem[i] = v;
            u = direction(v, beta, g, nesterov);
        }
        sum += static_cast<double>(u) * u;
    }
    sum = wave_sum(sum);
    if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0) partial[src.partial[w] + tile] = (sums[0] + sums[1]) + (sums[2] + sums[3]);
}

// X = u / |u| by rows and transposed, 64 x 64 entries a workgroup.  A matrix of zeros
// stays zero; one with an entry that is not finite becomes NaN.
template <bool BF16>
__global__ __launch_bounds__(256) void muon_start(const Sources src, float beta, int nesterov, const double* partial, char* ws) {
    __shared__ float tile[64][65];
    __shared__ double sums[4];
    const int w = find_segment(src.begin, src.count, blockIdx.x), t = blockIdx.x - src.begin[w];
    const int n = src.n[w], m = src.m[w], across = (m + 63) / 64;
    const int i0 = t / across * 64, j0 = t % across * 64;
    const void* const grad = src.grad[w];
    const float* const mem = src.mem[w];
    const int parts = static_cast<int>((static_cast<long long>(n) * m + MU_TILE - 1) / MU_TILE);
    double sum = 0.0;
    for (int p = threadIdx.x; p < parts; p += 256) sum += partial[src.partial[w] + p];
    sum = wave_sum(sum);
    if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = sum;
    __syncthreads();
    const double norm = sqrt((sums[0] + sums[1]) + (sums[2] + sums[3]));
    const double by = norm == 0.0 ? 0.0 : (norm < INFINITY ? SX / norm : static_cast<double>(NAN));
#pragma unroll 4
    for (int p = 0; p < 16; ++p) {
        const int i = p * 4 + (threadIdx.x >> 6), j = threadIdx.x & 63;
        float x = 0.0f;
        if (i0 + i < n && j0 + j < m) {
            const long long at = static_cast<long long>(i0 + i) * m + j0 + j;
            const float g = load_grad1<BF16>(grad, at);
            x = static_cast<float>((mem ? direction(mem[at], beta, g, nesterov) : g) * by);
        }
        tile[i][j] = x;
    }
    __syncthreads();
    const bool turned = n > m;
    const Shape s = {src.base[w], turned ? m : n, turned ? n : m};
    char* const by_rows = ws + (turned ? at_xt(s, 0) : at_x(s));
    char* const by_cols = ws + (turned ? at_x(s) : at_xt(s, 0));
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const int place = p * 256 + threadIdx.x, r = place >> 3, c = (place & 7) * 8;
        float v[8];
        if (i0 + r < n) {
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = tile[r][c + q];
            put8(by_rows + (i0 + r) * mu_groups(m) * 128, j0 + c, m, v);
        }
        if (j0 + r < m) {
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = tile[c + q][r];
            put8(by_cols + (j0 + r) * mu_groups(n) * 128, i0 + c, n, v);
        }
    }
}

// ---------------------------------------------------------------- products

enum { GRAM, GRAM_PART, POLY, APPLY, LAST_F32, LAST_BF16 };

// The I-th row and J-th column of the t-th tile on or below the diagonal.
__device__ __forceinline__ void below_diagonal(int t, int& I, int& J) {
    int i = static_cast<int>((sqrtf(8.0f * t + 1.0f) - 1.0f) * 0.5f);
    while (i * (i + 1) / 2 > t) --i;
    while ((i + 1) * (i + 2) / 2 <= t) ++i;
    I = i;
    J = t - i * (i + 1) / 2;
}

// A tile BM x BN of L R^T for held matrices L and R, the groups of k in LDS in a ring of
// RING, copied straight from memory; waves WM x WN.  A group is worked off in two stages of 16
// columns, and a wave reads the fragments of the next stage while its matrix instructions
// work on the present one.  LDS holds a row's 128 bytes together, its eight pieces permuted
// so that a fragment's reads meet no bank twice: piece b of row i of a fragment at slot
// b ^ (i >> 1 & 7).
template <int BM, int BN, int WM, int WN, int RING, int KIND>
__global__ __launch_bounds__(WM* WN * 64) void muon_product(const Batch batch, const Ends ends, char* ws, int turn, float ca, float cb,
                                                          float cc) {
    constexpr int NW = WM * WN, ROWS = BM + BN, MI = BM / WM / 32, NI = BN / WN / 32;
    constexpr int CP = ROWS / 8 / NW;                       // 8-row copies a wave makes for a group
    constexpr int GROUP = ROWS * 128;
    constexpr bool SYMMETRIC = KIND == GRAM || KIND == GRAM_PART || KIND == POLY;
    static_assert(CP * 8 * NW == ROWS && BM % (8 * NW) == 0 && NW % 4 == 0 && RING % 2 == 0 && (!SYMMETRIC || BM == BN), "tile and waves must fit");
    __shared__ __attribute__((aligned(1024))) unsigned char lds[RING * GROUP];
    const unsigned lds_at = static_cast<unsigned>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) unsigned char*)lds));
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = lane >> 5, i = lane & 31, wm = wave / WN, wn = wave % WN;

    const int block = static_cast<int>(xcd_place(blockIdx.x, gridDim.x));
    const int w = find_segment(batch.begin, batch.count, block);
    const Shape s = batch.s[w];
    int t = block - batch.begin[w], I, J, first = 0, groups, part = 0;
    if constexpr (SYMMETRIC) {
        const int side = (s.n + BM - 1) / BM, tiles = side * (side + 1) / 2;
        part = t / tiles;
        below_diagonal(t % tiles, I, J);
        groups = static_cast<int>(mu_groups(KIND == POLY ? s.n : s.m));
        if constexpr (KIND != POLY) {
            first = part * batch.per[w];
            groups = min(batch.per[w], groups - first);
        }
    } else {
        const int tiles_m = (s.n + BM - 1) / BM, tiles_n = (s.m + BN - 1) / BN;
        const int band = t / (4 * tiles_n), height = min(4, tiles_m - band * 4), in = t - band * 4 * tiles_n;
        I = band * 4 + in % height;
        J = in / height;
        groups = static_cast<int>(mu_groups(s.n));
    }
    I = __builtin_amdgcn_readfirstlane(I);
    J = __builtin_amdgcn_readfirstlane(J);
    const int i0 = I * BM, j0 = J * BN;
    const int rows_l = s.n, rows_r = SYMMETRIC ? s.n : s.m;
    const unsigned pitch = static_cast<unsigned>(mu_groups(KIND == GRAM || KIND == GRAM_PART ? s.m : s.n)) * 128;
    const char* const left = ws + (KIND == GRAM || KIND == GRAM_PART ? at_x(s) : KIND == POLY ? at_a(s) : at_p(s));
    const char* const right = SYMMETRIC ? left : ws + at_xt(s, turn);
    const unsigned char* const base_l = reinterpret_cast<const unsigned char*>(left) + static_cast<long long>(i0) * pitch + first * 128ll;
    const unsigned char* const base_r = reinterpret_cast<const unsigned char*>(right) + static_cast<long long>(j0) * pitch + first * 128ll;

    // Where this wave's copies come from: rows past the end are the last one again (their
    // results are not written); 256 rows of 2^24 bytes stay within 32 bits.
    unsigned off[CP];
    const unsigned piece = (lane & 7) ^ ((wave & 1) * 4 + (lane >> 4));
#pragma unroll
    for (int c = 0; c < CP; ++c) {
        const int r = (c * NW + wave) * 8 + (lane >> 3);
        off[c] = static_cast<unsigned>(c * 8 * NW < BM ? min(r, rows_l - 1 - i0) : min(r - BM, rows_r - 1 - j0)) * pitch + piece * 16;
    }
    auto copy = [&](int c, int group, int place) {
        copy16((c * 8 * NW < BM ? base_l : base_r) + min(group, groups - 1) * 128ll, off[c], lds_at + place * GROUP + (c * NW + wave) * 1024);
    };

    const int l_at = wm * MI * 4096 + i * 128, r_at = BM * 128 + wn * NI * 4096 + i * 128;
    int c_at[2][2];                                          // byte of a row, by stage, hi and lo
#pragma unroll
    for (int q = 0; q < 4; ++q) c_at[q >> 1][q & 1] = (((q & 1) * 4 + 2 * (q >> 1) + half) ^ ((i >> 1) & 7)) * 16;
    auto read = [&](auto& l, auto& r, int place, int stage) {
#pragma unroll
        for (int y = 0; y < NI; ++y)
#pragma unroll
            for (int h = 0; h < 2; ++h) r[y][h] = *reinterpret_cast<const f16x8*>(lds + place * GROUP + r_at + y * 4096 + c_at[stage][h]);
#pragma unroll
        for (int x = 0; x < MI; ++x)
#pragma unroll
            for (int h = 0; h < 2; ++h) l[x][h] = *reinterpret_cast<const f16x8*>(lds + place * GROUP + l_at + x * 4096 + c_at[stage][h]);
    };

    f32x16 acc[MI][NI];
#pragma unroll
    for (int x = 0; x < MI; ++x)
#pragma unroll
        for (int y = 0; y < NI; ++y)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[x][y][r] = 0.0f;

#pragma unroll
    for (int p = 0; p < RING; ++p)
#pragma unroll
        for (int c = 0; c < CP; ++c) copy(c, p, p);
    wait_for<(RING - 1) * CP>();
    meet();
    f16x8 l0[MI][2], r0[NI][2], l1[MI][2], r1[NI][2];
    read(l0, r0, 0, 0);

    // Group g + RING is copied in the second stage of group g, into g's place, and has landed
    // when its first fragments are read, in the second stage of group g + RING - 1.
    int g = 0, place = 0;
    auto stage = [&](auto second, auto& l, auto& r, auto& ln, auto& rn) {
        constexpr int G = decltype(second)::value;
        const int next = G ? (place == RING - 1 ? 0 : place + 1) : place;
        if constexpr (G == 1) {
            wait_for<(RING - 2) * CP>();                     // the next group has landed
            wait_reads();                                    // and nobody reads this one any more
            meet();
            __builtin_amdgcn_sched_barrier(0);
        }
        read(ln, rn, next, 1 - G);
        __builtin_amdgcn_sched_barrier(0);
        constexpr int SLOTS = 3 * MI;
#pragma unroll
        for (int t = 0; t < SLOTS; ++t) {
            const int x = t % MI, h = t / MI;                // hi hi, then hi lo, then lo hi
#pragma unroll
            for (int y = 0; y < NI; ++y) acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_f16(r[y][h == 1], l[x][h == 2], acc[x][y], 0, 0, 0);
            if constexpr (G == 1) {
#pragma unroll
                for (int c = t * CP / SLOTS; c < (t + 1) * CP / SLOTS; ++c) copy(c, g + RING, place);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (G == 1) place = next;
    };
    constexpr std::integral_constant<int, 0> k0{};
    constexpr std::integral_constant<int, 1> k1{};
    for (; g < groups; ++g) {
        stage(k0, l0, r0, l1, r1);
        stage(k1, l1, r1, l0, r0);
    }
    wait_for<0>();
    wait_reads();
    meet();                                                  // LDS is free

    // Results go through LDS, a row of fragments at a time in a region of the wave's own, and
    // leave by rows and transposed.
    constexpr int COLS = NI * 32, QUADS = COLS / 4;
    static_assert(NW * 32 * COLS * 4 <= RING * GROUP, "the results' regions must fit");
    float* const mine = reinterpret_cast<float*>(lds) + wave * 32 * COLS;
    const int row0 = i0 + wm * MI * 32, col0 = j0 + wn * COLS;
    const bool turned = KIND >= LAST_F32 && ends.turned[w];
#pragma unroll
    for (int x = 0; x < MI; ++x) {
#pragma unroll
        for (int y = 0; y < NI; ++y)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int quad = 8 * y + 2 * r + half;
                *reinterpret_cast<float4*>(mine + i * COLS + ((quad ^ i) & (QUADS - 1)) * 4) =
                    make_float4(acc[x][y][4 * r], acc[x][y][4 * r + 1], acc[x][y][4 * r + 2], acc[x][y][4 * r + 3]);
            }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        // by rows: eight columns a lane
        constexpr int PER_ROW = COLS / 8, AT_ONCE = 64 / PER_ROW;
        if (!turned) {
#pragma unroll
            for (int p = 0; p < 32 / AT_ONCE; ++p) {
                const int r = p * AT_ONCE + lane / PER_ROW, c = lane % PER_ROW * 8, row = row0 + x * 32 + r, col = col0 + c;
                float v[8];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float4* const at = reinterpret_cast<float4*>(mine + r * COLS + (((c / 4 + q) ^ r) & (QUADS - 1)) * 4);
                    const float4 f = *at;
                    v[4 * q] = f.x; v[4 * q + 1] = f.y; v[4 * q + 2] = f.z; v[4 * q + 3] = f.w;
                }
                if (row >= rows_l) continue;
                if constexpr (KIND == GRAM_PART) {
                    float* const to = reinterpret_cast<float*>(ws + at_parts(s)) + (static_cast<long long>(part) * s.n + row) * (mu_groups(s.n) * 32) + col;
                    if (col < mu_groups(s.n) * 32) {
                        reinterpret_cast<float4*>(to)[0] = make_float4(v[0], v[1], v[2], v[3]);
                        reinterpret_cast<float4*>(to)[1] = make_float4(v[4], v[5], v[6], v[7]);
                    }
                } else if constexpr (KIND == LAST_F32 || KIND == LAST_BF16) {
                    constexpr bool BF16 = KIND == LAST_BF16;
                    const float by = ends.scale[w] / (SP * SX);
                    const long long at = static_cast<long long>(row) * s.m + col;
#pragma unroll
                    for (int q = 0; q < 8; ++q) v[q] *= by;
                    if (col + 8 <= s.m) {
                        store_out<BF16>(ends.out[w], at, v);
                    } else {
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            if (col + q < s.m) store1<BF16>(ends.out[w], at + q, v[q]);
                    }
                } else {
                    if constexpr (KIND == GRAM) {
#pragma unroll
                        for (int q = 0; q < 8; ++q) v[q] *= SA / (SX * SX);
                    } else if constexpr (KIND == APPLY) {
#pragma unroll
                        for (int q = 0; q < 8; ++q) v[q] *= 1.0f / SP;
                    } else {
                        // c A^2 + b A + a I, all times SP
                        float old[8] = {};
                        if (col < s.n) {
                            const char* const from = ws + at_a(s) + row * mu_groups(s.n) * 128 + (col >> 5) * 128ll + (col & 31) * 2;
                            const f16x8 hi = *reinterpret_cast<const f16x8*>(from), lo = *reinterpret_cast<const f16x8*>(from + 64);
#pragma unroll
                            for (int q = 0; q < 8; ++q) old[q] = static_cast<float>(hi[q]) + static_cast<float>(lo[q]);
                        }
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            v[q] = cc * (SP / (SA * SA)) * v[q] + cb * (SP / SA) * old[q];
                            if (row == col + q) v[q] += ca * SP;
                        }
#pragma unroll
                        for (int q = 0; q < 2; ++q)          // for the transposed form
                            *reinterpret_cast<float4*>(mine + r * COLS + (((c / 4 + q) ^ r) & (QUADS - 1)) * 4) =
                                make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                    }
                    const int cols = SYMMETRIC ? s.n : s.m;
                    char* const to = ws + (KIND == GRAM ? at_a(s) : KIND == POLY ? at_p(s) : at_x(s));
                    put8(to + row * mu_groups(cols) * 128, col, cols, v);
                }
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
        // transposed: a column a lane, its 32 rows one group
        const bool mirror = KIND == APPLY || ((KIND == GRAM || KIND == POLY) && I != J) || turned;
        if (KIND != GRAM_PART && mirror) {
#pragma unroll
            for (int p = 0; p < (COLS + 63) / 64; ++p) {
                const int c = p * 64 + (COLS < 64 ? i : lane), col = col0 + c, row = row0 + x * 32;
                if (col >= rows_r || row >= rows_l || (COLS < 64 && half)) continue;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float v[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const int r = 8 * k + q;
                        v[q] = mine[r * COLS + (((c >> 2) ^ r) & (QUADS - 1)) * 4 + (c & 3)];
                        if constexpr (KIND == GRAM) v[q] *= SA / (SX * SX);
                        if constexpr (KIND == APPLY) v[q] *= 1.0f / SP;
                    }
                    if constexpr (KIND == LAST_F32 || KIND == LAST_BF16) {
                        constexpr bool BF16 = KIND == LAST_BF16;
                        const float by = ends.scale[w] / (SP * SX);
                        const long long at = static_cast<long long>(col) * s.n + row + 8 * k;
#pragma unroll
                        for (int q = 0; q < 8; ++q) v[q] *= by;
                        if (row + 8 * k + 8 <= s.n) {
                            store_out<BF16>(ends.out[w], at, v);
                        } else {
#pragma unroll
                            for (int q = 0; q < 8; ++q)
                                if (row + 8 * k + q < s.n) store1<BF16>(ends.out[w], at + q, v[q]);
                        }
                    } else {
                        char* const to = ws + (KIND == GRAM ? at_a(s) : KIND == POLY ? at_p(s) : at_xt(s, 1 - turn));
                        put8(to + col * mu_groups(s.n) * 128, row + 8 * k, s.n, v);
                    }
                }
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
}

// A from the parts of its k, added in order: 64 x 64 entries on or below the diagonal.
__global__ __launch_bounds__(256) void muon_join(const Batch batch, char* ws, int tile) {
    __shared__ float sums[64][65];
    const int w = find_segment(batch.begin, batch.count, blockIdx.x);
    const Shape s = batch.s[w];
    const int per = batch.per[w], parts = static_cast<int>((mu_groups(s.m) + per - 1) / per);
    int I, J;
    below_diagonal(blockIdx.x - batch.begin[w], I, J);
    const int i0 = I * 64, j0 = J * 64;
    const long long ld = mu_groups(s.n) * 32, stride = s.n * ld;
    const float* const from = reinterpret_cast<const float*>(ws + at_parts(s));
    char* const to = ws + at_a(s);
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const int place = p * 256 + threadIdx.x, r = place >> 3, c = (place & 7) * 8, row = i0 + r, col = j0 + c;
        float v[8] = {};
        // above the diagonal, within tiles of the product that have it, the parts are there too
        if (row < s.n && col < ld) {
            for (int k = 0; k < parts; ++k) {
                const float4* q = reinterpret_cast<const float4*>(from + k * stride + row * ld + col);
                const float4 a = q[0], b = q[1];
                v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
                v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
            }
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            v[q] *= SA / (SX * SX);
            sums[r][c + q] = v[q];
        }
        if (row < s.n) put8(to + row * mu_groups(s.n) * 128, col, s.n, v);
    }
    if (I == J) return;
    __syncthreads();
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const int place = p * 256 + threadIdx.x, r = place >> 3, c = (place & 7) * 8;
        if (j0 + r >= s.n) continue;
        float v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = sums[c + q][r];
        put8(to + (j0 + r) * mu_groups(s.n) * 128, i0 + c, s.n, v);
    }
}

// ---------------------------------------------------------------- host side

int64_t triangle(int64_t n, int64_t tile) { const int64_t k = (n + tile - 1) / tile; return k * (k + 1) / 2; }

Shape oriented(const gc_muon_mat& a) { return {0, std::min(a.n, a.m), std::max(a.n, a.m)}; }

bool mat_ok(const gc_muon_mat& a) {
    return a.n >= 1 && a.m >= 1 && a.n <= MU_MAX_SIDE && a.m <= MU_MAX_SIDE && static_cast<int64_t>(a.n) * a.m <= INT32_MAX;
}

// How the matrices of one launch are cut: parts of k for A = X X^T.
struct Cut {
    int per[MU_MAX];
    bool parts;
};
Cut cut_of(const gc_muon_mat* mats, int count) {
    Cut cut = {};
    for (int w = 0; w < count; ++w) cut.per[w] = static_cast<int>(mu_groups(oriented(mats[w]).m));
    return cut;
}

// Workspace of up to MU_MAX matrices: partial sums, then each matrix's parts.
int64_t layout(const gc_muon_mat* mats, int count, const Cut& cut, Shape* shapes, int* partial) {
    int64_t sums = 0;
    for (int w = 0; w < count; ++w) {
        if (partial) partial[w] = static_cast<int>(sums);
        sums += (static_cast<int64_t>(mats[w].n) * mats[w].m + MU_TILE - 1) / MU_TILE;
    }
    int64_t at = static_cast<int64_t>(round_up(sums * 8, 1024));
    for (int w = 0; w < count; ++w) {
        Shape s = oriented(mats[w]);
        s.base = at;
        if (shapes) shapes[w] = s;
        const int64_t parts = (mu_groups(s.m) + cut.per[w] - 1) / cut.per[w];
        at = at_parts(s) + (parts > 1 ? parts * s.n * mu_groups(s.n) * 128 : 0);
    }
    return at;
}

int64_t workspace(const gc_muon_mat* mats, int nmats) {
    int64_t need = 0;
    for (int f = 0; f < nmats; f += MU_MAX) {
        const int count = std::min(MU_MAX, nmats - f);
        need = std::max(need, layout(mats + f, count, cut_of(mats + f, count), nullptr, nullptr));
    }
    return need;
}

const float MU_COEFS[3] = {3.4445f, -4.7750f, 2.0315f};

// Whether X, A and P stay in the range that their pairs hold: with singular values up to
// `top`, the polynomial's largest value over them at each step, and P's.
bool coefs_ok(const float* coefs, int steps) {
    double top = 1.0;
    for (int k = 0; k < steps; ++k) {
        const double a = coefs[3 * k], b = coefs[3 * k + 1], c = coefs[3 * k + 2], t1 = top * top;
        if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c)) return false;
        double p = std::max(std::abs(a), std::abs(a + b * t1 + c * t1 * t1)), x = std::abs((a + b * t1 + c * t1 * t1) * top);
        auto value = [&](double t) {
            if (!(t > 0 && t < t1)) return;
            p = std::max(p, std::abs(a + b * t + c * t * t));
            x = std::max(x, std::abs((a + b * t + c * t * t) * std::sqrt(t)));
        };
        if (c != 0) {
            value(-b / (2 * c));
            const double d = 9 * b * b - 20 * a * c;
            if (d >= 0) value((-3 * b + std::sqrt(d)) / (10 * c)), value((-3 * b - std::sqrt(d)) / (10 * c));
        } else if (b != 0) {
            value(-a / (3 * b));
        }
        if (p > 16.0 || x > 4.0) return false;
        top = x;
    }
    return true;
}

template <int BM, int BN, int WM, int WN, int RING, int KIND>
void launch_product(Batch& batch, const Ends& ends, char* ws, int turn, const float* c, hipStream_t s) {
    constexpr bool SYMMETRIC = KIND == GRAM || KIND == GRAM_PART || KIND == POLY;
    int64_t blocks = 0;
    for (int w = 0; w < batch.count; ++w) {
        const Shape& m = batch.s[w];
        batch.begin[w] = static_cast<int>(blocks);
        const int64_t parts = KIND == GRAM_PART ? (mu_groups(m.m) + batch.per[w] - 1) / batch.per[w] : 1;
        blocks += SYMMETRIC ? triangle(m.n, BM) * parts : tiles_of(m.n, m.m, BM, BN);
    }
    TimedLaunch tl("muon_product", s);
    muon_product<BM, BN, WM, WN, RING, KIND><<<static_cast<unsigned>(blocks), WM * WN * 64, 0, s>>>(batch, ends, ws, turn, c[0], c[1], c[2]);
}

int run(const gc_muon_mat* mats, int count, int grad_dtype, int out_dtype, float beta, int nesterov, int steps, const float* coefs,
        char* ws, hipStream_t s) {
    const Cut cut = cut_of(mats, count);
    Sources src;
    Batch batch;
    Ends ends;
    src.count = batch.count = count;
    layout(mats, count, cut, batch.s, src.partial);
    int64_t sums = 0, tiles = 0;
    int begin[MU_MAX];
    for (int w = 0; w < count; ++w) {
        const gc_muon_mat& a = mats[w];
        src.grad[w] = a.grad;
        src.mem[w] = a.mem;
        src.n[w] = a.n;
        src.m[w] = a.m;
        src.base[w] = batch.s[w].base;
        src.begin[w] = static_cast<int>(sums);
        sums += (static_cast<int64_t>(a.n) * a.m + MU_TILE - 1) / MU_TILE;
        begin[w] = static_cast<int>(tiles);
        tiles += tiles_of(a.n, a.m, 64, 64);
        batch.per[w] = cut.per[w];
        ends.out[w] = a.out;
        ends.scale[w] = a.scale;
        ends.turned[w] = a.n > a.m;
    }
    double* const partial = reinterpret_cast<double*>(ws);
    {
        TimedLaunch tl("muon_moment", s);
        if (grad_dtype == GC_BF16) muon_moment<true><<<static_cast<unsigned>(sums), 256, 0, s>>>(src, beta, nesterov, partial);
        else muon_moment<false><<<static_cast<unsigned>(sums), 256, 0, s>>>(src, beta, nesterov, partial);
    }
    int rc = check_launch("gc_muon_step");
    if (rc != GC_OK) return rc;
    std::copy(begin, begin + count, src.begin);
    {
        TimedLaunch tl("muon_start", s);
        if (grad_dtype == GC_BF16) muon_start<true><<<static_cast<unsigned>(tiles), 256, 0, s>>>(src, beta, nesterov, partial, ws);
        else muon_start<false><<<static_cast<unsigned>(tiles), 256, 0, s>>>(src, beta, nesterov, partial, ws);
    }
    rc = check_launch("gc_muon_step");
    for (int k = 0; k < steps && rc == GC_OK; ++k) {
        const float* c = coefs ? coefs + 3 * k : MU_COEFS;
        launch_product<128, 128, 2, 2, 2, GRAM>(batch, ends, ws, k & 1, c, s);
        launch_product<128, 128, 2, 2, 2, POLY>(batch, ends, ws, k & 1, c, s);
        if (k + 1 < steps) launch_product<128, 128, 2, 2, 2, APPLY>(batch, ends, ws, k & 1, c, s);
        else if (out_dtype == GC_BF16) launch_product<128, 128, 2, 2, 2, LAST_BF16>(batch, ends, ws, k & 1, c, s);
        else launch_product<128, 128, 2, 2, 2, LAST_F32>(batch, ends, ws, k & 1, c, s);
        rc = check_launch("gc_muon_step");
    }
    return rc;
}

}  // namespace
}  // namespace gc

using namespace gc;

extern "C" {

size_t gc_muon_workspace_bytes(const gc_muon_mat* mats, int nmats) {
    if (!mats || nmats < 1) return 0;
    for (int w = 0; w < nmats; ++w)
        if (!mat_ok(mats[w])) return 0;
    return static_cast<size_t>(workspace(mats, nmats));
}

int gc_muon_step(const gc_muon_mat* mats, int nmats, int grad_dtype, int out_dtype, float beta, int nesterov, int steps,
                 const float* coefs, void* ws, size_t ws_bytes, void* stream) {
    if (!mats || nmats < 1) return fail(GC_ERR_ARG, "gc_muon_step: need at least one matrix");
    if (grad_dtype != GC_F32 && grad_dtype != GC_BF16) return fail(GC_ERR_DTYPE, "gc_muon_step: grad_dtype must be GC_F32 or GC_BF16");
    if (out_dtype != GC_F32 && out_dtype != GC_BF16) return fail(GC_ERR_DTYPE, "gc_muon_step: out_dtype must be GC_F32 or GC_BF16");
    if (steps < 1 || steps > MU_MAX_STEPS) return fail(GC_ERR_ARG, "gc_muon_step: steps must be in [1, 32]");
    if (coefs && !coefs_ok(coefs, steps))
        return fail(GC_ERR_ARG, "gc_muon_step: coefficients that take singular values past 4, or the factor of a step past 16");
    for (int w = 0; w < nmats; ++w) {
        const gc_muon_mat& a = mats[w];
        if (!mat_ok(a)) return fail(GC_ERR_ARG, "gc_muon_step: n and m must be in [1, 2^22], n * m at most 2^31 - 1");
        if (!a.grad || !a.out) return fail(GC_ERR_ARG, "gc_muon_step: null grad or out");
        if (!aligned16(a.grad) || !aligned16(a.out) || (a.mem && !aligned16(a.mem)))
            return fail(GC_ERR_ARG, "gc_muon_step: device pointers must be 16-byte aligned");
    }
    const size_t need = static_cast<size_t>(workspace(mats, nmats));
    if (!ws || !aligned16(ws)) return fail(GC_ERR_ARG, "gc_muon_step: ws is null or not 16-byte aligned");
    if (ws_bytes < need) return fail(GC_ERR_WORKSPACE, "gc_muon_step: workspace too small");
    // what is written overlaps nothing else
    struct Span { uintptr_t from, to; bool written; };
    const std::unique_ptr<Span[]> spans(new (std::nothrow) Span[3 * static_cast<size_t>(nmats) + 1]);
    if (!spans) return fail(GC_ERR_ARG, "gc_muon_step: out of host memory");
    size_t count = 0;
    auto add = [&](const void* p, size_t bytes, bool written) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(p);
        spans[count++] = {at, at + bytes, written};
    };
    for (int w = 0; w < nmats; ++w) {
        const size_t entries = static_cast<size_t>(mats[w].n) * mats[w].m;
        add(mats[w].grad, entries * (grad_dtype == GC_BF16 ? 2 : 4), false);
        add(mats[w].out, entries * (out_dtype == GC_BF16 ? 2 : 4), true);
        if (mats[w].mem) add(mats[w].mem, entries * 4, true);
    }
    add(ws, need, true);
    std::sort(spans.get(), spans.get() + count, [](const Span& a, const Span& b) { return a.from < b.from; });
    uintptr_t end = 0, written_end = 0;                      // of all spans so far, of the written ones
    for (size_t i = 0; i < count; ++i) {
        const Span& sp = spans[i];
        if (sp.from < (sp.written ? end : written_end)) return fail(GC_ERR_ARG, "gc_muon_step: buffers overlap");
        end = std::max(end, sp.to);
        if (sp.written) written_end = std::max(written_end, sp.to);
    }
    for (int f = 0; f < nmats; f += MU_MAX) {
        const int rc = run(mats + f, std::min(MU_MAX, nmats - f), grad_dtype, out_dtype, beta, nesterov != 0, steps, coefs,
                           static_cast<char*>(ws), static_cast<hipStream_t>(stream));
        if (rc != GC_OK) return rc;
    }
    return GC_OK;
}

}  // extern "C"
