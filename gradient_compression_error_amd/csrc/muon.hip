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
// hi = fl16(v 2^e), lo = fl16((v 2^e - hi) low), 22 to 24 bits together, and a product is three
// matrix instructions, hi hi + (hi lo + lo hi) / low, summed in float32: as good as float32
// products for entries that are not small.  A bf16 result is the float32 one rounded once.
// f16 has a least value, 2^-24, and so have the pairs.  Each step's powers of two (Step) are the
// largest that keep hi below f16's largest value, and with low = 2^11, which takes lo to hi's range,
// X and A are off by 2^-51 at most however small an entry is with the usual coefficients, P by 2^-50:
// half of the rows of 64 x 576 at 2^-24 of the others are 7e-7 off after five steps (float32 1e-7).
// The small products want sums of their own then, which tiles of 192 and 256 have no registers for
// (4096 x 4096: X X^T 200 us, with second sums 262, with a pass over k for them 239, by tiles of 128
// 238; P X 340, 445 with such a pass, 352 by 128).  Sets that take those tiles have low = 1: 2^-40 and 2^-39.
// f16 subnormals are kept by the matrix instructions.
//
// Layout.  A held matrix has rows of groups of 32 columns, 128 bytes each: 32 hi, then
// 32 lo, zeros behind the last column.  X is held by rows (for A) and transposed (for P X), A
// and P are symmetric: tiles on and below the diagonal are computed and written twice.
//
// Bounds, five steps to bf16: large matrices by the matrix units at the clock that power
// leaves (4096 x 4096 3.5 to 3.6 ms, 1.2 PFLOP/s of f16, units busy 61 to 74% of the cycles); a
// set of middling ones by rounds of tiles (a width-1024 layer's six 0.84 to 0.91 ms, units busy 27 to
// 53%); small ones by 17 to 22 dependent launches of 4 to 7 us (64 x 576 82 us).  Results in float32
// take as long.
#include <algorithm>
#include <cmath>
#include <memory>
#include <new>
#include <type_traits>

#include "entries.h"
#include "muon_plan.h"

namespace gc {
namespace {

constexpr int MU_SUMS = 1024;          // partial sums of squares of a matrix, at most
constexpr int MU_MAX_STEPS = 32;

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// ---------------------------------------------------------------- a call's matrices

// Entries of a partial sum of squares: a multiple of 1024, so that few sums are left to add
// for a large matrix and a small one still has several workgroups.
__host__ __device__ inline int mu_chunk(long long entries) {
    const long long even = (entries + MU_SUMS - 1) / MU_SUMS;
    return static_cast<int>(even <= 2048 ? 2048 : (even + 1023) / 1024 * 1024);
}
__host__ __device__ inline int mu_sums(long long entries) { return static_cast<int>((entries + mu_chunk(entries) - 1) / mu_chunk(entries)); }

// What a product's sums are multiplied by; for P also what A is, and what its diagonal gets; what lo is held times.
struct Factors {
    float out, old, one, low;
};

// A call's matrices.  The first kernel gets the table as an argument and leaves it at the
// workspace's start for the others: 17 launches with 2.4 KB of arguments each took the host 82
// us.  Workgroups from `..._at[i]` on are matrix i's.
struct Table {
    const void* grad[MU_MAX];
    float* mem[MU_MAX];
    void* out[MU_MAX];
    Shape s[MU_MAX];
    int sums_at[MU_MAX], start_at[MU_MAX], tile_at[3][MU_MAX], join_at[MU_MAX];
    int per[MU_MAX];                                         // groups of k of a part (A = X X^T)
    float scale[MU_MAX];
    unsigned char turned[MU_MAX];                            // X is the transposed matrix
    int count;
};
static_assert(sizeof(Table) % 4 == 0 && sizeof(Table) <= 4096 - 64, "a launch's arguments are at most 4 KB");
constexpr int64_t SUMS_AT = (sizeof(Table) + 1023) / 1024 * 1024;   // the partial sums, behind the table
constexpr int tile_kind(int kind) { return kind < APPLY ? kind : APPLY; }

// Eight values as pairs: two conversions and a mixed subtraction (exact) for two of them.
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ f16x8 halves(const float (&v)[8], float low, f16x8& lo) {
    f16x8 hi;
#pragma unroll
    for (int q = 0; q < 8; q += 2) {
        const f16x2 h = __builtin_convertvector((f32x2{v[q], v[q + 1]}), f16x2);
        const f16x2 l = __builtin_convertvector((f32x2{low * __builtin_fmaf(static_cast<float>(h[0]), -1.0f, v[q]),
                                                       low * __builtin_fmaf(static_cast<float>(h[1]), -1.0f, v[q + 1])}), f16x2);
        hi[q] = h[0]; hi[q + 1] = h[1];
        lo[q] = l[0]; lo[q + 1] = l[1];
    }
    return hi;
}

// Writes eight columns of a held row, `col` a multiple of 8; columns from `cols` on are zeros.
__device__ __forceinline__ void put8(char* row, int col, int cols, float (&v)[8], float low) {
    if (col >= ((cols + 31) & ~31)) return;
    if (col + 8 > cols) {
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (col + q >= cols) v[q] = 0.0f;
    }
    f16x8 lo;
    const f16x8 hi = halves(v, low, lo);
    char* const to = row + (col >> 5) * 128ll + (col & 31) * 2;
    *reinterpret_cast<f16x8*>(to) = hi;
    *reinterpret_cast<f16x8*>(to + 64) = lo;
}

// ---------------------------------------------------------------- momentum and norm

__device__ __forceinline__ float moved(float mem, float beta, float g) { return __fadd_rn(__fmul_rn(beta, mem), g); }
__device__ __forceinline__ float direction(float mem, float beta, float g, bool nesterov) {
    return nesterov ? __fadd_rn(g, __fmul_rn(beta, mem)) : mem;
}

// mem = beta mem + grad, and the sum of u^2 over a chunk of the entries in float64.  Bound by
// HBM: 12.6M float32 entries in 26 us (5.8 TB/s).
template <bool BF16>
__global__ __launch_bounds__(256) void muon_moment(const Table table, float beta, int nesterov, char* ws) {
    __shared__ double sums[4];
    if (blockIdx.x == 0) {
        for (unsigned i = threadIdx.x; i < sizeof(Table) / 4; i += 256)
            reinterpret_cast<unsigned*>(ws)[i] = reinterpret_cast<const unsigned*>(&table)[i];
    }
    const int w = find_segment(table.sums_at, table.count, blockIdx.x), chunk = blockIdx.x - table.sums_at[w];
    const void* const grad = table.grad[w];
    float* const mem = table.mem[w];
    const long long count = static_cast<long long>(table.s[w].n) * table.s[w].m, size = mu_chunk(count), first = chunk * size;
    const long long quads = min(count, first + size) / 4;
    double sum = 0.0;
#pragma unroll 4
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
    if (quads * 4 < first + size && i < count) {
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
    if (threadIdx.x == 0) reinterpret_cast<double*>(ws + SUMS_AT)[blockIdx.x] = (sums[0] + sums[1]) + (sums[2] + sums[3]);
}

// X = u / |u| (times sx) by rows and transposed, 64 x 64 entries a workgroup.  A matrix of zeros
// stays zero; one with an entry that is not finite becomes NaN.  Bound by HBM: 12.6M float32
// entries in 39 us (16 bytes each, 5.1 TB/s), the norm needed before any of it.
template <bool BF16>
__global__ __launch_bounds__(256) void muon_start(const Table* __restrict__ table, float beta, int nesterov, float sx, float low, char* ws) {
    __shared__ float tile[64][65];
    __shared__ double sums[4];
    const int w = find_segment(table->start_at, table->count, blockIdx.x), t = blockIdx.x - table->start_at[w];
    const Shape s = table->s[w];
    const bool turned = table->turned[w];
    const int n = turned ? s.m : s.n, m = turned ? s.n : s.m, across = (m + 63) / 64;
    const int i0 = t / across * 64, j0 = t % across * 64;
    const void* const grad = table->grad[w];
    const float* const mem = table->mem[w];
    // this thread's column of 16 rows, fetched together, and the partial sums
    float u[16], v[16];
    const int i1 = i0 + (threadIdx.x >> 6), j1 = j0 + (threadIdx.x & 63);
    const long long last = static_cast<long long>(n) * m - 1;
    auto place = [&](int p) { return min(static_cast<long long>(i1 + 4 * p) * m + j1, last); };
#pragma unroll
    for (int p = 0; p < 16; ++p) u[p] = load_grad1<BF16>(grad, place(p));
    if (mem) {
#pragma unroll
        for (int p = 0; p < 16; ++p) v[p] = mem[place(p)];
    }
    const int parts = mu_sums(static_cast<long long>(n) * m);
    double sum = 0.0;
    const double* const partial = reinterpret_cast<const double*>(ws + SUMS_AT) + table->sums_at[w];
    for (int p = threadIdx.x; p < parts; p += 256) sum += partial[p];
    sum = wave_sum(sum);
    if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = sum;
    __syncthreads();
    const double norm = sqrt((sums[0] + sums[1]) + (sums[2] + sums[3]));
    const double by = norm == 0.0 ? 0.0 : (norm < INFINITY ? sx / norm : static_cast<double>(NAN));
#pragma unroll
    for (int p = 0; p < 16; ++p) {
        const float x = mem ? direction(v[p], beta, u[p], nesterov) : u[p];
        tile[p * 4 + (threadIdx.x >> 6)][threadIdx.x & 63] = i1 + 4 * p < n && j1 < m ? static_cast<float>(x * by) : 0.0f;   // (by may be NaN)
    }
    __syncthreads();
    char* const by_rows = ws + (turned ? at_xt(s, 0) : at_x(s));
    char* const by_cols = ws + (turned ? at_x(s) : at_xt(s, 0));
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const int place = p * 256 + threadIdx.x, r = place >> 3, c = (place & 7) * 8;
        float v[8];
        if (i0 + r < n) {
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = tile[r][c + q];
            put8(by_rows + (i0 + r) * mu_groups(m) * 128, j0 + c, m, v, low);
        }
        if (j0 + r < m) {
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = tile[c + q][r];
            put8(by_cols + (j0 + r) * mu_groups(n) * 128, i0 + c, n, v, low);
        }
    }
}

// ---------------------------------------------------------------- products

// The I-th row and J-th column of the t-th tile on or below the diagonal.
__device__ __forceinline__ void below_diagonal(int t, int& I, int& J) {
    int i = static_cast<int>((sqrtf(8.0f * t + 1.0f) - 1.0f) * 0.5f);
    while (i * (i + 1) / 2 > t) --i;
    while ((i + 1) * (i + 2) / 2 <= t) ++i;
    I = i;
    J = t - i * (i + 1) / 2;
}

// One workgroup's product: a tile of L R^T at (i0, j0), over `groups` groups of k.
struct Job {
    Shape s;
    int w, i0, j0, groups;
    int part;                                                // of k, or -1: all of it
    bool diagonal;
    const unsigned char *left, *right;                       // the tile's first rows, at its first group
    int rows_l, rows_r;                                      // rows from there on
    unsigned pitch;
};
template <int KIND, int BM, int BN>
__device__ __forceinline__ Job job_of(const Table* __restrict__ table, char* ws, int turn) {
    Job b;
    const int block = static_cast<int>(xcd_place(blockIdx.x, gridDim.x));
    const auto& at = table->tile_at[tile_kind(KIND)];
    b.w = find_segment(at, table->count, block);
    b.s = table->s[b.w];
    const int t = block - at[b.w], per = KIND == GRAM ? table->per[b.w] : 0;
    int I, J, first = 0;
    b.part = -1;
    b.groups = static_cast<int>(mu_groups(KIND == GRAM ? b.s.m : b.s.n));
    b.pitch = static_cast<unsigned>(b.groups) * 128;
    if constexpr (symmetric(KIND)) {
        int tile = t;
        if (KIND == GRAM && per < b.groups) {     // in parts
            const int side = (b.s.n + BM - 1) / BM, tiles = side * (side + 1) / 2;
            b.part = t / tiles;
            tile = t - b.part * tiles;
            first = b.part * per;
            b.groups = min(per, b.groups - first);
        }
        below_diagonal(tile, I, J);
    } else {
        // bands of four tile rows, so that neighbours share operands
        const int tiles_m = (b.s.n + BM - 1) / BM, tiles_n = (b.s.m + BN - 1) / BN;
        const int band = t / (4 * tiles_n), height = min(4, tiles_m - band * 4), in = t - band * 4 * tiles_n;
        I = band * 4 + in % height;
        J = in / height;
    }
    I = __builtin_amdgcn_readfirstlane(I);
    J = __builtin_amdgcn_readfirstlane(J);
    b.i0 = I * BM;
    b.j0 = J * BN;
    b.diagonal = I == J;
    const char* const left = ws + (KIND == GRAM ? at_x(b.s) : KIND == POLY ? at_a(b.s) : at_p(b.s));
    const char* const right = symmetric(KIND) ? left : ws + at_xt(b.s, turn);
    b.left = reinterpret_cast<const unsigned char*>(left) + static_cast<long long>(b.i0) * b.pitch + first * 128ll;
    b.right = reinterpret_cast<const unsigned char*>(right) + static_cast<long long>(b.j0) * b.pitch + first * 128ll;
    b.rows_l = b.s.n - b.i0;
    b.rows_r = (symmetric(KIND) ? b.s.n : b.s.m) - b.j0;
    return b;
}

// The sums of 32 rows x COLS columns at (row0, col0), in LDS, to where they go: one wave's
// work.  Element (r, c) lies in the float4 (c / 4) ^ (r % 8) of row r.  They leave by rows, eight
// columns a lane, and (for X, and for A and P off the diagonal) transposed, eight rows of a
// column a lane, 32 rows one group.
template <int KIND, int COLS>
__device__ __forceinline__ void emit(float* region, const Job& b, int row0, int col0, const Table* __restrict__ table, char* ws, int turn,
                                     const Factors& f) {
    constexpr bool LAST = KIND == LAST_F32 || KIND == LAST_BF16, BF16 = KIND == LAST_BF16;
    const Shape& s = b.s;
    const int lane = threadIdx.x & 63, rows = s.n, cols = symmetric(KIND) ? s.n : s.m;
    if (row0 >= rows || col0 >= cols) return;
    const float by = KIND == GRAM && b.part >= 0 ? 1.0f : f.out;
    const float back = 1.0f / f.low;
    const float scale = LAST ? table->scale[b.w] : 1.0f;     // (not into `by`, which a small one would take below 2^-126)
    const bool turned = LAST && table->turned[b.w];
    if (!turned) {
        constexpr int PER_ROW = COLS / 8;
        f16x8 old[KIND == POLY ? COLS / 16 : 1][2];          // of A, fetched together
        if constexpr (KIND == POLY) {
#pragma unroll
            for (int p = 0; p < COLS / 16; ++p) {
                const int row = min(row0 + (p * 64 + lane) / PER_ROW, rows - 1), col = min(col0 + (p * 64 + lane) % PER_ROW * 8, (cols - 1) & ~7);
                const char* const from = ws + at_a(s) + row * mu_groups(s.n) * 128 + (col >> 5) * 128ll + (col & 31) * 2;
                old[p][0] = *reinterpret_cast<const f16x8*>(from);
                old[p][1] = *reinterpret_cast<const f16x8*>(from + 64);
            }
        }
#pragma unroll
        for (int p = 0; p < COLS / 16; ++p) {
            const int r = (p * 64 + lane) / PER_ROW, c = (p * 64 + lane) % PER_ROW * 8, row = row0 + r, col = col0 + c;
            float v[8];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const float4 sum = *reinterpret_cast<const float4*>(region + r * COLS + ((c / 4 + q) ^ (r & 7)) * 4);
                v[4 * q] = by * sum.x; v[4 * q + 1] = by * sum.y; v[4 * q + 2] = by * sum.z; v[4 * q + 3] = by * sum.w;
            }
            if (row >= rows) continue;
            if (KIND == GRAM && b.part >= 0) {
                const long long ld = mu_groups(s.n) * 32;
                if (col < ld) {
                    float4* const to = reinterpret_cast<float4*>(ws + at_parts(s) + ((static_cast<long long>(b.part) * s.n + row) * ld + col) * 4);
                    to[0] = make_float4(v[0], v[1], v[2], v[3]);
                    to[1] = make_float4(v[4], v[5], v[6], v[7]);
                }
                continue;
            }
            if constexpr (LAST) {
                const long long at = static_cast<long long>(row) * s.m + col;
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] *= scale;
                if (col + 8 <= s.m) {
                    store_out<BF16>(table->out[b.w], at, v);
                } else {
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        if (col + q < s.m) store1<BF16>(table->out[b.w], at + q, v[q]);
                }
            } else {
                if constexpr (KIND == POLY) {                // c A^2 + b A + a I
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        v[q] += f.old * __builtin_fmaf(static_cast<float>(old[p][1][q]), back, static_cast<float>(old[p][0][q]));
                        if (row == col + q) v[q] += f.one;
                    }
#pragma unroll
                    for (int q = 0; q < 2; ++q)              // for the transposed form
                        *reinterpret_cast<float4*>(region + r * COLS + ((c / 4 + q) ^ (r & 7)) * 4) =
                            make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                }
                put8(ws + (KIND == GRAM ? at_a(s) : KIND == POLY ? at_p(s) : at_x(s)) + row * mu_groups(cols) * 128, col, cols, v, f.low);
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    if constexpr (LAST) {
        if (!turned) return;
#pragma unroll
        for (int p = 0; p < COLS / 16; ++p) {                // eight rows of a column a lane
            const int c = p * 16 + (lane >> 2), k = (lane & 3) * 8, col = col0 + c;
            float v[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = scale * (by * region[(k + q) * COLS + ((c >> 2) ^ (k + q & 7)) * 4 + (c & 3)]);
            if (col >= cols) continue;
            const long long at = static_cast<long long>(col) * s.n + row0 + k;
            if (row0 + k + 8 <= s.n) {
                store_out<BF16>(table->out[b.w], at, v);
            } else {
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (row0 + k + q < s.n) store1<BF16>(table->out[b.w], at + q, v[q]);
            }
        }
    } else {
        if (symmetric(KIND) && (b.diagonal || b.part >= 0)) return;   // (a diagonal tile is its own mirror image)
        char* const to = ws + (KIND == GRAM ? at_a(s) : KIND == POLY ? at_p(s) : at_xt(s, 1 - turn));
        const long long pitch = mu_groups(s.n) * 128;
        const float factor = KIND == POLY ? 1.0f : by;
#pragma unroll
        for (int p = 0; p < COLS / 16; ++p) {                // eight rows of a column a lane
            const int c = p * 16 + (lane >> 2), k = (lane & 3) * 8, col = col0 + c;
            float v[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = factor * region[(k + q) * COLS + ((c >> 2) ^ (k + q & 7)) * 4 + (c & 3)];
            if (col < cols) put8(to + col * pitch, row0 + k, s.n, v, f.low);
        }
    }
}

// A 32 x 32 fragment of sums (column lane % 32 of the second factor's, so row lane % 32) to LDS.
template <int COLS>
__device__ __forceinline__ void lay(float* region, int y, const f32x16& acc) {
    const int lane = threadIdx.x & 63, i = lane & 31;
#pragma unroll
    for (int r = 0; r < 4; ++r)
        *reinterpret_cast<float4*>(region + i * COLS + ((8 * y + 2 * r + (lane >> 5)) ^ (i & 7)) * 4) =
            make_float4(acc[4 * r], acc[4 * r + 1], acc[4 * r + 2], acc[4 * r + 3]);
}

// A tile BM x BN, the groups of k in LDS in a ring of RING, copied straight from memory;
// waves WM x WN.  A group is worked off in two stages of 16 columns (one of 32, for the
// smallest tile), and a wave reads the fragments of the next stage while its matrix
// instructions work on the present one.  LDS
// holds a row's 128 bytes together, its eight pieces permuted so that a fragment's reads
// meet no bank twice: piece b of row i of a fragment at slot b ^ (i >> 1 & 7).
template <int BM, int BN, int WM, int WN, int RING, int KIND>
__global__ __launch_bounds__(WM* WN * 64, BM <= 128 ? 2 : 1) void muon_tile(const Table* __restrict__ table, char* ws, int turn, Factors f) {
    constexpr int NW = WM * WN, ROWS = BM + BN, MI = BM / WM / 32, NI = BN / WN / 32;
    constexpr int CP = ROWS / 8 / NW;                       // 8-row copies a wave makes for a group
    constexpr int GROUP = ROWS * 128;
    constexpr int S = MI * NI == 1 ? 2 : 1;                 // steps of 16 columns of a stage: enough work to cover LDS's latency
    static_assert(CP * 8 * NW == ROWS && BM % (8 * NW) == 0 && NW % 4 == 0 && (!symmetric(KIND) || BM == BN), "tile and waves must fit");
    __shared__ __attribute__((aligned(1024))) unsigned char lds[RING * GROUP];
    const unsigned lds_at = static_cast<unsigned>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) unsigned char*)lds));
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = lane >> 5, i = lane & 31, wm = wave / WN, wn = wave % WN;
    const Job b = job_of<KIND, BM, BN>(table, ws, turn);
    const int groups = b.groups;

    // Where this wave's copies come from: rows past the end are the last one again (their
    // results are not written); 256 rows of 2^24 bytes stay within 32 bits.
    unsigned off[CP];
    const unsigned piece = (lane & 7) ^ ((wave & 1) * 4 + (lane >> 4));
#pragma unroll
    for (int c = 0; c < CP; ++c) {
        const int r = (c * NW + wave) * 8 + (lane >> 3);
        off[c] = static_cast<unsigned>(c * 8 * NW < BM ? min(r, b.rows_l - 1) : min(r - BM, b.rows_r - 1)) * b.pitch + piece * 16;
    }
    auto copy = [&](int c, int group, int place) {           // groups past the end are the last again
        copy16((c * 8 * NW < BM ? b.left : b.right) + min(group, groups - 1) * 128ll, off[c], lds_at + place * GROUP + (c * NW + wave) * 1024);
    };

    const int l_at = wm * MI * 4096 + i * 128, r_at = BM * 128 + wn * NI * 4096 + i * 128;
    int c_at[2][2];                                          // byte of a row, by stage, hi and lo
#pragma unroll
    for (int q = 0; q < 4; ++q) c_at[q >> 1][q & 1] = (((q & 1) * 4 + 2 * (q >> 1) + half) ^ ((i >> 1) & 7)) * 16;
    auto read = [&](auto& l, auto& r, int place, int stage) {
#pragma unroll
        for (int k = 0; k < S; ++k) {
#pragma unroll
            for (int y = 0; y < NI; ++y)
#pragma unroll
                for (int h = 0; h < 2; ++h) r[k][y][h] = *reinterpret_cast<const f16x8*>(lds + place * GROUP + r_at + y * 4096 + c_at[stage * S + k][h]);
#pragma unroll
            for (int x = 0; x < MI; ++x)
#pragma unroll
                for (int h = 0; h < 2; ++h) l[k][x][h] = *reinterpret_cast<const f16x8*>(lds + place * GROUP + l_at + x * 4096 + c_at[stage * S + k][h]);
        }
    };

    // hi hi has sums of its own where registers allow (low may be anything then).  A matrix instruction
    // waits for the one before on the same sums: with few fragments hi lo and lo hi are apart too.
    constexpr int SETS = MI * NI < 4 ? 3 : MI * NI == 4 ? 2 : 1;
    f32x16 acc[SETS][MI][NI];
#pragma unroll
    for (int e = 0; e < SETS; ++e)
#pragma unroll
        for (int x = 0; x < MI; ++x)
#pragma unroll
            for (int y = 0; y < NI; ++y)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[e][x][y][r] = 0.0f;

#pragma unroll
    for (int p = 0; p < RING; ++p)
#pragma unroll
        for (int c = 0; c < CP; ++c) copy(c, p, p);
    wait_for<(RING - 1) * CP>();
    meet();
    f16x8 l0[S][MI][2], r0[S][NI][2], l1[S][MI][2], r1[S][NI][2];
    read(l0, r0, 0, 0);

    // Group g + RING is copied in the last stage of group g, into g's place, and has landed
    // when its first fragments are read, in the last stage of group g + RING - 1.
    int g = 0, place = 0;
    auto stage = [&](auto last_of_group, auto& l, auto& r, auto& ln, auto& rn) {
        constexpr int G = decltype(last_of_group)::value;
        const int next = G ? (place == RING - 1 ? 0 : place + 1) : place;
        if constexpr (G == 1) {
            wait_for<(RING - 2) * CP>();                     // the next group has landed
            wait_reads();                                    // and nobody reads this one any more
            meet();
            __builtin_amdgcn_sched_barrier(0);
        }
        read(ln, rn, next, S == 2 ? 0 : 1 - G);
        __builtin_amdgcn_sched_barrier(0);
        constexpr int SLOTS = S * 3 * MI;
#pragma unroll
        for (int t = 0; t < SLOTS; ++t) {
            // hi hi, then hi lo, then lo hi
            const int x = t % MI, h = t / MI % 3, k = t / MI / 3, hl = h == 2, hr = h == 1;
#pragma unroll
            for (int y = 0; y < NI; ++y) {
                f32x16& sum = acc[min(h, SETS - 1)][x][y];
                sum = __builtin_amdgcn_mfma_f32_32x32x16_f16(r[k][y][hr], l[k][x][hl], sum, 0, 0, 0);
            }
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
    if constexpr (S == 1) {
        for (; g < groups; ++g) {
            stage(k0, l0, r0, l1, r1);
            stage(k1, l1, r1, l0, r0);
        }
    } else {
        for (; g + 1 < groups; ++g) {
            stage(k1, l0, r0, l1, r1);
            ++g;
            stage(k1, l1, r1, l0, r0);
        }
        if (g < groups) stage(k1, l0, r0, l1, r1);
    }
    wait_for<0>();
    wait_reads();
    meet();                                                  // LDS is free

    // Results go through LDS, a row of fragments at a time in a region of the wave's own.
    constexpr int COLS = NI * 32;
    static_assert(NW * 32 * COLS * 4 <= RING * GROUP, "the results' regions must fit");
    float* const mine = reinterpret_cast<float*>(lds) + wave * 32 * COLS;
    const float back = 1.0f / f.low;
#pragma unroll
    for (int x = 0; x < MI; ++x) {
#pragma unroll
        for (int y = 0; y < NI; ++y) {
            if constexpr (SETS == 3) acc[1][x][y] += acc[2][x][y];
            if constexpr (SETS > 1) {
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[0][x][y][r] = __builtin_fmaf(acc[1][x][y][r], back, acc[0][x][y][r]);
            }
            lay<COLS>(mine, y, acc[0][x][y]);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        emit<KIND, COLS>(mine, b, b.i0 + (wm * MI + x) * 32, b.j0 + wn * COLS, table, ws, turn, f);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
}

// A from the parts of its k, added in order: 64 x 64 entries on or below the diagonal.  On it
// the entries above are those below (the parts may not have them).
__global__ __launch_bounds__(256) void muon_join(const Table* __restrict__ table, char* ws, float by, float low) {
    __shared__ float sums[64][65];
    const int w = find_segment(table->join_at, table->count, blockIdx.x);
    const Shape s = table->s[w];
    const int per = table->per[w], parts = static_cast<int>((mu_groups(s.m) + per - 1) / per);
    int I, J;
    below_diagonal(blockIdx.x - table->join_at[w], I, J);
    const int i0 = I * 64, j0 = J * 64;
    const long long ld = mu_groups(s.n) * 32, stride = s.n * ld, pitch = mu_groups(s.n) * 128;
    const float* const from = reinterpret_cast<const float*>(ws + at_parts(s));
    char* const to = ws + at_a(s);
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const int place = p * 256 + threadIdx.x, r = place >> 3, c = (place & 7) * 8, row = i0 + r, col = j0 + c;
        float v[8] = {};
        if (row < s.n && col <= row) {
#pragma unroll 4
            for (int k = 0; k < parts; ++k) {
                const float4* q = reinterpret_cast<const float4*>(from + k * stride + row * ld + col);
                const float4 a = q[0], b = q[1];
                v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
                v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
            }
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) sums[r][c + q] = v[q] * by;
    }
    __syncthreads();
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const int place = p * 256 + threadIdx.x, r = place >> 3, c = (place & 7) * 8;
        float v[8];
        if (i0 + r < s.n) {
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = I == J && c + q > r ? sums[c + q][r] : sums[r][c + q];
            put8(to + (i0 + r) * pitch, j0 + c, s.n, v, low);
        }
        if (I != J && j0 + r < s.n) {
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = sums[c + q][r];
            put8(to + (j0 + r) * pitch, i0 + c, s.n, v, low);
        }
    }
}

// ---------------------------------------------------------------- host side

// Workspace of up to MU_MAX matrices: the table, partial sums, then each matrix's parts.
int64_t layout(const gc_muon_mat* mats, int count, const Cut& cut, Shape* shapes) {
    int64_t sums = 0;
    for (int w = 0; w < count; ++w) sums += mu_sums(static_cast<int64_t>(mats[w].n) * mats[w].m);
    int64_t at = SUMS_AT + static_cast<int64_t>(round_up(sums * 8, 1024));
    for (int w = 0; w < count; ++w) {
        Shape s = oriented(mats[w]);
        s.base = at;
        if (shapes) shapes[w] = s;
        const int64_t parts = parts_of(s, cut.per[w]);
        at = at_parts(s) + (parts > 1 ? parts * s.n * mu_groups(s.n) * 128 : 0);
    }
    return at;
}

int64_t workspace(const gc_muon_mat* mats, int nmats) {
    int64_t need = 0;
    for (int f = 0; f < nmats; f += MU_MAX) {
        const int count = std::min(MU_MAX, nmats - f);
        need = std::max(need, layout(mats + f, count, cut_of(mats + f, count), nullptr));
    }
    return need;
}

const float MU_COEFS[3] = {3.4445f, -4.7750f, 2.0315f};

// A step's coefficients, and the powers of two that it holds X (which it starts from), A and P times.
struct Step {
    float a, b, c, sx, sa, sp;
};

// The largest power of two, 2^30 at most, that keeps values of up to `most` in f16's range, with
// a tenth of it left for roundings, which the bounds below do not know.
float power_for(double most) { return std::ldexp(1.0f, std::min(30, std::ilogb(59000.0 / std::max(most, 1e-6)))); }

// The steps of a call, and one more for the X of its result.  With singular values up to `top` at each
// step, the polynomial's largest value over them and P's say what X, A and P may reach: false
// where that leaves the range that pairs are good for.
bool steps_of(const float* coefs, int steps, Step* to) {
    double top = 1.0;
    for (int k = 0; k < steps; ++k) {
        const float* const f = coefs ? coefs + 3 * k : MU_COEFS;
        const double a = f[0], b = f[1], c = f[2], t1 = top * top;
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
        to[k] = {f[0], f[1], f[2], power_for(top), power_for(t1), power_for(p)};
        top = x;
    }
    to[steps].sx = power_for(top);
    return true;
}

// Adds up workgroups: where each matrix's begin, and how many there are.
template <typename F>
unsigned place(int (&at)[MU_MAX], int count, F blocks) {
    int64_t sum = 0;
    for (int w = 0; w < count; ++w) {
        at[w] = static_cast<int>(sum);
        sum += blocks(w);
    }
    return static_cast<unsigned>(sum);
}

template <int KIND>
void launch_product(Way way, unsigned grid, char* ws, int turn, const Factors& f, hipStream_t s) {
    TimedLaunch tl("muon_tile", s);
    auto go = [&](auto kernel, int threads) { kernel<<<grid, threads, 0, s>>>(reinterpret_cast<const Table*>(ws), ws, turn, f); };
    switch (way) {
        case TILE_64: go(muon_tile<64, 64, 2, 2, 4, KIND>, 256); break;
        case TILE_128: go(muon_tile<128, 128, 2, 4, 4, KIND>, 512); break;
        case TILE_128_PAIRED: go(muon_tile<128, 128, 2, 2, 2, KIND>, 256); break;
        case TILE_192: go(muon_tile<192, 192, 2, 2, 3, KIND>, 256); break;
        default:
            if constexpr (!symmetric(KIND)) go(muon_tile<256, 256, 2, 2, 2, KIND>, 256);
    }
}

int run(const gc_muon_mat* mats, int count, int grad_dtype, int out_dtype, float beta, int nesterov, int steps, const Step* step,
        char* ws, hipStream_t s) {
    const Cut cut = cut_of(mats, count);
    const float low = cut.low();
    Table table;
    table.count = count;
    layout(mats, count, cut, table.s);
    for (int w = 0; w < count; ++w) {
        const gc_muon_mat& a = mats[w];
        table.grad[w] = a.grad;
        table.mem[w] = a.mem;
        table.out[w] = a.out;
        table.per[w] = cut.per[w];
        table.scale[w] = a.scale;
        table.turned[w] = a.n > a.m;
    }
    const unsigned sums = place(table.sums_at, count, [&](int w) { return mu_sums(static_cast<int64_t>(mats[w].n) * mats[w].m); });
    const unsigned tiles = place(table.start_at, count, [&](int w) { return tiles_of(mats[w].n, mats[w].m, 64, 64); });
    const unsigned joins = place(table.join_at, count, [&](int w) { return parts_of(table.s[w], cut.per[w]) > 1 ? triangle(table.s[w].n, 64) : 0; });
    unsigned grid[3];
    for (int kind : {GRAM, POLY, APPLY})
        grid[kind] = place(table.tile_at[kind], count, [&](int w) { return blocks_of(kind, cut.way[kind], table.s[w], cut.per[w]); });
    const Table* const held = reinterpret_cast<const Table*>(ws);
    {
        TimedLaunch tl("muon_moment", s);
        if (grad_dtype == GC_BF16) muon_moment<true><<<sums, 256, 0, s>>>(table, beta, nesterov, ws);
        else muon_moment<false><<<sums, 256, 0, s>>>(table, beta, nesterov, ws);
    }
    {
        TimedLaunch tl("muon_start", s);
        if (grad_dtype == GC_BF16) muon_start<true><<<tiles, 256, 0, s>>>(held, beta, nesterov, step[0].sx, low, ws);
        else muon_start<false><<<tiles, 256, 0, s>>>(held, beta, nesterov, step[0].sx, low, ws);
    }
    int rc = check_launch("gc_muon_step");
    for (int k = 0; k < steps && rc == GC_OK; ++k) {
        const Step& t = step[k];
        const bool last = k + 1 == steps;
        const Factors gram = {t.sa / (t.sx * t.sx), 0, 0, low},
                      poly = {t.c * (t.sp / (t.sa * t.sa)), t.b * (t.sp / t.sa), t.a * t.sp, low},
                      apply = {(last ? 1.0f : step[k + 1].sx) / (t.sp * t.sx), 0, 0, low};
        launch_product<GRAM>(cut.way[GRAM], grid[GRAM], ws, k & 1, gram, s);
        if (joins > 0) {
            TimedLaunch tl("muon_join", s);
            muon_join<<<joins, 256, 0, s>>>(held, ws, gram.out, low);
        }
        launch_product<POLY>(cut.way[POLY], grid[POLY], ws, k & 1, poly, s);
        if (!last) launch_product<APPLY>(cut.way[APPLY], grid[APPLY], ws, k & 1, apply, s);
        else if (out_dtype == GC_BF16) launch_product<LAST_BF16>(cut.way[APPLY], grid[APPLY], ws, k & 1, apply, s);
        else launch_product<LAST_F32>(cut.way[APPLY], grid[APPLY], ws, k & 1, apply, s);
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
    Step step[MU_MAX_STEPS + 1];
    if (!steps_of(coefs, steps, step))
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
        const int rc = run(mats + f, std::min(MU_MAX, nmats - f), grad_dtype, out_dtype, beta, nesterov != 0, steps, step,
                           static_cast<char*>(ws), static_cast<hipStream_t>(stream));
        if (rc != GC_OK) return rc;
    }
    return GC_OK;
}

}  // extern "C"
