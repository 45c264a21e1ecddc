// Product of two 8-bit matrices: out[i, j] = [out +] sum_k A[i, k] * B[j, k].
//
// The f8f6f4 matrix instructions multiply E4M3 codes with one E8M0 scale per 32 codes and
// add in float32: 16 x 128 by 128 x 16 (fp8_wave) or 32 x 64 by 64 x 32 (fp8_tile).  A
// lane holds 32 codes of one row, and the scale byte of their block: one for a row's 128
// columns, so the order of the columns within a group of 128 is free as long as both
// operands have the same, and a word holds the scales of four groups.  B goes in as the
// first operand, so that a lane's results are neighbours in a row of out.
//
// These instructions add eight products at a time and cut each of them off 13 places
// below the largest one's leading bit; what they add up so far is kept in float32.  Sums
// of normal entries are off by 1.5e-5 then (relative, root of the mean square), a
// hundredth of what rounding to bf16 costs, but a hundred times float32's own rounding; next to
// products 2^13 times as large that cancel, small ones are lost altogether.  So
// they serve results in bf16, and results in float32 (EXACT) are summed by the bf16 matrix
// instructions, at half the rate: a code times its scale is a bf16 value, products are exact
// and sums are kept to 24 bits.
//
// Bounds: few rows by the read of B (1 x 8192 x 8192 12.5 us, 5.4 TB/s); 8192^3 to bf16 by
// the matrix units at the clock that power leaves (412 to 433 us by card, 2.5 to 2.7 PFLOP/s, units
// busy 66% of the cycles); 4096 x 1024 x 8192 added to float32 by conversions and matrix
// instructions of one wave a unit (63 to 66 us, 1.1 PFLOP/s; the library's bf16 rate would be 48).
#include <algorithm>
#include <type_traits>

#include "fp8_plan.h"

namespace gc {
namespace {

constexpr int E4M3 = 0;   // operand format of the f8f6f4 matrix instructions

__device__ __forceinline__ i32x8 joined(i32x4 a, i32x4 b) { return i32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}; }

__device__ __forceinline__ void arrived8(const i32x8& f) {
    arrived(__builtin_shufflevector(f, f, 0, 1, 2, 3));
    arrived(__builtin_shufflevector(f, f, 4, 5, 6, 7));
}

// Q picks the scale byte of either operand's word.
template <int Q>
__device__ __forceinline__ f32x4 mfma16(i32x8 a, i32x8 b, f32x4 c, int sa, int sb) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, E4M3, E4M3, Q, sa, Q, sb);
}
template <int Q>
__device__ __forceinline__ f32x16 mfma32(i32x8 a, i32x8 b, f32x16 c, int sa, int sb) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, E4M3, E4M3, Q, sa, Q, sb);
}

// Eight codes (two words) times their scale as bf16: exact down to 2^-133, bf16's least value.
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
__device__ __forceinline__ bf16x8 widened(int lo, int hi, float scale) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
// Byte Q of a word of scales as the conversions take it.
template <int Q>
__device__ __forceinline__ float scale_operand(unsigned word) {
    const unsigned s = word >> (8 * Q) & 255u;
    return __uint_as_float(s == 255u ? 0x7FC00000u : s << 23);
}

struct Operand {
    const unsigned char* codes;
    const unsigned char* scales;
    int rows;
    int shift;                                               // a row's scales are those of row >> shift
};

// ---------------------------------------------------------------- few tiles

// Where a 128 x 128 tile would leave most of the chip idle (few rows, or a small out): a
// workgroup takes 16 MI x 16 NI of out and its W waves share k, a unit of GU groups at a
// time (wave w takes units w, w + W, ...), operands straight from memory to registers.
// The waves' sums meet in LDS and are added in wave order.
//
// Lane l holds, of each group, the 16-byte pieces l / 16 and 4 + l / 16 of row l % 16, so
// that four lanes read 64 bytes of a row together, and one word with the scales of the
// four groups that the unit is in.
template <int MI, int NI, int W, int GU, bool EXACT>
__global__ __launch_bounds__(W * 64) void fp8_wave(const Operand A, const Operand B, int groups, int scale_pitch, void* out,
                                                   long long ldo, int add) {
    static_assert(GU == 1 || GU == 2 || GU == 4, "a unit lies in one scale word");
    constexpr int TM = 16 * MI, TN = 16 * NI;
    __shared__ __attribute__((aligned(16))) float sums[W][TM * TN];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i = lane & 15, quarter = lane >> 4;
    const int tiles_m = (A.rows + TM - 1) / TM;
    const unsigned t = xcd_place(blockIdx.x, gridDim.x);     // the tiles of one stretch of B on one XCD
    const int i0 = static_cast<int>(t % tiles_m) * TM, j0 = static_cast<int>(t / tiles_m) * TN;
    const int units = (groups + GU - 1) / GU;

    const unsigned char *pa[MI], *qa[MI], *pb[NI], *qb[NI];
#pragma unroll
    for (int x = 0; x < MI; ++x) {
        const int r = min(i0 + 16 * x + i, A.rows - 1);
        pa[x] = A.codes + static_cast<long long>(r) * groups * 128 + quarter * 16;
        qa[x] = A.scales + static_cast<long long>(r >> A.shift) * scale_pitch;
    }
#pragma unroll
    for (int y = 0; y < NI; ++y) {
        const int r = min(j0 + 16 * y + i, B.rows - 1);
        pb[y] = B.codes + static_cast<long long>(r) * groups * 128 + quarter * 16;
        qb[y] = B.scales + static_cast<long long>(r >> B.shift) * scale_pitch;
    }
    f32x4 acc[MI][NI];
#pragma unroll
    for (int x = 0; x < MI; ++x)
#pragma unroll
        for (int y = 0; y < NI; ++y) acc[x][y] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    // N groups from `first` on, all of them there and in one scale word
    auto unit = [&](auto count, int first) {
        constexpr int N = decltype(count)::value;
        i32x4 a[MI][N][2], b[NI][N][2];
        unsigned sa[MI], sb[NI];
#pragma unroll
        for (int y = 0; y < NI; ++y) {
#pragma unroll
            for (int u = 0; u < N; ++u)
#pragma unroll
                for (int h = 0; h < 2; ++h) b[y][u][h] = *reinterpret_cast<const i32x4*>(pb[y] + (first + u) * 128ll + h * 64);
            sb[y] = *reinterpret_cast<const unsigned*>(qb[y] + (first & ~3));
        }
#pragma unroll
        for (int x = 0; x < MI; ++x) {
#pragma unroll
            for (int u = 0; u < N; ++u)
#pragma unroll
                for (int h = 0; h < 2; ++h) a[x][u][h] = *reinterpret_cast<const i32x4*>(pa[x] + (first + u) * 128ll + h * 64);
            sa[x] = *reinterpret_cast<const unsigned*>(qa[x] + (first & ~3));
        }
        if constexpr (N < 4) {
            const int down = 8 * (first & 3);
#pragma unroll
            for (int x = 0; x < MI; ++x) sa[x] >>= down;
#pragma unroll
            for (int y = 0; y < NI; ++y) sb[y] >>= down;
        }
        auto group = [&](auto at) {
            constexpr int U = decltype(at)::value;
            if constexpr (U < N && !EXACT) {
#pragma unroll
                for (int x = 0; x < MI; ++x)
#pragma unroll
                    for (int y = 0; y < NI; ++y)
                        acc[x][y] = mfma16<U>(joined(b[y][U][0], b[y][U][1]), joined(a[x][U][0], a[x][U][1]), acc[x][y], sb[y], sa[x]);
            }
            if constexpr (U < N && EXACT) {
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    bf16x8 wide[NI];
#pragma unroll
                    for (int y = 0; y < NI; ++y)
                        wide[y] = widened(b[y][U][p >> 1][2 * (p & 1)], b[y][U][p >> 1][2 * (p & 1) + 1], scale_operand<U>(sb[y]));
#pragma unroll
                    for (int x = 0; x < MI; ++x) {
                        const bf16x8 w = widened(a[x][U][p >> 1][2 * (p & 1)], a[x][U][p >> 1][2 * (p & 1) + 1], scale_operand<U>(sa[x]));
#pragma unroll
                        for (int y = 0; y < NI; ++y) acc[x][y] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wide[y], w, acc[x][y], 0, 0, 0);
                    }
                }
            }
        };
        group(std::integral_constant<int, 0>{});
        group(std::integral_constant<int, 1>{});
        group(std::integral_constant<int, 2>{});
        group(std::integral_constant<int, 3>{});
    };
    for (int u = wave; u < units; u += W) {
        if (u * GU + GU <= groups) {
            unit(std::integral_constant<int, GU>{}, u * GU);
            continue;
        }
        for (int g = u * GU; g < groups; ++g) unit(std::integral_constant<int, 1>{}, g);   // the last unit, short
    }

    // row of fragment x: lane % 16; columns 4 * quarter .. of fragment y
#pragma unroll
    for (int x = 0; x < MI; ++x)
#pragma unroll
        for (int y = 0; y < NI; ++y) {
            const int r = 16 * x + i, quad = 4 * y + quarter;
            *reinterpret_cast<f32x4*>(&sums[wave][r * TN + ((quad ^ r) & (TN / 4 - 1)) * 4]) = acc[x][y];
        }
    __syncthreads();
    const int used = min(W, units);
    for (int q = threadIdx.x; q < TM * TN / 4; q += W * 64) {
        const int r = q / (TN / 4), quad = q % (TN / 4), at = r * TN + ((quad ^ r) & (TN / 4 - 1)) * 4;
        f32x4 v = *reinterpret_cast<const f32x4*>(&sums[0][at]);
        for (int w = 1; w < used; ++w) v += *reinterpret_cast<const f32x4*>(&sums[w][at]);
        const int row = i0 + r, col = j0 + quad * 4;
        if (row >= A.rows || col >= B.rows) continue;
        const long long to = row * ldo + col;
        put4<!EXACT>(out, to, v, B.rows - col, add);
    }
}

// ---------------------------------------------------------------- tiled kernel

// Workgroup tile BM x BN of out over one part of k, waves WM x WN.  A group of 128 columns
// of k is copied to LDS at a time, R groups in flight, and worked off in two stages of 64;
// a wave reads the fragments of the next stage while its matrix instructions work on the
// present one.
//   256 x 256, four waves of 128 x 128, R = 2: every operand byte read from LDS serves
//       128 rows, and a lane holds 256 accumulators.
//   128 x 128, four waves of 64 x 64, R = 4: a compute unit for each of up to 256 tiles.
//   128 x 128, eight waves of 64 x 32, R = 4: the same where k is short and starting counts.
//   128 x 128, four waves of 64 x 64, R = 2: two tiles a compute unit for more than 256, and
//       all of EXACT, whose conversions want a second wave on each unit's vector pipe.
//
// A fragment is 32 rows of a stage; lane l takes row l % 32 and 32 bytes, the 16-byte
// pieces 2 (l / 32) + 0, 1 of the stage's four.  LDS holds a row's 128 bytes of a group
// together, its eight pieces permuted so that a fragment's reads meet no bank twice:
// piece b of row i of a fragment at slot b ^ (i >> 1 & 7).  Scales come in words of four
// groups, each wave those of its own rows, a chunk of four groups ahead.
template <int BM, int BN, int WM, int WN, int R, int OUT, bool EXACT>
__global__ __launch_bounds__(WM* WN * 64) void fp8_tile(const Operand A, const Operand B, int row_groups, int scale_pitch,
                                                      int per_split, void* out, long long ldo, long long split_stride) {
    constexpr bool BF16 = OUT == OUT_BF16 || OUT == OUT_BF16_ADD, ADD = OUT == OUT_F32_ADD || OUT == OUT_BF16_ADD;
    constexpr int NW = WM * WN, ROWS = BM + BN;
    constexpr int MI = BM / WM / 32, NI = BN / WN / 32;      // fragments of a wave
    constexpr int CP = ROWS / 8 / NW;                       // 8-row copies of codes a wave makes for a group
    constexpr int SA = MI / 2, SB = (NI + 1) / 2;           // 64-row copies of scales a wave makes for a chunk
    static_assert(CP * 8 * NW == ROWS && (R == 2 || R == 4) && NI <= MI && MI % 2 == 0 && NW % 4 == 0 && BM % (8 * NW) == 0,
                  "tile and waves must fit");
    constexpr int GROUP = ROWS * 128, CHUNK = (SA + SB) * 256;   // bytes of a group, of a wave's scales of a chunk
    __shared__ __attribute__((aligned(1024))) unsigned char lds[R * GROUP + NW * 2 * CHUNK];
    const unsigned lds_at = static_cast<unsigned>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) unsigned char*)lds));

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int i0, j0, split;
    {
        // neighbouring tiles on one XCD, in bands of four tile rows
        const unsigned tiles_m = (A.rows + BM - 1) / BM, tiles_n = (B.rows + BN - 1) / BN, tiles = tiles_m * tiles_n;
        const unsigned place = xcd_place(blockIdx.x, gridDim.x);
        split = __builtin_amdgcn_readfirstlane(place / tiles);
        const unsigned t = place % tiles, band = t / (4 * tiles_n), first = band * 4, height = min(4u, tiles_m - first);
        const unsigned in = t - band * 4 * tiles_n;
        i0 = __builtin_amdgcn_readfirstlane((first + in % height) * BM);
        j0 = __builtin_amdgcn_readfirstlane(in / height * BN);
    }
    // this workgroup's part of k: per_split groups (a multiple of 4) from `begin` on
    const int begin = split * per_split, groups = min(per_split, row_groups - begin);
    const int half = lane >> 5, i = lane & 31, wm = wave / WN, wn = wave % WN;

    // With registers to spare (EARLY) both operands' fragments are held twice, so a
    // stage's reads are issued a whole stage ahead; else only B's, the smaller, are.
    constexpr bool EARLY = EXACT || MI * NI <= 4;
    // With groups to spare the second half of a group's codes is copied a stage later,
    // so that the copies are spread over all of the work.
    constexpr int LATER = EARLY && R > 2 ? CP / 2 : 0, NOW = CP - LATER;

    // A lane's part of out, 16 bytes of PER_ROW lanes a row.  What is added to is fetched
    // here, under the work, where there are registers for it (4096 x 1024 x 8192 to float32
    // in 63 us, fetched at the end 67; alone 60), else all together when the work is done.
    constexpr bool AHEAD = ADD && EARLY;
    constexpr int COLS = NI * 32, WIDE = BF16 ? 8 : 4, PER_ROW = COLS / WIDE, AT_ONCE = 64 / PER_ROW;
    const int col = j0 + wn * COLS + (lane % PER_ROW) * WIDE, row0 = i0 + wm * (BM / WM) + lane / PER_ROW;
    const int rows_left = A.rows - row0;                     // rows of this lane's from row0 on
    const bool whole = col + WIDE <= B.rows;                 // its 16 bytes are all there
    u32x4_any old[MI][32 / AT_ONCE];
    auto fetch = [&] {
#pragma unroll
        for (int x = 0; x < MI; ++x)
#pragma unroll
            for (int t = 0; t < 32 / AT_ONCE; ++t)
                if (whole && x * 32 + t * AT_ONCE < rows_left) old[x][t] = load16<BF16>(out, (row0 + x * 32 + t * AT_ONCE) * ldo + col);
    };
    if constexpr (AHEAD) fetch();

    // Where this wave's copies come from: a uniform base per operand and a lane's
    // offset (below 2^32: a tile's rows are at most 256 times 2^24 bytes).  Rows
    // past the operand are its last row again; their results are not written.
    const long long pitch = static_cast<long long>(row_groups) * 128;
    const unsigned char* const base_a = A.codes + i0 * pitch + begin * 128ll;
    const unsigned char* const base_b = B.codes + j0 * pitch + begin * 128ll;
    const unsigned left_a = A.rows - 1 - i0, left_b = B.rows - 1 - j0;
    // Rows of a B fragment are mixed (row 8 q + 4 h + s of the fragment is row
    // 16 (q / 2) + 8 h + 4 (q % 2) + s of the tile's 32), so that a lane's results are
    // twice eight neighbours of out.
    auto mixed = [](unsigned r) { return (r & ~15u) + ((r >> 2) & 1) * 8 + ((r >> 3) & 1) * 4 + (r & 3); };
    unsigned off[CP], soff_a[SA], soff_b[SB];
    const unsigned block = (lane & 7) ^ ((wave & 1) * 4 + (lane >> 4));   // of the eight of a group
#pragma unroll
    for (int c = 0; c < CP; ++c) {
        const unsigned r = (c * NW + wave) * 8 + (lane >> 3);   // of the stacked tile, BM of A over BN of B
        off[c] = (c * 8 * NW < BM ? min(r, left_a) : min(mixed(r - BM), left_b)) * static_cast<unsigned>(pitch) + block * 16;
    }
    const unsigned char* const sbase_a = A.scales + static_cast<long long>(i0 >> A.shift) * scale_pitch + begin;
    const unsigned char* const sbase_b = B.scales + static_cast<long long>(j0 >> B.shift) * scale_pitch + begin;
#pragma unroll
    for (int c = 0; c < SA; ++c) {
        const unsigned r = min(static_cast<unsigned>(wm * MI * 32 + c * 64 + lane), left_a);
        soff_a[c] = (((i0 + r) >> A.shift) - (i0 >> A.shift)) * scale_pitch;
    }
#pragma unroll
    for (int c = 0; c < SB; ++c) {
        const unsigned r = min(mixed(wn * NI * 32 + (NI == 1 ? i : c * 64 + lane)), left_b);
        soff_b[c] = (((j0 + r) >> B.shift) - (j0 >> B.shift)) * scale_pitch;
    }

    // Groups and chunks past the end are the last ones again.
    const int last_chunk = (groups - 1) / 4;
    auto copy_code = [&](int c, int group, int place) {
        copy16((c * 8 * NW < BM ? base_a : base_b) + min(group, groups - 1) * 128ll, off[c],
               lds_at + place * GROUP + (c * NW + wave) * 1024);
    };
    const unsigned scales_at = R * GROUP + wave * 2 * CHUNK;
    auto copy_scales = [&](int chunk, int place) {
        const unsigned at = lds_at + scales_at + place * CHUNK, word = min(chunk, last_chunk) * 4;
#pragma unroll
        for (int c = 0; c < SA; ++c) copy4(sbase_a, soff_a[c] + word, at + c * 256);
#pragma unroll
        for (int c = 0; c < SB; ++c) copy4(sbase_b, soff_b[c] + word, at + (SA + c) * 256);
    };

    // Where this wave's fragments lie.
    const int a_at = wm * MI * 4096 + i * 128, b_at = BM * 128 + wn * NI * 4096 + i * 128;
    int c_at[2][2];                                          // byte of a row, by stage and piece
#pragma unroll
    for (int q = 0; q < 4; ++q) c_at[q >> 1][q & 1] = (((q >> 1) * 4 + 2 * half + (q & 1)) ^ ((i >> 1) & 7)) * 16;
    auto read = [&](i32x8& f, int at, int place, int stage) {
        const i32x4 lo = *reinterpret_cast<const i32x4*>(lds + place * GROUP + at + c_at[stage][0]);
        const i32x4 hi = *reinterpret_cast<const i32x4*>(lds + place * GROUP + at + c_at[stage][1]);
        f = joined(lo, hi);
    };
    auto read_scales = [&](auto& sa, auto& sb, int place) {
        const unsigned char* const at = lds + scales_at + place * CHUNK;
#pragma unroll
        for (int x = 0; x < MI; ++x) sa[x] = *reinterpret_cast<const int*>(at + (x * 32 + i) * 4);
#pragma unroll
        for (int y = 0; y < NI; ++y) sb[y] = *reinterpret_cast<const int*>(at + SA * 256 + (y * 32 + i) * 4);
    };

    f32x16 acc[MI][NI];
#pragma unroll
    for (int x = 0; x < MI; ++x)
#pragma unroll
        for (int y = 0; y < NI; ++y)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[x][y][r] = 0.0f;

    // Chunk 0 of the scales and groups 0 .. R - 1 of the codes (the last without what the
    // loop's first stage copies).
    copy_scales(0, 0);
#pragma unroll
    for (int p = 0; p < R; ++p)
#pragma unroll
        for (int c = 0; c < (p == R - 1 ? NOW : CP); ++c) copy_code(c, p, p);
    wait_for<(R - 1) * CP - LATER>();
    meet();
    i32x8 fa0[MI], fa1[EARLY ? MI : 1], fb0[NI], fb1[NI];
    int sa[MI], sb[NI], san[MI], sbn[NI];
    read_scales(sa, sb, 0);
#pragma unroll
    for (int y = 0; y < NI; ++y) read(fb0[y], b_at + y * 4096, 0, 0);
#pragma unroll
    for (int x = 0; x < MI; ++x) read(fa0[x], a_at + x * 4096, 0, 0);

    bf16x8 wide_a[2][EXACT ? MI : 1], wide_b[2][EXACT ? NI : 1];
    if constexpr (EXACT) {
#pragma unroll
        for (int y = 0; y < NI; ++y) wide_b[0][y] = widened(fb0[y][0], fb0[y][1], scale_operand<0>(sb[y]));
#pragma unroll
        for (int x = 0; x < MI; ++x) wide_a[0][x] = widened(fa0[x][0], fa0[x][1], scale_operand<0>(sa[x]));
    }

    // One stage, the first or second (G) of a group, the Q-th of its chunk.  Group p + R
    // is copied from the second stage of group p on, into p's place, and has landed when
    // its first fragments are read, in the second stage of group p + R - 1.  Chunk c + 1
    // of the scales is copied in the first group of chunk c, behind its codes, and read in
    // the last.
    int chunk = 0;
    auto stage = [&](auto of_chunk, auto second, auto& fa, auto& fan, auto& fb, auto& fbn) {
        constexpr int Q = decltype(of_chunk)::value, G = decltype(second)::value;
        constexpr int HERE = Q % R, NEXT = G ? (Q + 1) % R : HERE;
        if constexpr (G == 1) {
            // the next group has landed: behind its codes were issued those of R - 2 more
            // groups, and the scales where one of their stages was a chunk's first
            constexpr int SCALES = R == 4 && (Q == 1 || Q == 2) ? SA + SB : 0;
            wait_for<(R - 2) * CP + SCALES>();
            if constexpr (EARLY) wait_reads();              // (issued a stage ago) and nobody reads this one any more
            meet();
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (Q == 3 && G == 1) read_scales(san, sbn, (chunk + 1) & 1);
        if constexpr (EARLY) {
#pragma unroll
            for (int y = 0; y < NI; ++y) read(fbn[y], b_at + y * 4096, NEXT, 1 - G);
#pragma unroll
            for (int x = 0; x < MI; ++x) read(fan[x], a_at + x * 4096, NEXT, 1 - G);
            __builtin_amdgcn_sched_barrier(0);
        }
        // The copies are spread over the matrix instructions: a wave that issues them
        // together waits for the address unit instead.
        if constexpr (EXACT) {
            // 16 columns of k a time.  The conversions of the next 16 (of the next stage, at the
            // end) are spread over the matrix instructions of the present ones.
            constexpr int PRODUCTS = MI * NI, FRAGMENTS = MI + NI, QN = G ? (Q + 1) & 3 : Q;
            auto& sa_next = [&]() -> auto& { if constexpr (Q == 3 && G == 1) return san; else return sa; }();
            auto& sb_next = [&]() -> auto& { if constexpr (Q == 3 && G == 1) return sbn; else return sb; }();
#pragma unroll
            for (int t = 0; t < 4 * PRODUCTS; ++t) {
                const int p = t / PRODUCTS, j = t % PRODUCTS, x = j / NI, y = j % NI, n = (p + 1) & 3;
                acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wide_b[p & 1][y], wide_a[p & 1][x], acc[x][y], 0, 0, 0);
#pragma unroll
                for (int f = j * FRAGMENTS / PRODUCTS; f < (j + 1) * FRAGMENTS / PRODUCTS; ++f) {
                    if (f < NI) {
                        const i32x8& from = p < 3 ? fb[f] : fbn[f];
                        wide_b[n & 1][f] = widened(from[2 * n], from[2 * n + 1], p < 3 ? scale_operand<Q>(sb[f]) : scale_operand<QN>(sb_next[f]));
                    } else {
                        const i32x8& from = p < 3 ? fa[f - NI] : fan[f - NI];
                        wide_a[n & 1][f - NI] = widened(from[2 * n], from[2 * n + 1], p < 3 ? scale_operand<Q>(sa[f - NI]) : scale_operand<QN>(sa_next[f - NI]));
                    }
                }
                constexpr int SLOTS = 4 * PRODUCTS;
                if constexpr (G == 1) {
#pragma unroll
                    for (int c = t * NOW / SLOTS; c < (t + 1) * NOW / SLOTS; ++c) copy_code(c, 4 * chunk + Q + R, HERE);
                    if (Q == 0 && t == SLOTS - 1) copy_scales(chunk + 1, (chunk + 1) & 1);
                } else {
#pragma unroll
                    for (int c = NOW + t * LATER / SLOTS; c < NOW + (t + 1) * LATER / SLOTS; ++c)
                        copy_code(c, 4 * chunk + Q - 1 + R, (Q + R - 1) % R);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        } else {
#pragma unroll
        for (int x = 0; x < MI; ++x) {
#pragma unroll
            for (int y = 0; y < NI; ++y) acc[x][y] = mfma32<Q>(fb[y], fa[x], acc[x][y], sb[y], sa[x]);
            if constexpr (!EARLY) {
                // a fragment of A gives way to the next stage's as soon as it is used
                read(fa[x], a_at + x * 4096, NEXT, 1 - G);
                if (x < NI) read(fbn[x], b_at + x * 4096, NEXT, 1 - G);
            }
            if constexpr (G == 1) {
                if (!EARLY && x == 0) {
                    // all of this stage's fragments are here (the next one's reads may
                    // still be out), so once every wave is here nobody reads this group
                    // any more
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int z = MI - 1; z >= 1; --z) arrived8(fa[z]);
#pragma unroll
                    for (int z = NI - 1; z >= 0; --z) arrived8(fb[z]);
                    meet();
                } else {
                    constexpr int FROM = EARLY ? 0 : 1;
#pragma unroll
                    for (int c = (x - FROM) * NOW / (MI - FROM); c < (x - FROM + 1) * NOW / (MI - FROM); ++c)
                        copy_code(c, 4 * chunk + Q + R, HERE);
                    if (Q == 0 && x == MI - 1) copy_scales(chunk + 1, (chunk + 1) & 1);
                }
            }
            if constexpr (G == 0 && LATER > 0) {
#pragma unroll
                for (int c = NOW + x * LATER / MI; c < NOW + (x + 1) * LATER / MI; ++c)
                    copy_code(c, 4 * chunk + Q - 1 + R, (Q + R - 1) % R);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        }
        if constexpr (Q == 3 && G == 1) {
#pragma unroll
            for (int x = 0; x < MI; ++x) sa[x] = san[x];
#pragma unroll
            for (int y = 0; y < NI; ++y) sb[y] = sbn[y];
        }
    };
    constexpr std::integral_constant<int, 0> k0{};
    constexpr std::integral_constant<int, 1> k1{};
    constexpr std::integral_constant<int, 2> k2{};
    constexpr std::integral_constant<int, 3> k3{};
    auto group = [&](auto q) {
        if constexpr (EARLY) {
            stage(q, k0, fa0, fa1, fb0, fb1);
            stage(q, k1, fa1, fa0, fb1, fb0);
        } else {
            stage(q, k0, fa0, fa0, fb0, fb1);
            stage(q, k1, fa0, fa0, fb1, fb0);
        }
    };
    for (; chunk < groups / 4; ++chunk) {
        group(k0);
        group(k1);
        group(k2);
        group(k3);
    }
    const int rest = groups & 3;
    if (rest > 0) group(k0);
    if (rest > 1) group(k1);
    if (rest > 2) group(k2);
    if constexpr (ADD && !AHEAD) fetch();
    wait_for<0>();
    meet();                                                  // every copy has landed, every fragment is read: LDS is free

    out = static_cast<char*>(out) + split * split_stride;

    // Results go through LDS, a row of fragments at a time in a region of the
    // wave's own, so that memory sees whole rows of the wave's columns.
    static_assert(NW * 32 * COLS * 4 <= R * GROUP, "the results' regions must fit");
    float* const mine = reinterpret_cast<float*>(lds) + wave * 32 * COLS;
#pragma unroll
    for (int x = 0; x < MI; ++x) {
#pragma unroll
        for (int y = 0; y < NI; ++y)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                // words 4 (r % 2) .. of the eight at columns 32 y + 16 (r / 2) + 8 half
                const int quad = (32 * y + 16 * (r >> 1) + 8 * half + 4 * (r & 1)) / 4;
                *reinterpret_cast<float4*>(mine + i * COLS + ((quad ^ i) & (COLS / 4 - 1)) * 4) =
                    make_float4(acc[x][y][4 * r], acc[x][y][4 * r + 1], acc[x][y][4 * r + 2], acc[x][y][4 * r + 3]);
            }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int t = 0; t < 32 / AT_ONCE; ++t) {
            const int r = t * AT_ONCE + lane / PER_ROW, row = row0 + x * 32 + t * AT_ONCE;
            float v[WIDE];
#pragma unroll
            for (int q = 0; q < WIDE / 4; ++q) {
                const int quad = (lane % PER_ROW) * (WIDE / 4) + q;
                const float4 f = *reinterpret_cast<const float4*>(mine + r * COLS + ((quad ^ r) & (COLS / 4 - 1)) * 4);
                v[4 * q] = f.x; v[4 * q + 1] = f.y; v[4 * q + 2] = f.z; v[4 * q + 3] = f.w;
            }
            if (row >= A.rows) continue;
            if (whole) {
                if constexpr (ADD) add16<BF16>(v, old[x][t]);
                store16<BF16, OUT != OUT_PART>(out, row * ldo + col, v);
            } else {
                put<BF16, ADD, WIDE>(out, row * ldo + col, v, B.rows - col);
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
}

template <bool BF16>
__global__ __launch_bounds__(256) void fp8_join(const float* parts, int splits, long long split_floats, int m, int n, int ldp,
                                                void* out, long long ldo, bool add) {
    join_parts<BF16>(parts, splits, split_floats, m, n, ldp, out, ldo, add);
}

// ---------------------------------------------------------------- launches

template <int MI, int NI, int W, int GU>
void launch_wave(const Operand& A, const Operand& B, int groups, int sp, void* out, int64_t ldo, int dtype, int add, hipStream_t s) {
    const unsigned grid = static_cast<unsigned>(tiles_of(A.rows, B.rows, 16 * MI, 16 * NI));
    TimedLaunch tl("fp8_wave", s);
    if (dtype == GC_BF16) fp8_wave<MI, NI, W, GU, false><<<grid, W * 64, 0, s>>>(A, B, groups, sp, out, ldo, add);
    else fp8_wave<MI, NI, W, GU, true><<<grid, W * 64, 0, s>>>(A, B, groups, sp, out, ldo, add);
}

template <int BM, int BN, int WM, int WN, int R, bool EXACT>
void launch_tile(const Plan& p, const Operand& A, const Operand& B, int groups, int sp, void* out, int64_t ldo, int add, void* ws,
                 hipStream_t s) {
    const unsigned grid = static_cast<unsigned>(tiles_of(A.rows, B.rows, BM, BN) * p.splits);
    const int64_t part = A.rows * p.ldp;
    TimedLaunch tl("fp8_tile", s);
    auto go = [&](auto kernel, void* to, int64_t ld, int64_t stride) {
        kernel<<<grid, WM * WN * 64, 0, s>>>(A, B, groups, sp, p.per_split, to, ld, stride);
    };
    if (p.splits > 1) {
        if constexpr (BM == 128 && (R == 4 || EXACT)) go(fp8_tile<BM, BN, WM, WN, R, OUT_PART, EXACT>, ws, p.ldp, part * 4);   // only these are split
    } else if (add) {
        go(fp8_tile<BM, BN, WM, WN, R, EXACT ? OUT_F32_ADD : OUT_BF16_ADD, EXACT>, out, ldo, 0);
    } else {
        go(fp8_tile<BM, BN, WM, WN, R, EXACT ? OUT_F32 : OUT_BF16, EXACT>, out, ldo, 0);
    }
}

}  // namespace
}  // namespace gc

using namespace gc;

extern "C" {

size_t gc_fp8_matmul_workspace_bytes(int64_t m, int64_t n, int64_t k) {
    if (!matmul_shape_ok(m, n, k)) return 0;
    int64_t need = 0;                                        // of either type of out
    for (const bool exact : {false, true}) {
        const Plan p = plan_of(m, n, k, exact);
        if (p.splits > 1) need = std::max(need, p.splits * m * p.ldp * 4);
    }
    return static_cast<size_t>(need);
}

int gc_fp8_matmul(const uint8_t* a_codes, const uint8_t* a_scales, int a_block_rows, const uint8_t* b_codes,
                  const uint8_t* b_scales, int b_block_rows, int64_t m, int64_t n, int64_t k, void* out, int64_t ldo,
                  int out_dtype, int accumulate, void* ws, size_t ws_bytes, void* stream) {
    const char* fn = "gc_fp8_matmul";
    int rc = mx_check_matrix(fn, "A", a_codes, a_scales);
    if (rc == GC_OK) rc = mx_check_matrix(fn, "B", b_codes, b_scales);
    if (rc != GC_OK) return rc;
    if (!f8_block_ok(a_block_rows) || !f8_block_ok(b_block_rows))
        return fail(GC_ERR_ARG, "gc_fp8_matmul: a_block_rows and b_block_rows must be 1 or 128");
    if (!out || !aligned16(out)) return fail(GC_ERR_ARG, "gc_fp8_matmul: out is null or not 16-byte aligned");
    if (out_dtype != GC_F32 && out_dtype != GC_BF16) return fail(GC_ERR_DTYPE, "gc_fp8_matmul: out_dtype must be GC_F32 or GC_BF16");
    if (!matmul_shape_ok(m, n, k)) return fail(GC_ERR_ARG, "gc_fp8_matmul: m, n or k out of range");
    if (ldo < n || ldo > MX_MAX_ENTRIES) return fail(GC_ERR_ARG, "gc_fp8_matmul: ldo must be in [n, 2^34]");
    if (m - 1 > MX_MAX_SPAN / ldo) return fail(GC_ERR_ARG, "gc_fp8_matmul: (m - 1) * ldo must be at most 2^40");
    const struct { const void* p; size_t n; } in[4] = {
        {a_codes, static_cast<size_t>(f8_code_bytes(m, k))}, {a_scales, static_cast<size_t>(f8_scale_bytes(m, k, a_block_rows))},
        {b_codes, static_cast<size_t>(f8_code_bytes(n, k))}, {b_scales, static_cast<size_t>(f8_scale_bytes(n, k, b_block_rows))}};
    const size_t ob = static_cast<size_t>((m - 1) * ldo + n) * (out_dtype == GC_BF16 ? 2 : 4);
    for (const auto& b : in)
        if (overlaps(out, ob, b.p, b.n)) return fail(GC_ERR_ARG, "gc_fp8_matmul: out overlaps an operand");
    const Plan p = plan_of(m, n, k, out_dtype == GC_F32);
    if (p.splits > 1) {
        const size_t need = static_cast<size_t>(p.splits * m * p.ldp * 4);
        if (!ws || !aligned16(ws)) return fail(GC_ERR_ARG, "gc_fp8_matmul: ws is null or not 16-byte aligned");
        if (ws_bytes < need) return fail(GC_ERR_WORKSPACE, "gc_fp8_matmul: workspace too small");
        for (const auto& b : in)
            if (overlaps(ws, need, b.p, b.n)) return fail(GC_ERR_ARG, "gc_fp8_matmul: ws overlaps a buffer");
        if (overlaps(ws, need, out, ob)) return fail(GC_ERR_ARG, "gc_fp8_matmul: ws overlaps a buffer");
    }
    const int groups = static_cast<int>(mx_groups(k)), sp = static_cast<int>(f8_scale_pitch(k));
    const Operand A = {a_codes, a_scales, static_cast<int>(m), f8_shift(a_block_rows)};
    const Operand B = {b_codes, b_scales, static_cast<int>(n), f8_shift(b_block_rows)};
    hipStream_t s = static_cast<hipStream_t>(stream);
    switch (p.kind) {
        case Plan::WAVE_1_1: launch_wave<1, 1, 8, 4>(A, B, groups, sp, out, ldo, out_dtype, accumulate, s); break;
        case Plan::WAVE_1_2: launch_wave<1, 2, 8, 4>(A, B, groups, sp, out, ldo, out_dtype, accumulate, s); break;
        case Plan::WAVE_2_1: launch_wave<2, 1, 8, 4>(A, B, groups, sp, out, ldo, out_dtype, accumulate, s); break;
        case Plan::WAVE_2_2: launch_wave<2, 2, 8, 4>(A, B, groups, sp, out, ldo, out_dtype, accumulate, s); break;
        case Plan::WAVE_2_4: launch_wave<2, 4, 8, 2>(A, B, groups, sp, out, ldo, out_dtype, accumulate, s); break;
        case Plan::WAVE_4_4: launch_wave<4, 4, 4, 2>(A, B, groups, sp, out, ldo, out_dtype, accumulate, s); break;
        case Plan::TILE_128: launch_tile<128, 128, 2, 2, 4, false>(p, A, B, groups, sp, out, ldo, accumulate, ws, s); break;
        case Plan::TILE_128_SHORT: launch_tile<128, 128, 2, 4, 4, false>(p, A, B, groups, sp, out, ldo, accumulate, ws, s); break;
        case Plan::TILE_128_PAIRED:
            if (out_dtype == GC_BF16) launch_tile<128, 128, 2, 2, 2, false>(p, A, B, groups, sp, out, ldo, accumulate, ws, s);
            else launch_tile<128, 128, 2, 2, 2, true>(p, A, B, groups, sp, out, ldo, accumulate, ws, s);
            break;
        case Plan::TILE_256: launch_tile<256, 256, 2, 2, 2, false>(p, A, B, groups, sp, out, ldo, accumulate, ws, s); break;
    }
    rc = check_launch(fn);
    if (rc != GC_OK || p.splits == 1) return rc;
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>((m * (p.ldp / 4) + 255) / 256, 8192));
    TimedLaunch tl("fp8_join", s);
    const float* parts = static_cast<const float*>(ws);
    if (out_dtype == GC_BF16) fp8_join<true><<<grid, 256, 0, s>>>(parts, p.splits, m * p.ldp, A.rows, B.rows, static_cast<int>(p.ldp), out, ldo, accumulate);
    else fp8_join<false><<<grid, 256, 0, s>>>(parts, p.splits, m * p.ldp, A.rows, B.rows, static_cast<int>(p.ldp), out, ldo, accumulate);
    return check_launch(fn);
}

}  // extern "C"
