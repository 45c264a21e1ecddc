// Product of two MXFP4 matrices: out[i, j] = [out +] sum_k A[i, k] * B[j, k].
//
// The f8f6f4 matrix instructions multiply E2M1 codes with one E8M0 scale per 32
// codes and add in float32: 16 x 128 by 128 x 16 (mxfp4_wave) or 32 x 64 by 64 x 32
// (mxfp4_tile).  A lane holds 32 consecutive codes of one row (16 bytes), which is
// one block, and the block's scale byte.  B goes in as the first operand, so that a
// lane's results are neighbours in a row of out.
//
// What bounds it.  Large products: 8192^3 with random codes takes 266 us (4.1 PFLOP/s),
// the matrix units busy for 59% of the cycles and the clock lowered to 1.7 GHz by the
// chip's power (158 us with codes of zero, 211 without the copies from memory).  About one
// 128 x 128 tile a compute unit: the copies into LDS and the matrix instructions, which
// overlap in part (4096 x 1024 x 8192: 25.0 us, either alone about 15; matrix units busy
// for 42% of the cycles).  Few rows: waiting for the read of B, two units of k one after
// the other (16 x 8192 x 8192: 10.0 us, 3.6 TB/s; one row 8.4; the waves wait for 60% of
// their time).  Small calls: the launch (1 x 4096 x 1024: 2.5 us).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "matmul.h"
#include "mxfp4.h"

namespace gc {
namespace {

constexpr int E2M1 = 4;   // operand format of the f8f6f4 matrix instructions

__device__ __forceinline__ f32x4 mfma16(i32x4 a, i32x4 b, f32x4 c, int sa, int sb) {
    const i32x8 x = {a[0], a[1], a[2], a[3], 0, 0, 0, 0}, y = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, E2M1, E2M1, 0, sa, 0, sb);
}

// 32 x 64 by 64 x 32: half the operand reads an operation of the above.  A lane
// holds one block of row lane % 32; U picks the scale byte.
template <int U>
__device__ __forceinline__ f32x16 mfma32(i32x4 a, i32x4 b, f32x16 c, int sa, int sb) {
    const i32x8 x = {a[0], a[1], a[2], a[3], 0, 0, 0, 0}, y = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, E2M1, E2M1, U, sa, U, sb);
}

struct Operand {
    const unsigned char* codes;
    const unsigned char* scales;
    int rows;
};

// ---------------------------------------------------------------- few tiles

// Where a 128 x 128 tile would leave most of the chip idle (few rows, or a small
// out): a workgroup takes 16 MI x 16 NI of out and its W waves share k, a unit at a
// time (wave w takes units w, w + W, ...), operands straight from memory to registers.
// The waves' sums meet in LDS and are added in wave order.  It is bound by one trip to
// memory and back, and for few rows by the read of B.  Units of four groups against
// units of two: 16 x 1024 x 8192 6.7 and 7.5 us, 16 x 8192 x 8192 11.6 and 13.4; the
// largest tile has registers for two.
//
// A unit of k is GU groups.  Lane l holds, of each group, block l / 16 of row l % 16
// (four lanes read 64 bytes of a row), and all of the row's scales of the unit, of
// which it shifts its own byte down.
template <int MI, int NI, int W, int GU>
__global__ __launch_bounds__(W * 64) void mxfp4_wave(const Operand A, const Operand B, int groups, void* out, long long ldo,
                                                     int bf16, int add) {
    constexpr int TM = 16 * MI, TN = 16 * NI;
    __shared__ __attribute__((aligned(16))) float sums[W][TM * TN];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i = lane & 15, quarter = lane >> 4;
    const int tiles_m = (A.rows + TM - 1) / TM;
    const unsigned t = xcd_place(blockIdx.x, gridDim.x);     // the tiles of one stretch of B on one XCD
    const int i0 = static_cast<int>(t % tiles_m) * TM, j0 = static_cast<int>(t / tiles_m) * TN;
    const int units = (groups + GU - 1) / GU;

    // scales are 4-byte aligned only
    typedef unsigned scales_t __attribute__((ext_vector_type(GU), aligned(4)));
    const unsigned char *pa[MI], *qa[MI], *pb[NI], *qb[NI];
#pragma unroll
    for (int x = 0; x < MI; ++x) {
        const long long r = static_cast<long long>(min(i0 + 16 * x + i, A.rows - 1)) * groups;
        pa[x] = A.codes + r * 64 + quarter * 16;
        qa[x] = A.scales + r * 4;
    }
#pragma unroll
    for (int y = 0; y < NI; ++y) {
        const long long r = static_cast<long long>(min(j0 + 16 * y + i, B.rows - 1)) * groups;
        pb[y] = B.codes + r * 64 + quarter * 16;
        qb[y] = B.scales + r * 4;
    }
    f32x4 acc[MI][NI];
#pragma unroll
    for (int x = 0; x < MI; ++x)
#pragma unroll
        for (int y = 0; y < NI; ++y) acc[x][y] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    auto unit = [&](int first) {                             // GU groups from `first` on, all of them there
        i32x4 a[MI][GU], b[NI][GU];
        scales_t sa[MI], sb[NI];
#pragma unroll
        for (int y = 0; y < NI; ++y) {
#pragma unroll
            for (int u = 0; u < GU; ++u) b[y][u] = *reinterpret_cast<const i32x4*>(pb[y] + (first + u) * 64ll);
            sb[y] = *reinterpret_cast<const scales_t*>(qb[y] + first * 4ll);
        }
#pragma unroll
        for (int x = 0; x < MI; ++x) {
#pragma unroll
            for (int u = 0; u < GU; ++u) a[x][u] = *reinterpret_cast<const i32x4*>(pa[x] + (first + u) * 64ll);
            sa[x] = *reinterpret_cast<const scales_t*>(qa[x] + first * 4ll);
        }
#pragma unroll
        for (int u = 0; u < GU; ++u)
#pragma unroll
            for (int x = 0; x < MI; ++x)
#pragma unroll
                for (int y = 0; y < NI; ++y)
                    acc[x][y] = mfma16(b[y][u], a[x][u], acc[x][y], sb[y][u] >> (8 * quarter), sa[x][u] >> (8 * quarter));
    };
    for (int u = wave; u < units; u += W) {
        if (u * GU + GU <= groups) {
            unit(u * GU);
            continue;
        }
        for (int g = u * GU; g < groups; ++g) {              // the last unit, short
            i32x4 a[MI], b[NI];
            int sa[MI], sb[NI];
#pragma unroll
            for (int y = 0; y < NI; ++y) {
                b[y] = *reinterpret_cast<const i32x4*>(pb[y] + g * 64ll);
                sb[y] = qb[y][g * 4ll + quarter];
            }
#pragma unroll
            for (int x = 0; x < MI; ++x) {
                a[x] = *reinterpret_cast<const i32x4*>(pa[x] + g * 64ll);
                sa[x] = qa[x][g * 4ll + quarter];
            }
#pragma unroll
            for (int x = 0; x < MI; ++x)
#pragma unroll
                for (int y = 0; y < NI; ++y) acc[x][y] = mfma16(b[y], a[x], acc[x][y], sb[y], sa[x]);
        }
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
        if (bf16) put4<true>(out, to, v, B.rows - col, add);
        else put4<false>(out, to, v, B.rows - col, add);
    }
}

// ---------------------------------------------------------------- tiled kernel

// Workgroup tile BM x BN of out over one part of k, waves WM x WN.  Stages of 128
// columns of k (one group) are copied to LDS in pairs, R pairs at a time; a wave
// reads the fragments of the next stage while its matrix instructions work on the
// present one.  Pairs, since eight lanes then fetch 128 neighbouring bytes of a row:
// with stages of 64, eight waves and direct stores of the results 8192^3 took 329 us,
// with pairs, four waves and results by way of LDS 278, with bands of tiles and
// streaming stores 260.
//   256 x 256, four waves of 128 x 128, R = 2: every operand byte read from LDS serves
//       128 rows, and a lane holds 256 accumulators; with eight waves 290 against 278 us.
//   128 x 128, eight waves of 64 x 32, R = 4: a compute unit for each of up to 256 tiles.
//       4096 x 1024 x 8192: 23.8 us (25.0 on other cards), 30.9 with the next, 48.8 with the
//       first; 25.5 with two teams of four 64 x 64 waves that share k, which read a third
//       less from LDS.
//   128 x 128, four waves of 64 x 64, R = 2: two tiles a compute unit for more than 256.
//       4096 x 2048 x 8192: 43.8 us, 51.8 with the one before, 53.0 with the first.
//
// A fragment is 32 rows of a stage; lane l takes row l % 32 and, of the group's
// four blocks, 2 (l / 32) + u in matrix instruction u = 0, 1, so that one 16-bit
// read brings the scale bytes of both.  LDS holds a row's 128 bytes of a pair
// together, its eight blocks permuted so that a fragment's reads meet no bank
// twice: block b of row i of a fragment at slot b ^ (i >> 1 & 7).  Scales come in
// chunks of four groups (16 bytes of a row), half a chunk with each pair, with
// group q of row i at word (q + (i >> 3)) & 3.
template <int BM, int BN, int WM, int WN, int R, int OUT>
__global__ __launch_bounds__(WM* WN * 64) void mxfp4_tile(const Operand A, const Operand B, int row_groups, int per_split,
                                                        void* out, long long ldo, long long split_stride) {
    constexpr bool BF16 = OUT == OUT_BF16 || OUT == OUT_BF16_ADD, ADD = OUT == OUT_F32_ADD || OUT == OUT_BF16_ADD;
    constexpr int NW = WM * WN, ROWS = BM + BN;
    constexpr int MI = BM / WM / 32, NI = BN / WN / 32;      // fragments of a wave
    constexpr int CP = ROWS / 8 / NW;                       // 8-row copies of codes a wave makes for a pair
    constexpr int SP = ROWS / 16 / NW;                      // 16-row copies of scales a wave makes for a chunk
    static_assert(CP * 8 * NW == ROWS && SP * 16 * NW == ROWS && SP % 2 == 0 && R % 2 == 0 && NI <= MI && MI >= 2 && NW % 4 == 0 &&
                      BM % (16 * NW) == 0, "tile and waves must fit");
    constexpr int D = (R + 2) / 2;                          // chunks of scales in flight
    constexpr int PAIR = ROWS * 128, CHUNK = ROWS * 16;
    __shared__ __attribute__((aligned(1024))) unsigned char lds[R * PAIR + (D + 1) * CHUNK];
    unsigned char* const scale_lds = lds + R * PAIR;
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

    // With registers to spare (EARLY) both operands' fragments are held twice, so a
    // stage's reads are issued a whole stage ahead; else only B's, the smaller, are.
    constexpr bool EARLY = MI * NI <= 4;
    // With pairs to spare the second half of a pair's codes is copied a stage later,
    // so that the copies are spread over all of the work (24.6 us -> 23.8).
    constexpr int LATER = EARLY && R > 2 ? CP / 2 : 0, NOW = CP - LATER;

    // A lane's part of out, 16 bytes of PER_ROW lanes a row.  What is added to is
    // fetched here, under the work, where a workgroup has a compute unit to itself and
    // registers for it (4096 x 1024 x 8192 added to float32: 29.4 us, 30.8 fetched at the end; 28.0 now).
    constexpr bool AHEAD = ADD && EARLY && R == 4;
    constexpr int COLS = NI * 32, WIDE = BF16 ? 8 : 4, PER_ROW = COLS / WIDE, AT_ONCE = 64 / PER_ROW;
    const int wm = wave / WN, wn = wave % WN;
    const int col = j0 + wn * COLS + (lane % PER_ROW) * WIDE, row0 = i0 + wm * (BM / WM) + lane / PER_ROW;
    const bool inside = i0 + BM <= A.rows && j0 + BN <= B.rows;
    u32x4_any old[AHEAD ? MI : 1][32 / AT_ONCE];
    if (AHEAD && inside) {
#pragma unroll
        for (int x = 0; x < MI; ++x)
#pragma unroll
            for (int t = 0; t < 32 / AT_ONCE; ++t) old[x][t] = load16<BF16>(out, (row0 + x * 32 + t * AT_ONCE) * ldo + col);
    }

    // Where this wave's copies come from: a uniform base per operand and a lane's
    // offset (below 2^32: a tile's rows are at most 256 times 2^23 bytes).  Rows
    // past the operand are its last row again; their results are not written.
    const long long pitch = static_cast<long long>(row_groups) * 64;
    const unsigned char* const base_a = A.codes + i0 * pitch + begin * 64ll;
    const unsigned char* const base_b = B.codes + j0 * pitch + begin * 64ll;
    const unsigned char* const sbase_a = A.scales + i0 * (pitch / 16) + begin * 4ll;
    const unsigned char* const sbase_b = B.scales + j0 * (pitch / 16) + begin * 4ll;
    const unsigned left_a = A.rows - 1 - i0, left_b = B.rows - 1 - j0;
    // Row r of the stacked tile, BM of A over BN of B.  Rows of a B fragment are
    // mixed (row 8 q + 4 h + s of the fragment is row 16 (q / 2) + 8 h + 4 (q % 2) + s of
    // the tile's 32), so that a lane's results are twice eight neighbours of out.
    auto row_offset = [&](unsigned r, bool a, unsigned row_bytes) {
        if (a) return min(r, left_a) * row_bytes;
        r -= BM;
        return min((r & ~15u) + ((r >> 2) & 1) * 8 + ((r >> 3) & 1) * 4 + (r & 3), left_b) * row_bytes;
    };
    unsigned off[CP], soff[SP];
    const unsigned block = (lane & 7) ^ ((wave & 1) * 4 + (lane >> 4));   // of the eight of a pair
#pragma unroll
    for (int c = 0; c < CP; ++c)
        off[c] = row_offset((c * NW + wave) * 8 + (lane >> 3), c * 8 * NW < BM, static_cast<unsigned>(pitch)) + block * 16;
    const unsigned second = block & 4 ? 64 : 0;              // what leads from the pair's second group back to its first
#pragma unroll
    for (int c = 0; c < SP; ++c)
        soff[c] = row_offset((c * NW + wave) * 16 + (lane >> 2), c * 16 * NW < BM, static_cast<unsigned>(pitch / 16));
    const int sgroup = (lane - 2 * wave - (lane >> 5)) & 3;   // which group of a chunk this lane copies scales of

    // Pairs and chunks past the end are the last ones again, the second group of a
    // pair that has one only is the first again.
    const int last_pair = (groups - 1) / 2;
    auto copy_code = [&](int c, int pair, int place) {
        const int p = min(pair, last_pair);
        const unsigned back = 2 * p + 1 < groups ? 0 : second;
        copy16((c * 8 * NW < BM ? base_a : base_b) + static_cast<long long>(p) * 128, off[c] - back,
               lds_at + place * PAIR + (c * NW + wave) * 1024);
    };
    auto copy_scale = [&](int c, int chunk, int ring) {
        const unsigned g = min(chunk * 4 + sgroup, groups - 1) * 4;
        copy4(c * 16 * NW < BM ? sbase_a : sbase_b, soff[c] + g, lds_at + R * PAIR + ring * CHUNK + (c * NW + wave) * 256);
    };

    // Where this wave's fragments lie.
    const int half = lane >> 5, i = lane & 31;
    const int a_at = wm * MI * 4096 + i * 128, b_at = BM * 128 + wn * NI * 4096 + i * 128;
    const int as_at = wm * MI * 512 + i * 16 + 2 * half, bs_at = BM * 16 + wn * NI * 512 + i * 16 + 2 * half;
    int c_at[2][2];                                          // byte of a row, by group of the pair and u
#pragma unroll
    for (int q = 0; q < 4; ++q) c_at[q >> 1][q & 1] = (((q >> 1) * 4 + 2 * half + (q & 1)) ^ ((i >> 1) & 7)) * 16;

    struct Place {
        int pair, ring;                                      // LDS place of a stage's codes and scales,
        int group, word;                                     // and where it lies in its pair and chunk
    };
    auto read_a = [&](auto& a, auto& sa, int x, Place s) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
            a[x][u] = *reinterpret_cast<const i32x4*>(lds + s.pair * PAIR + a_at + c_at[s.group][u] + x * 4096);
        sa[x] = *reinterpret_cast<const unsigned short*>(scale_lds + s.ring * CHUNK + as_at + ((s.word + (i >> 3)) & 3) * 4 + x * 512);
    };
    auto read_b = [&](auto& b, auto& sb, int y, Place s) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
            b[y][u] = *reinterpret_cast<const i32x4*>(lds + s.pair * PAIR + b_at + c_at[s.group][u] + y * 4096);
        sb[y] = *reinterpret_cast<const unsigned short*>(scale_lds + s.ring * CHUNK + bs_at + ((s.word + (i >> 3)) & 3) * 4 + y * 512);
    };

    f32x16 acc[MI][NI];
#pragma unroll
    for (int x = 0; x < MI; ++x)
#pragma unroll
        for (int y = 0; y < NI; ++y)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[x][y][r] = 0.0f;

    // Pairs 0 .. R - 1 (without what the loop's first stage copies) and chunks 0 .. D - 1,
    // from pair 2 on in the order of the loop, so that its wait counts hold from the start.
#pragma unroll
    for (int p = 0; p < R; ++p) {
        if (p < 2) {
#pragma unroll
            for (int c = 0; c < SP; ++c) copy_scale(c, p, p);
        } else {
#pragma unroll
            for (int c = 0; c < SP / 2; ++c) copy_scale((p & 1) * (SP / 2) + c, 2 + (p - 2) / 2, 2 + (p - 2) / 2);
        }
#pragma unroll
        for (int c = 0; c < (p == R - 1 ? NOW : CP); ++c) copy_code(c, p, p);
    }
    wait_for<(D - 1) * SP + (R - 1) * CP - LATER>();
    meet();
    i32x4 fa0[MI][2], fa1[EARLY ? MI : 1][2], fb0[NI][2], fb1[NI][2];
    int sa0[MI], sa1[EARLY ? MI : 1], sb0[NI], sb1[NI];
#pragma unroll
    for (int y = 0; y < NI; ++y) read_b(fb0, sb0, y, {0, 0, 0, 0});
#pragma unroll
    for (int x = 0; x < MI; ++x) read_a(fa0, sa0, x, {0, 0, 0, 0});

    // One stage, the first or second (G) of a pair, the first or second (P) of a
    // chunk.  Pair p + R is copied from the second stage of pair p on, into p's place,
    // and has landed when its first fragments are read, in the second stage of pair
    // p + R - 1.  Chunk c + D comes with the two pairs of chunk c, where chunk c - 1 was.
    int chunk = 0, ring = 0, pair = 0;                       // chunk, and the places of chunk and pair
    auto stage = [&](auto second_pair, auto second_stage, auto& fa, auto& sa, auto& fan, auto& san, auto& fb, auto& sb,
                     auto& fbn, auto& sbn) {
        constexpr int P = decltype(second_pair)::value, G = decltype(second_stage)::value;
        const int ring1 = ring == D ? 0 : ring + 1, pair1 = pair == R - 1 ? 0 : pair + 1;
        const Place next = {G ? pair1 : pair, P && G ? ring1 : ring, 1 - G, (2 * P + G + 1) & 3};
        if constexpr (G == 1) {
            wait_for<(R - 2) * (CP + SP / 2)>();            // the next pair has landed
            if constexpr (EARLY) wait_reads();              // (issued a stage ago) and nobody reads this one any more
            meet();
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (EARLY) {
#pragma unroll
            for (int y = 0; y < NI; ++y) read_b(fbn, sbn, y, next);
#pragma unroll
            for (int x = 0; x < MI; ++x) read_a(fan, san, x, next);
            __builtin_amdgcn_sched_barrier(0);
        }
        // The copies are spread over the matrix instructions: a wave that issues them
        // together waits for the address unit instead.
#pragma unroll
        for (int x = 0; x < MI; ++x) {
#pragma unroll
            for (int y = 0; y < NI; ++y) acc[x][y] = mfma32<0>(fb[y][0], fa[x][0], acc[x][y], sb[y], sa[x]);
#pragma unroll
            for (int y = 0; y < NI; ++y) acc[x][y] = mfma32<1>(fb[y][1], fa[x][1], acc[x][y], sb[y], sa[x]);
            if constexpr (!EARLY) {
                // a fragment of A gives way to the next stage's as soon as it is used
                read_a(fa, sa, x, next);
                if (x < NI) read_b(fbn, sbn, x, next);
            }
            if constexpr (G == 1) {
                if (!EARLY && x == 0) {
                    // all of this stage's fragments are here (the next one's reads, six
                    // so far, may still be out), so once every wave is here nobody reads
                    // this pair any more
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int z = MI - 1; z >= 1; --z) arrived(sa[z]), arrived(fa[z][1]), arrived(fa[z][0]);
#pragma unroll
                    for (int z = NI - 1; z >= 0; --z) arrived(sb[z]), arrived(fb[z][1]), arrived(fb[z][0]);
                    meet();
                } else {
                    constexpr int FROM = EARLY ? 0 : 1;
#pragma unroll
                    for (int c = (x - FROM) * NOW / (MI - FROM); c < (x - FROM + 1) * NOW / (MI - FROM); ++c)
                        copy_code(c, 2 * chunk + P + R, pair);
                    if (x == MI - 1) {
#pragma unroll
                        for (int c = 0; c < SP / 2; ++c) copy_scale(P * (SP / 2) + c, chunk + D, ring == 0 ? D : ring - 1);
                    }
                }
            }
            if constexpr (G == 0 && LATER > 0) {
#pragma unroll
                for (int c = NOW + x * LATER / MI; c < NOW + (x + 1) * LATER / MI; ++c)
                    copy_code(c, 2 * chunk + P - 1 + R, pair == 0 ? R - 1 : pair - 1);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (G == 1) pair = pair1;
        if constexpr (P == 1 && G == 1) ring = ring1;
    };
    auto even = [&](auto p, auto g) {
        if constexpr (EARLY) stage(p, g, fa0, sa0, fa1, sa1, fb0, sb0, fb1, sb1);
        else stage(p, g, fa0, sa0, fa0, sa0, fb0, sb0, fb1, sb1);
    };
    auto odd = [&](auto p, auto g) {
        if constexpr (EARLY) stage(p, g, fa1, sa1, fa0, sa0, fb1, sb1, fb0, sb0);
        else stage(p, g, fa0, sa0, fa0, sa0, fb1, sb1, fb0, sb0);
    };
    constexpr std::integral_constant<int, 0> k0{};
    constexpr std::integral_constant<int, 1> k1{};
    for (; chunk < groups / 4; ++chunk) {
        even(k0, k0);
        odd(k0, k1);
        even(k1, k0);
        odd(k1, k1);
    }
    const int rest = groups & 3;
    if (rest > 0) even(k0, k0);
    if (rest > 1) odd(k0, k1);
    if (rest > 2) even(k1, k0);
    wait_for<0>();
    meet();                                                  // every copy has landed, every fragment is read: LDS is free

    out = static_cast<char*>(out) + split * split_stride;

    // Results go through LDS, a row of fragments at a time in a region of the
    // wave's own, so that memory sees whole rows of the wave's columns.
    static_assert(NW * 32 * COLS * 4 <= 2 * PAIR, "the results' regions must fit");
    float* const mine = reinterpret_cast<float*>(lds) + wave * 32 * COLS;
#pragma unroll
    for (int x = 0; x < MI; ++x) {
        if (ADD && !AHEAD && inside) {
#pragma unroll
            for (int t = 0; t < 32 / AT_ONCE; ++t) old[0][t] = load16<BF16>(out, (row0 + x * 32 + t * AT_ONCE) * ldo + col);
        }
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
            if (inside) {
                if constexpr (ADD) add16<BF16>(v, old[AHEAD ? x : 0][t]);
                store16<BF16, OUT != OUT_PART>(out, row * ldo + col, v);
            } else if (row < A.rows) {
                put<BF16, ADD, WIDE>(out, row * ldo + col, v, B.rows - col);
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
}

// 1024 x 1024 x 32768 takes 31 us with its join, 63 in one part.
template <bool BF16>
__global__ __launch_bounds__(256) void mxfp4_join(const float* parts, int splits, long long split_floats, int m, int n, int ldp,
                                                  void* out, long long ldo, bool add) {
    join_parts<BF16>(parts, splits, split_floats, m, n, ldp, out, ldo, add);
}

// ---------------------------------------------------------------- choice of the kernel

struct Plan {
    enum Kind { WAVE_1_1, WAVE_1_2, WAVE_2_1, WAVE_2_2, WAVE_2_4, WAVE_4_4, TILE_128, TILE_128_PAIRED, TILE_256 } kind;
    int splits, per_split;                                   // parts of k, groups of each
    int64_t ldp;                                             // entries between the rows of a part
};

bool matmul_shape_ok(int64_t m, int64_t n, int64_t k) {
    return m <= MX_MAX_DIM && n <= MX_MAX_DIM && k <= MX_MAX_K && mx_shape_ok(m, k) && mx_shape_ok(n, k) && mx_shape_ok(m, n);
}

// The cheapest kernel by times (in us) fitted to measurements of every kernel over
// m of 1 .. 8192, n of 16 .. 100000 and k of 256 .. 32768; a round is what 256 compute
// units take at once.  Both sides at some borders: 16 x 8192 x 8192: 12.8 (1 x 1), 10.4
// (1 x 2); 64 x 4096 x 1024: 5.0 (1 x 1), 3.8 (2 x 1), 3.5 (2 x 2), 4.3 (2 x 4); 777 x 1001 x
// 1155: 9.2 (2 x 4), 7.3 (4 x 4), 9.9 (128); 512 x 4096 x 1024: 12.1 (4 x 4), 6.3 (128);
// 1024 x 1024 x 16384: 35 (128), 26 (in two parts), 23 (in four); 2048 x 4096 x 4096: 28.5
// (128), 25.0 (128, two a unit), 31.7 (256); 4096 x 4096 x 4096: 57.6, 47.1, 38.0;
// 6144 x 4096 x 1024: 34.6, 26.2, 28.7.
Plan plan_of(int64_t m, int64_t n, int64_t k) {
    const int groups = static_cast<int>(mx_groups(k));
    const double g = groups;
    Plan best = {Plan::TILE_256, 1, (groups + 3) / 4 * 4, (n + 3) / 4 * 4};
    double least = INFINITY;
    auto offer = [&](Plan::Kind kind, double us, int splits) {
        if (us >= least) return;
        least = us;
        best.kind = kind;
        best.per_split = ((groups + splits - 1) / splits + 3) / 4 * 4;
        best.splits = (groups + best.per_split - 1) / best.per_split;
    };
    // several of these fit a compute unit, the last two alone: whole rounds.  A launch
    // holds fewer than 2^32 threads, 512 a workgroup.
    auto wave = [&](Plan::Kind kind, int mi, int ni, double per_group, bool whole) {
        const int64_t tiles = tiles_of(m, n, 16 * mi, 16 * ni);
        if (tiles > int64_t(1) << 22) return;
        const double r = std::max(1.0, tiles / 256.0);
        offer(kind, 2.5 + per_group * g * (whole ? std::ceil(r) : r), 1);
    };
    wave(Plan::WAVE_1_1, 1, 1, 0.08, false);
    wave(Plan::WAVE_1_2, 1, 2, 0.12, false);
    wave(Plan::WAVE_2_1, 2, 1, 0.11, false);
    wave(Plan::WAVE_2_2, 2, 2, 0.15, false);
    wave(Plan::WAVE_2_4, 2, 4, 0.24, true);
    wave(Plan::WAVE_4_4, 4, 4, 0.42, true);
    // A part costs its write and read back, and a launch; at most 256 workgroups.
    const int64_t t128 = tiles_of(m, n, 128, 128), t256 = tiles_of(m, n, 256, 256);
    for (int s = 1; s <= MAX_SPLITS && t128 * s <= 256 && (s == 1 || groups >= 16 * s); s *= 2) {
        const double parts = s > 1 ? 5.0 + 0.55e-6 * 4.0 * s * static_cast<double>(m) * best.ldp : 0.0;
        offer(Plan::TILE_128, 4.2 + (t128 * s > 128 ? 0.31 : 0.26) * std::ceil(g / s) + parts, s);
    }
    auto rounds = [](double x) { return x <= 1 ? 1.0 : (x + std::ceil(x)) / 2; };
    if (t128 > 256) {
        offer(Plan::TILE_128_PAIRED, rounds(t128 / 512.0) * (3.5 + 0.66 * g), 1);
        offer(Plan::TILE_256, rounds(t256 / 256.0) * (8.0 + 0.95 * g), 1);
    }
    return best;
}

template <int MI, int NI, int W, int GU>
void launch_wave(const Operand& A, const Operand& B, int groups, void* out, int64_t ldo, int dtype, int add, hipStream_t s) {
    const unsigned grid = static_cast<unsigned>(tiles_of(A.rows, B.rows, 16 * MI, 16 * NI));
    TimedLaunch tl("mxfp4_wave", s);
    mxfp4_wave<MI, NI, W, GU><<<grid, W * 64, 0, s>>>(A, B, groups, out, ldo, dtype == GC_BF16, add);
}

template <int BM, int BN, int WM, int WN, int R>
void launch_tile(const Plan& p, const Operand& A, const Operand& B, int groups, void* out, int64_t ldo, int dtype, int add,
                 void* ws, hipStream_t s) {
    const unsigned grid = static_cast<unsigned>(tiles_of(A.rows, B.rows, BM, BN) * p.splits);
    const int64_t part = A.rows * p.ldp;
    const int kind = p.splits > 1 ? OUT_PART : dtype == GC_BF16 ? (add ? OUT_BF16_ADD : OUT_BF16) : (add ? OUT_F32_ADD : OUT_F32);
    TimedLaunch tl("mxfp4_tile", s);
    switch (kind) {
        case OUT_F32: mxfp4_tile<BM, BN, WM, WN, R, OUT_F32><<<grid, WM * WN * 64, 0, s>>>(A, B, groups, p.per_split, out, ldo, 0); break;
        case OUT_F32_ADD: mxfp4_tile<BM, BN, WM, WN, R, OUT_F32_ADD><<<grid, WM * WN * 64, 0, s>>>(A, B, groups, p.per_split, out, ldo, 0); break;
        case OUT_BF16: mxfp4_tile<BM, BN, WM, WN, R, OUT_BF16><<<grid, WM * WN * 64, 0, s>>>(A, B, groups, p.per_split, out, ldo, 0); break;
        case OUT_BF16_ADD: mxfp4_tile<BM, BN, WM, WN, R, OUT_BF16_ADD><<<grid, WM * WN * 64, 0, s>>>(A, B, groups, p.per_split, out, ldo, 0); break;
        default:
            if constexpr (BM == 128 && R == 4)               // only this one is split
                mxfp4_tile<BM, BN, WM, WN, R, OUT_PART><<<grid, WM * WN * 64, 0, s>>>(A, B, groups, p.per_split, ws, p.ldp, part * 4);
    }
}

}  // namespace
}  // namespace gc

using namespace gc;

extern "C" {

size_t gc_mxfp4_matmul_workspace_bytes(int64_t m, int64_t n, int64_t k) {
    if (!matmul_shape_ok(m, n, k)) return 0;
    const Plan p = plan_of(m, n, k);
    return p.splits > 1 ? static_cast<size_t>(p.splits * m * p.ldp * 4) : 0;
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
    if (!matmul_shape_ok(m, n, k))
        return fail(GC_ERR_ARG, "gc_mxfp4_matmul: m, n or k out of range");
    if (ldo < n || ldo > MX_MAX_ENTRIES) return fail(GC_ERR_ARG, "gc_mxfp4_matmul: ldo must be in [n, 2^34]");
    if (m - 1 > MX_MAX_SPAN / ldo) return fail(GC_ERR_ARG, "gc_mxfp4_matmul: (m - 1) * ldo must be at most 2^40");
    const size_t ob = static_cast<size_t>((m - 1) * ldo + n) * (out_dtype == GC_BF16 ? 2 : 4);
    if (overlaps(out, ob, a_codes, mx_code_bytes(m, k)) || overlaps(out, ob, a_scales, mx_scale_bytes(m, k)) ||
        overlaps(out, ob, b_codes, mx_code_bytes(n, k)) || overlaps(out, ob, b_scales, mx_scale_bytes(n, k)))
        return fail(GC_ERR_ARG, "gc_mxfp4_matmul: out overlaps an operand");
    const Plan p = plan_of(m, n, k);
    if (p.splits > 1) {
        const size_t need = static_cast<size_t>(p.splits * m * p.ldp * 4);
        if (!ws || !aligned16(ws)) return fail(GC_ERR_ARG, "gc_mxfp4_matmul: ws is null or not 16-byte aligned");
        if (ws_bytes < need) return fail(GC_ERR_WORKSPACE, "gc_mxfp4_matmul: workspace too small");
        if (overlaps(ws, need, out, ob) || overlaps(ws, need, a_codes, mx_code_bytes(m, k)) ||
            overlaps(ws, need, a_scales, mx_scale_bytes(m, k)) || overlaps(ws, need, b_codes, mx_code_bytes(n, k)) ||
            overlaps(ws, need, b_scales, mx_scale_bytes(n, k)))
            return fail(GC_ERR_ARG, "gc_mxfp4_matmul: ws overlaps a buffer");
    }
    const int groups = static_cast<int>(mx_groups(k));
    const Operand A = {a_codes, a_scales, static_cast<int>(m)}, B = {b_codes, b_scales, static_cast<int>(n)};
    hipStream_t s = static_cast<hipStream_t>(stream);
    switch (p.kind) {
        case Plan::WAVE_1_1: launch_wave<1, 1, 8, 4>(A, B, groups, out, ldo, out_dtype, accumulate, s); break;
        case Plan::WAVE_1_2: launch_wave<1, 2, 8, 4>(A, B, groups, out, ldo, out_dtype, accumulate, s); break;
        case Plan::WAVE_2_1: launch_wave<2, 1, 8, 4>(A, B, groups, out, ldo, out_dtype, accumulate, s); break;
        case Plan::WAVE_2_2: launch_wave<2, 2, 8, 4>(A, B, groups, out, ldo, out_dtype, accumulate, s); break;
        case Plan::WAVE_2_4: launch_wave<2, 4, 8, 4>(A, B, groups, out, ldo, out_dtype, accumulate, s); break;
        case Plan::WAVE_4_4: launch_wave<4, 4, 4, 2>(A, B, groups, out, ldo, out_dtype, accumulate, s); break;
        case Plan::TILE_128: launch_tile<128, 128, 2, 4, 4>(p, A, B, groups, out, ldo, out_dtype, accumulate, ws, s); break;
        case Plan::TILE_128_PAIRED: launch_tile<128, 128, 2, 2, 2>(p, A, B, groups, out, ldo, out_dtype, accumulate, ws, s); break;
        case Plan::TILE_256: launch_tile<256, 256, 2, 2, 2>(p, A, B, groups, out, ldo, out_dtype, accumulate, ws, s); break;
    }
    rc = check_launch(fn);
    if (rc != GC_OK || p.splits == 1) return rc;
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>((m * (p.ldp / 4) + 255) / 256, 8192));
    TimedLaunch tl("mxfp4_join", s);
    const float* parts = static_cast<const float*>(ws);
    if (out_dtype == GC_BF16) mxfp4_join<true><<<grid, 256, 0, s>>>(parts, p.splits, m * p.ldp, A.rows, B.rows, static_cast<int>(p.ldp), out, ldo, accumulate);
    else mxfp4_join<false><<<grid, 256, 0, s>>>(parts, p.splits, m * p.ldp, A.rows, B.rows, static_cast<int>(p.ldp), out, ldo, accumulate);
    return check_launch(fn);
}

}  // extern "C"
