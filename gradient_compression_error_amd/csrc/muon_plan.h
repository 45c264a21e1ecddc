// How the matrices of an orthogonalised update lie in the workspace and are cut into tiles and parts (host, and
// places for the device).
#pragma once

#include <algorithm>
#include <cmath>

#include "matmul.h"

namespace gc {
namespace {

constexpr int MU_MAX = 32;             // matrices of a launch: their table fits a launch's arguments
constexpr int64_t MU_MAX_SIDE = int64_t(1) << 22;
constexpr int MU_MAX_PARTS = 64;

enum { GRAM, POLY, APPLY, LAST_F32, LAST_BF16 };
constexpr bool symmetric(int kind) { return kind == GRAM || kind == POLY; }

// Where a matrix's parts lie in the workspace, n <= m the oriented sides.
struct Shape {
    long long base;
    int n, m;
};
__host__ __device__ inline int64_t mu_groups(int64_t cols) { return (cols + 31) / 32; }
__host__ __device__ inline long long at_x(const Shape& s) { return s.base; }
__host__ __device__ inline long long at_xt(const Shape& s, int which) {
    return at_x(s) + s.n * mu_groups(s.m) * 128 + which * (s.m * mu_groups(s.n) * 128);
}
__host__ __device__ inline long long at_a(const Shape& s) { return at_xt(s, 2); }
__host__ __device__ inline long long at_p(const Shape& s) { return at_a(s) + s.n * mu_groups(s.n) * 128; }
__host__ __device__ inline long long at_parts(const Shape& s) { return at_p(s) + s.n * mu_groups(s.n) * 128; }

int64_t triangle(int64_t n, int64_t tile) { const int64_t k = (n + tile - 1) / tile; return k * (k + 1) / 2; }

Shape oriented(const gc_muon_mat& a) { return {0, std::min(a.n, a.m), std::max(a.n, a.m)}; }

bool mat_ok(const gc_muon_mat& a) {
    return a.n >= 1 && a.m >= 1 && a.n <= MU_MAX_SIDE && a.m <= MU_MAX_SIDE && static_cast<int64_t>(a.n) * a.m <= INT32_MAX;
}

// The tile that a workgroup takes.
enum Way { TILE_64, TILE_128, TILE_128_PAIRED, TILE_192, TILE_256, WAYS };
constexpr int SIDE[WAYS] = {64, 128, 128, 192, 256};

int64_t parts_of(const Shape& s, int per) { return (mu_groups(s.m) + per - 1) / per; }

int64_t blocks_of(int kind, Way way, const Shape& s, int per) {
    return symmetric(kind) ? triangle(s.n, SIDE[way]) * (kind == GRAM ? parts_of(s, per) : 1) : tiles_of(s.n, s.m, SIDE[way], SIDE[way]);
}

// A launch's time in us, by fits to measurements over matrices of 64 x 576 to 4096 x 4096,
// alone and in sets: START, a tile's start and end, and what a group takes a workgroup alone
// and with every compute unit busy (the copies out of the L2 bound the smallest tile, the
// matrix units at the clock that the power allows the largest).  Both sides of some
// choices, X X^T and P X: 64 x 576 6.4 and 5.2 (64), 12.1 and 6.3 (128); 1024 x 1024 13.1 and
// 13.4 (64), 20.8 and 22.2 (128), 26.8 and 27.0 (paired); 2048 x 2048 46 and 65 (64), 48 and 56
// (128), 58 and 65 (paired), 81 and 85 (192); 4096 x 4096 329 and 515 (64), 238 and 349
// (paired), 194 and 366 (192), 246 and 321 (256).  256 x 256 is not offered to A and P, whose
// triangles it fills worst.
double time_of(int kind, Way way, const Shape* shapes, const int* per, int count) {
    constexpr double START = 3.0, FIXED[WAYS] = {3.0, 4.5, 5.5, 12.5, 19.0}, ALONE[WAYS] = {0.2, 0.43, 0.57, 0.85, 1.4},
                     BUSY[WAYS] = {0.28, 0.66, 0.62, 1.35, 2.35};
    constexpr bool PAIRED[WAYS] = {true, false, true, false, false};
    double blocks = 0, work = 0, longest = 0, bytes = 0;
    for (int w = 0; w < count; ++w) {
        const double b = blocks_of(kind, way, shapes[w], per[w]), n = shapes[w].n;
        const double g = kind == GRAM ? std::min<int64_t>(per[w], mu_groups(shapes[w].m)) : mu_groups(shapes[w].n);
        blocks += b;
        work += b * g;
        longest = std::max(longest, g);
        if (kind == GRAM && parts_of(shapes[w], per[w]) > 1) bytes += parts_of(shapes[w], per[w]) * n * n * 4;
    }
    const double x = blocks / 256, rounds = way == TILE_64 ? std::max(1.0, x) : std::ceil(x);
    const double alone = longest * (ALONE[way] + (BUSY[way] - ALONE[way]) * std::min(1.0, x));
    const double busy = work / blocks * BUSY[way] * rounds;
    const double fixed = FIXED[way] * std::ceil(x / (PAIRED[way] ? 2 : 1));
    return START + fixed + std::max(alone, x > 1 ? busy : 0.0) + (bytes > 0 ? 4.5 + bytes / 4e6 : 0.0);   // with the join
}

// How the matrices of one launch are cut: the tile of each product, and for A = X X^T the
// groups of a part, so that few tiles of a long k do not leave the chip idle, nor long ones
// run on behind the others.
struct Cut {
    Way way[3];                                              // A, P, P X
    int per[MU_MAX];
    // what a pair's lo is held times: 1 where a tile has one set of sums for all products of a pair
    float low() const { return std::max({way[GRAM], way[POLY], way[APPLY]}) < TILE_192 ? 2048.0f : 1.0f; }
};
Cut cut_of(const gc_muon_mat* mats, int count) {
    Shape shapes[MU_MAX];
    Cut cut;
    int per[MU_MAX];
    int64_t longest = 0;
    for (int w = 0; w < count; ++w) {
        shapes[w] = oriented(mats[w]);
        longest = std::max(longest, mu_groups(shapes[w].m));
    }
    for (int kind : {GRAM, POLY, APPLY}) {
        double least = INFINITY;
        for (int64_t most = longest;; most = (most + 1) / 2) {   // groups of a part
            for (int w = 0; w < count; ++w) {
                const int64_t g = mu_groups(shapes[w].m), parts = std::min<int64_t>(MU_MAX_PARTS, (g + most - 1) / most);
                per[w] = static_cast<int>((g + parts - 1) / parts);
            }
            for (int way = 0; way < (symmetric(kind) ? TILE_256 : WAYS); ++way) {
                const double us = time_of(kind, static_cast<Way>(way), shapes, per, count);
                if (us >= least) continue;
                least = us;
                cut.way[kind] = static_cast<Way>(way);
                if (kind == GRAM) std::copy(per, per + count, cut.per);
            }
            if (kind != GRAM || most <= 8) break;
        }
    }
    return cut;
}

}  // namespace
}  // namespace gc
