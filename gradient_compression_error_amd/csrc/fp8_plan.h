// The choice of the kernel of an 8-bit product, from its sizes and the type of its result alone (host only).
#pragma once

#include <algorithm>
#include <cmath>

#include "fp8.h"
#include "matmul.h"

namespace gc {
namespace {

struct Plan {
    enum Kind { WAVE_1_1, WAVE_1_2, WAVE_2_1, WAVE_2_2, WAVE_2_4, WAVE_4_4, TILE_128, TILE_128_SHORT, TILE_128_PAIRED, TILE_256 } kind;
    int splits, per_split;                                   // parts of k, groups of each
    int64_t ldp;                                             // entries between the rows of a part
};

bool matmul_shape_ok(int64_t m, int64_t n, int64_t k) {
    return m <= MX_MAX_DIM && n <= MX_MAX_DIM && k <= MX_MAX_K && mx_shape_ok(m, k) && mx_shape_ok(n, k) && mx_shape_ok(m, n);
}

// The cheapest kernel by times (in us) fitted to measurements over m of 1 .. 8192, n of 512 ..
// 8192 and k of 300 .. 16384, in graphs; a round is what 256 compute units take at once.
// Both sides at some borders, bf16 out: 4 x 8192 x 8192 14.6 (1 x 1), 13.2 (1 x 2); 64 x 4096 x
// 1024 5.6 (1 x 2), 4.9 (2 x 2), 5.8 (2 x 4); 777 x 1001 x 1155 10.0 (4 x 4), 8.4 (128); 1024 x
// 1024 x 16384 47.9 (128), 27.3 (in four parts); 1024 x 1024 x 1024 7.1 (128), 6.7 (128, short),
// 2048 x 2048 x 2048 13.0 and 14.7; 2048 x 4096 x 4096 37.1 (128), 34.2 (128, two a
// unit), 47.0 (256); 4096 x 4096 x 4096 68.1 (two a unit), 55.6 (256).  float32 out: 1024 x
// 1024 x 1024 8.8 (4 x 4), 10.2 (128); eight waves of 64 x 32 with four groups in flight took 5%
// more than four of 64 x 64 with two (4096 x 1024 x 8192 62.6 and 58.6).  256 x 256 is not for
// float32, whose operands' wide forms leave it no registers.
Plan plan_of(int64_t m, int64_t n, int64_t k, bool exact) {
    const int groups = static_cast<int>(mx_groups(k));
    const double g = groups;
    Plan best = {Plan::TILE_128_PAIRED, 1, (groups + 3) / 4 * 4, (n + 3) / 4 * 4};
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
    wave(Plan::WAVE_1_1, 1, 1, 0.12, false);
    wave(Plan::WAVE_1_2, 1, 2, 0.17, false);
    wave(Plan::WAVE_2_1, 2, 1, 0.18, false);
    wave(Plan::WAVE_2_2, 2, 2, 0.23, false);
    wave(Plan::WAVE_2_4, 2, 4, 0.36, true);
    wave(Plan::WAVE_4_4, 4, 4, 0.67, true);
    // A part costs its write and read back, and a launch; at most 256 workgroups.
    const int64_t t128 = tiles_of(m, n, 128, 128), t256 = tiles_of(m, n, 256, 256);
    for (int s = 1; s <= MAX_SPLITS && t128 * s <= 256 && (s == 1 || groups >= 8 * s); s *= 2) {
        const double parts = s > 1 ? 3.0 + 0.35e-6 * 4.0 * s * static_cast<double>(m) * best.ldp : 0.0;
        const double mine = std::ceil(g / s), one = exact ? (t128 * s > 128 ? 0.83 : 0.68) : (t128 * s > 128 ? 0.42 : 0.34);
        if (exact) offer(Plan::TILE_128_PAIRED, 5.2 + one * mine + parts, s);
        else offer(mine <= 13 ? Plan::TILE_128_SHORT : Plan::TILE_128, 4.8 + one * mine + parts, s);
    }
    auto rounds = [](double x) { return x <= 1 ? 1.0 : (x + std::ceil(x)) / 2; };
    if (t128 > 256) {
        offer(Plan::TILE_128_PAIRED, rounds(t128 / 512.0) * (exact ? 5.0 + 1.58 * g : 4.5 + 0.95 * g), 1);
        if (!exact) offer(Plan::TILE_256, rounds(t256 / 256.0) * (8.0 + 1.48 * g), 1);
    }
    return best;
}

}  // namespace
}  // namespace gc
