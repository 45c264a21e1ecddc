"""Which kernels a call gets, asked of the library's own rules: their headers, compiled for the host (not a test module)."""
import functools
import os
import subprocess
import tempfile

from gradient_compression_error_amd import build

FP8 = r"""
#include <cstdio>
#include "fp8_plan.h"
int main() {
    using namespace gc;
    const char* const names[] = {"WAVE_1_1", "WAVE_1_2", "WAVE_2_1", "WAVE_2_2", "WAVE_2_4", "WAVE_4_4", "TILE_128", "TILE_128_SHORT",
                                 "TILE_128_PAIRED", "TILE_256"};
    long long m, n, k;
    int exact;
    while (scanf("%lld %lld %lld %d", &m, &n, &k, &exact) == 4) {
        const Plan p = plan_of(m, n, k, exact != 0);
        printf("%s %d %d\n", names[p.kind], p.splits, p.per_split);
    }
}
"""

MUON = r"""
#include <cstdio>
#include <vector>
#include "muon_plan.h"
int main() {
    using namespace gc;
    const char* const names[] = {"TILE_64", "TILE_128", "TILE_128_PAIRED", "TILE_192", "TILE_256"};
    int count;
    while (scanf("%d", &count) == 1) {
        std::vector<gc_muon_mat> mats(count);
        for (auto& a : mats)
            if (scanf("%d %d", &a.n, &a.m) != 2) return 1;
        const Cut cut = cut_of(mats.data(), count);
        printf("%d %s %s %s", static_cast<int>(cut.low()), names[cut.way[GRAM]], names[cut.way[POLY]], names[cut.way[APPLY]]);
        for (int w = 0; w < count; ++w) printf(" %d", static_cast<int>(parts_of(oriented(mats[w]), cut.per[w])));
        printf("\n");
    }
}
"""


@functools.lru_cache(None)
def _program(source):
    folder = tempfile.TemporaryDirectory()
    src, exe = os.path.join(folder.name, "plan.hip"), os.path.join(folder.name, "plan")
    with open(src, "w") as f:
        f.write(source)
    build._run([build.HIPCC, *build.CFLAGS, "--offload-host-only", f"-I{build.CSRC}", src, "-o", exe])
    return folder, exe                                       # (the folder goes with the last reference)


def _asked(source, lines):
    got = subprocess.run([_program(source)[1]], input="\n".join(lines) + "\n", text=True, stdout=subprocess.PIPE, check=True)
    return [line.split() for line in got.stdout.splitlines()]


def fp8_plans(shapes):
    """[(m, n, k, float32 out)] -> [(kernel, parts of k, groups of a part)]."""
    return [(a, int(b), int(c)) for a, b, c in _asked(FP8, [f"{m} {n} {k} {int(e)}" for m, n, k, e in shapes])]


def muon_cuts(sets):
    """[[(n, m), ...] of at most 32] -> [((tile of X X^T, of P, of P X), [parts of k of each matrix])]."""
    return [(tuple(g[1:4]), [int(v) for v in g[4:]]) for g in _muon(sets)]


def muon_lows(sets):
    """What a pair's lo is held times, for each set."""
    return [int(g[0]) for g in _muon(sets)]


def _muon(sets):
    return _asked(MUON, [f"{len(s)} " + " ".join(f"{n} {m}" for n, m in s) for s in sets])
