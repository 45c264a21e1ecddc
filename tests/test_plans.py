"""The rules that choose kernels (no GPU): the shapes that the GPU tests take reach every kernel that can be chosen, so that
a new fit of the rules' times does not leave one untested without a word."""
import os
import re

from gradient_compression_error_amd import build
from plan_util import FP8, MUON, fp8_plans, muon_cuts, muon_lows
from test_gpu_fp8_kernels import LARGE, SHAPES
from test_gpu_muon_kernels import SETS

WAVES = {"WAVE_1_1", "WAVE_1_2", "WAVE_2_1", "WAVE_2_2", "WAVE_2_4", "WAVE_4_4"}


def fp8_reached(shapes, exact):
    """{(kernel, in parts?, remainder of the last part's groups by four)}."""
    out = set()
    for (m, n, k), (kind, splits, per) in zip(shapes, fp8_plans([(*s, exact) for s in shapes])):
        out.add((kind, splits > 1, (-(-k // 128) - (splits - 1) * per) % 4))
    return out


def test_fp8_names():
    """The kinds here are the header's, in its order."""
    with open(os.path.join(build.CSRC, "fp8_plan.h")) as f:
        kinds = re.search(r"enum Kind \{([^}]*)\}", f.read()).group(1).replace(" ", "").split(",")
    assert re.findall(r'"(\w+)"', FP8.split("names[]")[1].split(";")[0]) == kinds


def test_fp8_kernels_are_reached():
    rests = range(4)
    whole = {(kind, False, r) for kind in WAVES for r in rests}
    bf16 = whole | {(kind, False, r) for kind in ("TILE_128", "TILE_128_SHORT", "TILE_128_PAIRED", "TILE_256") for r in rests} | \
        {(kind, True, r) for kind in ("TILE_128", "TILE_128_SHORT") for r in rests}
    f32 = whole | {("TILE_128_PAIRED", parts, r) for parts in (False, True) for r in rests}
    assert bf16 - fp8_reached(SHAPES, False) == set()
    assert f32 - fp8_reached(SHAPES, True) == set()
    # tiles of 256: exactly one chunk of four groups, and several
    groups = [-(-k // 128) for (m, n, k), p in zip(LARGE, fp8_plans([(*s, False) for s in LARGE])) if p[0] == "TILE_256"]
    assert 4 in groups and any(g % 4 == 0 and g > 4 for g in groups)


def test_fp8_reach_of_random_shapes():
    """No other kernel, and none of these in another form, is chosen over a wide range of sizes."""
    import random
    r = random.Random(3)
    shapes = [tuple(int(2 ** r.uniform(0, top)) for top in (13, 13, 15)) for _ in range(20000)]
    for exact in (False, True):
        chosen = {(k, s > 1) for k, s, _ in fp8_plans([(*s, exact) for s in shapes])}
        assert chosen <= {(k, p) for k, p, _ in fp8_reached(SHAPES, exact)}


def muon_reached(sets):
    """({(tile of X X^T, in parts?)}, {tile of P}, {tile of P X})."""
    cuts = muon_cuts(sets)
    return {(w[0], p > 1) for w, parts in cuts for p in parts}, {w[1] for w, _ in cuts}, {w[2] for w, _ in cuts}


def test_muon_names():
    with open(os.path.join(build.CSRC, "muon_plan.h")) as f:
        ways = re.search(r"enum Way \{([^}]*), WAYS \}", f.read()).group(1).replace(" ", "").split(",")
    assert re.findall(r'"(TILE\w+)"', MUON) == ways


def test_muon_kernels_are_reached():
    small = {"TILE_64", "TILE_128", "TILE_128_PAIRED", "TILE_192"}
    gram, poly, apply = muon_reached(SETS)
    assert gram == {(w, parts) for w in small for parts in (False, True)}
    assert poly == small and apply == small | {"TILE_256"}
    # pairs of either kind; what test_gpu_muon_accuracy says of its shapes
    assert set(muon_lows(SETS)) == {1, 2048}
    assert muon_lows([[s] for s in [(64, 576), (576, 64), (33, 31), (130, 257), (300, 1111), (1500, 1400), (3010, 2990)]]) == [2048] * 6 + [1]
    # a layer's set: the long matrices' X X^T in parts on the paired tile, the square ones' whole
    assert muon_cuts(SETS[:1])[0][0][0] == "TILE_128_PAIRED" and muon_cuts(SETS[:1])[0][1] == [1, 1, 1, 1, 4, 4]


def test_a_set_cut_as_each_alone():
    """test_gpu_muon.test_a_set_is_each_alone asks for the bits of each matrix alone, which the entry point does not promise:
    here why it gets them.  X X^T of its matrices comes in as many parts, and the two smallest tiles add alike: hi hi, hi lo
    and lo hi along k in sums of their own, added at the end."""
    import gen
    r = gen.rng(0, gen.KIND_MISC, 1100 + 6, 0)
    shapes = [(int(r.integers(1, 200)), int(r.integers(1, 260))) for _ in range(68)] + [(300, 900), (700, 520)]
    cuts, alone = muon_cuts([shapes[f:f + 32] for f in range(0, 70, 32)]), muon_cuts([[s] for s in shapes])
    assert [p for c in cuts for p in c[1]] == [c[1][0] for c in alone]
    assert {way for c in cuts + alone for way in c[0]} <= {"TILE_64", "TILE_128"}
