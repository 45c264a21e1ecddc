"""The rules that choose kernels (no GPU): the shapes that the GPU tests take reach every kernel that can be chosen, so that
a new fit of the rules' times does not leave one untested without a word."""
import os
import re

from gradient_compression_error_amd import build
from plan_util import FP8, fp8_plans
from test_gpu_fp8_kernels import LARGE, SHAPES

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
