"""GPU: the 8-bit product's tests of numerics on every kernel that the present rules choose, each with every remainder of its
(last part's) groups by four.  test_plans.py asks the rules that the shapes reach them."""
import pytest
import torch

import test_gpu_fp8 as base
from gpu_util import DEV, lib, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


# waves that share k, for either type of out
WAVES = [(37, 300, 899), (1, 1000, 515), (90, 17, 641), (64, 500, 782),
         (247, 356, 993), (263, 337, 541), (267, 343, 650), (287, 322, 777),
         (773, 163, 397), (826, 162, 518), (812, 163, 653), (858, 162, 263), (779, 175, 946),
         (512, 346, 969), (451, 365, 586), (445, 401, 688), (384, 473, 801),
         (655, 631, 391), (579, 708, 555), (777, 538, 653), (700, 584, 259), (428, 897, 905),
         (731, 1049, 415), (862, 903, 532), (987, 775, 655), (1198, 644, 264), (1123, 641, 783)]
# tiles of 128 x 128, all of k in one: bf16 of eight waves, of four; two a compute unit (all of float32)
TILES = [(793, 869, 1022), (1075, 979, 517), (1430, 712, 655), (1123, 641, 783),
         (763, 722, 1995), (645, 821, 2169), (594, 1061, 1747), (792, 742, 1843),
         (1667, 2362, 940), (2753, 1428, 535), (3264, 1172, 684), (2245, 1821, 806)]
# the same in parts of k
PARTS = [(385, 449, 7121), (418, 331, 7253), (407, 422, 6796), (485, 296, 7012),
         (274, 664, 5513), (468, 708, 4666), (377, 506, 5795), (447, 421, 5905),
         (654, 931, 3973), (779, 955, 3130), (615, 1189, 3328), (1421, 488, 3359), (343, 281, 11191)]
# tiles of 256 x 256 (bf16): one chunk of four groups, one and a rest, several whole ones
LARGE = [(3603, 3091, 431), (2706, 3998, 564), (3636, 3002, 702), (3869, 3036, 289), (4001, 3970, 1024), (3970, 4000, 1500)]
SHAPES = WAVES + TILES + PARTS + LARGE


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_exact(m, n, k):
    base.test_product_exact(m, n, k)


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_bound(m, n, k):
    base.test_product_bound(m, n, k)


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_scale_ends_and_nan(m, n, k):
    base.test_product_scale_ends_and_nan(m, n, k)


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_repeats_bitwise(m, n, k):
    """Three times the same product, alone and added to the same values: the same bits."""
    gc = lib()
    print(f"case: fp8 matmul determinism {m}x{n}x{k}", flush=True)
    r = base.rng(7, m, n, k)
    a, b = (base.held_from(*base.random_held(r, rows, k, 100, 140, 1, True)) for rows in (m, n))
    ws = torch.empty(max(16, gc.gc_fp8_matmul_workspace_bytes(m, n, k)), dtype=torch.uint8, device=DEV)
    for dt in (torch.float32, torch.bfloat16):
        for add in (False, True):
            outs = [torch.full((m, n), 3.0, device=DEV, dtype=dt) for _ in range(3)]
            for out in outs:
                gc.gc_fp8_matmul(*a, *b, k, out, ws, accumulate=add)
            assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
