"""GPU: what gc_muon_step's results are accurate to, beyond the bounds of test_gpu_muon."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, require_gpu
from test_gpu_muon import matrix, step

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


SETS = [[(1, 1), (33, 31)], [(64, 576)], [(100, 64)], [(130, 257), (300, 200), (257, 1000)], [(1024, 1024)], [(2048, 300)],
        [(2100, 2300)], [(4097, 4000)]]


@pytest.mark.parametrize("steps", [1, 5])
@pytest.mark.parametrize("shapes", SETS, ids=lambda s: "+".join(f"{n}x{m}" for n, m in s))
def test_bf16_is_the_float32_result_rounded_once(shapes, steps):
    """Every step is the same for either type of out; the tiles of each product, odd and even groups of k."""
    print(f"case: muon bf16 against float32 {shapes} steps {steps}", flush=True)
    grads = [matrix(n, m, "low", 40) for n, m in shapes]
    exact, _ = step(grads, steps=steps)
    got, _ = step(grads, steps=steps, out_dtype=torch.bfloat16)
    for w, g in zip(exact, got):
        assert torch.equal(g, w.to(torch.bfloat16))
