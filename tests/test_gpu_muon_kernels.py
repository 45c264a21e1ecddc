"""GPU: one step of gc_muon_step with every tile of each product, X X^T whole and in parts: every matrix of each set within
test_gpu_muon's bounds.  test_plans.py asks the rules that the sets reach them."""
import pytest
import torch

from gpu_util import DEV, lib, require_gpu
from test_gpu_muon import USUAL, one_step_on_device, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


# a transformer layer's six matrices of width 1024 among them
SETS = [[(1024, 1024)] * 4 + [(4096, 1024), (1024, 4096)], [(452, 453)] * 32, [(463, 466)] * 16, [(3823, 835)], [(2278, 1289)] * 4,
        [(978, 904)] * 16, [(2851, 2826)], [(325, 5690)], [(267, 5618)] * 4, [(1860, 2413)], [(4357, 520)] * 4, [(3116, 929)] * 4,
        [(964, 12)], [(8, 8), (40, 33)], [(46, 21), (3365, 193)] * 3]


@pytest.mark.parametrize("shapes", SETS, ids=lambda s: f"{len(s)}:" + "+".join(f"{n}x{m}" for n, m in dict.fromkeys(s)))
def test_every_matrix_of_a_set(shapes):
    gc = lib()
    print(f"case: muon set {shapes}", flush=True)
    g = torch.Generator(device=DEV)
    g.manual_seed(7 * len(shapes) + shapes[0][0])
    us = [torch.randn(s, generator=g, device=DEV) * torch.exp2(torch.randint(-3, 1, (s[0], 1), generator=g, device=DEV)) for s in shapes]
    for coefs in (USUAL, (0.0, 1.0, 0.0)):
        got = {}
        for dt in (torch.float32, torch.bfloat16):
            outs = [torch.full((s[0] * s[1] + 8,), 7.0, dtype=dt, device=DEV) for s in shapes]
            mats = gc.MuonArray([gc.MuonMat(u, o[:-8].view(u.shape)) for u, o in zip(us, outs)])
            ws = workspace(mats)
            gc.gc_muon_step(mats, 0.9, ws[: ws.numel() - 64], steps=1, coefs=coefs)
            assert bool((ws[ws.numel() - 64:] == 255).all()) and all(bool((o[-8:] == 7.0).all()) for o in outs), "written past a buffer"
            got[dt] = [o[:-8].view(u.shape) for u, o in zip(us, outs)]
        for i, u in enumerate(us):
            want, bound = one_step_on_device(u, coefs, False)
            assert bool(((got[torch.float32][i].double() - want).abs() <= bound).all()), (i, coefs)
            assert torch.equal(got[torch.bfloat16][i], got[torch.float32][i].to(torch.bfloat16))
