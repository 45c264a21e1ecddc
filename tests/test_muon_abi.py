"""gc_muon_step without a GPU: sizes, refusals of the C call and of the binding.

The C calls get made-up aligned addresses and fail validation before any HIP
call; they are skipped where a GPU is visible."""
import ctypes as C

import numpy as np
import pytest

from test_abi import gcl, no_gpu  # noqa: F401

G, M, O, W = 0x10000000, 0x20000000, 0x30000000, 0x40000000


def array(gcl, *mats):  # noqa: F811
    return (gcl.gc_muon_mat * len(mats))(*(gcl.gc_muon_mat(*m) for m in mats))


def test_struct_size(gcl):  # noqa: F811
    assert C.sizeof(gcl.gc_muon_mat) == 40


def test_sizes(gcl):  # noqa: F811
    size = lambda *mats: gcl.lib.gc_muon_workspace_bytes(array(gcl, *mats), len(mats))    # noqa: E731
    one = size((G, M, O, 64, 576, 1.0))
    assert one >= 12 * 64 * 576 + 8 * 64 * 64
    assert size((G, M, O, 576, 64, 1.0)) == one
    assert one < size((G, M, O, 64, 576, 1.0), (G, M, O, 64, 576, 1.0)) <= 2 * one
    for n, m in [(0, 5), (5, 0), (-1, 5), (2**22 + 1, 1), (1, 2**22 + 1), (2**16, 2**15)]:
        assert size((G, M, O, n, m, 1.0)) == 0
        assert size((G, M, O, 4, 4, 1.0), (G, M, O, n, m, 1.0)) == 0
    assert size((G, M, O, 2**22, 511, 1.0)) > 0
    assert gcl.lib.gc_muon_workspace_bytes(None, 1) == 0
    assert gcl.lib.gc_muon_workspace_bytes(array(gcl, (G, M, O, 4, 4, 1.0)), 0) == 0
    assert "muon_tile" in gcl.gc_kernel_names()


@no_gpu
def test_refusals(gcl):  # noqa: F811
    def call(mats=((G, M, O, 100, 50, 1.0),), count=None, dt=0, odt=1, steps=5, coefs=None, ws=W, wsb=1 << 30):
        c = None if coefs is None else np.asarray(coefs, np.float32).ctypes.data_as(C.POINTER(C.c_float))
        return gcl.lib.gc_muon_step(array(gcl, *mats), len(mats) if count is None else count, dt, odt, 0.9, 1, steps, c, ws, wsb, None)

    ok = (G, M, O, 100, 50, 1.0)                              # grad and mem 20000 bytes, out 10000
    second = (G + 2**20, M + 2**20, O + 2**20, 100, 50, 1.0)
    assert gcl.lib.gc_muon_step(None, 1, 0, 1, 0.9, 1, 5, None, W, 1 << 30, None) == gcl.GC_ERR_ARG
    for kw in [dict(count=0), dict(count=-1), dict(steps=0), dict(steps=33), dict(steps=-1), dict(ws=None), dict(ws=W + 8)]:
        assert call(**kw) == gcl.GC_ERR_ARG, kw
    assert call(dt=2) == gcl.GC_ERR_DTYPE and call(odt=5) == gcl.GC_ERR_DTYPE
    for bad in [(None, M, O, 100, 50, 1.0), (G, M, None, 100, 50, 1.0), (G + 4, M, O, 100, 50, 1.0), (G, M + 8, O, 100, 50, 1.0),
                (G, M, O + 2, 100, 50, 1.0), (G, M, O, 0, 50, 1.0), (G, M, O, 100, -5, 1.0), (G, M, O, 2**22 + 1, 1, 1.0),
                (G, M, O, 2**16, 2**15, 1.0)]:
        assert call(mats=(bad,)) == gcl.GC_ERR_ARG, bad
        assert call(mats=(second, bad)) == gcl.GC_ERR_ARG, bad
    for bad in [(G, G, O, 100, 50, 1.0), (G, G + 19984, O, 100, 50, 1.0), (G, M, G + 19984, 100, 50, 1.0), (G, M, M + 16, 100, 50, 1.0),
                (G, M, O + 2**20 + 9984, 100, 50, 1.0), (G, M + 2**20 - 19984, O, 100, 50, 1.0), (G, M, G + 2**20, 100, 50, 1.0),
                (G, M, M + 2**20 - 16, 100, 50, 1.0), (G, M, W + 64, 100, 50, 1.0), (G, W, O, 100, 50, 1.0), (W, M, O, 100, 50, 1.0)]:
        assert call(mats=(second, bad)) == gcl.GC_ERR_ARG, bad
        assert "overlap" in gcl.gc_last_error()
    need = gcl.lib.gc_muon_workspace_bytes(array(gcl, ok), 1)
    assert call(wsb=need - 1) == gcl.GC_ERR_WORKSPACE
    # coefficients that leave the range: singular values past 4, the factor past 16, at a later step, not finite
    # (the first of them: 1.99 after the first step, where the usual ones make it 33)
    usual, first = [3.4445, -4.7750, 2.0315], [8.2872, -23.5959, 17.3004]
    for bad in (first + usual * 4, [4.5, 0, 0] * 5, [17, -16.5, 0] * 5, usual * 4 + [0, 0, 5.0], usual * 2 + [float("nan"), 0, 0] + usual * 2,
                [float("inf"), 0, 0] * 5, [2.0, 0, 0] * 5, [0, 16.1, 0] * 5, [-4.2, 0, 0] * 5):
        assert call(coefs=bad) == gcl.GC_ERR_ARG, bad
        assert "coefficients" in gcl.gc_last_error()
    # what is in the range gets past that check, to the workspace's
    for good in (usual * 5, [1.5, -0.5, 0] * 5, [2, -1.5, 0.5] * 5, first + [4.1071, -2.9478, 0.5448] * 4, [1, 0, 0] * 5, [0, 1, 0] * 5):
        assert call(coefs=good, wsb=16) == gcl.GC_ERR_WORKSPACE, good


def test_binding_refusals(gcl):  # noqa: F811
    import torch
    f = lambda *s: torch.zeros(*s)                                  # noqa: E731
    mat = lambda g=None, o=None, m=None: gcl.MuonMat(f(4, 5) if g is None else g, f(4, 5) if o is None else o, m)    # noqa: E731
    with pytest.raises(ValueError, match="at least one"):
        gcl.MuonArray([])
    with pytest.raises(ValueError, match="2-D"):
        gcl.MuonArray([mat(g=f(5))])
    with pytest.raises(ValueError, match="2-D"):
        gcl.MuonArray([mat(g=f(0, 5), o=f(0, 5))])
    with pytest.raises(ValueError, match="out must have grad's shape"):
        gcl.MuonArray([mat(o=f(5, 4))])
    with pytest.raises(ValueError, match="mem must have grad's shape"):
        gcl.MuonArray([mat(m=f(20))])
    with pytest.raises(ValueError, match="contiguous"):
        gcl.MuonArray([mat(g=f(5, 4).t())])
    with pytest.raises(TypeError, match="mem"):
        gcl.MuonArray([mat(m=f(4, 5).double())])
    with pytest.raises(TypeError, match="not supported"):
        gcl.MuonArray([mat(g=f(4, 5).half())])
    with pytest.raises(ValueError, match="gradient must have"):
        gcl.MuonArray([mat(), mat(g=f(4, 5).bfloat16())])
    with pytest.raises(ValueError, match="out must have the first"):
        gcl.MuonArray([mat(), mat(o=f(4, 5).bfloat16())])
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="coefs"):
        gcl.gc_muon_step([mat()], 0.9, ws, coefs=(1.0, 2.0))
    with pytest.raises(ValueError, match="coefs"):
        gcl.gc_muon_step([mat()], 0.9, ws, steps=4, coefs=[(1.0, 0.0, 0.0)] * 5)
    with pytest.raises(ValueError, match="steps"):
        gcl.gc_muon_step([mat()], 0.9, ws, steps=40, coefs=(1.0, 0.0, 0.0))
    with pytest.raises(ValueError, match="device tensor"):
        gcl.gc_muon_step([mat()], 0.9, ws)
    assert gcl.gc_muon_workspace_bytes([mat()]) > 0
