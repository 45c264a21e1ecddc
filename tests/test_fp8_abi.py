"""8-bit entry points without a GPU: sizes, refusals of the C calls and of the binding.

The C calls get made-up aligned addresses and fail validation before any HIP
call; they are skipped where a GPU is visible."""
import pytest

from test_abi import gcl, no_gpu  # noqa: F401


def test_sizes(gcl):  # noqa: F811
    for rows, cols, g, p in [(1, 1, 1, 4), (1, 128, 1, 4), (1, 129, 2, 4), (7, 1155, 10, 12), (30522, 1024, 8, 8), (129, 513, 5, 8)]:
        assert gcl.gc_fp8_code_bytes(rows, cols) == rows * 128 * g
        assert gcl.gc_fp8_scale_bytes(rows, cols) == rows * p
        assert gcl.gc_fp8_scale_bytes(rows, cols, 128) == -(-rows // 128) * p
    for rows, cols in [(0, 1), (1, 0), (-1, 5), (1, 2**34 + 1), (2**34, 1), (2**27 + 1, 1)]:
        assert gcl.gc_fp8_code_bytes(rows, cols) == 0 and gcl.gc_fp8_scale_bytes(rows, cols) == 0
    for block in (0, 2, 64, 127, 129, -1):
        assert gcl.gc_fp8_scale_bytes(5, 5, block) == 0
    assert gcl.gc_fp8_code_bytes(1, 2**34) == 2**34 and gcl.gc_fp8_code_bytes(2**27, 128) == 2**34
    assert gcl.gc_fp8_matmul_workspace_bytes(0, 5, 5) == 0
    assert gcl.gc_fp8_matmul_workspace_bytes(2**31, 5, 5) == 0
    assert "fp8_tiles" in gcl.gc_kernel_names()


C, S, X = 0x3000000, 0x4000000, 0x5000000


@no_gpu
def test_quantize_refusals(gcl):  # noqa: F811
    T, U = 0x6000000, 0x7000000

    def call(x=X, dt=0, rows=10, cols=200, ld=200, block=1, c=C, s=S, t=T, u=U):
        return gcl.lib.gc_fp8_quantize(x, dt, rows, cols, ld, block, c, s, t, u, None)

    # 10 x 200: x 8000 bytes, codes 2560, scales 40; transposed 25600 and 800
    for kw in [dict(x=None), dict(x=X + 4), dict(c=None), dict(s=None), dict(t=None), dict(u=None),
               dict(c=None, s=None, t=None, u=None), dict(rows=0), dict(cols=0), dict(ld=199), dict(ld=2**35),
               dict(rows=2**27, cols=32, ld=2**34), dict(c=C + 8), dict(u=U + 8), dict(rows=2**20, cols=2**20, ld=2**20),
               dict(rows=1, cols=2**30, ld=2**30),                    # the transposed form of one long row is too large
               dict(block=0), dict(block=2), dict(block=127), dict(block=-128),
               dict(c=X + 16), dict(s=X + 7984), dict(t=C + 2544), dict(u=S + 32), dict(t=X + 7984), dict(u=T + 25584)]:
        assert call(**kw) == gcl.GC_ERR_ARG, kw
    assert call(dt=7) == gcl.GC_ERR_DTYPE


@no_gpu
def test_dequantize_refusals(gcl):  # noqa: F811
    def call(c=C, s=S, block=1, rows=10, cols=200, out=X, ldo=200, dt=0):
        return gcl.lib.gc_fp8_dequantize(c, s, block, rows, cols, out, ldo, dt, None)

    for kw in [dict(c=None), dict(s=None), dict(out=None), dict(c=C + 8), dict(s=S + 8), dict(out=X + 8), dict(block=3),
               dict(rows=0), dict(cols=0), dict(rows=2**30, cols=2**20, ldo=2**20), dict(ldo=199), dict(ldo=2**35),
               dict(rows=2**27, cols=32, ldo=2**34), dict(out=C + 2544), dict(out=S + 32), dict(out=S - 7984)]:
        assert call(**kw) == gcl.GC_ERR_ARG, kw
    assert call(dt=2) == gcl.GC_ERR_DTYPE


@no_gpu
def test_matmul_refusals(gcl):  # noqa: F811
    AC, AS, BC, BS, W = 0x1000000, 0x2000000, 0x3000000, 0x4000000, 0x6000000

    def call(ac=AC, as_=AS, ab=1, bc=BC, bs=BS, bb=128, m=100, n=50, k=300, out=X, ldo=50, dt=0, ws=W, wsb=1 << 30):
        return gcl.lib.gc_fp8_matmul(ac, as_, ab, bc, bs, bb, m, n, k, out, ldo, dt, 0, ws, wsb, None)

    for kw in [dict(ac=None), dict(as_=None), dict(bc=None), dict(bs=None), dict(out=None), dict(ac=AC + 8),
               dict(bs=BS + 4), dict(out=X + 8), dict(m=0), dict(n=0), dict(k=0), dict(m=2**31), dict(n=2**31),
               dict(k=2**31), dict(k=2**24 + 1), dict(m=2**26, k=2**20), dict(m=2**20, n=2**20), dict(ldo=49), dict(ldo=2**35),
               dict(m=2**27, n=32, k=32, ldo=2**34), dict(ab=0), dict(bb=64), dict(ab=256), dict(bb=-1),
               dict(out=AC + 64), dict(out=AS), dict(out=BC + 64), dict(out=BS - 16)]:
        assert call(**kw) == gcl.GC_ERR_ARG, kw
    assert call(dt=4) == gcl.GC_ERR_DTYPE
    # a product in parts: its workspace missing, misaligned, short or over a buffer
    big = dict(m=256, n=512, k=32768, ldo=512)
    need = gcl.gc_fp8_matmul_workspace_bytes(256, 512, 32768)
    assert need > 0
    assert call(**big, ws=None) == gcl.GC_ERR_ARG and call(**big, ws=W + 8) == gcl.GC_ERR_ARG
    assert call(**big, wsb=16) == gcl.GC_ERR_WORKSPACE
    assert call(**big, ws=X + 16) == gcl.GC_ERR_ARG and call(**big, ws=AS) == gcl.GC_ERR_ARG


def test_binding_refusals(gcl):  # noqa: F811
    import torch
    f = lambda *s: torch.zeros(*s)                                  # noqa: E731
    b = lambda *s: torch.zeros(*s, dtype=torch.uint8)               # noqa: E731
    with pytest.raises(ValueError, match="no output"):
        gcl.gc_fp8_quantize(f(4, 5))
    with pytest.raises(ValueError, match="codes and scales"):
        gcl.gc_fp8_quantize(f(4, 5), b(512))
    with pytest.raises(ValueError, match="contiguous rows"):
        gcl.gc_fp8_quantize(f(5, 4).t(), b(512), b(16))
    with pytest.raises(ValueError, match="overlap"):
        gcl.gc_fp8_quantize(f(1, 5).expand(4, 5), b(512), b(16))
    with pytest.raises(ValueError, match="row codes"):
        gcl.gc_fp8_quantize(f(4, 5), b(511), b(16))
    with pytest.raises(ValueError, match="row scales"):
        gcl.gc_fp8_quantize(f(4, 5), b(512), b(15))
    with pytest.raises(ValueError, match="column codes"):
        gcl.gc_fp8_quantize(f(4, 5), None, None, b(512), b(20))
    with pytest.raises(ValueError, match="column scales"):
        gcl.gc_fp8_quantize(f(4, 5), None, None, b(640), b(3), block_rows=128)
    with pytest.raises(ValueError, match="block rows"):
        gcl.gc_fp8_quantize(f(4, 5), b(512), b(16), block_rows=64)
    with pytest.raises(TypeError, match="row codes"):
        gcl.gc_fp8_quantize(f(4, 5), f(512), b(16))
    with pytest.raises(ValueError, match="matrix with entries"):
        gcl.gc_fp8_quantize(f(0, 5), b(512), b(16))
    with pytest.raises(ValueError, match="matrix scales"):
        gcl.gc_fp8_dequantize(b(512), b(12), f(4, 5))
    with pytest.raises(ValueError, match="contiguous"):
        gcl.gc_fp8_dequantize(b(2, 512)[:, ::2], b(16), f(4, 5))
    with pytest.raises(TypeError, match="not supported"):
        gcl.gc_fp8_dequantize(b(512), b(16), f(4, 5).double())
    with pytest.raises(ValueError, match="B scales"):
        gcl.gc_fp8_matmul(b(512), b(16), b(640), b(16), 100, f(4, 5))
    with pytest.raises(ValueError, match="A codes"):
        gcl.gc_fp8_matmul(b(511), b(16), b(640), b(20), 100, f(4, 5))
    with pytest.raises(ValueError, match="block rows"):
        gcl.gc_fp8_matmul(b(512), b(16), b(640), b(20), 100, f(4, 5), a_block_rows=0)
    with pytest.raises(ValueError, match="device tensor"):
        gcl.gc_fp8_matmul(b(512), b(16), b(640), b(4), 100, f(4, 5), b_block_rows=128)
    with pytest.raises(ValueError, match="k must be"):
        gcl.gc_fp8_matmul(b(512), b(16), b(640), b(20), 0, f(4, 5))
