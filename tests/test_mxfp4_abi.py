"""MXFP4 entry points without a GPU: sizes, refusals of the C calls and of the binding.

The C calls get made-up aligned addresses and fail validation before any HIP
call; they are skipped where a GPU is visible."""
import pytest

from test_abi import gcl, no_gpu  # noqa: F401


def test_sizes(gcl):  # noqa: F811
    for rows, cols, g in [(1, 1, 1), (1, 128, 1), (1, 129, 2), (7, 1155, 10), (30522, 1024, 8)]:
        assert gcl.gc_mxfp4_code_bytes(rows, cols) == rows * 64 * g
        assert gcl.gc_mxfp4_scale_bytes(rows, cols) == rows * 4 * g
    for rows, cols in [(0, 1), (1, 0), (-1, 5), (1, 2**34 + 1), (2**34, 1), (2**27 + 1, 1)]:
        assert gcl.gc_mxfp4_code_bytes(rows, cols) == 0 and gcl.gc_mxfp4_scale_bytes(rows, cols) == 0
    assert gcl.gc_mxfp4_code_bytes(1, 2**34) == 2**33 and gcl.gc_mxfp4_code_bytes(2**27, 128) == 2**33
    assert gcl.gc_mxfp4_matmul_workspace_bytes(0, 5, 5) == 0
    assert gcl.gc_mxfp4_matmul_workspace_bytes(2**31, 5, 5) == 0
    assert "mxfp4_rows" in gcl.gc_kernel_names()


G, M, C, S, X = 0x1000000, 0x2000000, 0x3000000, 0x4000000, 0x5000000


@no_gpu
def test_ef_encode_refusals(gcl):  # noqa: F811
    def call(grad=G, dt=0, mem=M, d=1000, codes=C, scales=S):
        return gcl.lib.gc_mxfp4_ef_encode(grad, dt, mem, d, 1.0, codes, scales, None)

    for kw in [dict(grad=None), dict(mem=None), dict(codes=None), dict(scales=None), dict(d=0), dict(d=-4),
               dict(d=2**34 + 1), dict(grad=G + 4), dict(mem=M + 8), dict(codes=C + 4), dict(scales=S + 4)]:
        assert call(**kw) == gcl.GC_ERR_ARG, kw
    assert call(dt=2) == gcl.GC_ERR_DTYPE
    # 1000 entries: 4000 bytes of mem and grad, 512 of codes, 32 of scales
    for kw in [dict(mem=G), dict(mem=G + 3984), dict(codes=G + 16), dict(scales=G + 3984), dict(codes=M - 496),
               dict(scales=M + 3984), dict(scales=C + 496)]:
        assert call(**kw) == gcl.GC_ERR_ARG, kw
        assert "overlap" in gcl.gc_last_error()


@no_gpu
def test_decode_refusals(gcl):  # noqa: F811
    def call(codes=C, scales=S, nmsg=1, cs=0, ss=0, rows=4, cols=200, out=X, dt=0, acc=0):
        return gcl.lib.gc_mxfp4_decode(codes, scales, nmsg, cs, ss, rows, cols, 1.0, out, dt, acc, None)

    for kw in [dict(codes=None), dict(scales=None), dict(out=None), dict(codes=C + 8), dict(scales=S + 8),
               dict(out=X + 8), dict(rows=0), dict(cols=0), dict(rows=2**30, cols=2**20), dict(nmsg=0), dict(nmsg=-1),
               dict(nmsg=2, cs=496, ss=32), dict(nmsg=2, cs=520, ss=32), dict(nmsg=2, cs=512, ss=28),
               dict(nmsg=2, cs=512, ss=33), dict(nmsg=2, cs=2**41, ss=32), dict(nmsg=2, cs=-512, ss=32),
               dict(out=C + 256), dict(out=S + 16), dict(nmsg=2, cs=1024, ss=32, out=C + 1040)]:
        assert call(**kw) == gcl.GC_ERR_ARG, kw
    assert call(dt=2) == gcl.GC_ERR_DTYPE


@no_gpu
def test_extents_past_64_bits_are_refused(gcl):  # noqa: F811
    """Sizes whose last byte has no 64-bit offset: messages, rows of x and rows of out far apart."""
    lib_ = gcl.lib
    args = (2**40, 2**40, 1, 32, 1.0, X, 0, 0, None)
    for nmsg in (2**31 - 1, 2**20 + 1):
        assert lib_.gc_mxfp4_decode(C, S, nmsg, *args) == gcl.GC_ERR_ARG and "2^20" in gcl.gc_last_error(), nmsg
    for rows in (2**27, 66):
        assert lib_.gc_mxfp4_quantize(X, 0, rows, 32, 2**34, C, S, None, None, None) == gcl.GC_ERR_ARG
        assert "2^40" in gcl.gc_last_error(), rows
        assert lib_.gc_mxfp4_matmul(C, S, C, S, rows, 32, 32, X, 2**34, 0, 0, None, 0, None) == gcl.GC_ERR_ARG
        assert "2^40" in gcl.gc_last_error(), rows


@no_gpu
def test_quantize_refusals(gcl):  # noqa: F811
    T, U = 0x6000000, 0x7000000

    def call(x=X, dt=0, rows=10, cols=200, ld=200, c=C, s=S, t=T, u=U):
        return gcl.lib.gc_mxfp4_quantize(x, dt, rows, cols, ld, c, s, t, u, None)

    for kw in [dict(x=None), dict(x=X + 4), dict(c=None), dict(s=None), dict(t=None), dict(u=None),
               dict(c=None, s=None, t=None, u=None), dict(rows=0), dict(cols=0), dict(ld=199), dict(ld=2**35),
               dict(c=C + 8), dict(u=U + 8), dict(rows=2**20, cols=2**20, ld=2**20),
               dict(rows=1, cols=2**30, ld=2**30),                    # the transposed form of one long row is too large
               dict(c=X + 16), dict(s=X + 7984), dict(t=C + 16), dict(u=S), dict(t=X + 7984), dict(u=T + 128)]:
        assert call(**kw) == gcl.GC_ERR_ARG, kw
    assert call(dt=7) == gcl.GC_ERR_DTYPE


@no_gpu
def test_matmul_refusals(gcl):  # noqa: F811
    AC, AS, BC, BS, W = 0x1000000, 0x2000000, 0x3000000, 0x4000000, 0x6000000

    def call(ac=AC, as_=AS, bc=BC, bs=BS, m=100, n=50, k=300, out=X, ldo=50, dt=0, ws=W, wsb=1 << 30):
        return gcl.lib.gc_mxfp4_matmul(ac, as_, bc, bs, m, n, k, out, ldo, dt, 0, ws, wsb, None)

    for kw in [dict(ac=None), dict(as_=None), dict(bc=None), dict(bs=None), dict(out=None), dict(ac=AC + 8),
               dict(bs=BS + 4), dict(out=X + 8), dict(m=0), dict(n=0), dict(k=0), dict(m=2**31), dict(n=2**31),
               dict(k=2**31), dict(k=2**24 + 1), dict(m=2**26, k=2**20), dict(m=2**20, n=2**20), dict(ldo=49), dict(ldo=2**35),
               dict(out=AC + 64), dict(out=AS), dict(out=BC + 64), dict(out=BS - 16)]:
        assert call(**kw) == gcl.GC_ERR_ARG, kw
    assert call(dt=4) == gcl.GC_ERR_DTYPE


def test_binding_refusals(gcl):  # noqa: F811
    import torch
    f = lambda *s: torch.zeros(*s)                                  # noqa: E731
    b = lambda *s: torch.zeros(*s, dtype=torch.uint8)               # noqa: E731
    with pytest.raises(ValueError, match="same number of entries"):
        gcl.gc_mxfp4_ef_encode(f(5), f(6), 1.0, b(64), b(4))
    with pytest.raises(ValueError, match="same number of entries"):
        gcl.gc_mxfp4_ef_encode(f(0), f(0), 1.0, b(64), b(4))
    with pytest.raises(TypeError, match="mem"):
        gcl.gc_mxfp4_ef_encode(f(5), f(5).double(), 1.0, b(64), b(4))
    with pytest.raises(ValueError, match="codes need"):
        gcl.gc_mxfp4_ef_encode(f(129), f(129), 1.0, b(127), b(8))
    with pytest.raises(ValueError, match="scales need"):
        gcl.gc_mxfp4_ef_encode(f(129), f(129), 1.0, b(128), b(7))
    with pytest.raises(TypeError, match="codes"):
        gcl.gc_mxfp4_ef_encode(f(5), f(5), 1.0, f(64), b(4))
    with pytest.raises(ValueError, match="one row per message"):
        gcl.gc_mxfp4_decode(b(2, 64), b(3, 4), f(5))
    with pytest.raises(ValueError, match="a message"):
        gcl.gc_mxfp4_decode(b(2, 64), b(2, 4), f(2, 5))
    with pytest.raises(ValueError, match="contiguous"):
        gcl.gc_mxfp4_decode(b(64, 2).t(), b(2, 4), f(5))
    with pytest.raises(ValueError, match="no output"):
        gcl.gc_mxfp4_quantize(f(4, 5))
    with pytest.raises(ValueError, match="codes and scales"):
        gcl.gc_mxfp4_quantize(f(4, 5), b(256))
    with pytest.raises(ValueError, match="contiguous rows"):
        gcl.gc_mxfp4_quantize(f(5, 4).t(), b(256), b(16))
    with pytest.raises(ValueError, match="overlap"):
        gcl.gc_mxfp4_quantize(f(1, 5).expand(4, 5), b(256), b(16))
    with pytest.raises(ValueError, match="column codes"):
        gcl.gc_mxfp4_quantize(f(4, 5), None, None, b(256), b(20))
    with pytest.raises(ValueError, match="B codes"):
        gcl.gc_mxfp4_matmul(b(256), b(16), b(256), b(20), 100, f(4, 5))
    with pytest.raises(ValueError, match="matrix with entries"):
        gcl.gc_mxfp4_matmul(b(256), b(16), b(320), b(20), 100, f(0, 5))
    with pytest.raises(ValueError, match="device tensor"):
        gcl.gc_mxfp4_matmul(b(256), b(16), b(320), b(20), 100, f(4, 5))
    with pytest.raises(ValueError, match="k must be"):
        gcl.gc_mxfp4_matmul(b(256), b(16), b(320), b(20), 0, f(4, 5))
