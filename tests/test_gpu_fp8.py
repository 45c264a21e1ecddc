"""GPU: the 8-bit operators against the 64-bit oracle.

The quantiser and the values are compared bit for bit.  Products are compared
exactly where no sum rounds whatever its order, and within derived bounds
elsewhere.  A sum of K terms in float32 differs from the exact one by at most
K * 2^-23 * sum |a b|, one last place an addition.  Results in bf16 are summed by
the 8-bit matrix instructions, which cut each of eight products off 13 places below
the largest one's leading bit: at most 7 of every eight lose, each less than 2^-13
times that product, so another 7 * 2^-13 * sum |a b|; then the rounding, 2^-8 of the
result.
"""
import numpy as np
import pytest
import torch

import gen
import oracle
from gpu_util import DEV, f32_bits, lib, require_gpu, to_dev

pytestmark = pytest.mark.gpu

GUARD = 0xA5


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def rng(which, *of):
    return gen.rng(0, gen.KIND_MISC, 900 + which, sum(v * w for v, w in zip(of, (31, 7, 1))))


class Held:
    """An 8-bit matrix's buffers with guards."""

    def __init__(self, rows, cols, block=1):
        gc = lib()
        self.rows, self.cols, self.block = rows, cols, block
        self.nc, self.ns = gc.gc_fp8_code_bytes(rows, cols), gc.gc_fp8_scale_bytes(rows, cols, block)
        self.c, self.s = (torch.full((n + 64,), GUARD, dtype=torch.uint8, device=DEV) for n in (self.nc, self.ns))

    @property
    def pair(self):
        return self.c[: self.nc], self.s[: self.ns]

    def host(self):
        c, s = self.c.cpu().numpy(), self.s.cpu().numpy()
        assert np.all(c[self.nc:] == GUARD) and np.all(s[self.ns:] == GUARD), "written past the buffers"
        return c[: self.nc].reshape(self.rows, -1), s[: self.ns].reshape(-(-self.rows // self.block), -1)

    def values(self):
        return oracle.fp8_values(*self.host(), self.cols, self.block)


def held_from(codes, scales):
    return tuple(torch.from_numpy(np.ascontiguousarray(a).ravel()).to(DEV) for a in (codes, scales))


def same(held, ref):
    c, s = held.host()
    assert np.array_equal(s, ref[1]), "scales differ"
    assert np.array_equal(c, ref[0]), "codes differ"


def wide_matrix(rows, cols, seed):
    """Values over many binades, with rounding borders, scale borders and zeros among them."""
    r = rng(0, seed)
    x = r.standard_normal((rows, cols), dtype=np.float32)
    x *= np.exp2(r.integers(-8, 8, (rows, 1))).astype(np.float32)
    grid = np.array([448, 449, 447, 224, 1.0625, 1.1875, 17, 19, 2.0 ** -10, 3 * 2.0 ** -10, 0.0, -0.0], np.float32)
    put = r.uniform(size=x.shape) < 0.3
    x[put] = (grid[r.integers(0, grid.size, x.shape)] * np.sign(r.standard_normal(x.shape)).astype(np.float32))[put]
    return x


def both_types(x, dtype):
    return gen.f32_to_bf16_bits(x) if dtype == "bf16" else x


SHAPES = [(1, 1), (1, 7), (1, 128), (1, 129), (1, 513), (1, 2049), (31, 5), (32, 64), (127, 130), (128, 128), (129, 96),
          (5, 4096), (3, 5000), (300, 257), (260, 1155), (640, 512)]


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize_shapes(rows, cols, dtype, block):
    gc = lib()
    print(f"case: fp8 quantize {rows}x{cols} {dtype} block {block}", flush=True)
    x = both_types(wide_matrix(rows, cols, rows * 7919 + cols), dtype)
    xt = to_dev(x.ravel()).view(rows, cols)
    r, c, r2, c2 = (Held(*s, block) for s in ((rows, cols), (cols, rows)) * 2)
    gc.gc_fp8_quantize(xt, *r.pair, block_rows=block)
    gc.gc_fp8_quantize(xt, None, None, *c.pair, block_rows=block)
    gc.gc_fp8_quantize(xt, *r2.pair, *c2.pair, block_rows=block)
    by_rows, by_cols = oracle.fp8_quantize(x, block), oracle.fp8_quantize(np.ascontiguousarray(x.T), block)
    same(r, by_rows)
    same(c, by_cols)
    same(r2, by_rows)
    same(c2, by_cols)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols,pitch", [(8301, 700, 700), (8193, 1001, 1016), (4099, 1024, 1024), (1, 4300001, 4300001)])
def test_quantize_large_rows(rows, cols, pitch, dtype):
    """Where a thread takes two units at a time: the same bits as the matrix in pieces of few rows (or columns), with guards."""
    gc = lib()
    print(f"case: fp8 quantize large {rows}x{cols} pitch {pitch} {dtype}", flush=True)
    g = torch.Generator(device=DEV)
    g.manual_seed(rows + cols)
    x = torch.randn((rows, pitch), generator=g, device=DEV).to(dtype)[:, :cols]
    r = Held(rows, cols)
    gc.gc_fp8_quantize(x, *r.pair)
    codes, scales = r.host()
    codes, scales = codes.reshape(rows, -1), scales.reshape(rows, -1)
    at = range(0, rows, 1500) if rows > 1 else range(0, cols, 512 * 2000)
    for f in at:
        piece = x[f:f + 1500] if rows > 1 else x[:, f:f + 512 * 2000].contiguous()
        p = Held(*piece.shape)
        gc.gc_fp8_quantize(piece, *p.pair)
        c, s = (t.reshape(piece.shape[0], -1) for t in p.host())
        if rows > 1:
            assert np.array_equal(codes[f:f + 1500], c) and np.array_equal(scales[f:f + 1500], s)
        else:
            assert np.array_equal(codes[:, f:f + c.shape[1]], c) and np.array_equal(scales[:, f // 128:f // 128 + s.shape[1]], s)


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols,pitch", [(70, 129, 136), (70, 129, 131), (200, 512, 1024), (33, 64, 65), (1, 50, 99)])
def test_pitch(rows, cols, pitch, dtype, block):
    """Rows apart, in what is quantised and in where the values go; what lies between is not read and not written."""
    gc = lib()
    print(f"case: fp8 quantize {rows}x{cols} pitch {pitch} {dtype} block {block}", flush=True)
    x = wide_matrix(rows, pitch, 5)
    x[:, cols:] = 1e30
    x = both_types(x, dtype)
    xt = to_dev(x.ravel()).view(rows, pitch)[:, :cols]
    r, r1, c = Held(rows, cols, block), Held(rows, cols, block), Held(cols, rows, block)
    gc.gc_fp8_quantize(xt, *r.pair, *c.pair, block_rows=block)
    gc.gc_fp8_quantize(xt, *r1.pair, block_rows=block)
    inner = np.ascontiguousarray(x[:, :cols])
    want = oracle.fp8_quantize(inner, block)
    same(r, want)
    same(r1, want)
    same(c, oracle.fp8_quantize(np.ascontiguousarray(inner.T), block))
    out = torch.full((rows, pitch), 7.0, dtype=xt.dtype, device=DEV)
    gc.gc_fp8_dequantize(*r.pair, out[:, :cols], block_rows=block)
    assert bool((out[:, cols:] == 7.0).all())
    # E4M3 values in these scales are bf16 values
    assert np.array_equal(out[:, :cols].float().cpu().numpy(), oracle.fp8_values(*want, cols, block).astype(np.float32))


def extremes():
    """Rows of 128: rounding borders and their neighbours at several scales, subnormals, the largest values, not finite ones."""
    mags = np.array([(8 + m) * 2.0 ** (e - 10) if e else m * 2.0 ** -9 for e in (0, 1, 2, 7, 14, 15) for m in range(8)][:47])
    mids = ((mags[:-1] + mags[1:]) / 2).astype(np.float32)[::2]
    near = np.concatenate([np.nextafter(mids, np.float32(0)), mids, np.nextafter(mids, np.float32(999))])
    base = np.concatenate([[448.0], near, [0.0, -0.0, 1e-30, -1e-30]]).astype(np.float32)
    with np.errstate(over="ignore"):
        rows = [base * np.float32(2.0) ** np.float32(e) for e in (0, 1, -1, 40, -40, 119, -119, -126)]
    rows += [np.left_shift(np.uint32(1), np.arange(128, dtype=np.uint32) % 23).view(np.float32),        # subnormals
             np.full(128, 2.0 ** -126, np.float32), np.full(128, 3.4028235e38, np.float32), np.full(128, 2.0 ** -127, np.float32),
             np.zeros(128, np.float32), np.full(128, -0.0, np.float32), np.full(128, 448.00003, np.float32)]
    for bad in (np.inf, -np.inf, np.nan):
        r = np.ones(128, np.float32)
        r[17] = bad
        rows.append(r)
    out = np.zeros((len(rows), 128), np.float32)
    for i, r in enumerate(rows):
        out[i, : r.size] = r
    out[1::2] *= np.float32(-1)
    return out


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantize_extremes(dtype, block):
    gc = lib()
    x = extremes()
    if dtype == "bf16":                                      # cut to bf16 bits, so that borders and subnormals stay among them
        nan = np.isnan(x)
        x = (x.view(np.uint32) >> 16).astype(np.uint16)
        x[nan] = 0x7FC0
    # each row a block of its own; all in one row; each row a block along the columns; the finite rows one by one as square blocks
    for a in [x, np.ascontiguousarray(x.reshape(1, -1)), np.ascontiguousarray(x.T)] + [x[i:i + 1] for i in range(x.shape[0]) if block == 128]:
        print(f"case: fp8 quantize extremes {a.shape} {dtype} block {block}", flush=True)
        r, r1, c = Held(*a.shape, block), Held(*a.shape, block), Held(*a.shape[::-1], block)
        at = to_dev(np.ascontiguousarray(a).ravel()).view(*a.shape)
        gc.gc_fp8_quantize(at, *r1.pair, block_rows=block)
        gc.gc_fp8_quantize(at, *r.pair, *c.pair, block_rows=block)
        want = oracle.fp8_quantize(a, block)
        same(r, want)
        same(r1, want)
        same(c, oracle.fp8_quantize(np.ascontiguousarray(a.T), block))


def test_every_code_and_scale():
    """The values of all 256 codes at all 256 scales, in float32 (exact up to an infinity at the top) and in bf16 (rounded once)."""
    gc = lib()
    print("case: fp8 values of every code and scale", flush=True)
    codes = np.tile(np.arange(256, dtype=np.uint8), (256, 1))
    scales = np.zeros((256, 4), np.uint8)
    scales[:, :2] = np.arange(256, dtype=np.uint8)[:, None]
    with np.errstate(over="ignore"):
        want = torch.from_numpy(oracle.fp8_values(codes, scales, 256).astype(np.float32))
    for dt in (torch.float32, torch.bfloat16):
        out = torch.empty(256, 256, dtype=dt, device=DEV)
        gc.gc_fp8_dequantize(*held_from(codes, scales), out)
        assert torch.equal(out.cpu().nan_to_num(nan=7.5), want.to(dt).nan_to_num(nan=7.5))
        assert torch.equal(out.cpu().isnan(), want.isnan())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 1000), (5, 130), (64, 512), (33, 1155), (257, 1024), (130, 7)])
def test_dequantize_shapes(rows, cols, block, dtype):
    gc = lib()
    print(f"case: fp8 values {rows}x{cols} block {block}", flush=True)
    a = random_held(rng(1, rows, cols), rows, cols, 100, 150, block, wide=True)
    out = torch.full((rows * cols + 16,), 7.0, dtype=dtype, device=DEV)
    gc.gc_fp8_dequantize(*held_from(*a), out[: rows * cols].view(rows, cols), block_rows=block)
    assert bool((out[rows * cols:] == 7.0).all())
    assert np.array_equal(out[: rows * cols].view(rows, cols).float().cpu().numpy(), oracle.fp8_values(*a, cols, block).astype(np.float32))


# ---------------------------------------------------------------- products

def random_held(r, rows, cols, low, high, block=1, wide=False):
    """Random codes with scale bytes in [low, high], pads zero, as (codes, scales) on the host.  wide: every finite code;
    else two binades, whose products are multiples of 2^-8 up to 900 of them."""
    g, down = -(-cols // 128), -(-rows // block)
    codes = np.zeros((rows, g * 128), np.uint8)
    c = r.integers(0, 127, (rows, cols)) if wide else r.integers(6 * 8, 8 * 8, (rows, cols))
    codes[:, :cols] = c | (r.integers(0, 2, (rows, cols)) << 7)
    scales = np.zeros((down, -(-g // 4) * 4), np.uint8)
    scales[:, :g] = r.integers(low, high + 1, (down, g))
    return codes, scales


def product(a, b, m, n, k, dtype=torch.float32, old=None, pitch=None, ab=1, bb=1):
    """The product through the entry point, on a pitched out whose gaps must stay."""
    gc = lib()
    pitch = n if pitch is None else pitch
    out = torch.full((m, pitch), 3.0, dtype=dtype, device=DEV)
    view = out[:, :n]
    if old is not None:
        view.copy_(to_dev(old))
    ws = torch.full((gc.gc_fp8_matmul_workspace_bytes(m, n, k) + 64,), GUARD, dtype=torch.uint8, device=DEV)
    gc.gc_fp8_matmul(*held_from(*a), *held_from(*b), k, view, ws[: ws.numel() - 64], a_block_rows=ab, b_block_rows=bb,
                     accumulate=old is not None)
    assert bool((out[:, n:] == 3.0).all()), "written between the rows"
    assert bool((ws[ws.numel() - 64:] == GUARD).all()), "written past the workspace"
    return view.cpu()


# every path's edges: single rows, tiles of 16 to 256, one group of k to many, sizes one off a tile, parts of k
PRODUCTS = [(1, 1, 1), (1, 5, 33), (2, 16, 128), (1, 4096, 1024), (3, 1000, 2000), (16, 16, 129), (17, 33, 257),
            (15, 700, 4100), (16, 4096, 1024), (31, 129, 1155), (32, 512, 4096), (64, 64, 64), (65, 100, 640), (100, 1024, 1024),
            (128, 128, 256), (129, 127, 385), (200, 3000, 300), (255, 257, 512), (256, 256, 128), (257, 255, 1),
            (300, 520, 8192), (1000, 1155, 777), (512, 2048, 1024), (1024, 1024, 2048), (2049, 1025, 1030),
            (1, 20000, 300), (16, 9000, 1000), (30, 9000, 200), (777, 1001, 1155), (1100, 1500, 1500), (300, 520, 16384),
            (601, 1001, 16000), (2100, 2001, 100), (2100, 2001, 130), (2050, 2100, 700), (2100, 2000, 1000), (4000, 3970, 384),
            (4001, 3900, 520), (3900, 4000, 1200), (3841, 4095, 1155), (2300, 2200, 4400),
            (9001, 10, 1000), (1100, 1500, 2000), (1001, 1901, 1900), (500, 1500, 500), (354, 1220, 100), (1050, 1030, 4300)]


def exact_operands(m, n, k, ab, bb):
    """Products that are multiples of 2^-10, at most 3600 of them (of 2^-8, at most 900, where k is long): a sum of k and an
    old value below 64 stay under 2^24 multiples for k < 4640 (18400)."""
    r = rng(2, m, n, k)
    low = 126 if k < 4600 else 127
    return r, random_held(r, m, k, low, 127, ab), random_held(r, n, k, low, 127, bb)


@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_product_exact(m, n, k):
    bb = 128 if (m + n) % 2 else 1
    ab = 128 if (m + k) % 3 == 0 else 1
    print(f"case: fp8 matmul exact {m}x{n}x{k} blocks {ab} {bb}", flush=True)
    r, a, b = exact_operands(m, n, k, ab, bb)
    want = torch.from_numpy(oracle.fp8_matmul(a, b, k, ab, bb).astype(np.float32))
    kw = dict(ab=ab, bb=bb)
    assert torch.equal(product(a, b, m, n, k, **kw), want)
    old = torch.from_numpy(r.integers(-1000, 1000, (m, n)).astype(np.float32) / np.float32(16))
    assert torch.equal(product(a, b, m, n, k, old=old.numpy(), pitch=n + 3, **kw), want + old)
    assert torch.equal(product(a, b, m, n, k, dtype=torch.bfloat16, pitch=n + 8, **kw), want.to(torch.bfloat16))
    old16 = old.to(torch.bfloat16)
    got = product(a, b, m, n, k, dtype=torch.bfloat16, old=old16.float().numpy(), pitch=-(-n // 8) * 8, **kw)
    assert torch.equal(got, (want + old16.float()).to(torch.bfloat16))


def within(got, want, size, k, exact):
    got = got.double().numpy()
    tol = k * 2.0 ** -23 * size
    if not exact:
        tol = (1 + 2.0 ** -8) * (tol + 7 * 2.0 ** -13 * size) + 2.0 ** -8 * np.abs(want)
    return np.all(np.abs(got - want) <= tol)


# a shape for each kernel and the parts of k, each with every remainder of groups by four
KERNELS = [(1, 300, 1000), (16, 1024, 4096), (31, 500, 900), (64, 700, 1900), (100, 130, 8192), (300, 260, 1155), (600, 1024, 16384),
           (1100, 1500, 1500), (2100, 2001, 1300), (3900, 4000, 1155), (3841, 4095, 1700)]


@pytest.mark.parametrize("m,n,k", KERNELS)
def test_product_bound(m, n, k):
    """Every finite code, scales over 24 binades, so that the sums round."""
    print(f"case: fp8 matmul bound {m}x{n}x{k}", flush=True)
    r = rng(3, m, n, k)
    a, b = random_held(r, m, k, 110, 133, 1, True), random_held(r, n, k, 110, 133, 1, True)
    va, vb = (torch.from_numpy(oracle.fp8_values(*h, k)).to(DEV) for h in (a, b))
    want, size = (va @ vb.t().contiguous()).cpu().numpy(), (va.abs() @ vb.abs().t().contiguous()).cpu().numpy()
    assert within(product(a, b, m, n, k), want, size, k, True)
    assert within(product(a, b, m, n, k, dtype=torch.bfloat16), want, size, k, False)


@pytest.mark.parametrize("m,n,k", KERNELS)
def test_product_scale_ends_and_nan(m, n, k):
    """A least scale against a large one, exactly; a NaN scale and a NaN code reach their row and column and nothing else."""
    print(f"case: fp8 matmul scale ends and NaN {m}x{n}x{k}", flush=True)
    r = rng(4, m, n, k)
    a, b = random_held(r, m, k, 127, 127), random_held(r, n, k, 127, 127)
    want = torch.from_numpy(oracle.fp8_matmul(a, b, k).astype(np.float32))
    g = -(-k // 128)
    for sa, sb in ((7, 247), (247, 7)):
        a[1][:, :g], b[1][:, :g] = sa, sb
        assert torch.equal(product(a, b, m, n, k), want)
        assert torch.equal(product(a, b, m, n, k, dtype=torch.bfloat16), want.to(torch.bfloat16))
    a[1][:, :g], b[1][:, :g] = 127, 127
    a[1][m - 1, g - 1] = 255
    a[0][m - 1, (g - 1) * 128:] = 0                          # zero codes do not hide a NaN scale
    b[0][n // 2, k // 2] = 0x7F
    a2, b2 = (a[0], a[1].copy()), (b[0].copy(), b[1])
    bad = np.zeros((m, n), bool)
    bad[m - 1, :], bad[:, n // 2] = True, True
    a2[1][m - 1, g - 1] = 127
    b2[0][n // 2, k // 2] = 0
    want = oracle.fp8_matmul(a2, b2, k).astype(np.float32)
    for dt in (torch.float32, torch.bfloat16):
        got = product(a, b, m, n, k, dtype=dt)
        assert bool(got[torch.from_numpy(bad)].isnan().all())
        assert torch.equal(got[torch.from_numpy(~bad)], torch.from_numpy(want[~bad]).to(dt))


@pytest.mark.parametrize("m,n,k", [(3, 40, 256), (600, 512, 300), (2100, 2001, 128)])
def test_product_least_scale(m, n, k):
    """Values below float32's least normal one: in a float32 result they count as multiples of 2^-133."""
    print(f"case: fp8 matmul at the least scale {m}x{n}x{k}", flush=True)
    r = rng(11, m, n, k)
    a, b = random_held(r, m, k, 0, 0), random_held(r, n, k, 230, 230)
    a[0][:, :k] &= 0x8F                                      # exponent fields 0 and 1: multiples of 2^-136 below 2^-132
    va = torch.from_numpy(oracle.fp8_values(*a, k))
    held = (torch.round(va * 2.0 ** 133) * 2.0 ** -133).numpy()
    assert np.any(held != va.numpy())
    want = held @ oracle.fp8_values(*b, k).T                 # multiples of 2^-133 2^99, at most 2^4 (2^8 k) of them: exact
    assert torch.equal(product(a, b, m, n, k), torch.from_numpy(want.astype(np.float32)))


def test_product_infinite():
    print("case: fp8 matmul past float32's range", flush=True)
    for m, n, k in [(4, 50, 256), (300, 260, 256), (2100, 2001, 256)]:
        r = rng(5)
        a, b = random_held(r, m, k, 200, 200), random_held(r, n, k, 200, 200)
        a[0][:], b[0][:] = 0x38, 0x38                        # all ones: 256 * 2^146
        for dt in (torch.float32, torch.bfloat16):
            assert bool(torch.isposinf(product(a, b, m, n, k, dtype=dt)).all())


def test_products_repeat_bitwise():
    """The same product three times gives the same bits."""
    gc = lib()
    print("case: fp8 matmul determinism", flush=True)
    r = rng(6)
    for m, n, k in KERNELS:
        a, b = held_from(*random_held(r, m, k, 100, 140, 1, True)), held_from(*random_held(r, n, k, 100, 140, 1, True))
        ws = torch.empty(max(16, gc.gc_fp8_matmul_workspace_bytes(m, n, k)), dtype=torch.uint8, device=DEV)
        for dt in (torch.float32, torch.bfloat16):
            outs = [torch.empty(m, n, device=DEV, dtype=dt) for _ in range(3)]
            for out in outs:
                gc.gc_fp8_matmul(*a, *b, k, out, ws)
            assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_workspace_refusals_and_turns():
    """Products in parts of k: a short or missing workspace is refused; two of them in turn on one workspace."""
    gc = lib()
    shapes = [s for s in [(256, 512, 16384), (385, 641, 14400), (300, 520, 16384)] if gc.gc_fp8_matmul_workspace_bytes(*s) > 0]
    assert len(shapes) >= 2
    ws = torch.full((max(gc.gc_fp8_matmul_workspace_bytes(*s) for s in shapes),), 0xFF, dtype=torch.uint8, device=DEV)
    held, want = [], []
    for m, n, k in shapes:
        print(f"case: fp8 matmul in parts {m}x{n}x{k}", flush=True)
        _, a, b = exact_operands(m, n, k, 1, 1)
        held.append((held_from(*a), held_from(*b)))
        want.append(torch.from_numpy(oracle.fp8_matmul(a, b, k).astype(np.float32)))
        out = torch.full((m, n), 3.0, device=DEV)
        need = gc.gc_fp8_matmul_workspace_bytes(m, n, k)
        refused = 0
        for dt, small in [(torch.float32, need - 16), (torch.bfloat16, need - 16), (torch.float32, None), (torch.bfloat16, None)]:
            out = torch.full((m, n), 3.0, device=DEV, dtype=dt)
            try:
                gc.gc_fp8_matmul(*held[-1][0], *held[-1][1], k, out, None if small is None else ws[:small])
            except gc.GCError as e:
                refused += 1
                assert e.status == (gc.GC_ERR_ARG if small is None else gc.GC_ERR_WORKSPACE) and bool((out == 3.0).all())
        assert refused >= 2                                  # one of the types needs all of it
    for i in (0, 1, 0, 0, 1):
        m, n, k = shapes[i]
        for dt in (torch.float32, torch.bfloat16):
            out = torch.empty(m, n, device=DEV, dtype=dt)
            gc.gc_fp8_matmul(*held[i][0], *held[i][1], k, out, ws)
            assert torch.equal(out.cpu(), want[i].to(dt))


# ---------------------------------------------------------------- together, as they are used

def quantized(x, block=1):
    r, c = Held(*x.shape, block), Held(*x.shape[::-1], block)
    lib().gc_fp8_quantize(x, *r.pair, *c.pair, block_rows=block)
    return r, c


def mm(a, b, k, out, accumulate=False):
    gc = lib()
    ws = torch.empty(max(16, gc.gc_fp8_matmul_workspace_bytes(*out.shape, k)), dtype=torch.uint8, device=DEV)
    gc.gc_fp8_matmul(*a.pair, *b.pair, k, out, ws, a_block_rows=a.block, b_block_rows=b.block, accumulate=accumulate)
    return out


@pytest.mark.parametrize("tokens,fin,fout", [(1, 64, 96), (70, 200, 130), (512, 256, 384)])
def test_linear_layer_step(tokens, fin, fout):
    """Forward (bf16), both gradients (the input's in bf16, the weight's in float32 over two micro-batches), then the weight's
    gradient through a compressor; every result against the oracle on what the quantiser held."""
    gc = lib()
    print(f"case: fp8 linear layer {tokens}x{fin}x{fout}", flush=True)
    r = rng(7, tokens)
    x, w, dy = (r.standard_normal(s, dtype=np.float32) * np.float32(f) for s, f in
                [((tokens, fin), 1.0), ((fout, fin), 0.05), ((tokens, fout), 1e-2)])
    xr, xc = quantized(to_dev(x))
    wr, wc = quantized(to_dev(w), 128)
    gr, gcol = quantized(to_dev(dy))
    # the weight has the same values both ways
    assert np.array_equal(wr.values(), wc.values().T)
    cases = [(xr, wr, fin, (tokens, fout), torch.bfloat16), (gr, wc, fout, (tokens, fin), torch.bfloat16),
             (gcol, xc, tokens, (fout, fin), torch.float32)]
    for a, b, k, shape, dt in cases:
        out = mm(a, b, k, torch.empty(shape, dtype=dt, device=DEV))
        va, vb = a.values(), b.values()
        assert within(out.cpu(), va @ vb.T, np.abs(va) @ np.abs(vb).T, k, dt == torch.float32)
    once = out.clone()
    mm(gcol, xc, tokens, out, accumulate=True)
    assert np.array_equal(f32_bits(out), f32_bits(once + once))
    d, k = out.numel(), max(1, out.numel() // 100)
    host = out.cpu().numpy()
    mem, idx, val = torch.zeros(d, device=DEV), torch.empty(k, dtype=torch.int32, device=DEV), torch.empty(k, device=DEV)
    gc.gc_topk_ef_encode(out.view(-1), mem, 0.5, k, idx, val,
                         torch.empty(gc.gc_topk_workspace_bytes(d, k), dtype=torch.uint8, device=DEV))
    assert np.array_equal(idx.cpu().numpy(), oracle.topk_ef_step(np.zeros(d, np.float32), host.ravel(), 0.5, k)["idx"])


def test_gradients_against_differences():
    """y = x W^T with entries that E4M3 holds exactly in either direction; L = sum(dy * y).  The gradient products are the
    formula's exactly, and the differences of L by single entries (L is linear in each) give them too."""
    print("case: fp8 gradients against differences", flush=True)
    r = rng(8)
    t, fi, fo = 150, 70, 140
    # whole numbers up to 15: exact in every block, whatever its scale (largest 448 = 28 * 16)
    x, w, dy = (r.integers(-15, 16, s).astype(np.float32) for s in ((t, fi), (fo, fi), (t, fo)))

    def forward(xh):
        xr, _ = quantized(to_dev(xh))
        wr, _ = quantized(to_dev(w), 128)
        return mm(xr, wr, fi, torch.empty(t, fo, device=DEV)).cpu().numpy().astype(np.float64)

    _, xc = quantized(to_dev(x))
    _, wc = quantized(to_dev(w), 128)
    gr, gcol = quantized(to_dev(dy))
    dx = mm(gr, wc, fo, torch.empty(t, fi, device=DEV)).cpu().numpy()
    dw = mm(gcol, xc, t, torch.empty(fo, fi, device=DEV)).cpu().numpy()
    assert np.array_equal(dx, dy.astype(np.float64) @ w) and np.array_equal(dw, dy.T.astype(np.float64) @ x)
    for i, j in [(0, 1), (13, 40), (149, 69), (128, 32)]:
        up, low = x.copy(), x.copy()
        up[i, j], low[i, j] = 4.0, 1.0
        diff = (np.sum(dy * forward(up)) - np.sum(dy * forward(low))) / 3.0
        assert diff == dx[i, j]


@pytest.mark.parametrize("t,fi,fo", [(300, 512, 256), (16384, 512, 256)])
def test_side_stream_and_graph(t, fi, fo):
    """The chain (the longer one has its product in parts of k) on another stream, then in two graphs with a workspace each,
    replayed with eager work between: every result equals the eager one bit for bit."""
    gc = lib()
    print(f"case: fp8 chain on a side stream and in graphs {t}x{fi}x{fo}", flush=True)
    r = rng(9, t)
    x, dy = r.standard_normal((t, fi), dtype=np.float32), r.standard_normal((t, fo), dtype=np.float32) * np.float32(1e-2)
    if t > 10000:
        assert gc.gc_fp8_matmul_workspace_bytes(fo, fi, t) > 0

    class Chain:
        def __init__(self):
            self.x, self.dy = torch.empty(t, fi, device=DEV), torch.empty(t, fo, device=DEV)
            self.xc, self.dyc, self.dyr = Held(fi, t), Held(fo, t), Held(t, fo)
            self.dw, self.back = torch.zeros(fo, fi, device=DEV), torch.zeros(t, fo, dtype=torch.bfloat16, device=DEV)
            self.ws = torch.empty(max(16, gc.gc_fp8_matmul_workspace_bytes(fo, fi, t)), dtype=torch.uint8, device=DEV)

        def load(self, step):
            self.x.copy_(to_dev(np.roll(x, step, 0)))
            self.dy.copy_(to_dev(dy * np.float32(1 + step)))
            self.dw.fill_(0.25)

        def run(self):
            gc.gc_fp8_quantize(self.x, None, None, *self.xc.pair)
            gc.gc_fp8_quantize(self.dy, *self.dyr.pair, *self.dyc.pair)
            gc.gc_fp8_matmul(*self.dyc.pair, *self.xc.pair, t, self.dw, self.ws, accumulate=True)
            gc.gc_fp8_dequantize(*self.dyr.pair, self.back)

        def bits(self):
            torch.cuda.synchronize()
            return [f32_bits(self.dw), f32_bits(self.back.float())]

    eager, steps = Chain(), []
    for s in range(4):
        eager.load(s)
        eager.run()
        steps.append(eager.bits())
    side, other = torch.cuda.Stream(), Chain()
    for s in range(4):
        other.load(s)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other.run()
        torch.cuda.current_stream().wait_stream(side)
        assert all(np.array_equal(p, q) for p, q in zip(other.bits(), steps[s]))
    graphs = []
    for _ in range(2):
        c = Chain()
        c.load(0)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            c.run()
        graphs.append((g, c))
    for s in range(4):
        for g, c in graphs:
            c.load(s)
            g.replay()
        torch.ones(1000, device=DEV).sum().item()
        for _, c in graphs:
            assert all(np.array_equal(p, q) for p, q in zip(c.bits(), steps[s]))


# ---------------------------------------------------------------- past 32 bits

def test_past_32_bits():
    """More than 2^32 bytes of codes, as one row and as many: quantised, read back and multiplied."""
    gc = lib()
    rows, k = (1 << 25) + 77, 130
    print(f"case: fp8 quantize {rows}x{k} bf16, values, matmul with one row", flush=True)
    r = rng(10)
    part = both_types(r.standard_normal((4096, k), dtype=np.float32), "bf16")
    x = to_dev(part.ravel()).view(4096, k).repeat(-(-rows // 4096), 1)[:rows]
    codes = torch.empty(gc.gc_fp8_code_bytes(rows, k), dtype=torch.uint8, device=DEV)
    scales = torch.empty(gc.gc_fp8_scale_bytes(rows, k), dtype=torch.uint8, device=DEV)
    gc.gc_fp8_quantize(x, codes, scales)
    ref = oracle.fp8_quantize(part)
    full = rows // 4096 * 4096
    for got, want, width in ((codes, ref[0], 256), (scales, ref[1], 4)):
        want = torch.from_numpy(want).to(DEV)
        assert torch.equal(got.view(rows, width)[:full].view(-1, 4096, width), want[None].expand(full // 4096, 4096, width))
        assert torch.equal(got.view(rows, width)[full:], want[: rows - full])
    out = torch.empty(1, rows, dtype=torch.bfloat16, device=DEV)
    a = random_held(r, 1, k, 127, 127)
    gc.gc_fp8_matmul(*held_from(*a), codes, scales, k, out)
    small = torch.empty(1, 4096, dtype=torch.bfloat16, device=DEV)
    gc.gc_fp8_matmul(*held_from(*a), *held_from(*ref), k, small)
    va, vb = oracle.fp8_values(*a, k), oracle.fp8_values(*ref, k)
    assert within(small.cpu(), va @ vb.T, np.abs(va) @ np.abs(vb).T, k, False)
    assert within(out[:, :4096].cpu(), va @ vb.T, np.abs(va) @ np.abs(vb).T, k, False)
    assert torch.equal(out[0, :full].view(-1, 4096), out[:, :4096].expand(full // 4096, 4096))
    x.zero_()
    gc.gc_fp8_dequantize(codes, scales, x)
    want = torch.from_numpy(vb.astype(np.float32)).to(DEV).to(torch.bfloat16)
    assert torch.equal(x[:full].view(-1, 4096, k), want[None].expand(full // 4096, 4096, k)) and torch.equal(x[full:], want[: rows - full])
    del x, codes, scales, out
    torch.cuda.empty_cache()
    d = 2**32 + 1000
    print(f"case: fp8 quantize 1x{d} bf16 and values", flush=True)
    flat = to_dev(part[:, :128].ravel()).repeat(-(-d // (4096 * 128)))[:d]
    codes = torch.empty(gc.gc_fp8_code_bytes(1, d), dtype=torch.uint8, device=DEV)
    scales = torch.empty(gc.gc_fp8_scale_bytes(1, d), dtype=torch.uint8, device=DEV)
    gc.gc_fp8_quantize(flat, codes, scales)
    ref = oracle.fp8_quantize(np.ascontiguousarray(part[:, :128]))
    want = torch.from_numpy(oracle.fp8_values(*ref, 128).astype(np.float32)).to(DEV).to(torch.bfloat16).view(-1)
    flat.zero_()
    gc.gc_fp8_dequantize(codes, scales, flat)
    full = d // want.numel() * want.numel()
    assert torch.equal(flat[:full].view(-1, want.numel()), want[None].expand(full // want.numel(), want.numel()))
    # the last block is cut short, so its scale may be another one
    cut = oracle.fp8_quantize(np.ascontiguousarray(part[:, :128].ravel()[: d - full].reshape(1, -1)))
    assert np.array_equal(flat[full:].float().cpu().numpy(), oracle.fp8_values(*cut, d - full)[0].astype(np.float32))
    del flat, codes, scales
    torch.cuda.empty_cache()
