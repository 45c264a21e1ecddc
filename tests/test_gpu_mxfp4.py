"""GPU: the MXFP4 operators against the 64-bit oracle.

The quantiser, the step with memory and the decode are compared bit for bit:
each is defined down to its float32 roundings.  Products are compared exactly
where every partial sum is a whole multiple of a quantum with fewer than 24
bits (then no order of the additions rounds), and within a derived bound
elsewhere: a sum of K terms differs from the exact one by at most
K * 2^-23 * sum |a b|, one last place an addition, whatever its order.
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


def byte_buffer(n, guard=64):
    """n bytes for the call and `guard` more behind them that it must not touch."""
    return torch.full((n + guard,), GUARD, dtype=torch.uint8, device=DEV)


class Held:
    """An MXFP4 matrix's buffers with guards."""

    def __init__(self, rows, cols):
        gc = lib()
        self.rows, self.cols = rows, cols
        self.nc, self.ns = gc.gc_mxfp4_code_bytes(rows, cols), gc.gc_mxfp4_scale_bytes(rows, cols)
        self.c, self.s = byte_buffer(self.nc), byte_buffer(self.ns)

    @property
    def pair(self):
        return self.c[: self.nc], self.s[: self.ns]

    def host(self):
        c, s = self.c.cpu().numpy(), self.s.cpu().numpy()
        assert np.all(c[self.nc:] == GUARD) and np.all(s[self.ns:] == GUARD), "written past the buffers"
        return c[: self.nc].reshape(self.rows, -1), s[: self.ns].reshape(self.rows, -1)


def held_from(codes, scales):
    """Host codes and scales on the device."""
    return (torch.from_numpy(np.ascontiguousarray(codes).ravel()).to(DEV),
            torch.from_numpy(np.ascontiguousarray(scales).ravel()).to(DEV))


def same(held, ref):
    c, s = held.host()
    assert np.array_equal(s, ref[1]), "scales differ"
    assert np.array_equal(c, ref[0]), "codes differ"


def bf16(a):
    return gen.f32_to_bf16_bits(a)


def wide_matrix(rows, cols, seed):
    """Values over many binades, with exact rounding borders and zeros among them."""
    r = gen.rng(0, gen.KIND_MISC, 400, seed)
    x = r.standard_normal((rows, cols), dtype=np.float32)
    x *= np.exp2(r.integers(-8, 8, (rows, 1))).astype(np.float32)
    grid = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 0.0, -0.0], np.float32)
    put = r.uniform(size=x.shape) < 0.3
    x[put] = (grid[r.integers(0, grid.size, x.shape)] * np.sign(r.standard_normal(x.shape)).astype(np.float32))[put]
    return x


SHAPES = [(1, 1), (1, 31), (1, 32), (1, 33), (1, 127), (1, 128), (1, 129), (1, 1025), (31, 5), (32, 64), (33, 65),
          (127, 130), (129, 96), (5, 4096), (3, 5000), (300, 257), (260, 1155)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize_shapes(rows, cols, dtype):
    gc = lib()
    print(f"case: mxfp4 quantize {rows}x{cols} {dtype}", flush=True)
    x = wide_matrix(rows, cols, rows * 7919 + cols)
    x = bf16(x) if dtype == "bf16" else x
    xt = to_dev(x.ravel()).view(rows, cols)
    r, c, r2, c2 = Held(rows, cols), Held(cols, rows), Held(rows, cols), Held(cols, rows)
    gc.gc_mxfp4_quantize(xt, *r.pair)
    gc.gc_mxfp4_quantize(xt, None, None, *c.pair)
    gc.gc_mxfp4_quantize(xt, *r2.pair, *c2.pair)
    by_rows, by_cols = oracle.mxfp4_quantize(x), oracle.mxfp4_quantize(np.ascontiguousarray(x.T))
    same(r, by_rows)
    same(c, by_cols)
    same(r2, by_rows)
    same(c2, by_cols)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols,pitch", [(70, 129, 136), (70, 129, 131), (200, 512, 1024), (33, 64, 65), (1, 50, 99)])
def test_quantize_pitch(rows, cols, pitch, dtype):
    gc = lib()
    print(f"case: mxfp4 quantize {rows}x{cols} pitch {pitch} {dtype}", flush=True)
    x = wide_matrix(rows, pitch, 5)
    x[:, cols:] = np.nan                                     # between the rows: not part of the matrix
    x = bf16(np.nan_to_num(x, nan=1e30)) if dtype == "bf16" else x
    xt = to_dev(x.ravel()).view(rows, pitch)[:, :cols]
    r, c = Held(rows, cols), Held(cols, rows)
    gc.gc_mxfp4_quantize(xt, *r.pair, *c.pair)
    same(r, oracle.mxfp4_quantize(np.ascontiguousarray(x[:, :cols])))
    same(c, oracle.mxfp4_quantize(np.ascontiguousarray(x[:, :cols].T)))


def extremes():
    """Rows of 32: borders and their neighbours at several scales, subnormals, the largest values, not finite ones."""
    b = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.999], np.float32)
    near = np.concatenate([np.nextafter(b, np.float32(0)), b, np.nextafter(b, np.float32(9))])
    base = np.concatenate([[np.float32(4.0)], near, [0.0, -0.0, 1e-30, -1e-30]]).astype(np.float32)
    rows = [base * np.float32(2.0) ** e for e in (0, 1, -1, 40, -40, 120, -120, -126)]
    tiny = np.arange(32, dtype=np.uint32)
    rows += [np.left_shift(np.uint32(1), np.minimum(tiny, 22)).view(np.float32),              # subnormals
             np.full(32, 2.0 ** -126, np.float32), np.full(32, 3.4028235e38, np.float32),
             np.zeros(32, np.float32), np.full(32, -0.0, np.float32)]
    for bad in (np.inf, -np.inf, np.nan):
        r = np.ones(32, np.float32)
        r[17] = bad
        rows.append(r)
    out = np.zeros((len(rows), 32), np.float32)
    for i, r in enumerate(rows):
        out[i, : r.size] = r
    out[1::2] *= np.float32(-1)
    return out


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantize_extremes(dtype):
    gc = lib()
    x = extremes()
    if dtype == "bf16":                                      # cut to bf16 bits, so that borders and subnormals stay among them
        x = (x.view(np.uint32) >> 16).astype(np.uint16)
        x[np.isnan(extremes())] = 0x7FC0
    for a in (x, np.ascontiguousarray(x.reshape(1, -1)), np.ascontiguousarray(x.T)):
        print(f"case: mxfp4 quantize extremes {a.shape} {dtype}", flush=True)
        r, c = Held(*a.shape), Held(*a.shape[::-1])
        at = to_dev(np.ascontiguousarray(a).ravel()).view(*a.shape)
        gc.gc_mxfp4_quantize(at, *r.pair)
        same(r, oracle.mxfp4_quantize(a))
        gc.gc_mxfp4_quantize(at, *r.pair, *c.pair)
        same(r, oracle.mxfp4_quantize(a))
        same(c, oracle.mxfp4_quantize(np.ascontiguousarray(a.T)))


def test_every_code_and_scale():
    """Decode of all 16 codes at all 256 scales, to float32 and bf16 (both exact up to an infinity at the top)."""
    gc = lib()
    print("case: mxfp4 decode of every code and scale", flush=True)
    codes = np.tile((np.arange(16, dtype=np.uint8).reshape(-1, 2) * [1, 16]).sum(1).astype(np.uint8), (256, 8))
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 4, axis=1)
    want = oracle.mxfp4_values(codes, scales, 128)
    for dt in (torch.float32, torch.bfloat16):
        out = torch.empty(256, 128, dtype=dt, device=DEV)
        gc.gc_mxfp4_decode(*held_from(codes, scales), out)
        got = out.float().cpu().numpy()
        with np.errstate(over="ignore"):
            assert np.array_equal(got, want.astype(np.float32), equal_nan=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [1, 2, 7, 8, 31, 33, 128, 129, 1000, 2047, 2049, 10_000, 100_003, 1_000_001])
def test_ef_steps(d, dtype):
    """Three steps from a memory that is not zero: message and memory bit for bit, nothing behind d touched."""
    gc = lib()
    print(f"case: mxfp4 ef encode d={d} {dtype}", flush=True)
    mem_h = gen.gaussian_vector(d, 3, 0.1)
    mem = torch.full((d + 8,), 77.0, device=DEV)
    mem[:d] = to_dev(mem_h)
    for t in range(3):
        g = gen.gaussian_vector(d, 50 + t)
        g = bf16(g) if dtype == "bf16" else g
        msg = Held(1, d)
        gc.gc_mxfp4_ef_encode(to_dev(g), mem[:d], 0.1, *msg.pair)
        ref = oracle.mxfp4_ef_step(mem_h, g, 0.1)
        same(msg, (ref["codes"], ref["scales"]))
        assert np.array_equal(f32_bits(mem[:d]), f32_bits(ref["mem"]))
        out = torch.empty(d, device=DEV)
        gc.gc_mxfp4_decode(*msg.pair, out)
        assert np.array_equal(out.cpu().numpy(), ref["g"].astype(np.float32))
        mem_h = ref["mem"]
    assert bool((mem[d:] == 77.0).all())


def test_ef_not_finite_stays_in_its_block():
    gc = lib()
    print("case: mxfp4 ef encode with inf and nan", flush=True)
    d = 300
    g = gen.gaussian_vector(d, 9)
    g[40], g[200] = np.inf, np.nan
    mem = torch.zeros(d, device=DEV)
    msg = Held(1, d)
    gc.gc_mxfp4_ef_encode(to_dev(g), mem, 1.0, *msg.pair)
    ref = oracle.mxfp4_ef_step(np.zeros(d, np.float32), g, 1.0)
    same(msg, (ref["codes"], ref["scales"]))
    got = mem.cpu().numpy()
    bad = np.zeros(d, bool)
    bad[32:64] = bad[192:224] = True
    assert np.isnan(got[bad]).all() and np.array_equal(got[~bad], ref["mem"][~bad])


def sums32(codes, scales, cols, weight, old):
    """The decode's definition in float32, operation by operation."""
    total = oracle.mxfp4_values(codes[0], scales[0], cols).astype(np.float32)
    for c, s in zip(codes[1:], scales[1:]):
        total = total + oracle.mxfp4_values(c, s, cols).astype(np.float32)
    total = total * np.float32(weight)
    return total if old is None else old + total


@pytest.mark.parametrize("nmsg", [1, 2, 3, 8])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 1000), (5, 130), (64, 128), (33, 1155), (7, 2056)])
def test_decode_messages(rows, cols, nmsg):
    """Gathered messages in one buffer (codes, then scales, each): weighted sums to both types, over and onto out."""
    gc = lib()
    print(f"case: mxfp4 decode {nmsg} x {rows}x{cols}", flush=True)
    nc, ns = gc.gc_mxfp4_code_bytes(rows, cols), gc.gc_mxfp4_scale_bytes(rows, cols)
    stride = -(-(nc + ns) // 16) * 16
    host = np.full((nmsg, stride), 0xFF, np.uint8)
    codes, scales = [], []
    for i in range(nmsg):
        c, s = oracle.mxfp4_quantize(wide_matrix(rows, cols, 60 + i))
        codes.append(c)
        scales.append(s)
        host[i, :nc], host[i, nc:nc + ns] = c.ravel(), s.ravel()
    buf = torch.from_numpy(host).to(DEV)
    weight = 1.0 / nmsg
    old = gen.gaussian_mat(rows, cols, 4)
    for dt in (torch.float32, torch.bfloat16):
        for add in (False, True):
            out = torch.full((rows * cols + 16,), 5.0, dtype=dt, device=DEV)
            view = out[: rows * cols].view(rows, cols)
            view.copy_(to_dev(old))
            before = view.float().cpu().numpy()
            gc.gc_mxfp4_decode(buf[:, :nc], buf[:, nc:nc + ns], view, weight=weight, accumulate=add)
            want = torch.from_numpy(sums32(codes, scales, cols, weight, before if add else None)).to(dt)
            assert torch.equal(view.cpu(), want)
            assert bool((out[rows * cols:] == 5.0).all())


# ---------------------------------------------------------------- products

def random_held(r, rows, cols, low, high):
    """Random codes with scale bytes in [low, high], pads zero, as (codes, scales) on the host."""
    g = -(-cols // 128)
    nib = np.zeros((rows, g * 128), np.uint8)
    nib[:, :cols] = r.integers(0, 16, (rows, cols))
    scales = np.zeros((rows, g * 4), np.uint8)
    blocks = -(-cols // 32)
    scales[:, :blocks] = r.integers(low, high + 1, (rows, blocks))
    return nib[:, 0::2] | (nib[:, 1::2] << 4), scales


def product(a, b, m, n, k, dtype=torch.float32, old=None, pitch=None):
    """The product through the entry point, on a pitched out whose gaps must stay."""
    gc = lib()
    pitch = n if pitch is None else pitch
    out = torch.full((m, pitch), 3.0, dtype=dtype, device=DEV)
    view = out[:, :n]
    if old is not None:
        view.copy_(to_dev(old))
    ws = torch.full((gc.gc_mxfp4_matmul_workspace_bytes(m, n, k) + 64,), GUARD, dtype=torch.uint8, device=DEV)
    gc.gc_mxfp4_matmul(*held_from(*a), *held_from(*b), k, view, ws[: ws.numel() - 64], accumulate=old is not None)
    assert bool((out[:, n:] == 3.0).all()), "written between the rows"
    assert bool((ws[ws.numel() - 64:] == GUARD).all()), "written past the workspace"
    return view.cpu()


# every path's edges: single rows, tiles of 16 to 256, one group of k to many, sizes one off a tile
PRODUCTS = [(1, 1, 1), (1, 5, 33), (2, 16, 128), (1, 4096, 1024), (3, 1000, 2000), (16, 16, 129), (17, 33, 257),
            (15, 700, 4100), (16, 4096, 1024), (31, 129, 1155), (32, 512, 4096), (64, 64, 64), (65, 100, 640), (100, 1024, 1024),
            (128, 128, 256), (129, 127, 385), (200, 3000, 300), (255, 257, 512), (256, 256, 128), (257, 255, 1),
            (300, 520, 8192), (1000, 1155, 777), (512, 2048, 1024), (1024, 1024, 2048), (2049, 1025, 1030)]


@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_product_exact(m, n, k):
    """Scale bytes 126 and 127: every product is a multiple of 2^-4 below 36, so a sum of K of them, and an old value that
    is a multiple of 2^-4, need log2(36 * 16 * K) < 24 bits: exact in float32 for K < 2^14."""
    print(f"case: mxfp4 matmul exact {m}x{n}x{k}", flush=True)
    r = gen.rng(0, gen.KIND_MISC, 500, m * 31 + n * 7 + k)
    a, b = random_held(r, m, k, 126, 127), random_held(r, n, k, 126, 127)
    want = oracle.mxfp4_matmul(a, b, k)
    assert np.array_equal(product(a, b, m, n, k).numpy(), want)
    old = r.integers(-1000, 1000, (m, n)).astype(np.float32) / np.float32(16)
    assert np.array_equal(product(a, b, m, n, k, old=old, pitch=n + 3).numpy(), want + old)
    half = product(a, b, m, n, k, dtype=torch.bfloat16, pitch=n + 8)
    assert torch.equal(half, torch.from_numpy(want).to(torch.float32).to(torch.bfloat16))
    old16 = torch.from_numpy(old).to(torch.bfloat16)
    half = product(a, b, m, n, k, dtype=torch.bfloat16, old=old16.float().numpy(), pitch=n + 5)
    assert torch.equal(half, (torch.from_numpy(want).float() + old16.float()).to(torch.bfloat16))


# the kernels for larger outs: few rows of many columns, one and several parts of k, both tile sizes at few and many groups
LARGE_PRODUCTS = [(1, 20000, 300), (16, 9000, 1000), (30, 9000, 200), (500, 1000, 1000), (777, 1001, 1155), (1100, 1500, 1500),
                  (300, 520, 16384), (601, 1001, 20000), (1500, 1100, 16400), (2100, 2001, 100), (2100, 2001, 130),
                  (2050, 2100, 700), (2100, 2000, 1000), (4000, 3970, 384), (4000, 4001, 400), (4001, 3900, 520),
                  (4000, 3970, 700), (3900, 4000, 900), (3841, 4095, 1155), (8000, 8000, 200)]


@pytest.mark.parametrize("m,n,k", LARGE_PRODUCTS)
def test_large_product_exact(m, n, k):
    """As above (K < 2^14.8: 36 * 16 * K < 2^24)."""
    print(f"case: mxfp4 matmul exact {m}x{n}x{k}", flush=True)
    r = gen.rng(0, gen.KIND_MISC, 507, m * 31 + n * 7 + k)
    a, b = random_held(r, m, k, 126, 127), random_held(r, n, k, 126, 127)
    want = torch.from_numpy(oracle.mxfp4_matmul(a, b, k).astype(np.float32))
    old = torch.from_numpy(r.integers(-1000, 1000, (m, n)).astype(np.float32) / np.float32(16))
    assert torch.equal(product(a, b, m, n, k, old=old.numpy(), pitch=n + n % 2), want + old)
    assert torch.equal(product(a, b, m, n, k), want)
    assert torch.equal(product(a, b, m, n, k, dtype=torch.bfloat16, pitch=n + 8), want.to(torch.bfloat16))
    old16 = old.to(torch.bfloat16)
    got = product(a, b, m, n, k, dtype=torch.bfloat16, old=old16.float().numpy(), pitch=-(-n // 8) * 8)
    assert torch.equal(got, (want + old16.float()).to(torch.bfloat16))


@pytest.mark.parametrize("m,n,k", [(1, 300, 1000), (16, 1024, 4096), (100, 130, 8192), (300, 260, 1155), (600, 1024, 16384)])
def test_product_bound(m, n, k):
    """Scales over 24 binades, so that the sums round."""
    print(f"case: mxfp4 matmul bound {m}x{n}x{k}", flush=True)
    r = gen.rng(0, gen.KIND_MISC, 501, m + n + k)
    a, b = random_held(r, m, k, 110, 133), random_held(r, n, k, 110, 133)
    want = oracle.mxfp4_matmul(a, b, k)
    size = np.abs(oracle.mxfp4_values(*a, k)) @ np.abs(oracle.mxfp4_values(*b, k)).T
    got = product(a, b, m, n, k).numpy().astype(np.float64)
    assert np.all(np.abs(got - want) <= k * 2.0 ** -23 * size)


@pytest.mark.parametrize("m,n,k", [(1, 64, 256), (20, 40, 300), (300, 300, 512), (600, 512, 4096)])
def test_product_scale_range_and_nan(m, n, k):
    """The ends of the scale range (a product of two least scales is below float32's least subnormal: zero), and NaN."""
    print(f"case: mxfp4 matmul scale range {m}x{n}x{k}", flush=True)
    r = gen.rng(0, gen.KIND_MISC, 502, m + n + k)
    a, b = random_held(r, m, k, 127, 127), random_held(r, n, k, 127, 127)
    a[1][:], b[1][:] = 0, 254
    want = oracle.mxfp4_matmul(a, b, k)                      # 2^-127 * 2^127
    assert np.array_equal(product(a, b, m, n, k).numpy(), want)
    b[1][:] = 127
    want = oracle.mxfp4_matmul(a, b, k)                      # values near 2^-127: subnormal sums may be flushed
    got = product(a, b, m, n, k).numpy().astype(np.float64)
    assert np.all(np.abs(got - want) <= 2 * k * 2.0 ** -126)         # a flush loses less than 2^-126: k products, k sums
    b[1][:] = 0
    assert np.all(product(a, b, m, n, k).numpy() == 0)
    a[1][:], b[1][:] = 127, 127
    a[1][m - 1, 1] = 255
    b[1][n // 2, 0] = 255
    if k > 256:
        a[0][m - 1, 16:32] = 0                               # zero codes do not hide a NaN scale
    got = product(a, b, m, n, k).numpy()
    bad = np.zeros((m, n), bool)
    bad[m - 1, :], bad[:, n // 2] = True, True
    good = (np.where(a[1] == 255, 127, a[1]).astype(np.uint8), np.where(b[1] == 255, 127, b[1]).astype(np.uint8))
    want = oracle.mxfp4_matmul((a[0], good[0]), (b[0], good[1]), k)
    assert np.isnan(got[bad]).all() and np.array_equal(got[~bad], want[~bad])


def test_product_infinite():
    print("case: mxfp4 matmul past float32's range", flush=True)
    r = gen.rng(0, gen.KIND_MISC, 503)
    a, b = random_held(r, 40, 256, 200, 200), random_held(r, 50, 256, 200, 200)
    a[0][:], b[0][:] = 0x22, 0x22                            # all ones: 256 * 2^146
    assert np.all(np.isposinf(product(a, b, 40, 50, 256).numpy()))


def test_products_repeat_bitwise():
    """The same product twice, and with another in between on the same workspace, gives the same bits."""
    gc = lib()
    print("case: mxfp4 matmul determinism", flush=True)
    r = gen.rng(0, gen.KIND_MISC, 504)
    for m, n, k in [(4, 1024, 8192), (256, 512, 16384), (300, 700, 5000), (2100, 2000, 500), (4000, 3970, 384)]:
        a, b = held_from(*random_held(r, m, k, 100, 140)), held_from(*random_held(r, n, k, 100, 140))
        ws = torch.empty(max(16, gc.gc_mxfp4_matmul_workspace_bytes(m, n, k)), dtype=torch.uint8, device=DEV)
        outs = []
        for _ in range(3):
            out = torch.empty(m, n, device=DEV)
            gc.gc_mxfp4_matmul(*a, *b, k, out, ws)
            outs.append(out)
        assert np.array_equal(f32_bits(outs[0]), f32_bits(outs[1])) and np.array_equal(f32_bits(outs[0]), f32_bits(outs[2]))


def test_workspace_too_small():
    gc = lib()
    shapes = [(m, n, k) for m, n, k in LARGE_PRODUCTS if gc.gc_mxfp4_matmul_workspace_bytes(m, n, k) > 0]
    assert shapes
    for m, n, k in shapes:
        r = gen.rng(0, gen.KIND_MISC, 505)
        a, b = held_from(*random_held(r, m, k, 127, 127)), held_from(*random_held(r, n, k, 127, 127))
        out = torch.full((m, n), 3.0, device=DEV)
        need = gc.gc_mxfp4_matmul_workspace_bytes(m, n, k)
        with pytest.raises(gc.GCError) as e:
            gc.gc_mxfp4_matmul(*a, *b, k, out, torch.empty(need - 16, dtype=torch.uint8, device=DEV))
        assert e.value.status == gc.GC_ERR_WORKSPACE
        with pytest.raises(gc.GCError) as e:
            gc.gc_mxfp4_matmul(*a, *b, k, out)
        assert e.value.status == gc.GC_ERR_ARG and bool((out == 3.0).all())


# ---------------------------------------------------------------- together, as they are used

def linear_setup(tokens, fin, fout):
    r = gen.rng(0, gen.KIND_MISC, 600)
    x = r.standard_normal((tokens, fin), dtype=np.float32)
    w = r.standard_normal((fout, fin), dtype=np.float32) * np.float32(0.05)
    dy = r.standard_normal((tokens, fout), dtype=np.float32) * np.float32(1e-2)
    return x, w, dy


def quantized(x):
    """x by rows and by columns through the entry point."""
    r, c = Held(*x.shape), Held(*x.shape[::-1])
    lib().gc_mxfp4_quantize(x, *r.pair, *c.pair)
    return r, c


def mm(a, b, k, out, accumulate=False):
    gc = lib()
    m, n = out.shape
    ws = torch.empty(max(16, gc.gc_mxfp4_matmul_workspace_bytes(m, n, k)), dtype=torch.uint8, device=DEV)
    gc.gc_mxfp4_matmul(*a.pair, *b.pair, k, out, ws, accumulate=accumulate)
    return out


@pytest.mark.parametrize("tokens,fin,fout", [(1, 64, 96), (70, 200, 130), (512, 256, 384)])
def test_linear_layer_step(tokens, fin, fout):
    """Forward, both gradients over two micro-batches, then the weight's gradient through every compressor that takes it;
    the product's inputs and outputs against the oracle on what the quantiser held."""
    gc = lib()
    print(f"case: mxfp4 linear layer {tokens}x{fin}x{fout}", flush=True)
    x, w, dy = linear_setup(tokens, fin, fout)
    xr, xc = quantized(to_dev(x))
    wr, wc = quantized(to_dev(w))
    gr, gcol = quantized(to_dev(dy))
    val = lambda h: oracle.mxfp4_values(*h.host(), h.cols)           # noqa: E731
    cases = [(xr, wr, fin, torch.empty(tokens, fout, device=DEV)), (gr, wc, fout, torch.empty(tokens, fin, device=DEV)),
             (gcol, xc, tokens, torch.empty(fout, fin, device=DEV))]
    for a, b, k, out in cases:
        mm(a, b, k, out)
        va, vb = val(a), val(b)
        assert np.all(np.abs(out.cpu().numpy() - va @ vb.T) <= k * 2.0 ** -23 * (np.abs(va) @ np.abs(vb).T))
    dw = cases[2][3]
    once = dw.clone()
    mm(gcol, xc, tokens, dw, accumulate=True)
    assert np.array_equal(f32_bits(dw), f32_bits(once + once))
    # the gradient into the compressors: 4-bit with memory, top-k, PowerSGD
    d = dw.numel()
    host = dw.cpu().numpy()
    mem, msg = torch.zeros(d, device=DEV), Held(1, d)
    gc.gc_mxfp4_ef_encode(dw.view(-1), mem, 0.5, *msg.pair)
    ref = oracle.mxfp4_ef_step(np.zeros(d, np.float32), host.ravel(), 0.5)
    same(msg, (ref["codes"], ref["scales"]))
    assert np.array_equal(f32_bits(mem), f32_bits(ref["mem"]))
    k = max(1, d // 100)
    tmem, idx, tval = torch.zeros(d, device=DEV), torch.empty(k, dtype=torch.int32, device=DEV), torch.empty(k, device=DEV)
    gc.gc_topk_ef_encode(dw.view(-1), tmem, 0.5, k, idx, tval,
                         torch.empty(gc.gc_topk_workspace_bytes(d, k), dtype=torch.uint8, device=DEV))
    assert np.array_equal(idx.cpu().numpy(), oracle.topk_ef_step(np.zeros(d, np.float32), host.ravel(), 0.5, k)["idx"])
    # a message of a matrix whose rows are whole groups is that matrix's MXFP4 form
    if fin % 128 == 0:
        direct = Held(fout, fin)
        gc.gc_mxfp4_quantize((dw * 0.5), *direct.pair)
        assert torch.equal(direct.pair[0], msg.pair[0]) and torch.equal(direct.pair[1], msg.pair[1])
        y, vx = torch.empty(tokens, fout, device=DEV), val(xr)
        ws = torch.empty(max(16, gc.gc_mxfp4_matmul_workspace_bytes(tokens, fout, fin)), dtype=torch.uint8, device=DEV)
        gc.gc_mxfp4_matmul(*xr.pair, *msg.pair, fin, y, ws)
        g = ref["g"].reshape(fout, fin)
        assert np.all(np.abs(y.cpu().numpy() - vx @ g.T) <= fin * 2.0 ** -23 * (np.abs(vx) @ np.abs(g).T))


def test_gradients_against_differences():
    """y = x W^T with entries that MXFP4 holds exactly in either direction; L = sum(dy * y).  The two gradient products are
    the formula's exactly, and the differences of L by single entries (L is linear in each) give them too."""
    print("case: mxfp4 gradients against differences", flush=True)
    r = gen.rng(0, gen.KIND_MISC, 601)
    t, fi, fo = 40, 70, 50
    grid = np.array([-6, -4, -3, -2, -1.5, -1, -0.5, 0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float32)

    def held_exactly(rows, cols):
        a = grid[r.integers(0, grid.size, (rows, cols))]
        for i in range(0, rows, 32):
            for j in range(cols):
                a[min(i + (j * 7) % 32, rows - 1), j] = 6.0            # every column block's largest
        for i in range(rows):
            for j in range(0, cols, 32):
                a[i, min(j + (i * 5) % 32, cols - 1)] = 6.0            # every row block's largest
        return a

    x, w, dy = held_exactly(t, fi), held_exactly(fo, fi), held_exactly(t, fo)

    def forward(xh):
        xr, _ = quantized(to_dev(xh))
        wr, _ = quantized(to_dev(w))
        return mm(xr, wr, fi, torch.empty(t, fo, device=DEV)).cpu().numpy().astype(np.float64)

    _, xc = quantized(to_dev(x))
    _, wc = quantized(to_dev(w))
    gr, gcol = quantized(to_dev(dy))
    dx = mm(gr, wc, fo, torch.empty(t, fi, device=DEV)).cpu().numpy()
    dw = mm(gcol, xc, t, torch.empty(fo, fi, device=DEV)).cpu().numpy()
    assert np.array_equal(dx, dy.astype(np.float64) @ w) and np.array_equal(dw, dy.T.astype(np.float64) @ x)
    for i, j in [(0, 1), (13, 40), (39, 69), (31, 32)]:
        up, low = x.copy(), x.copy()
        up[i, j], low[i, j] = 4.0, 1.0                       # both exact while the row block keeps a 6 or a 4
        diff = (np.sum(dy * forward(up)) - np.sum(dy * forward(low))) / 3.0
        assert diff == dx[i, j]


def test_side_stream_and_graph():
    """The chain on another stream, then captured (one launch sequence per graph, two graphs with a workspace each) and
    replayed with eager work between: every replay equals the eager chain bit for bit."""
    gc = lib()
    print("case: mxfp4 chain on a side stream and in graphs", flush=True)
    t, fi, fo = 300, 512, 256
    x, _, dy = linear_setup(t, fi, fo)

    class Chain:
        def __init__(self):
            self.x, self.dy = torch.empty(t, fi, device=DEV), torch.empty(t, fo, device=DEV)
            self.xc, self.gc_ = Held(fi, t), Held(fo, t)
            self.dw, self.mem = torch.zeros(fo, fi, device=DEV), torch.zeros(fo * fi, device=DEV)
            self.msg, self.out = Held(1, fo * fi), torch.zeros(fo, fi, device=DEV)
            self.ws = torch.empty(max(16, gc.gc_mxfp4_matmul_workspace_bytes(fo, fi, t)), dtype=torch.uint8, device=DEV)

        def load(self, seed):
            self.x.copy_(to_dev(np.roll(x, seed, 0)))
            self.dy.copy_(to_dev(dy * np.float32(1 + seed)))

        def run(self):
            gc.gc_mxfp4_quantize(self.x, None, None, *self.xc.pair)
            gc.gc_mxfp4_quantize(self.dy, None, None, *self.gc_.pair)
            gc.gc_mxfp4_matmul(*self.gc_.pair, *self.xc.pair, t, self.dw, self.ws)
            gc.gc_mxfp4_ef_encode(self.dw.view(-1), self.mem, 0.3, *self.msg.pair)
            gc.gc_mxfp4_decode(*self.msg.pair, self.out)

        def bits(self):
            torch.cuda.synchronize()
            return [f32_bits(self.dw), f32_bits(self.mem), f32_bits(self.out)]

    eager = Chain()
    steps = []
    for s in range(4):
        eager.load(s)
        eager.run()
        steps.append(eager.bits())
    side = torch.cuda.Stream()
    other = Chain()
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

def test_ef_past_32_bits():
    """More than 2^31 entries: the ends and a slice across 2^31 against the oracle."""
    gc = lib()
    d = 2**31 + 5000 * 32 + 13
    print(f"case: mxfp4 ef encode d={d} bf16", flush=True)
    grad = torch.empty(d, dtype=torch.bfloat16, device=DEV)
    piece = to_dev(bf16(gen.gaussian_vector(1 << 20, 12)))
    for i in range(0, d, 1 << 20):
        n = min(1 << 20, d - i)
        grad[i:i + n] = piece[:n]
    mem = torch.full((d,), 0.125, device=DEV)
    codes = torch.empty(gc.gc_mxfp4_code_bytes(1, d), dtype=torch.uint8, device=DEV)
    scales = torch.empty(gc.gc_mxfp4_scale_bytes(1, d), dtype=torch.uint8, device=DEV)
    gc.gc_mxfp4_ef_encode(grad, mem, 1.0, codes, scales)
    out = torch.empty(d, dtype=torch.bfloat16, device=DEV)
    gc.gc_mxfp4_decode(codes, scales, out)
    for lo in (0, 2**31 - 3200, d // 32 * 32 - 3200):
        hi = min(d, lo + 6400)
        g = grad[lo:hi].view(torch.int16).cpu().numpy().view(np.uint16)
        ref = oracle.mxfp4_ef_step(np.full(hi - lo, 0.125, np.float32), g, 1.0)
        assert np.array_equal(f32_bits(mem[lo:hi]), f32_bits(ref["mem"]))
        assert np.array_equal(out[lo:hi].float().cpu().numpy(), ref["g"].astype(np.float32))
    del grad, mem, codes, scales, out
    torch.cuda.empty_cache()


@pytest.mark.parametrize("turned", [False, True])
def test_product_of_a_vector_and_2_27_rows(turned):
    """The most rows of an operand against one: 2^23 tiles of 16 x 16 would be 2^32 threads of one launch."""
    gc = lib()
    rows, k = 1 << 27, 32
    print(f"case: mxfp4 matmul {1 if turned else rows}x{rows if turned else 1}x{k}", flush=True)
    r = gen.rng(0, gen.KIND_MISC, 507)
    a, part = random_held(r, 1, k, 126, 127), random_held(r, 4096, k, 126, 127)
    bc = torch.from_numpy(part[0].reshape(4096, 64)).to(DEV).repeat(rows // 4096, 1)
    bs = torch.from_numpy(part[1].reshape(4096, 4)).to(DEV).repeat(rows // 4096, 1)
    out = torch.empty((1, rows) if turned else (rows, 1), device=DEV)
    m, n = out.shape
    ws = torch.empty(max(16, gc.gc_mxfp4_matmul_workspace_bytes(m, n, k)), dtype=torch.uint8, device=DEV)
    one, many = held_from(*a), (bc.view(-1), bs.view(-1))
    gc.gc_mxfp4_matmul(*(one + many if turned else many + one), k, out, ws)
    want = torch.from_numpy(oracle.mxfp4_matmul(part, a, k).astype(np.float32)).to(DEV).view(-1)
    assert torch.equal(out.view(-1, 4096), want[None].expand(rows // 4096, 4096))
    del bc, bs, many, out
    torch.cuda.empty_cache()


@pytest.mark.parametrize("m", [1, 40])
def test_product_past_32_bits(m):
    """An operand of more than 2^32 bytes of codes: rows at its start, across the border and at its end."""
    gc = lib()
    n, k = (1 << 20) + 77, 8192
    print(f"case: mxfp4 matmul {m}x{n}x{k}", flush=True)
    r = gen.rng(0, gen.KIND_MISC, 506, m)
    a, part = random_held(r, m, k, 126, 127), random_held(r, 4096, k, 126, 127)
    bc = torch.empty(n, k // 2, dtype=torch.uint8, device=DEV)
    bs = torch.empty(n, k // 32, dtype=torch.uint8, device=DEV)
    pc, ps = torch.from_numpy(part[0]).to(DEV), torch.from_numpy(part[1]).to(DEV)
    for i in range(0, n, 4096):
        c = min(4096, n - i)
        bc[i:i + c], bs[i:i + c] = pc[:c], ps[:c]
    out = torch.empty(m, n, device=DEV)
    ws = torch.empty(max(16, gc.gc_mxfp4_matmul_workspace_bytes(m, n, k)), dtype=torch.uint8, device=DEV)
    gc.gc_mxfp4_matmul(*held_from(*a), bc.view(-1), bs.view(-1), k, out, ws)
    want = torch.from_numpy(oracle.mxfp4_matmul(a, part, k).astype(np.float32)).to(DEV)
    full = n // 4096 * 4096
    assert torch.equal(out[:, :full].reshape(m, -1, 4096), want[:, None, :].expand(m, full // 4096, 4096))
    assert torch.equal(out[:, full:], want[:, : n - full])
    del bc, bs, out
    torch.cuda.empty_cache()
