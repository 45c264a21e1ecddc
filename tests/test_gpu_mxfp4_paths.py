"""GPU: the MXFP4 product's kernels on the paths that few or shallow sums do not reach, and the operators together.

Products are compared exactly where no order of the additions rounds: with scale bytes in [low, high] every term is a
whole multiple of 2^-2 * 2^(2 (low - 127)) and at most 36 * 2^(2 (high - 127)), so a sum of K terms is exact in float32
for 144 * K * 4^(high - low) < 2^24.
"""
import numpy as np
import pytest
import torch

import gen
import oracle
from gpu_util import DEV, f32_bits, lib, rel_err, require_gpu, to_dev
from test_gpu_mxfp4 import Held, held_from, linear_setup, product, random_held, same, sums32

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def rng(which, m=0, n=0, k=0):
    return gen.rng(0, gen.KIND_MISC, 700 + which, m * 31 + n * 7 + k)


# Outs that take the 256 x 256 tile, the 128 x 128 tile with two on a compute unit, that tile alone, and in parts of k.
# A place for scales in LDS is first read after it was written again from group 13, 13 and 17 of 128 columns on; the
# groups past the last whole four are 0 to 3.
DEEP = [(4000, 3970, 3000), (4000, 3970, 3100), (4000, 3970, 3300), (3841, 4095, 3400),
        (2100, 2000, 1650), (2100, 2000, 1700), (2049, 2100, 1900), (2100, 2000, 2000),
        (700, 900, 2100), (700, 900, 2200), (700, 900, 2400), (700, 900, 2500),
        (385, 641, 14400)]


@pytest.mark.parametrize("m,n,k", DEEP)
def test_deep_product_exact(m, n, k):
    """Three scales within a factor of four (144 * 3400 * 16 < 2^24; two for the deepest: 144 * 14400 * 4 < 2^24)."""
    print(f"case: mxfp4 matmul deep {m}x{n}x{k}", flush=True)
    r = rng(1, m, n, k)
    low = 125 if k < 7000 else 126
    a, b = random_held(r, m, k, low, 127), random_held(r, n, k, low, 127)
    want = torch.from_numpy(oracle.mxfp4_matmul(a, b, k).astype(np.float32))
    assert torch.equal(product(a, b, m, n, k), want)
    assert torch.equal(product(a, b, m, n, k, dtype=torch.bfloat16, pitch=n + 6), want.to(torch.bfloat16))
    old = torch.from_numpy(r.integers(-1000, 1000, (m, n)).astype(np.float32))
    assert torch.equal(product(a, b, m, n, k, old=old.numpy()), want + old)
    old16 = old.to(torch.bfloat16)
    assert torch.equal(product(a, b, m, n, k, dtype=torch.bfloat16, old=old16.float().numpy()), (want + old16.float()).to(torch.bfloat16))


# One out for each tile of the product, and one in parts of k; the first for the kernel of few tiles.
TILES = [(300, 300, 512), (700, 900, 2100), (300, 520, 16384), (2100, 2000, 1000), (4000, 3970, 1700)]


@pytest.mark.parametrize("m,n,k", TILES)
def test_scale_ends_on_every_tile(m, n, k):
    """The least and the largest scale against each other: the terms are those of scales 2^0 and 2^0 (their scale bytes
    add up to 254), 144 * K < 2^24."""
    print(f"case: mxfp4 matmul scale ends {m}x{n}x{k}", flush=True)
    r = rng(2, m, n, k)
    a, b = random_held(r, m, k, 127, 127), random_held(r, n, k, 127, 127)
    want = torch.from_numpy(oracle.mxfp4_matmul(a, b, k).astype(np.float32))
    blocks = -(-k // 32)
    for sa, sb in [(0, 254), (254, 0)]:
        a[1][:, :blocks], b[1][:, :blocks] = sa, sb
        assert torch.equal(product(a, b, m, n, k), want)
    # by blocks: byte s against 254 - s
    s = r.integers(0, 255, blocks).astype(np.uint8)
    a[1][:, :blocks], b[1][:, :blocks] = s, 254 - s
    assert torch.equal(product(a, b, m, n, k), want)


@pytest.mark.parametrize("m,n,k", TILES)
def test_nan_scales_on_every_tile(m, n, k):
    """A NaN scale in the first and the last block of a row makes that row (or column) of out NaN, zero codes or not, and
    nothing else."""
    print(f"case: mxfp4 matmul NaN scales {m}x{n}x{k}", flush=True)
    r = rng(3, m, n, k)
    a, b = random_held(r, m, k, 127, 127), random_held(r, n, k, 127, 127)
    want = torch.from_numpy(oracle.mxfp4_matmul(a, b, k).astype(np.float32))
    last = (k - 1) // 32
    bad = torch.zeros(m, n, dtype=torch.bool)
    for row, block in [(0, last), (m // 2, last // 2), (m - 1, 0)]:
        a[1][row, block] = 255
        bad[row] = True
    for col, block in [(1, 0), (n // 3, last), (n - 1, last)]:
        b[1][col, block] = 255
        bad[:, col] = True
    a[0][0, last * 16:last * 16 + 16] = 0
    b[0][1, :16] = 0
    got = product(a, b, m, n, k)
    assert bool(got[bad].isnan().all())
    assert torch.equal(got[~bad], want[~bad])


@pytest.mark.parametrize("m,n,k", TILES)
def test_bound_on_every_tile(m, n, k):
    """Scales over 24 binades, so that the sums round: at most one last place of the magnitudes' sum an addition."""
    print(f"case: mxfp4 matmul bound {m}x{n}x{k}", flush=True)
    r = rng(4, m, n, k)
    a, b = random_held(r, m, k, 110, 133), random_held(r, n, k, 110, 133)
    va, vb = oracle.mxfp4_values(*a, k), oracle.mxfp4_values(*b, k)
    err = np.abs(product(a, b, m, n, k).numpy() - va @ vb.T)
    assert np.all(err <= k * 2.0 ** -23 * (np.abs(va) @ np.abs(vb).T))


@pytest.mark.parametrize("m,n,k", [(1, 64, 256), (20, 40, 300), (300, 300, 512), (600, 512, 4096)] + TILES[1:])
def test_least_scales_exact(m, n, k):
    """Terms below float32's least normal value are kept: with scales 2^-127 and 2^b they are whole multiples of
    2^(b - 129), which float32 holds down to 2^-149, and a sum of K is exact for 144 * K < 2^24."""
    print(f"case: mxfp4 matmul least scales {m}x{n}x{k}", flush=True)
    r = rng(5, m, n, k)
    a, b = random_held(r, m, k, 127, 127), random_held(r, n, k, 127, 127)
    blocks = -(-k // 32)
    a[1][:, :blocks] = 0
    for power in (0, -10, -20):
        b[1][:, :blocks] = 127 + power
        want = oracle.mxfp4_matmul(a, b, k)
        assert np.abs(want).max() >= 2.0 ** (power - 126)
        assert np.array_equal(product(a, b, m, n, k).numpy().astype(np.float64), want)


def test_products_in_turn_on_one_workspace():
    """Two products in parts of k, another number and size of them, on one workspace in turn: what one left there does
    not reach the other's result."""
    gc = lib()
    shapes = [(256, 512, 16384), (385, 641, 14400)]
    need = [gc.gc_mxfp4_matmul_workspace_bytes(*s) for s in shapes]
    assert min(need) > 0
    ws = torch.full((max(need),), 0xFF, dtype=torch.uint8, device=DEV)
    r = rng(6)
    held, want = [], []
    for m, n, k in shapes:
        a, b = random_held(r, m, k, 126, 127), random_held(r, n, k, 126, 127)
        held.append((held_from(*a), held_from(*b)))
        want.append(torch.from_numpy(oracle.mxfp4_matmul(a, b, k).astype(np.float32)))
    outs = []
    for i in (0, 1, 0, 0, 1):
        m, n, k = shapes[i]
        print(f"case: mxfp4 matmul in turn {m}x{n}x{k}", flush=True)
        out = torch.empty(m, n, device=DEV)
        gc.gc_mxfp4_matmul(*held[i][0], *held[i][1], k, out, ws)
        outs.append((i, out))
    for i, out in outs:
        assert torch.equal(out.cpu(), want[i])


def test_product_in_parts_on_a_side_stream_and_in_graphs():
    """A weight's gradient over many tokens, its product in parts of k (a workspace for each user): on another stream,
    then in two graphs that are replayed with eager work between; every result equals the eager one bit for bit."""
    gc = lib()
    t, fi, fo = 16384, 512, 256
    print(f"case: mxfp4 product in parts, side stream and graphs {fo}x{fi}x{t}", flush=True)
    assert gc.gc_mxfp4_matmul_workspace_bytes(fo, fi, t) > 0
    x, _, dy = linear_setup(t, fi, fo)

    class Layer:
        def __init__(self):
            self.x, self.dy = torch.empty(t, fi, device=DEV), torch.empty(t, fo, device=DEV)
            self.xc, self.dyc = Held(fi, t), Held(fo, t)
            self.dw = torch.zeros(fo, fi, device=DEV)
            self.ws = torch.empty(gc.gc_mxfp4_matmul_workspace_bytes(fo, fi, t), dtype=torch.uint8, device=DEV)

        def load(self, step):
            self.x.copy_(to_dev(np.roll(x, step, 0)))
            self.dy.copy_(to_dev(dy * np.float32(1 + step)))
            self.dw.fill_(0.25)

        def run(self):
            gc.gc_mxfp4_quantize(self.x, None, None, *self.xc.pair)
            gc.gc_mxfp4_quantize(self.dy, None, None, *self.dyc.pair)
            gc.gc_mxfp4_matmul(*self.dyc.pair, *self.xc.pair, t, self.dw, self.ws, accumulate=True)

    eager, steps = Layer(), []
    for s in range(4):
        eager.load(s)
        eager.run()
        steps.append(f32_bits(eager.dw))
    va, vb = (oracle.mxfp4_values(*h.host(), t) for h in (eager.dyc, eager.xc))
    err = np.abs(eager.dw.cpu().numpy() - (va @ vb.T + 0.25))
    assert np.all(err <= (t + 1) * 2.0 ** -23 * (np.abs(va) @ np.abs(vb).T + 0.25))
    side, other = torch.cuda.Stream(), Layer()
    for s in range(4):
        other.load(s)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other.run()
        torch.cuda.current_stream().wait_stream(side)
        assert np.array_equal(f32_bits(other.dw), steps[s])
    graphs = []
    for _ in range(2):
        layer = Layer()
        layer.load(0)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            layer.run()
        graphs.append((g, layer))
    for s in range(4):
        for g, layer in graphs:
            layer.load(s)
            g.replay()
        torch.ones(1000, device=DEV).sum().item()
        for _, layer in graphs:
            assert np.array_equal(f32_bits(layer.dw), steps[s])


def test_layer_gradients_exchanged():
    """Four workers: a layer's weight gradient from MXFP4 products over two micro-batches, its message with memory, the
    gathered messages' mean, for two steps; and the same gradient through PowerSGD with memory."""
    gc = lib()
    workers, t, fi, fo, eta = 4, 96, 160, 72, 0.5
    print(f"case: mxfp4 layer gradients of {workers} workers {t}x{fi}x{fo}", flush=True)
    d = fo * fi
    nc, ns = gc.gc_mxfp4_code_bytes(1, d), gc.gc_mxfp4_scale_bytes(1, d)
    x, _, dy = linear_setup(t, fi, fo)
    mems = [torch.zeros(d, device=DEV) for _ in range(workers)]
    host_mems = [np.zeros(d, np.float32) for _ in range(workers)]
    gathered = torch.full((workers, -(-(nc + ns) // 16) * 16), 0xFF, dtype=torch.uint8, device=DEV)
    ws = torch.empty(max(16, gc.gc_mxfp4_matmul_workspace_bytes(fo, fi, t)), dtype=torch.uint8, device=DEV)
    mean = torch.empty(d, device=DEV)
    for step in range(2):
        codes, scales = [], []
        for w in range(workers):
            dw = torch.zeros(fo, fi, device=DEV)
            total, size = np.zeros((fo, fi)), np.zeros((fo, fi))
            for micro in range(2):
                shift = 8 * step + 2 * w + micro
                xh, dyh = np.roll(x, shift, 0), np.roll(dy, 3 * shift, 1)
                xc, dyc = Held(fi, t), Held(fo, t)
                gc.gc_mxfp4_quantize(to_dev(xh), None, None, *xc.pair)
                gc.gc_mxfp4_quantize(to_dev(dyh), None, None, *dyc.pair)
                same(xc, oracle.mxfp4_quantize(np.ascontiguousarray(xh.T)))
                same(dyc, oracle.mxfp4_quantize(np.ascontiguousarray(dyh.T)))
                gc.gc_mxfp4_matmul(*dyc.pair, *xc.pair, t, dw, ws, accumulate=True)
                va, vb = oracle.mxfp4_values(*dyc.host(), t), oracle.mxfp4_values(*xc.host(), t)
                total, size = total + va @ vb.T, size + np.abs(va) @ np.abs(vb).T
            # t additions a micro-batch, and one to what was there
            assert np.all(np.abs(dw.cpu().numpy() - total) <= 2 * (t + 1) * 2.0 ** -23 * size)
            message = gathered[w, :nc], gathered[w, nc:nc + ns]
            gc.gc_mxfp4_ef_encode(dw.view(-1), mems[w], eta, *message)
            ref = oracle.mxfp4_ef_step(host_mems[w], dw.cpu().numpy().ravel(), eta)
            assert np.array_equal(message[0].cpu().numpy(), ref["codes"][0]) and np.array_equal(message[1].cpu().numpy(), ref["scales"][0])
            assert np.array_equal(f32_bits(mems[w]), f32_bits(ref["mem"]))
            host_mems[w] = ref["mem"]
            codes.append(ref["codes"])
            scales.append(ref["scales"])
        gc.gc_mxfp4_decode(gathered[:, :nc], gathered[:, nc:nc + ns], mean, weight=1.0 / workers)
        assert np.array_equal(f32_bits(mean), f32_bits(sums32(codes, scales, d, 1.0 / workers, None).ravel()))
    # the last worker's gradient as a matrix of a low-rank step
    mem, q, out = torch.zeros(fo, fi, device=DEV), to_dev(gen.q_init(0, 0, fi)), torch.zeros(fo, fi, device=DEV)
    q_before = q.cpu().numpy()
    mats = [gc.Mat(grad=dw, mem=mem, q=q, rank=2, p=torch.zeros(4, fo, device=DEV), out=out)]
    gc.gc_powersgd_ef_step(mats, eta, torch.empty(gc.gc_powersgd_workspace_bytes(mats), dtype=torch.uint8, device=DEV))
    ref = oracle.powersgd_ef_step(dw.cpu().numpy(), np.zeros((fo, fi), np.float32), q_before.T, eta, 2)
    # the low-rank step's tolerance: float32 sums of at most 160 terms, twice over, through a well-conditioned P
    assert rel_err(out.cpu().numpy(), ref["out"]) <= 1e-4 and rel_err(mem.cpu().numpy(), ref["mem"]) <= 1e-4
