"""GPU: gc_muon_step against the 64-bit oracle.

The momentum is compared bit for bit.  One step's update is held to a bound entry by
entry.  X, A = X X^T and P = a I + b A + c A A are pairs of f16, so a held value is off by
2^-23 of itself (hi is off by 2^-11 at most, lo by 2^-12 of that), a product of two pairs by 2^-22 more (lo lo is left out), and a sum
of k terms in float32 by k 2^-23 of the sum of their magnitudes, three for each.  With
|X| the matrix of magnitudes and B = |b| |X||X|^T + |c| (|X||X|^T)^2, the step's result is off by
at most e B |X| + d |a| |X|, e = 9 * 2^-22 + 3 * (m + 2 n) 2^-23: the roundings of X (three
times at most, in c A A X five), of A (twice), of P, the products and the sums (of length m for A,
n for the others), each times at most two; d = 9 * 2^-22 + 3 n 2^-23, without the sum where
nothing else is added (b = c = 0).  Beside that a small lo is rounded to multiples of
f16's least value, 2^-24: held times 2^12 (X) or 2^11 (A, P), so X is off by 2^-37 and A and P
by 2^-36 more, whatever their size; `floors` follows them through the step: A is off by
|X| dX^T + dX |X|^T + 2^-36, P by |b| dA + |c| (|A| dA + dA |A|) + 2^-36, the result by |P| dX + dP |X|.
The tests take twice all of that.

After more steps: the polynomial's slope over the singular values that occur is at most 4
(3.4445 at zero), so what a step is off by grows 4 times with each that follows, and the
norm of the sum is at most the sum of the norms.  There (`steps_bound`) the roundings are
taken as independent: in a product V W of k terms they are at most 3 * 2^-22 + sqrt(3 k) 2^-23
of |V W| and of the root of the sum of its terms' squares, each in the Frobenius norm, and an error
E of a factor is one of at most |E| times the other's largest singular value.  The tests take
twice that too.

A bf16 result's last step takes A = X X^T and P X from the hi parts alone, each off by 2^-11 of
itself at most.  Its result is off by 2^-11 times 2 |a| |X| (P's rounding and X's), 4 |b| |X||X|^T |X|
(the two X of A as well) and 6 |c| (|X||X|^T)^2 |X| more, entry by entry; as independent roundings by
(|b| + 2 |c| |A|_2) |X|_2 times 2 * 2^-11 of the root of the sum of X X^T's terms' squares, and 2^-11 of
|P|_F |X|_2 + |P|_2 |X|_F.  Then 2^-8 of each entry for the rounding.
"""
import numpy as np
import pytest
import torch

import gen
import oracle
from gpu_util import DEV, f32_bits, lib, require_gpu, to_dev

pytestmark = pytest.mark.gpu

USUAL = (3.4445, -4.7750, 2.0315)


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def rng(which, *of):
    return gen.rng(0, gen.KIND_MISC, 1100 + which, sum(v * w for v, w in zip(of, (31, 7, 1))))


def matrix(n, m, kind="gauss", which=0):
    r = rng(which, n, m)
    g = r.standard_normal((n, m), dtype=np.float32)
    if kind == "low":                                        # three strong directions over a little noise
        g = (r.standard_normal((n, 3)) @ r.standard_normal((3, m)) + 1e-3 * g).astype(np.float32)
    elif kind == "rows":                                     # rows of very different sizes
        g *= np.exp2(r.integers(-20, 1, (n, 1))).astype(np.float32)
    return g


def workspace(mats):
    """Poisoned (every float NaN), with a guard behind."""
    need = lib().gc_muon_workspace_bytes(mats)
    return torch.full((need + 64,), 255, dtype=torch.uint8, device=DEV)


def step(grads, mems=None, beta=0.9, out_dtype=torch.float32, scales=None, **kw):
    """One call on copies: (outs, mems), on the host; guards behind every buffer that is written."""
    gc = lib()
    mats, outs, held = [], [], []
    for i, g in enumerate(grads):
        n, m = g.shape
        out = torch.full((n * m + 8,), 7.0, dtype=out_dtype, device=DEV)
        mem = None
        if mems is not None and mems[i] is not None:
            mem = torch.full((n * m + 4,), 7.0, device=DEV)
            mem[: n * m] = to_dev(mems[i]).view(-1)
        outs.append(out)
        held.append(mem)
        mats.append(gc.MuonMat(to_dev(g.ravel()).view(n, m), out[: n * m].view(n, m), None if mem is None else mem[: n * m].view(n, m),
                               1.0 if scales is None else scales[i]))
    ws = workspace(mats)
    gc.gc_muon_step(mats, beta, ws[: ws.numel() - 64], **kw)
    torch.cuda.synchronize()
    assert bool((ws[ws.numel() - 64:] == 255).all()), "written past the workspace"
    for g, out, mem in zip(grads, outs, held):
        assert bool((out[g.size:] == 7.0).all()) and (mem is None or bool((mem[g.size:] == 7.0).all())), "written past a buffer"
    return ([o[: g.size].view(g.shape).cpu() for g, o in zip(grads, outs)],
            [None if h is None else h[: g.size].view(g.shape).cpu().numpy() for g, h in zip(grads, held)])


def floors(x, big, p, b, c):
    """What the least value of the pairs puts on a step's result, entry by entry: x, big, p the magnitudes of X, A and P."""
    n, m = x.shape
    dx = np.full((n, m), 2.0 ** -37)
    da = x @ dx.T + dx @ x.T + 2.0 ** -36
    dp = b * da + c * (big @ da + da @ big) + 2.0 ** -36
    return p @ dx + dp @ x


def one_step_bound(u, coefs, bf16=False):
    """(the step's result, what it may be off by) in float64, n <= m or not."""
    x = np.asarray(u, np.float64)
    x = x / np.linalg.norm(x)
    turned = x.shape[0] > x.shape[1]
    x = x.T if turned else x
    n, m = x.shape
    a, b, c = (abs(float(np.float32(v))) for v in coefs)
    big = np.abs(x) @ np.abs(x).T
    p = b * big + c * (big @ big)
    e = 9 * 2.0 ** -22 + 3 * (m + 2 * n) * 2.0 ** -23
    d = 9 * 2.0 ** -22 + (3 * n * 2.0 ** -23 if b or c else 0.0)
    bound = 2 * (e * (p @ np.abs(x)) + d * a * np.abs(x) + floors(np.abs(x), big, p + a * np.eye(n), b, c))
    want = oracle.newton_schulz(u, 1, coefs)
    if bf16:
        bound += 2.0 ** -11 * 1.01 * (2 * a * np.abs(x) + (4 * b * big + 6 * c * (big @ big)) @ np.abs(x))
    bound = bound.T if turned else bound
    return want, bound * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want) if bf16 else bound


def steps_bound(u, steps, coefs=USUAL, bf16=False):
    """2-norm (Frobenius) by which `steps` steps may be off when roundings are independent."""
    x = np.asarray(u, np.float64)
    x = (x.T if x.shape[0] > x.shape[1] else x) / np.linalg.norm(x)
    a, b, c = coefs
    norm, most = np.linalg.norm, lambda v: np.linalg.norm(v, 2)                          # noqa: E731

    def product_off(v, w, k):
        return (3 * 2.0 ** -22 + (3 * k) ** 0.5 * 2.0 ** -23) * (norm(v @ w) + norm(np.sqrt((v * v) @ (w * w))))

    off = 0.0
    for k in range(steps):
        n, m = x.shape
        g = x @ x.T
        gg = g @ g
        p = a * np.eye(n) + b * g + c * gg
        g2, p2 = most(g), most(p)
        x2 = g2 ** 0.5
        off_g = product_off(x, x.T, m) + 2 * x2 * 2.0 ** -22 * norm(x) + 2.0 ** -22 * norm(g)
        off_p = abs(b) * off_g + abs(c) * (2 * g2 * off_g + product_off(g, g, n)) + 2.0 ** -22 * norm(p)
        here = off_p * x2 + p2 * 2.0 ** -22 * norm(x) + product_off(p, x, n)
        big = np.abs(x) @ np.abs(x).T
        least = floors(np.abs(x), big, np.abs(p), abs(b), abs(c))
        if bf16 and k == steps - 1:
            one = 2.0 ** -10 * norm(np.sqrt((x * x) @ (x * x).T))
            here += (abs(b) + 2 * abs(c) * g2) * one * x2 + 2.0 ** -11 * (norm(p) * x2 + p2 * norm(x))
        off = 4 * off + 2 * (here + norm(least))
        x = p @ x
    return off * (1 + 2.0 ** -8) + 2.0 ** -8 * norm(x) if bf16 else off


SHAPES = [(1, 1), (1, 2), (2, 1), (1, 700), (700, 1), (3, 5), (31, 33), (32, 32), (33, 31), (64, 576), (576, 64), (63, 65), (65, 129),
          (128, 128), (129, 127), (130, 257), (200, 300), (300, 200), (257, 1000), (1000, 130)]


@pytest.mark.parametrize("coefs", [USUAL, (1.0, 0.0, 0.0), (0.0, 1.0, 0.0), (0.0, 0.0, 1.0)], ids=["usual", "X", "AX", "AAX"])
@pytest.mark.parametrize("n,m", SHAPES)
def test_one_step(n, m, coefs):
    print(f"case: muon one step {n}x{m} {coefs}", flush=True)
    for kind in ("gauss", "low", "rows"):
        u = matrix(n, m, kind)
        want, bound = one_step_bound(u, coefs)
        (got,), _ = step([u], steps=1, coefs=coefs)
        assert np.all(np.abs(got.numpy() - want) <= bound), kind
        assert np.linalg.norm(got.numpy() - want) <= steps_bound(u, 1, coefs), kind
        (got,), _ = step([u], steps=1, coefs=coefs, out_dtype=torch.bfloat16)
        assert np.all(np.abs(got.double().numpy() - want) <= one_step_bound(u, coefs, True)[1]), kind
        assert np.linalg.norm(got.double().numpy() - want) <= steps_bound(u, 1, coefs, True), kind


@pytest.mark.parametrize("n,m", [(3, 5), (33, 31), (300, 200)])
def test_what_the_bounds_notice(n, m):
    """X, A or P without its lo part is past the one-step bounds: in the oracle, each rounded to f16."""
    half = lambda v, s: (v * s).astype(np.float16).astype(np.float64) / s                # noqa: E731
    u = matrix(n, m)
    x = u.astype(np.float64) / np.linalg.norm(u)
    x = x.T if n > m else x
    want, bound = one_step_bound(u, (1.0, 0.0, 0.0))
    assert np.mean(np.abs((half(x, 4096).T if n > m else half(x, 4096)) - want) > bound) > 0.9
    a = half(x @ x.T, 2048)
    assert np.linalg.norm(a @ x - x @ x.T @ x) > 2 * steps_bound(u, 1, (0.0, 1.0, 0.0))
    if max(n, m) < 100:                                      # (A A X of the larger one is near the pairs' least value)
        assert np.linalg.norm(a @ a @ x - x @ x.T @ (x @ x.T @ x)) > 2 * steps_bound(u, 1, (0.0, 0.0, 1.0))
    p = half(3.4445 * np.eye(x.shape[0]) - 4.775 * x @ x.T + 2.0315 * x @ x.T @ (x @ x.T), 2048)
    exact = oracle.newton_schulz(u, 1)
    assert np.linalg.norm(p @ x - (exact.T if n > m else exact)) > 2 * steps_bound(u, 1)


@pytest.mark.parametrize("kind", ["gauss", "low"])
@pytest.mark.parametrize("n,m", SHAPES + [(1024, 1024), (512, 2048), (2048, 300), (700, 1111)])
def test_five_steps(n, m, kind):
    print(f"case: muon five steps {n}x{m} {kind}", flush=True)
    u = matrix(n, m, kind, 1)
    want, off = oracle.newton_schulz(u), steps_bound(u, 5)
    (got,), _ = step([u])
    assert np.linalg.norm(got.numpy() - want) <= off
    (got,), _ = step([u], out_dtype=torch.bfloat16)
    assert np.linalg.norm(got.double().numpy() - want) <= steps_bound(u, 5, bf16=True)


@pytest.mark.parametrize("steps", [1, 2, 3, 6])
def test_steps_and_coefficients(steps):
    print(f"case: muon {steps} steps, coefficients of their own", flush=True)
    u = matrix(100, 160, "gauss", 2)
    coefs = [(1.5, -0.5, 0.0), (2.0, -1.5, 0.5), (3.0, -3.0, 1.0), (1.0, 0.25, -0.25), (1.875, -1.25, 0.375), (0.5, 0.0, 0.0)][:steps]
    want = oracle.newton_schulz(u, steps, coefs)
    (got,), _ = step([u], steps=steps, coefs=coefs, scales=[-2.5])
    # slopes at most 4 here too; a step's own error as the usual coefficients'
    assert np.linalg.norm(got.numpy() / -2.5 - want) <= steps_bound(u, steps)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("nesterov", [True, False])
def test_momentum_bits(dtype, nesterov):
    """The memory bit for bit, the update of u = what the oracle says; lengths that leave one to three entries behind the fours."""
    print(f"case: muon momentum {dtype} nesterov {nesterov}", flush=True)
    shapes = [(1, 1), (3, 3), (5, 7), (2, 9), (127, 131), (130, 128), (1, 16385), (129, 129)]
    grads = [matrix(n, m, "gauss", 3) * np.float32(1e-3) for n, m in shapes]
    grads = [gen.f32_to_bf16_bits(g) for g in grads] if dtype == "bf16" else grads
    mems = [matrix(n, m, "rows", 4) for n, m in shapes]
    mems[3] = None
    outs, after = step(grads, mems, beta=0.95, nesterov=nesterov)
    for g, mem, out, got in zip(grads, mems, outs, after):
        ref = oracle.muon_step(g, mem, 0.95, nesterov)
        assert mem is None or np.array_equal(f32_bits(got), f32_bits(ref["mem"]))
        assert np.linalg.norm(out.numpy() - ref["out"]) <= steps_bound(ref["u"], 5)


def test_zero_not_finite_and_far_scales():
    """Each matrix of a call by itself: zeros, an entry that is not finite, entries near float32's ends."""
    print("case: muon zeros, not finite, far scales", flush=True)
    base = matrix(70, 90, "gauss", 5)
    mats = [base, np.zeros((40, 30), np.float32), base * np.float32(1e-37), base * np.float32(7e37), np.zeros((1, 1), np.float32),
            (base * np.float32(1e-44)).astype(np.float32)]
    for bad in (np.nan, np.inf, -np.inf):
        mats.append(base.copy())
        mats[-1][69, 89] = bad
    outs, _ = step(mats)
    want = oracle.newton_schulz(base)
    off = steps_bound(base, 5)
    for i in (0, 2, 3):
        # the scaling's own rounding is at most 2^-24 of each entry (2^-149 below float32's least normal one)
        exact = oracle.newton_schulz(mats[i])
        assert np.linalg.norm(outs[i].numpy() - exact) <= off
    assert np.linalg.norm(outs[0].numpy() - want) <= off
    assert bool((outs[1] == 0).all()) and bool((outs[4] == 0).all())
    assert bool(outs[5].isfinite().all()) and np.linalg.norm(outs[5].numpy() - oracle.newton_schulz(mats[5])) <= steps_bound(mats[5], 5)
    for o in outs[6:]:
        assert bool(o.isnan().all())


def test_a_set_is_each_alone():
    """More matrices than a launch takes, of many shapes: the same bits as each in a call of its own, twice."""
    print("case: muon 70 matrices in one call", flush=True)
    r = rng(6)
    shapes = [(int(r.integers(1, 200)), int(r.integers(1, 260))) for _ in range(68)] + [(300, 900), (700, 520)]
    grads = [matrix(n, m, "gauss", 6) for n, m in shapes]
    scales = [0.5 + i for i in range(len(shapes))]
    outs, _ = step(grads, scales=scales, out_dtype=torch.bfloat16)
    again, _ = step(grads, scales=scales, out_dtype=torch.bfloat16)
    for i, g in enumerate(grads):
        (alone,), _ = step([g], scales=scales[i:i + 1], out_dtype=torch.bfloat16)
        assert torch.equal(outs[i], again[i]) and torch.equal(outs[i], alone), shapes[i]


def test_side_stream_and_graph():
    """The step on another stream, then in two graphs with buffers of their own, replayed with eager work between: every
    result equals the eager one bit for bit."""
    gc = lib()
    print("case: muon on a side stream and in graphs", flush=True)
    shapes = [(96, 200), (256, 64), (130, 130), (200, 1500)]
    grads = [[matrix(n, m, "gauss", 10 + t) for n, m in shapes] for t in range(4)]

    class Opt:
        def __init__(self):
            self.g = [torch.empty(s, device=DEV) for s in shapes]
            self.m = [torch.zeros(s, device=DEV) for s in shapes]
            self.o = [torch.empty(s, dtype=torch.bfloat16, device=DEV) for s in shapes]
            self.mats = gc.MuonArray([gc.MuonMat(g, o, m) for g, o, m in zip(self.g, self.o, self.m)])
            self.ws = workspace(self.mats)

        def load(self, t):
            for dst, src in zip(self.g, grads[t]):
                dst.copy_(to_dev(src))

        def run(self):
            gc.gc_muon_step(self.mats, 0.9, self.ws)

        def bits(self):
            torch.cuda.synchronize()
            return [f32_bits(t.float()) for t in self.o + self.m]

    eager, steps = Opt(), []
    for t in range(4):
        eager.load(t)
        eager.run()
        steps.append(eager.bits())
    side, other = torch.cuda.Stream(), Opt()
    for t in range(4):
        other.load(t)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other.run()
        torch.cuda.current_stream().wait_stream(side)
        assert all(np.array_equal(p, q) for p, q in zip(other.bits(), steps[t]))
    graphs = []
    for _ in range(2):
        c = Opt()
        c.load(0)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            c.run()
        graphs.append((g, c))
    for t in range(4):
        for g, c in graphs:
            c.load(t)
            g.replay()
        torch.ones(1000, device=DEV).sum().item()
        for _, c in graphs:
            assert all(np.array_equal(p, q) for p, q in zip(c.bits(), steps[t]))


def test_short_workspace():
    gc = lib()
    out = torch.full((64, 96), 3.0, device=DEV)
    mats = gc.MuonArray([gc.MuonMat(to_dev(matrix(64, 96)), out)])
    need = gc.gc_muon_workspace_bytes(mats)
    with pytest.raises(gc.GCError) as e:
        gc.gc_muon_step(mats, 0.9, torch.empty(need - 1, dtype=torch.uint8, device=DEV))
    assert e.value.status == gc.GC_ERR_WORKSPACE
    torch.cuda.synchronize()
    assert bool((out == 3.0).all())


# ---------------------------------------------------------------- together, as they are used

def test_training_steps_in_8_bits():
    """A linear layer over three steps: 8-bit operands from activations, weight and output gradients, the weight's gradient
    over two micro-batches, sent in MXFP4 with memory, decoded, and the orthogonalised update applied; every stage against
    the oracle on what the one before left."""
    gc = lib()
    t, fi, fo = 200, 256, 150
    print(f"case: layer in 8 bits, MXFP4 message, muon update {t}x{fi}x{fo}", flush=True)
    r = rng(20)
    w = to_dev(r.standard_normal((fo, fi), dtype=np.float32) * np.float32(0.05))
    mem, ef = torch.zeros(fo, fi, device=DEV), torch.zeros(fo * fi, device=DEV)
    byte = lambda n: torch.empty(max(16, n), dtype=torch.uint8, device=DEV)          # noqa: E731
    held = lambda a, b, k=1: (byte(gc.gc_fp8_code_bytes(a, b)), byte(gc.gc_fp8_scale_bytes(a, b, k)))    # noqa: E731
    xr, xc, wr, dc = held(t, fi), held(fi, t), held(fo, fi, 128), held(fo, t)
    y, dw, grad = torch.empty(t, fo, dtype=torch.bfloat16, device=DEV), torch.empty(fo, fi, device=DEV), torch.empty(fo, fi, device=DEV)
    msg = (byte(gc.gc_mxfp4_code_bytes(1, fo * fi)), byte(gc.gc_mxfp4_scale_bytes(1, fo * fi)))
    update = torch.empty(fo, fi, dtype=torch.bfloat16, device=DEV)
    mats = gc.MuonArray([gc.MuonMat(grad, update, mem, 0.2)])
    ws, fws = workspace(mats), byte(gc.gc_fp8_matmul_workspace_bytes(fo, fi, t))
    hmem, hef = np.zeros((fo, fi), np.float32), np.zeros(fo * fi, np.float32)
    for s in range(3):
        want = np.zeros((fo, fi))
        for b in range(2):
            x, target = (r.standard_normal(shape, dtype=np.float32) for shape in ((t, fi), (t, fo)))
            gc.gc_fp8_quantize(w, *wr, block_rows=128)
            gc.gc_fp8_quantize(to_dev(x), *xr, *xc)
            gc.gc_fp8_matmul(*xr, *wr, fi, y, b_block_rows=128)
            dy = (y.float() - to_dev(target)) / t
            gc.gc_fp8_quantize(dy, None, None, *dc)
            gc.gc_fp8_matmul(*dc, *xc, t, dw, fws, accumulate=b > 0)
            vx = oracle.fp8_values(*oracle.fp8_quantize(np.ascontiguousarray(x.T)), t)
            vd = oracle.fp8_values(*oracle.fp8_quantize(np.ascontiguousarray(dy.cpu().numpy().T)), t)
            want += vd @ vx.T
        size = np.abs(vd) @ np.abs(vx).T
        got = dw.cpu().numpy()
        assert np.all(np.abs(got - want) <= (2 * t + 2) * 2.0 ** -23 * (2 * size + size.max()))
        gc.gc_mxfp4_ef_encode(dw.view(-1), ef, 1.0, *msg)
        gc.gc_mxfp4_decode(*msg, grad.view(-1))
        ref = oracle.mxfp4_ef_step(hef, got.ravel(), 1.0)
        hef = ref["mem"]
        assert np.array_equal(f32_bits(grad.view(-1)), f32_bits(ref["g"].astype(np.float32)))
        gc.gc_muon_step(mats, 0.9, ws)
        ref = oracle.muon_step(grad.cpu().numpy(), hmem, 0.9, True, scale=0.2)
        hmem = ref["mem"]
        assert np.array_equal(f32_bits(mem), f32_bits(hmem))
        assert np.linalg.norm(update.double().cpu().numpy() - ref["out"]) <= 0.2 * steps_bound(ref["u"], 5, bf16=True)
        w -= 0.02 * update.float()
    # an orthogonalised update beside PowerSGD's factors: the same message through a rank-4 step
    q = to_dev(r.standard_normal((4, fi), dtype=np.float32))
    low = gc.Mat(grad=grad, mem=torch.zeros(fo, fi, device=DEV), q=q, rank=4, out=torch.empty(fo, fi, device=DEV))
    gc.gc_powersgd_ef_step([low], 1.0, byte(gc.gc_powersgd_workspace_bytes([low])))
    again = gc.MuonArray([gc.MuonMat(low.out, update)])
    gc.gc_muon_step(again, 0.0, workspace(again))
    u = low.out.cpu().numpy()
    exact = oracle.newton_schulz(u)
    assert np.linalg.norm(update.double().cpu().numpy() - exact) <= steps_bound(u, 5, bf16=True)


# ---------------------------------------------------------------- large

def one_step_on_device(u, coefs, bf16):
    """one_step_bound in float64 on the device: (the step's result, what it may be off by)."""
    x = u.double()
    x = x / torch.linalg.vector_norm(x)
    turned = x.shape[0] > x.shape[1]
    x = x.t().contiguous() if turned else x
    n, m = x.shape
    a, b, c = (float(np.float32(v)) for v in coefs)
    g = x @ x.t().contiguous()
    p = b * g + c * (g @ g)
    p.diagonal().add_(a)
    want = p @ x
    del g, p
    ax = x.abs()
    big = ax @ ax.t().contiguous()
    square = big @ big
    # the entries of `floors`, at most: every dX is 2^-37
    dx = 2.0 ** -37
    da = dx * (ax.sum(1)[:, None] + ax.sum(1)[None, :]) + 2.0 ** -36
    dp = abs(b) * da + abs(c) * (big @ da + da @ big) + 2.0 ** -36
    pa = abs(b) * big + abs(c) * square
    e = 9 * 2.0 ** -22 + 3 * (m + 2 * n) * 2.0 ** -23
    d = 9 * 2.0 ** -22 + (3 * n * 2.0 ** -23 if b or c else 0.0)
    bound = 2 * (e * (pa @ ax) + d * abs(a) * ax + dx * (pa.sum(1, keepdim=True) + abs(a)) + dp @ ax)
    if bf16:
        bound += 2.0 ** -11 * 1.01 * (2 * abs(a) * ax + (4 * abs(b) * big + 6 * abs(c) * square) @ ax)
    want, bound = (want.t(), bound.t()) if turned else (want, bound)
    return want, bound * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs() if bf16 else bound


# each tile for each product, whole k and parts of it, the last tile cut short, tall ones, sets of both
LARGE = [[(1024, 1024)], [(1000, 4100)], [(700, 5000)], [(2048, 2048)], [(3500, 3000)], [(4097, 4000)], [(5000, 5003)], [(256, 30001)],
         [(1024, 1000), (1024, 1024), (4096, 1024), (1000, 4096), (64, 64)], [(512, 520)] * 16, [(2001, 8000)]]


@pytest.mark.parametrize("shapes", LARGE, ids=lambda s: "+".join(f"{n}x{m}" for n, m in dict.fromkeys(s)))
def test_large_shapes(shapes):
    gc = lib()
    print(f"case: muon large {shapes}", flush=True)
    g = torch.Generator(device=DEV)
    g.manual_seed(len(shapes) + shapes[0][0])
    us = [torch.randn(s, generator=g, device=DEV) * torch.exp2(torch.randint(-3, 1, (s[0], 1), generator=g, device=DEV)) for s in shapes]
    for coefs in (USUAL, (0.0, 1.0, 0.0)):
        for dt in (torch.float32, torch.bfloat16):
            outs = [torch.full((s[0] * s[1] + 8,), 7.0, dtype=dt, device=DEV) for s in shapes]
            mats = gc.MuonArray([gc.MuonMat(u, o[:-8].view(u.shape)) for u, o in zip(us, outs)])
            ws = workspace(mats)
            gc.gc_muon_step(mats, 0.9, ws[: ws.numel() - 64], steps=1, coefs=coefs)
            assert bool((ws[ws.numel() - 64:] == 255).all()) and all(bool((o[-8:] == 7.0).all()) for o in outs), "written past a buffer"
            for u, o in zip(us[:1] + us[-3:], outs[:1] + outs[-3:]):
                want, bound = one_step_on_device(u, coefs, dt == torch.bfloat16)
                assert bool(((o[:-8].view(u.shape).double() - want).abs() <= bound).all())
    # five steps, twice: the same bits, near the formula's in float32
    outs = [[torch.empty_like(u) for u in us] for _ in range(2)]
    for o in outs:
        mats = gc.MuonArray([gc.MuonMat(u, t) for u, t in zip(us, o)])
        gc.gc_muon_step(mats, 0.9, workspace(mats))
    assert all(torch.equal(p, q) for p, q in zip(*outs))
    a, b, c = (float(np.float32(v)) for v in USUAL)
    for u, o in zip(us[-1:], outs[0][-1:]):
        x = (u.t().contiguous() if u.shape[0] > u.shape[1] else u).double()
        x = x / torch.linalg.vector_norm(x)
        for _ in range(5):
            s = x @ x.t().contiguous()
            x = a * x + (b * s + c * (s @ s)) @ x
        x = x.t() if u.shape[0] > u.shape[1] else x
        # what a step rounds, at most 8 * 2^-22 of X with independent roundings, grows four times in each that follows: 341 of them
        assert float((o.double() - x).norm() / x.norm()) <= 341 * 8 * 2.0 ** -22

def test_past_32_bits():
    """The largest square: parts of the workspace and of a held matrix past 2^32 bytes.  One step that gives X back."""
    gc = lib()
    n = m = 40000
    print(f"case: muon {n}x{m}, one step of coefficients 1, 0, 0", flush=True)
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    x = torch.randn(n, m, generator=g, device=DEV, dtype=torch.bfloat16)
    out = torch.empty(n, m, dtype=torch.bfloat16, device=DEV)
    mats = gc.MuonArray([gc.MuonMat(x, out)])
    ws = torch.empty(gc.gc_muon_workspace_bytes(mats), dtype=torch.uint8, device=DEV)
    assert ws.numel() > 2**34
    gc.gc_muon_step(mats, 0.0, ws, steps=1, coefs=(1.0, 0.0, 0.0))
    norm = torch.zeros((), dtype=torch.float64, device=DEV)
    for i in range(0, n, 4000):
        norm += x[i:i + 4000].double().square().sum()
    norm = norm.sqrt()
    for i in range(0, n, 4000):
        want = x[i:i + 4000].double() / norm
        # 2^-8 for the rounding to bf16, 2^-11 for X's hi part, and its least value's half, 2^-37 (P is 1: exact)
        assert bool(((out[i:i + 4000].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -10) * want.abs() + 2.0 ** -36).all())
    del x, out, ws, mats
    torch.cuda.empty_cache()


@pytest.mark.parametrize("n,m", [(1, 1 << 22), (1 << 22, 3), (40, 1 << 20)])
def test_long_sides(n, m):
    print(f"case: muon {n}x{m}", flush=True)
    u = matrix(n, m, "gauss", 30)
    want, bound = one_step_bound(u, USUAL)
    (got,), _ = step([u], steps=1, coefs=USUAL)
    assert np.all(np.abs(got.numpy() - want) <= bound)
