"""The 8-bit operators and the orthogonalised update as they are measured: quantisation, product, and the update step.

An 8-bit matrix of `rows` x `cols` entries holds one E4M3 code a byte, row by row, each row in groups of 128 columns; codes
past `cols` in the last group are zero.  One E8M0 byte s stands for the scale 2^(s - 127) of a block: 128 columns of one
row (`block` 1), or of 128 rows (`block` 128).  The scale bytes of a row of blocks are padded with zeros to a multiple of 4.

A block's scale is the least power of two, 2^-127 at least, that takes its largest magnitude to at most 448; codes are the
entries over the scale, rounded to the nearest E4M3 value (ties to the even code).

The update step: mem = beta mem + grad; u = grad + beta mem (Nesterov) or mem; X = u / |u|, |u| the root of the sum of its
squares; then `steps` times, with A = X X^T, X = a X + (b A + c A A) X; the update is scale X.
"""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
_COEFS = (3.4445, -4.7750, 2.0315)


def listed():
    return [
        # the activations of a few tokens, on the way to a product: latency counts
        {"name": "quantize 16x1024 bf16", "op": "quantize", "rows": 16, "cols": 1024, "pitch": 1024, "dtype": "bf16", "form": "rows", "block": 1},
        # odd sizes, rows further apart than their length, both directions in one call
        {"name": "quantize 1003x1155 f32", "op": "quantize", "rows": 1003, "cols": 1155, "pitch": 1160, "dtype": "f32", "form": "both", "block": 1},
        # a 4096 x 1024 weight in blocks of 128 x 128, for the forward product and for the input's gradient
        {"name": "quantize tiles 4096x1024 f32", "op": "quantize", "rows": 4096, "cols": 1024, "pitch": 1024, "dtype": "f32", "form": "both", "block": 128},
        # the activations of 8192 tokens: along the features for the forward product, along the tokens for the weight's gradient
        {"name": "quantize 8192x4096 bf16", "op": "quantize", "rows": 8192, "cols": 4096, "pitch": 4096, "dtype": "bf16", "form": "both", "block": 1},
        # one token through a 4096 x 1024 layer
        {"name": "matmul 1x4096x1024", "op": "matmul", "m": 1, "n": 4096, "k": 1024, "block": 128, "dtype": "bf16", "add": False},
        # odd sizes in every direction
        {"name": "matmul 777x1001x1155", "op": "matmul", "m": 777, "n": 1001, "k": 1155, "block": 128, "dtype": "bf16", "add": False},
        # the gradient of a 4096 x 1024 weight over 8192 tokens, added to the one of earlier micro-batches
        {"name": "matmul add 4096x1024x8192", "op": "matmul", "m": 4096, "n": 1024, "k": 8192, "block": 1, "dtype": "f32", "add": True},
        # the largest product
        {"name": "matmul 8192x8192x8192", "op": "matmul", "m": 8192, "n": 8192, "k": 8192, "block": 128, "dtype": "bf16", "add": False},
        # one small weight (a 64 x 576 convolution): latency counts
        {"name": "muon 64x576", "op": "muon", "shapes": "64x576", "dtype": "f32", "beta": 0.95, "nesterov": True},
        # a set of odd shapes, wide and tall, bf16 gradients, no Nesterov term
        {"name": "muon odd set", "op": "muon", "shapes": "777x301,130x1155,1001x67,300x300", "dtype": "bf16", "beta": 0.9, "nesterov": False},
        # the six matrices of a transformer layer of width 1024
        {"name": "muon layer 1024", "op": "muon", "shapes": "1024x1024,1024x1024,1024x1024,1024x1024,4096x1024,1024x4096", "dtype": "f32", "beta": 0.95, "nesterov": True},
        # the largest: one 4096 x 4096 matrix
        {"name": "muon 4096x4096", "op": "muon", "shapes": "4096x4096", "dtype": "bf16", "beta": 0.95, "nesterov": True},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["quantize", "matmul", "matmul", "muon"])
    dtype = rng.choice(["f32", "bf16"])
    if op == "quantize":
        cols = _log(rng, 64, 8192)
        pitch = cols + rng.choice([0, 0, 1, 8, 64])
        return {"op": op, "rows": _log(rng, 1, 30_000_000 // cols), "cols": cols, "pitch": pitch, "dtype": dtype,
                "form": rng.choice(["rows", "columns", "both"]), "block": rng.choice([1, 1, 128])}
    if op == "matmul":
        m, n, k = _log(rng, 1, 6000), _log(rng, 256, 6000), _log(rng, 128, 8192)
        return {"op": op, "m": m, "n": n, "k": k, "block": rng.choice([1, 128]), "dtype": dtype, "add": rng.random() < 0.3}
    shapes, left = [], 9e10
    for _ in range(rng.choice([1, 1, 2, 3, 6])):
        n, m = _log(rng, 32, 2048), _log(rng, 32, 4096)
        left -= min(n, m) ** 2 * max(n, m)
        if left > 0 or not shapes:
            shapes.append("%dx%d" % (n, m))
    return {"op": op, "shapes": ",".join(shapes), "dtype": dtype, "beta": rng.choice([0.9, 0.95]), "nesterov": rng.random() < 0.7}


def _shapes(case):
    return [tuple(int(v) for v in s.split("x")) for s in case["shapes"].split(",")]


# ---------------------------------------------------------------- the plain form

def _power(biased):
    """2^(biased - 127) in float32 from its bits, for biased in 0 .. 254."""
    return torch.where(biased > 0, biased << 23, torch.full_like(biased, 1 << 22)).view(torch.float32)


def _quantize(x, block):
    """float32 [rows, cols] -> (scaled and rounded entries, scale bytes), in blocks [row blocks, block, groups, 128]."""
    rows, cols = x.shape
    b = torch.nn.functional.pad(x, (0, -cols % 128, 0, -rows % block)).reshape(-(-rows // block), block, -1, 128)
    top = b.abs().amax((1, 3), keepdim=True)
    f, e = torch.frexp(top)                                  # top = f 2^e, f in [0.5, 1): 448 is 0.875 * 2^9
    byte = torch.where(top > 0, e - 9 + (f > 0.875).int() + 127, torch.zeros_like(e)).clamp_min(0)
    v = b * _power(254 - byte)
    step = _power(torch.frexp(v).exponent.clamp_min(-5) - 4 + 127)   # of the binade, at least that of 2^-6
    return torch.round(v / step) * step, byte


def _values(v, byte, rows, cols):
    """The float32 values that scaled entries and scales stand for, [rows, cols]."""
    return (v * _power(byte)).reshape(-1, v.shape[2] * 128)[:rows, :cols]


def _pack(v, byte, rows):
    """A matrix as it is held: uint8 [rows, 128 groups] and [row blocks, groups padded to a multiple of 4]."""
    codes = v.reshape(-1, v.shape[2] * 128)[:rows].to(torch.float8_e4m3fn).view(torch.uint8).contiguous()
    scales = torch.nn.functional.pad(byte[:, 0, :, 0], (0, -v.shape[2] % 4)).to(torch.uint8).contiguous()
    return codes, scales


def _unpack(codes, scales, block, cols):
    """The float32 values of a held matrix, [rows, cols]."""
    rows, groups = codes.shape[0], codes.shape[1] // 128
    s = _power(scales[:, :groups].int()).repeat_interleave(block, 0)[:rows]
    return (codes.view(torch.float8_e4m3fn).float().reshape(rows, groups, 128) * s[..., None]).reshape(rows, -1)[:, :cols]


# ---------------------------------------------------------------- inputs

def _gaussian(gen, rows, cols, sigma, dtype=torch.float32):
    """Normal values whose spread differs from row to row, as a layer's gradients and activations have them."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    s = torch.exp(torch.randn(rows, 1, generator=gen, device="cuda")) * sigma
    return (x * s).to(dtype)


def _gradient(gen, rows, cols, dtype):
    """A weight's gradient: a few strong directions over noise."""
    r = min(16, rows, cols)
    s = 2.0 ** -torch.arange(r, device="cuda", dtype=torch.float32)
    g = (torch.randn(rows, r, generator=gen, device="cuda") * s) @ torch.randn(r, cols, generator=gen, device="cuda")
    return ((g + torch.randn(rows, cols, generator=gen, device="cuda") * 0.3) * 1e-3).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op, dtype = case["op"], _TYPES[case["dtype"]]
    state = {"case": case}
    if op == "quantize":
        state["x"] = _gaussian(gen, case["rows"], case["pitch"], 1.0, dtype)[:, : case["cols"]]
    elif op == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        state["a"] = _pack(*_quantize(_gaussian(gen, m, k, 1.0), 1), m)
        state["b"] = _pack(*_quantize(_gaussian(gen, n, k, 0.02), case["block"]), n)
        state["out"] = _gaussian(gen, m, n, 1.0, dtype)
    else:
        state["grad"] = [_gradient(gen, n, m, dtype) for n, m in _shapes(case)]
        state["mem"] = [_gradient(gen, n, m, torch.float32) for n, m in _shapes(case)]
    return state


# ---------------------------------------------------------------- one pass

def _orthogonal(u):
    """Five Newton-Schulz steps on a float32 matrix, on its shorter side."""
    a, b, c = _COEFS
    x = u / u.double().square().sum().sqrt().float()
    x = x.t().contiguous() if x.shape[0] > x.shape[1] else x
    for _ in range(5):
        g = x @ x.t()
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.t() if u.shape[0] > u.shape[1] else x


def _run_plain(state):
    case = state["case"]
    op, dtype = case["op"], _TYPES[case["dtype"]]
    if op == "quantize":
        x, got, block = state["x"].float(), {}, case["block"]
        if case["form"] != "columns":
            got["rows"] = _values(*_quantize(x, block), case["rows"], case["cols"])
        if case["form"] != "rows":
            got["columns"] = _values(*_quantize(x.t().contiguous(), block), case["cols"], case["rows"])
        return {name: v.to(torch.bfloat16) for name, v in got.items()}
    if op == "matmul":
        y = _unpack(*state["a"], 1, case["k"]) @ _unpack(*state["b"], case["block"], case["k"]).t()
        state["out"].copy_(state["out"].float() + y if case["add"] else y)
        return state["out"]
    update = []
    for grad, mem in zip(state["grad"], state["mem"]):
        g = grad.float()
        mem.mul_(case["beta"]).add_(g)
        update.append(_orthogonal(g + case["beta"] * mem if case["nesterov"] else mem).to(torch.bfloat16))
    return {"update": update, "mem": state["mem"]}


def _kept(state):
    """What a program keeps beside its data: outputs, workspace, and the step's prepared matrices."""
    import gradient_compression_error_amd as gc
    case = state["case"]
    op = case["op"]
    byte = lambda n: torch.empty(max(16, n), dtype=torch.uint8, device="cuda")  # noqa: E731
    held = lambda r, c: (byte(gc.gc_fp8_code_bytes(r, c)), byte(gc.gc_fp8_scale_bytes(r, c, case["block"])))  # noqa: E731
    kept = {"gc": gc}
    if op == "quantize":
        rows, cols = case["rows"], case["cols"]
        if case["form"] != "columns":
            kept["rows"] = held(rows, cols)
            kept["rows values"] = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
        if case["form"] != "rows":
            kept["columns"] = held(cols, rows)
            kept["columns values"] = torch.empty(cols, rows, dtype=torch.bfloat16, device="cuda")
    elif op == "matmul":
        kept["ws"] = byte(gc.gc_fp8_matmul_workspace_bytes(case["m"], case["n"], case["k"]))
    else:
        kept["update"] = [torch.empty(n, m, dtype=torch.bfloat16, device="cuda") for n, m in _shapes(case)]
        mats = [gc.MuonMat(g, out, mem) for g, out, mem in zip(state["grad"], kept["update"], state["mem"])]
        kept["mats"] = gc.MuonArray(mats)
        kept["ws"] = byte(gc.gc_muon_workspace_bytes(kept["mats"]))
    return kept


def _run_own(state):
    case = state["case"]
    op = case["op"]
    if "kept" not in state:
        state["kept"] = _kept(state)
    kept = state["kept"]
    gc = kept["gc"]
    if op == "quantize":
        # the matrices are returned as the values that they stand for (every one of them is a bf16 value)
        gc.gc_fp8_quantize(state["x"], *kept.get("rows", (None, None)), *kept.get("columns", (None, None)), block_rows=case["block"])
        got = {}
        for name in ("rows", "columns"):
            if name in kept:
                gc.gc_fp8_dequantize(*kept[name], kept[name + " values"], block_rows=case["block"])
                got[name] = kept[name + " values"]
        return got
    if op == "matmul":
        gc.gc_fp8_matmul(*state["a"], *state["b"], case["k"], state["out"], kept["ws"], b_block_rows=case["block"], accumulate=case["add"])
        return state["out"]
    gc.gc_muon_step(kept["mats"], case["beta"], kept["ws"], nesterov=case["nesterov"], steps=5)
    return {"update": kept["update"], "mem": state["mem"]}


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    op, size = case["op"], 4 if case["dtype"] == "f32" else 2
    if op == "quantize":
        # the matrix read, each form written; the form read, its values written
        n, forms = case["rows"] * case["cols"], 2 if case["form"] == "both" else 1
        return {"bytes": n * (size + forms * 4), "flops": n * forms * 8}
    if op == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": (m + n) * k + m * n * size * (2 if case["add"] else 1), "flops": 2 * m * n * k}
    # gradient read, memory read and written, update written; a step multiplies X by its transpose and A by itself, both
    # symmetric (half of the entries), and the result by X
    sizes = [(min(s), max(s)) for s in _shapes(case)]
    return {"bytes": sum(n * m for n, m in sizes) * (size + 8 + 2), "flops": sum(5 * (3 * n * n * m + n ** 3) for n, m in sizes)}


# ---------------------------------------------------------------- the definition in 64 bits

def _power64(e):
    """2^e in float64 for whole e, from its bits (a library's pow may be off in the last place)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _round64(x, block):
    """float64 [rows, cols] -> the values of its 8-bit form: each entry to the nearest multiple of its binade's step."""
    rows, cols = x.shape
    down, along = -(-rows // block), -(-cols // 128)
    b = torch.zeros(down * block, along * 128, dtype=torch.float64, device=x.device)
    b[:rows, :cols] = x
    top = b.abs().view(down, block, along, 128).amax(3).amax(1)
    # the entries are float32 values, so a logarithm is either whole or at least 2^-24 from a whole number: what is
    # subtracted or added keeps the last bit of log2 from mattering
    near = 2.0 ** -40
    scale = torch.ceil(torch.log2((top / 448).clamp_min(2.0 ** -200)) - near).clamp(-127, 127)
    scale = scale.repeat_interleave(block, 0).repeat_interleave(128, 1)
    v = b * _power64(-scale)
    binade = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6)) + near)
    step = _power64(binade - 3)
    return (torch.round(v / step) * step * _power64(scale))[:rows, :cols]


def _decode64(codes, scales, block, cols):
    """A held matrix in float64, from the fields of its codes: sign, four exponent bits, three mantissa bits."""
    c = codes.long()
    e, mant = (c // 8) % 16, (c % 8).double()
    v = torch.where(e == 0, mant * 2.0 ** -9, (8 + mant) * _power64(e - 10))
    v = torch.where(c >= 128, -v, v)
    s = _power64(scales.int() - 127).repeat_interleave(128, 1)[:, : c.shape[1]]
    return (v * s[torch.arange(c.shape[0], device=c.device) // block])[:, :cols]


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x, got = state["x"].double(), {}
        if case["form"] != "columns":
            got["rows"] = _round64(x, case["block"])
        if case["form"] != "rows":
            got["columns"] = _round64(x.t(), case["block"])
        return got
    if op == "matmul":
        a, b = _decode64(*state["a"], 1, case["k"]), _decode64(*state["b"], case["block"], case["k"])
        y = a @ b.t().contiguous()
        return state["out"].double() + y if case["add"] else y
    update, kept = [], []
    for grad, mem in zip(state["grad"], state["mem"]):
        beta = case["beta"]
        m = beta * mem.double() + grad.double()
        u = beta * m + grad.double() if case["nesterov"] else m
        tall = u.shape[0] > u.shape[1]
        x = (u.t() if tall else u).contiguous() / torch.linalg.vector_norm(u)
        for _ in range(5):
            # x (a I + b S + c S S), S = x^T x, is the same polynomial from the other side; here from the shorter one
            s = x @ x.t().contiguous()
            p = _COEFS[2] * (s @ s) + _COEFS[1] * s
            p.diagonal().add_(_COEFS[0])
            x = p @ x
        update.append(x.t().contiguous() if tall else x)
        kept.append(m)
    return {"update": update, "mem": kept}
