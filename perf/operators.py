"""The MXFP4 operators as they are measured: error-feedback encode, decode, quantisation of matrices, and the product.

An MXFP4 matrix of `rows` x `cols` entries is held row by row in groups of 128 columns: 64 bytes of E2M1 codes
(two a byte, the lower column in the low four bits) and 4 scale bytes (E8M0, one per 32 columns) a group.  Columns past
`cols` in the last group are zero codes; a block without entries has the scale byte 0.  A vector is one row.

A block's scale byte is max(E - 2, 0), E the biased float32 exponent of its largest magnitude; codes are the entries
over the scale 2^(byte - 127), rounded to the nearest E2M1 value (ties to the even code), at most 6 in magnitude.
"""
import math

import numpy as np
import torch

own = False

_LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # a small vector with its memory (10,000 entries, the smallest step of the benchmark): latency counts
        {"name": "ef encode 10000 f32", "op": "ef", "d": 10_000, "dtype": "f32", "eta": 0.1},
        # the benchmark's flat gradient of 25.6M entries
        {"name": "ef encode 25.6M f32", "op": "ef", "d": 25_600_000, "dtype": "f32", "eta": 1.0},
        # the gradient of BERT-large's embedding, 30522 x 1024
        {"name": "ef encode 31.3M bf16", "op": "ef", "d": 30522 * 1024, "dtype": "bf16", "eta": 1.0},
        # one message added to a gradient vector of odd length
        {"name": "decode add 100003 f32", "op": "decode", "rows": 1, "cols": 100_003, "msgs": 1, "dtype": "f32", "add": True},
        # the messages of eight workers for a 4096 x 1024 layer, averaged
        {"name": "decode mean 8x4096x1024", "op": "decode", "rows": 4096, "cols": 1024, "msgs": 8, "dtype": "f32", "add": False},
        # the activations of a few tokens, along the features
        {"name": "quantize 16x1024 bf16", "op": "quantize", "rows": 16, "cols": 1024, "pitch": 1024, "dtype": "bf16", "form": "rows"},
        # odd sizes, rows further apart than their length, both directions in one call
        {"name": "quantize 1003x1155 f32", "op": "quantize", "rows": 1003, "cols": 1155, "pitch": 1160, "dtype": "f32", "form": "both"},
        # the activations of 8192 tokens: along the features for the forward product, along the tokens for the weight's gradient
        {"name": "quantize 8192x4096 bf16", "op": "quantize", "rows": 8192, "cols": 4096, "pitch": 4096, "dtype": "bf16", "form": "both"},
        # one token through a 4096 x 1024 layer
        {"name": "matmul 1x4096x1024", "op": "matmul", "m": 1, "n": 4096, "k": 1024, "dtype": "bf16", "add": False},
        # odd sizes in every direction
        {"name": "matmul 777x1001x1155", "op": "matmul", "m": 777, "n": 1001, "k": 1155, "dtype": "bf16", "add": False},
        # the gradient of a 4096 x 1024 weight over 8192 tokens, added to the one of earlier micro-batches
        {"name": "matmul add 4096x1024x8192", "op": "matmul", "m": 4096, "n": 1024, "k": 8192, "dtype": "f32", "add": True},
        # the largest product
        {"name": "matmul 8192x8192x8192", "op": "matmul", "m": 8192, "n": 8192, "k": 8192, "dtype": "bf16", "add": False},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["ef", "decode", "quantize", "matmul", "matmul"])
    dtype = rng.choice(["f32", "bf16"])
    if op == "ef":
        return {"op": op, "d": _log(rng, 1000, 30_000_000), "dtype": dtype, "eta": rng.choice([1.0, 0.1])}
    if op == "decode":
        cols, msgs = _log(rng, 64, 8192), rng.choice([1, 1, 2, 3, 4, 8])
        return {"op": op, "rows": _log(rng, 1, 33_000_000 // (cols * msgs)), "cols": cols, "msgs": msgs, "dtype": dtype, "add": rng.random() < 0.5}
    if op == "quantize":
        cols = _log(rng, 64, 8192)
        pitch = cols + rng.choice([0, 0, 1, 8, 64])
        return {"op": op, "rows": _log(rng, 1, 30_000_000 // cols), "cols": cols, "pitch": pitch, "dtype": dtype,
                "form": rng.choice(["rows", "columns", "both"])}
    m, n, k = _log(rng, 1, 6000), _log(rng, 256, 6000), _log(rng, 128, 8192)
    return {"op": op, "m": m, "n": n, "k": k, "dtype": dtype, "add": rng.random() < 0.3}


# ---------------------------------------------------------------- the plain form

def _blocks(x):
    """float32 [rows, cols] -> [rows, groups * 4, 32], zeros past the columns."""
    rows, cols = x.shape
    return torch.nn.functional.pad(x, (0, -cols % 128)).reshape(rows, -1, 32)


def _power(biased):
    """2^(biased - 127) in float32 from its bits, for biased in 0 .. 254."""
    return torch.where(biased > 0, biased << 23, torch.full_like(biased, 1 << 22)).view(torch.float32)


def _quantize(x):
    """float32 [rows, cols] -> (E2M1 code indices as int8 with the sign in bit 3 [rows, blocks, 32], scale bytes [rows, blocks])."""
    b = _blocks(x)
    top = b.abs().amax(2)
    exponent = torch.frexp(top).exponent - 1 + 127 - 2
    byte = torch.where(top > 0, exponent, torch.zeros_like(exponent)).clamp_min(0)
    v = b * _power(254 - byte)[..., None]
    a = v.abs()
    code = ((a > 0.25).to(torch.int8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5))
    return torch.where(v < 0, code + 8, code), byte


def _values(code, byte, cols):
    """The float32 values that codes and scales stand for, [rows, cols]."""
    level = torch.tensor(_LEVELS + tuple(-v for v in _LEVELS), device=code.device)[code.long()]
    return (level * _power(byte)[..., None]).reshape(code.shape[0], -1)[:, :cols]


def _pack(code, byte):
    """Code indices and scale bytes as they are held: uint8 [rows, 64 groups] and [rows, 4 groups]."""
    c = code.reshape(code.shape[0], -1).to(torch.uint8)
    return c[:, 0::2] | (c[:, 1::2] << 4), byte.to(torch.uint8)


def _unpack(codes, scales, cols):
    """The float32 values of a held matrix, [rows, cols]."""
    c = torch.stack((codes & 15, codes >> 4), dim=2).reshape(codes.shape[0], -1, 32)
    return _values(c, scales.int(), cols)


# ---------------------------------------------------------------- inputs

def _gaussian(gen, rows, cols, sigma, dtype=torch.float32):
    """Normal values whose spread differs from row to row, as a layer's gradients and activations have them."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    s = torch.exp(torch.randn(rows, 1, generator=gen, device="cuda")) * sigma
    return (x * s).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op, dtype = case["op"], _TYPES[case["dtype"]]
    state = {"case": case}
    if op == "ef":
        state["grad"] = _gaussian(gen, 1, case["d"], 1e-3, dtype)[0]
        state["mem"] = _gaussian(gen, 1, case["d"], 3e-4)[0]
    elif op == "decode":
        rows, cols, msgs = case["rows"], case["cols"], case["msgs"]
        held = _pack(*_quantize(_gaussian(gen, msgs * rows, cols, 1e-3)))
        state["codes"], state["scales"] = held[0].reshape(msgs, -1), held[1].reshape(msgs, -1)
        state["out"] = _gaussian(gen, rows, cols, 1e-3, dtype)
    elif op == "quantize":
        state["x"] = _gaussian(gen, case["rows"], case["pitch"], 1.0, dtype)[:, : case["cols"]]
    else:
        m, n, k = case["m"], case["n"], case["k"]
        state["a"] = _pack(*_quantize(_gaussian(gen, m, k, 1.0)))
        state["b"] = _pack(*_quantize(_gaussian(gen, n, k, 0.02)))
        state["out"] = _gaussian(gen, m, n, 1.0, dtype)
    return state


# ---------------------------------------------------------------- one pass

def _run_plain(state):
    case = state["case"]
    op, dtype = case["op"], _TYPES[case["dtype"]]
    if op == "ef":
        step = state["grad"].float() * torch.tensor(case["eta"], dtype=torch.float32).item()
        acc = state["mem"] + step
        value = _values(*_quantize(acc[None]), case["d"])[0]
        state["mem"].copy_(acc - value)
        return {"sent": value, "mem": state["mem"]}
    if op == "decode":
        rows, cols, msgs = case["rows"], case["cols"], case["msgs"]
        value = _unpack(state["codes"].reshape(msgs * rows, -1), state["scales"].reshape(msgs * rows, -1), cols)
        total = value.reshape(msgs, rows, cols).sum(0) * (1.0 / msgs)
        state["out"].copy_(state["out"].float() + total if case["add"] else total)
        return state["out"]
    if op == "quantize":
        x, got = state["x"].float(), {}
        if case["form"] != "columns":
            got["rows"] = _values(*_quantize(x), case["cols"])
        if case["form"] != "rows":
            got["columns"] = _values(*_quantize(x.t().contiguous()), case["rows"])
        return {name: v.to(torch.bfloat16) for name, v in got.items()}
    a, b = _unpack(*state["a"], case["k"]), _unpack(*state["b"], case["k"])
    y = a @ b.t()
    state["out"].copy_(state["out"].float() + y if case["add"] else y)
    return state["out"]


def _kept(state):
    """The buffers that a program keeps beside its data: messages, workspace, outputs."""
    import gradient_compression_error_amd as gc
    case = state["case"]
    op = case["op"]
    byte = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")  # noqa: E731
    held = lambda r, c: (byte(gc.gc_mxfp4_code_bytes(r, c)), byte(gc.gc_mxfp4_scale_bytes(r, c)))  # noqa: E731
    kept = {"gc": gc}
    if op == "ef":
        kept["message"] = held(1, case["d"])
        kept["sent"] = torch.empty(case["d"], device="cuda")
    elif op == "quantize":
        rows, cols = case["rows"], case["cols"]
        if case["form"] != "columns":
            kept["rows"] = held(rows, cols)
            kept["rows values"] = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
        if case["form"] != "rows":
            kept["columns"] = held(cols, rows)
            kept["columns values"] = torch.empty(cols, rows, dtype=torch.bfloat16, device="cuda")
    elif op == "matmul":
        kept["ws"] = byte(max(16, gc.gc_mxfp4_matmul_workspace_bytes(case["m"], case["n"], case["k"])))
    return kept


def _run_own(state):
    case = state["case"]
    op = case["op"]
    if "kept" not in state:
        state["kept"] = _kept(state)
    kept = state["kept"]
    gc = kept["gc"]
    if op == "ef":
        # the step of one worker: its message, and the values that the message stands for
        gc.gc_mxfp4_ef_encode(state["grad"], state["mem"], case["eta"], *kept["message"])
        gc.gc_mxfp4_decode(*kept["message"], kept["sent"])
        return {"sent": kept["sent"], "mem": state["mem"]}
    if op == "decode":
        gc.gc_mxfp4_decode(state["codes"], state["scales"], state["out"], weight=1.0 / case["msgs"], accumulate=case["add"])
        return state["out"]
    if op == "quantize":
        # the matrices are returned as the values that they stand for (every one of them is a bf16 value)
        gc.gc_mxfp4_quantize(state["x"], *kept.get("rows", (None, None)), *kept.get("columns", (None, None)))
        got = {}
        for name in ("rows", "columns"):
            if name in kept:
                gc.gc_mxfp4_decode(*kept[name], kept[name + " values"])
                got[name] = kept[name + " values"]
        return got
    gc.gc_mxfp4_matmul(*state["a"], *state["b"], case["k"], state["out"], kept["ws"], accumulate=case["add"])
    return state["out"]


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    op, size = case["op"], 4 if case["dtype"] == "f32" else 2
    held = 17 / 32
    if op == "ef":
        # gradient and memory read, memory and message written; the message read, its values written
        return {"bytes": case["d"] * (size + 8 + 2 * held + 4), "flops": case["d"] * 10}
    if op == "decode":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (case["msgs"] * held + size * (2 if case["add"] else 1)), "flops": n * (2 * case["msgs"] + 1)}
    if op == "quantize":
        # the matrix read, each form written; the form read, its values written
        n, forms = case["rows"] * case["cols"], 2 if case["form"] == "both" else 1
        return {"bytes": n * (size + forms * (2 * held + 2)), "flops": n * forms * 8}
    m, n, k = case["m"], case["n"], case["k"]
    return {"bytes": (m + n) * k * held + m * n * size * (2 if case["add"] else 1), "flops": 2 * m * n * k}


# ---------------------------------------------------------------- the definition in 64 bits

def _power64(e):
    """2^e in float64 for whole e, from its bits (a library's pow may be off in the last place)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _round64(x, cols):
    """float64 [rows, cols] -> the values of its MXFP4 form: each entry to the nearest multiple of its binade's step."""
    rows = x.shape[0]
    b = torch.zeros(rows, -(-cols // 32) * 32, dtype=torch.float64, device=x.device)
    b[:, :cols] = x
    b = b.view(rows, -1, 32)
    # the entries are float32 values, so a logarithm is either whole or at least 2^-24 below a whole number: what is
    # added keeps the last bit of log2 from mattering
    near = 2.0 ** -40
    scale = torch.floor(torch.log2(b.abs().amax(2).clamp_min(2.0 ** -200)) + near).clamp(-125, 127) - 2
    v = b * _power64(-scale)[..., None]
    binade = torch.floor(torch.log2(v.abs().clamp_min(0.5)) + near).clamp(0, 2)
    step = _power64(binade - 1)
    r = (torch.round(v / step) * step).clamp(-6, 6)
    return (r * _power64(scale)[..., None]).reshape(rows, -1)[:, :cols]


def _decode64(codes, scales, cols):
    """A held matrix in float64, from the fields of its codes: sign, exponent and mantissa bit."""
    c = torch.empty(codes.shape[0], codes.shape[1] * 2, dtype=torch.int64, device=codes.device)
    c[:, 0::2], c[:, 1::2] = codes % 16, codes // 16
    e, mant = (c // 2) % 4, (c % 2).double()
    v = torch.where(e == 0, 0.5 * mant, (1 + 0.5 * mant) * _power64(e - 1))
    v = torch.where(c >= 8, -v, v)
    return (v * _power64(scales.int() - 127).repeat_interleave(32, dim=1))[:, :cols]


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "ef":
        # the step and the sum are defined with one float32 rounding each
        step = (state["grad"].double() * float(np.float32(case["eta"]))).float().double()
        acc = (state["mem"].double() + step).float().double()
        value = _round64(acc[None], case["d"])[0]
        return {"sent": value, "mem": acc - value}
    if op == "decode":
        rows, cols, msgs = case["rows"], case["cols"], case["msgs"]
        total = torch.zeros(rows, cols, dtype=torch.float64, device="cuda")
        for codes, scales in zip(state["codes"], state["scales"]):
            total += _decode64(codes.view(rows, -1), scales.view(rows, -1), cols)
        total /= msgs
        return state["out"].double() + total if case["add"] else total
    if op == "quantize":
        x, got = state["x"].double(), {}
        if case["form"] != "columns":
            got["rows"] = _round64(x, case["cols"])
        if case["form"] != "rows":
            got["columns"] = _round64(x.t(), case["rows"])
        return got
    a, b = _decode64(*state["a"], case["k"]), _decode64(*state["b"], case["k"])
    y = a @ b.t().contiguous()
    return state["out"].double() + y if case["add"] else y
