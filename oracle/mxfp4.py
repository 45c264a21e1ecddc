"""MXFP4 quantiser, decode, error-feedback step and product (oracle, test infrastructure).

Source: the OCP Microscaling Formats specification (MXFP4: blocks of 32 E2M1
values with one E8M0 scale) for the format and the scale rule; "Sparsified SGD
with Memory", method section, for the memory: g_t = comp(m_t + eta_t grad_t),
m_{t+1} = m_t + eta_t grad_t - g_t, with comp = the quantiser.

Readings taken:
  * the scale exponent is floor(log2(max |x|)) - 2, at least -127; a block of
    zeros has the least scale; a block with an entry that is not finite has the
    NaN scale (byte 255) and zero codes;
  * codes round to nearest, ties to the even code, saturate at 6 and keep the
    entry's sign;
  * rows are held in groups of 128 columns, pads are zero codes and zero bytes.
"""
from __future__ import annotations

import numpy as np

from .topk_ef import ef_accumulate

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _nearest_code(a: np.ndarray) -> np.ndarray:
    """Index of the magnitude nearest to a >= 0; between two the even index."""
    d = np.abs(a[..., None] - MAGNITUDES)
    best = d.min(-1, keepdims=True)
    tied = d == best
    even = tied & (np.arange(8) % 2 == 0)
    pick = np.where(even.any(-1, keepdims=True), even, tied)
    return pick.argmax(-1)


def mxfp4_quantize(x: np.ndarray):
    """[rows, cols] (float32, or uint16 bf16 bits) -> (codes [rows, 64 G], scales [rows, 4 G])."""
    if x.dtype == np.uint16:
        x = (x.astype(np.uint32) << 16).view(np.float32)
    rows, cols = x.shape
    groups = -(-cols // 128)
    b = np.zeros((rows, groups * 4, 32))
    with np.errstate(invalid="ignore"):
        b.reshape(rows, -1)[:, :cols] = np.asarray(x, np.float64)
    codes = np.zeros((rows, groups * 4, 32), np.uint8)
    scales = np.zeros((rows, groups * 4), np.uint8)
    fine = np.isfinite(b).all(-1)
    top = np.where(fine, np.abs(np.where(np.isfinite(b), b, 0.0)).max(-1), 0.0)
    _, ex = np.frexp(top)                                     # top = f * 2^ex, f in [0.5, 1)
    e = np.where(top > 0, np.maximum(ex - 1 - 2, -127), -127)
    scales[:] = np.where(fine, e + 127, 255)
    v = np.ldexp(np.where(fine[..., None], b, 0.0), -e[..., None])
    codes[:] = _nearest_code(np.abs(v)) + 8 * (np.signbit(b) & fine[..., None])
    flat = codes.reshape(rows, -1)
    return flat[:, 0::2] | (flat[:, 1::2] << 4), scales


def mxfp4_values(codes: np.ndarray, scales: np.ndarray, cols: int) -> np.ndarray:
    """The float64 values of a held matrix, [rows, cols]."""
    rows = scales.shape[0]
    c = np.empty((rows, codes.shape[1] * 2), np.uint8)
    c[:, 0::2], c[:, 1::2] = codes & 15, codes >> 4
    v = np.where(c & 8, -1.0, 1.0) * MAGNITUDES[c & 7]
    s = np.repeat(scales.astype(np.int64), 32, axis=1)
    return np.where(s == 255, np.nan, np.ldexp(v, s - 127))[:, :cols]


def mxfp4_ef_step(mem: np.ndarray, grad: np.ndarray, eta: float) -> dict:
    """One step with memory: {"codes", "scales", "g", "mem"}."""
    acc = ef_accumulate(mem, grad, eta)
    codes, scales = mxfp4_quantize(acc.reshape(1, -1))
    g = mxfp4_values(codes, scales, acc.size)[0]
    return {"acc": acc, "codes": codes, "scales": scales, "g": g,
            "mem": (acc.astype(np.float64) - g).astype(np.float32)}


def mxfp4_decode(codes: np.ndarray, scales: np.ndarray, cols: int, weight: float = 1.0) -> np.ndarray:
    """weight * the sum of the messages' values (codes [nmsg, rows, 64 G], scales [nmsg, rows, 4 G]), float64."""
    total = sum(mxfp4_values(c, s, cols) for c, s in zip(codes, scales))
    return float(np.float32(weight)) * total


def mxfp4_matmul(a, b, k: int) -> np.ndarray:
    """D(A) D(B)^T in float64 for held matrices a = (codes, scales), b = (codes, scales)."""
    return mxfp4_values(*a, k) @ mxfp4_values(*b, k).T

