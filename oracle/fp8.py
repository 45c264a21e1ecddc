"""8-bit quantiser in blocks of 128, its values and the product (oracle, test infrastructure).

Source: the OCP 8-bit Floating Point specification for the element type (E4M3:
bias 7, no infinity, 0x7F / 0xFF NaN, largest magnitude 448), the OCP
Microscaling Formats specification for the scale type (E8M0).

Readings taken:
  * a block is 128 columns of 1 or of 128 rows; its scale is the least power of
    two, at least 2^-127, that takes the largest magnitude to at most 448; a
    block of zeros has the least scale; a block with an entry that is not finite
    has the NaN scale (byte 255) and zero codes;
  * codes round to nearest, ties to the even code, and keep the entry's sign;
    what would so become 2^128, past float32's range, is the value below it;
  * rows are held in groups of 128 columns, pads are zero codes; a row of blocks
    has its scale bytes padded with zeros to a multiple of four.
"""
from __future__ import annotations

import numpy as np


def _magnitudes() -> np.ndarray:
    """The 127 magnitudes in code order, from the fields of the codes."""
    out = []
    for code in range(127):
        e, m = code >> 3, code & 7
        out.append(m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(out)


MAGNITUDES8 = _magnitudes()


def _nearest_code(a: np.ndarray) -> np.ndarray:
    """Index of the magnitude nearest to a in [0, 448]; between two the even index."""
    low = np.clip(np.searchsorted(MAGNITUDES8, a, side="right") - 1, 0, 125)
    d0, d1 = a - MAGNITUDES8[low], MAGNITUDES8[low + 1] - a
    return np.where(d0 < d1, low, np.where(d0 > d1, low + 1, low + (low & 1)))


def fp8_quantize(x: np.ndarray, block_rows: int = 1):
    """[rows, cols] (float32, or uint16 bf16 bits) -> (codes [rows, 128 G], scales [row blocks, 4 ceil(G / 4)])."""
    if x.dtype == np.uint16:
        x = (x.astype(np.uint32) << 16).view(np.float32)
    rows, cols = x.shape
    groups, down = -(-cols // 128), -(-rows // block_rows)
    b = np.zeros((down * block_rows, groups * 128))
    with np.errstate(invalid="ignore"):
        b[:rows, :cols] = np.asarray(x, np.float64)
    b = b.reshape(down, block_rows, groups, 128)
    fine = np.isfinite(b).all((1, 3))
    top = np.where(fine, np.abs(np.where(np.isfinite(b), b, 0.0)).max((1, 3)), 0.0)
    e = np.full(top.shape, -127)
    some = top > 0
    f, ex = np.frexp(top[some] / 448.0)                      # the least e with top / 448 <= 2^e
    guess = np.where(f == 0.5, ex - 1, ex)
    guess = np.where(np.ldexp(448.0, guess - 1) >= top[some], guess - 1, guess)     # (the division may have rounded)
    guess = np.where(np.ldexp(448.0, guess) < top[some], guess + 1, guess)
    e[some] = np.maximum(guess, -127)
    scales = np.zeros((down, -(-groups // 4) * 4), np.uint8)
    scales[:, :groups] = np.where(fine, e + 127, 255)
    ok = fine[:, None, :, None]
    v = np.ldexp(np.where(ok, b, 0.0), -e[:, None, :, None])
    codes = _nearest_code(np.abs(v))
    codes = np.where((codes == 0x78) & (e == 120)[:, None, :, None], 0x77, codes) + 128 * (np.signbit(b) & ok)
    return codes.astype(np.uint8).reshape(down * block_rows, groups * 128)[:rows], scales


def fp8_values(codes: np.ndarray, scales: np.ndarray, cols: int, block_rows: int = 1) -> np.ndarray:
    """The float64 values of a held matrix, [rows, cols]."""
    rows, groups = codes.shape[0], codes.shape[1] // 128
    mags = np.append(MAGNITUDES8, np.nan)
    v = np.where(codes & 128, -1.0, 1.0) * mags[codes & 127]
    s = np.repeat(np.repeat(scales[:, :groups].astype(np.int64), 128, axis=1), block_rows, axis=0)[:rows]
    return np.where(s == 255, np.nan, np.ldexp(v, s - 127))[:, :cols]


def fp8_matmul(a, b, k: int, a_block_rows: int = 1, b_block_rows: int = 1) -> np.ndarray:
    """D8(A) D8(B)^T in float64 for held matrices a = (codes, scales), b = (codes, scales)."""
    return fp8_values(*a, k, a_block_rows) @ fp8_values(*b, k, b_block_rows).T
