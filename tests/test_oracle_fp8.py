"""The 8-bit oracle (CPU): hand-worked blocks, the rounding borders, scales and invariants."""
import numpy as np
import pytest

import gen
import oracle
from oracle.fp8 import MAGNITUDES8


def codes_of(row):
    c, s = oracle.fp8_quantize(np.asarray([row], np.float32))
    return c[0, : len(row)].tolist(), int(s[0, 0])


def test_magnitudes():
    # E4M3: 2^-9 steps below 2^-6, largest 448, one at code 0x38
    assert MAGNITUDES8[0] == 0 and MAGNITUDES8[1] == 2.0 ** -9 and MAGNITUDES8[8] == 2.0 ** -6
    assert MAGNITUDES8[0x38] == 1.0 and MAGNITUDES8[126] == 448.0 and np.all(np.diff(MAGNITUDES8) > 0)


def test_hand_block():
    # largest 448: scale 1; the magnitudes are their own codes
    c, s = codes_of([448.0, 1.0, -1.0, 1.125, 0.0, -0.0, 2.0 ** -9, 2.0 ** -6, -448.0])
    assert s == 127 and c == [126, 0x38, 0xB8, 0x39, 0, 128, 1, 8, 254]
    # a hair above 448 takes the next scale, a hair below the same
    assert codes_of([np.nextafter(np.float32(448), np.float32(999))])[1] == 128
    assert codes_of([np.nextafter(np.float32(448), np.float32(0))]) == ([126], 127)
    # 224 still has the scale one half
    assert codes_of([224.0]) == ([126], 126) and codes_of([225.0])[1] == 127


def test_rounding_borders():
    # scale 1: ties between neighbours go to the even code
    mids = (MAGNITUDES8[:-1] + MAGNITUDES8[1:]) / 2
    near = np.stack([np.nextafter(mids.astype(np.float32), np.float32(0)), mids.astype(np.float32),
                     np.nextafter(mids.astype(np.float32), np.float32(999))], 1)
    x = np.full((126, 4), 448, np.float32)
    x[:, 1:] = near
    c, s = oracle.fp8_quantize(x)
    i = np.arange(126)
    assert np.all(s[:, 0] == 127)
    assert np.array_equal(c[:, 1], i) and np.array_equal(c[:, 2], i + (i & 1)) and np.array_equal(c[:, 3], i + 1)


def test_scale_range():
    assert codes_of([3.4028235e38])[1] == 247               # 2^120 * 448 holds it: float32's largest is below 2^128
    assert codes_of([2.0 ** -127]) == ([0x38], 0)           # scale 2^-127
    assert codes_of([2.0 ** -136]) == ([1], 0) and codes_of([2.0 ** -137]) == ([0], 0)
    assert codes_of([0.0, -0.0]) == ([0, 128], 0)


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_not_finite(bad):
    x = np.ones((130, 300), np.float32)
    x[3, 140] = bad
    c, s = oracle.fp8_quantize(x)
    assert s[3].tolist() == [119, 255, 119, 0] and s[4].tolist() == [119, 119, 119, 0] and np.all(c[3, 128:256] == 0)
    c, s = oracle.fp8_quantize(x, 128)
    assert s.tolist() == [[119, 255, 119, 0], [119, 119, 119, 0]]
    v = oracle.fp8_values(c, s, 300, 128)
    assert np.isnan(v[:128, 128:256]).all() and np.all(v[:, :128] == 1) and np.all(v[128:] == 1)


@pytest.mark.parametrize("block", [1, 128])
def test_invariants(block):
    r = gen.rng(0, gen.KIND_MISC, 800, block)
    x = (r.standard_normal((200, 300)) * np.exp2(r.integers(-20, 20, (200, 1)))).astype(np.float32)
    c, s = oracle.fp8_quantize(x, block)
    v = oracle.fp8_values(c, s, 300, block)
    groups = np.repeat(np.repeat(s[:, :3].astype(np.int64), 128, 1), block, 0)[:200, :300]
    step = np.ldexp(1.0, groups - 127)
    # at most half a step: 2^-4 of the magnitude, or 2^-10 scales where the code has no exponent
    assert np.all(np.abs(v - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * step))
    # what is held is held again, bit for bit; the transposed matrix in square blocks has the same values
    c2, s2 = oracle.fp8_quantize(v.astype(np.float32), block)
    assert np.array_equal(oracle.fp8_values(c2, s2, 300, block), v)
    ct, st = oracle.fp8_quantize(np.ascontiguousarray(x.T), 128)
    if block == 128:
        assert np.array_equal(oracle.fp8_values(ct, st, 200, 128), v.T) and np.array_equal(st[:, :2], s[:, :3].T)
