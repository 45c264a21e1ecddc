"""The largest float32 values in 8 bits: what is finite stays finite.  The oracle here; the kernels on the GPU."""
import numpy as np
import pytest
import torch

import gen
import oracle

FIRST = np.float32(1.9375 * 2.0 ** 127)                      # 248 at the scale 2^120: the tie between 240 and 256
LAST = np.float32(3.4028235e38)
LARGE = np.array([FIRST, np.nextafter(FIRST, np.float32(0)), LAST, -LAST, -FIRST, 1.875 * 2.0 ** 127, 1.76 * 2.0 ** 127, 2.0 ** 127,
                  1.0, 0.0, -0.0, 3 * 2.0 ** 112], np.float32)
WANT = np.array([0x77, 0x77, 0x77, 0xF7, 0xF7, 0x77, 0x76, 0x70, 0x00, 0x00, 0x80, 0x06], np.uint8)


def test_oracle():
    for block in (1, 128):
        c, s = oracle.fp8_quantize(LARGE[None], block)
        assert s[0, 0] == 247 and np.array_equal(c[0, : LARGE.size], WANT)
        v = oracle.fp8_values(c, s, LARGE.size, block)
        assert np.all(np.isfinite(v.astype(np.float32))) and v.max() == 1.875 * 2.0 ** 127
    # one binade down, the same fractions have a scale of their own and round as anywhere
    c, s = oracle.fp8_quantize((LARGE[:4] / 2)[None])
    assert s[0, 0] == 246 and np.array_equal(c[0, :4], [0x78, 0x77, 0x78, 0xF8])


@pytest.mark.gpu
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 600), (130, 257), (2100, 2048)])
def test_kernels(rows, cols, dtype, block):
    """Codes and scales bit for bit in both directions, finite values, and finite products in either type of out."""
    from gpu_util import DEV, lib, require_gpu, to_dev
    from test_gpu_fp8 import Held, held_from, same
    require_gpu()
    gc = lib()
    print(f"case: fp8 largest values {rows}x{cols} {dtype} block {block}", flush=True)
    r = gen.rng(0, gen.KIND_MISC, 990, rows)
    x = np.where(r.uniform(size=(rows, cols)) < 0.1, LARGE[r.integers(0, LARGE.size, (rows, cols))], 0).astype(np.float32)
    if dtype == "bf16":                                      # cut to bf16: the largest is 1.9921875 * 2^127
        x = (x.view(np.uint32) >> 16).astype(np.uint16)
    xt = to_dev(x.ravel()).view(rows, cols)
    a, b, c = Held(rows, cols, block), Held(rows, cols, block), Held(cols, rows, block)
    gc.gc_fp8_quantize(xt, *a.pair, block_rows=block)
    gc.gc_fp8_quantize(xt, *b.pair, *c.pair, block_rows=block)
    want = oracle.fp8_quantize(x, block)
    same(a, want)
    same(b, want)
    same(c, oracle.fp8_quantize(np.ascontiguousarray(x.T), block))
    for dt in (torch.float32, torch.bfloat16):
        out = torch.empty(rows, cols, dtype=dt, device=DEV)
        gc.gc_fp8_dequantize(*a.pair, out, block_rows=block)
        assert bool(out.isfinite().all())
    # against one code of 2^-6 at the scale 2^-100 in each column's place: sums of up to 2048 terms stay in range
    n = 40
    codes, scales = np.full((n, -(-cols // 128) * 128), 0x08, np.uint8), np.zeros((n, -(-cols // 512) * 4), np.uint8)
    codes[:, cols:] = 0
    scales[:, : -(-cols // 128)] = 27
    for dt in (torch.float32, torch.bfloat16):
        out = torch.empty(rows, n, dtype=dt, device=DEV)
        ws = torch.empty(gc.gc_fp8_matmul_workspace_bytes(rows, n, cols) + 16, dtype=torch.uint8, device=DEV)
        gc.gc_fp8_matmul(*a.pair, *held_from(codes, scales), cols, out, ws, a_block_rows=block)
        assert bool(out.isfinite().all())
