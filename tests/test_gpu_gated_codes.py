"""Codes of the gated block's h: those of the binary64 value, but where it lies within the f32 evaluation's error of the
border between two codes.

gate and up are sums of MXFP4 products that f32 holds exactly.  s = 1 / (1 + exp(-z)) is within 6 + 0.05 |z| units of
2^-24, and the three products of w (g s u) round by one unit each: h is within (9 + 0.05 |z|) 2^-24 of its value before
it is quantized, which is one rounding.
"""
import numpy as np
import pytest
import torch

from block_scaled_precision_token_amd import ops
from tests import mx_reference as mx
from tests.gpu_util import to_dev

pytestmark = pytest.mark.gpu

GRIDS = {ops.FMT_MXFP8: (mx.E4M3[:127], 448.0, 119), ops.FMT_MXFP4: (mx.VALUES, 6.0, 125)}


def check_codes(codes, scales, h, tol, fmt):
    """tol: relative error of each value of h before its rounding.  Returns how many codes are not h's own."""
    grid, top, last = GRIDS[fmt]
    blocks = lambda a: a.reshape(a.shape[0], a.shape[1] // 32, 32).max(2)  # noqa: E731
    k = scales.astype(np.int64) - 127
    assert (k <= mx.block_exponent(blocks(np.abs(h) * (1 + tol)), top, -127, last)).all()
    assert (k >= mx.block_exponent(blocks(np.abs(h) * (1 - tol)), top, -127, last)).all()
    y = np.minimum(np.abs(h) * np.exp2(-k.astype(np.float64)).repeat(32, 1), top)
    if fmt == ops.FMT_MXFP4:
        codes = np.stack([codes & 15, codes >> 4], -1).reshape(h.shape)
    sign = 8 if fmt == ops.FMT_MXFP4 else 128
    mag = codes & (sign - 1)
    assert ((codes >= sign) == np.signbit(h))[y > 0].all()
    mid = np.concatenate([[-1.0], (grid[1:] + grid[:-1]) / 2, [np.inf]])
    lo, hi = mid[mag], mid[mag + 1]
    bad = (y * (1 + tol) < lo) | (y * (1 - tol) > hi)
    assert not bad.any(), (int(bad.sum()), y[bad][:4], mag[bad][:4])
    return int(((y < lo) | (y > hi)).sum())


@pytest.mark.parametrize("h_fmt", [ops.FMT_MXFP8, ops.FMT_MXFP4])
@pytest.mark.parametrize("tile", [32, 128])
@pytest.mark.parametrize("far", [False, True])
def test_codes_of_h(far, tile, h_fmt):
    """far: gates between -78 and -5, each shared by a block of 32 columns, so that no value is lost beside its block's
    maximum; else gates of a few units."""
    R, I, K = 4096, 512, 32
    rng = np.random.default_rng(11)
    ac = rng.integers(0, 256, (R, K // 2)).astype(np.uint8)
    wc = rng.integers(0, 256, (2 * I, K // 2)).astype(np.uint8)
    as_ = np.full((R, 1), 127, np.uint8)
    ws = np.full((2 * I, 1), 124, np.uint8)
    if far:
        wc[:I] = wc[:I:32].repeat(32, 0)
        ac &= 0x77                         # positive tokens, negative gate weights
        wc[:I] |= 0x88
        wc[:I, :3] = 0
        ws[:I] = 125
    else:
        ws[:I] = 121
    av, wv = mx.mxfp4_values(ac, as_), mx.mxfp4_values(wc, ws)
    h13 = av @ wv.T
    g = h13[:, :I]
    if far:
        assert -85 < g.min() < -70 and g.max() < 0
    w = (rng.random(R) + 0.1).astype(np.float32)
    out = ops.moe_gated(ops.FMT_MXFP4, *(to_dev(t) for t in (ac, as_, wc, ws, np.array([0, R], np.int64))), I, K,
                        row_weights=to_dev(w), h_fmt=h_fmt, tile=tile)
    h, _, _ = mx.gated(h13, w)
    check_codes(out["codes"].cpu().numpy(), out["scales"].cpu().numpy(), h, (9 + 0.05 * np.abs(g)) * 2.0 ** -24, h_fmt)
