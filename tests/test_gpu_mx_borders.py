"""Codes at the borders between them: for every border of E4M3 and E2M1, at exponents over the whole range, the border
itself (ties to even) and its f32 neighbours, both signs, as gate or up of the checkpoint and as h.

A value n 2^e is given to the block exactly: the digits of n in base 16 lie in K blocks whose scales are 2^e, 2^(e + 4), ..
and up's row c of the weights takes column c of each.  Its digits add up to 24 significant bits, so f32 holds every partial
sum.  gate is 128 from one more block: silu(128) = 128 in f32, so h = 128 up.
"""
import numpy as np
import pytest

from block_scaled_precision_token_amd import ops
from tests import mx_reference as mx
from tests.gpu_util import assert_bytes_equal, to_dev

pytestmark = pytest.mark.gpu

DIGITS, I = 13, 32
K = 32 * (DIGITS + 1)
EXPONENTS = [-90, -77, -50, -13, -1, 0, 1, 7, 40, 77, 100, 110]
NIBBLES = np.array([int(np.argmax(mx.E4M3[:127] == v)) for v in range(16)], np.uint8)


def rows_of(grid, top):
    """(n [R, 32], e [R]): per exponent and binade of borders their values and neighbours, and the block's maximum."""
    mids = (grid[1:] + grid[:-1]) / 2
    binade = np.floor(np.log2(mids)).astype(int)
    rng = np.random.default_rng(1)
    n, e = [], []
    for k in EXPONENTS:
        for b in np.unique(binade):
            t = (mids[binade == b] * 2.0 ** (23 - b)).astype(np.int64)       # 24 bits
            v = np.concatenate([[int(top * 2.0 ** (23 - b))], t, t - 1, t + 1])
            row = np.zeros(32, np.int64)
            row[:len(v)] = v * rng.choice([-1, 1], len(v))
            n.append(row)
            e.append(k + b - 23)
    return np.stack(n), np.array(e)


def operands(n, e, bits):
    R = len(n)
    codes, scales = np.zeros((R, K), np.uint8), np.full((R, K // 32), 127, np.uint8)
    for j in range(DIGITS):
        digit = (np.abs(n) >> (4 * j)) & 15
        codes[:, 32 * j:32 * j + 32] = NIBBLES[digit] | (128 * (n < 0)).astype(np.uint8)
        scales[:, j] = np.where(digit.any(1), 127 + e + 4 * j, 127)
    assert (np.abs(n) >> (4 * DIGITS) == 0).all()
    codes[:, 32 * DIGITS] = 0x70                                             # 128
    one = np.zeros((2 * I, K), np.uint8)
    one[:I, 32 * DIGITS] = 1
    for j in range(DIGITS):
        one[I + np.arange(I), 32 * j + np.arange(I)] = 1
    w = 0x38 * one if bits == 8 else 2 * one[:, ::2] | 32 * one[:, 1::2]
    return codes, scales, w.astype(np.uint8), np.full((2 * I, K // 32), 127, np.uint8)


@pytest.mark.parametrize("h_fmt", [ops.FMT_MXFP8, ops.FMT_MXFP4])
@pytest.mark.parametrize("fmt,bits", [(ops.FMT_MXFP8_MXFP4, 4), (ops.FMT_MXFP8, 8)])
@pytest.mark.parametrize("tile", [32, 128])
def test_codes(tile, fmt, bits, h_fmt):
    n, e = rows_of(mx.E4M3[:127], 448.0) if h_fmt == ops.FMT_MXFP8 else rows_of(mx.VALUES, 6.0)
    values = n * np.exp2(e.astype(float))[:, None]
    assert np.array_equal(values, values.astype(np.float32))
    args = [to_dev(t) for t in (*operands(n, e, bits), np.array([0, len(n)], np.int64))]
    out = ops.moe_gated(fmt, *args, I, K, h_fmt=h_fmt, checkpoint=True, tile=tile)
    c, s = mx.mxfp8(values)
    # a digit's zero may have either sign: what is 0 in the end is +0
    assert_bytes_equal(out["ckpt_codes"].cpu().numpy()[:, I:][n != 0], c[n != 0])
    assert_bytes_equal(out["ckpt_scales"].cpu().numpy()[:, 1:], s)
    assert (out["ckpt_codes"].cpu().numpy()[:, :I] == mx.mxfp8(np.full((1, 32), 128.0))[0][0, 0]).all()
    if h_fmt == ops.FMT_MXFP8:
        c, s = mx.mxfp8(128 * values)
        assert_bytes_equal(out["codes"].cpu().numpy()[n != 0], c[n != 0])
    else:
        c, s = mx.mxfp4(128 * values)
        unpack = lambda b: np.stack([b & 15, b >> 4], -1).reshape(n.shape)  # noqa: E731
        assert_bytes_equal(unpack(out["codes"].cpu().numpy())[n != 0], unpack(c)[n != 0])
    assert_bytes_equal(out["scales"].cpu().numpy(), s)
