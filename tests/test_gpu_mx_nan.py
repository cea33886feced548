"""NaN and infinities through the MX operators: a NaN stays one and stays where it is, an infinity saturates, whatever
the other rows of the batch hold."""
import numpy as np
import pytest
import torch

from block_scaled_precision_token_amd import ops
from tests import mx_reference as mx
from tests.gpu_util import DEV, host, to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu

ROWS, I, K = 40, 32, 64
NAN_ROW, TOP_ROW, LARGE_ROW, INF_ROW = 3, 5, 7, 20
NAN_COLUMNS = [4, I + 9]


def tokens(special):
    """MXFP8 tokens: row 3 with a NaN, row 5 in the largest blocks; special: row 7 makes products past these, row 20
    overflows."""
    rng = np.random.default_rng(1)
    c, s = mx.mxfp8(rng.standard_normal((ROWS, K)))
    c[NAN_ROW, 5] = 0x7F
    c[TOP_ROW], s[TOP_ROW] = 0, 246
    c[TOP_ROW, :2] = 0x70                     # twice 128 x 2^119 times 1.5: 384 x 2^119
    if special:
        c[[LARGE_ROW, INF_ROW]], s[[LARGE_ROW, INF_ROW]] = 0, 246
        c[LARGE_ROW, 0] = 0x7A                # 320 x 2^119, times 1.5: finite, and more than 448 x 2^119
        c[INF_ROW, 0] = 0x7E                  # 448 x 2^119, times 1.5: past 2^128
    return c, s


def weights(bits):
    """1.5 or -1.5 (the first two of a row alike), MXFP8 or MXFP4, and two rows of NaN."""
    sign = np.random.default_rng(2).integers(0, 2, (2 * I, K)).astype(np.uint8)
    sign[:, 1] = sign[:, 0]
    s = np.full((2 * I, K // 32), 127, np.uint8)
    if bits == 8:
        c = 0x3C | (sign << 7)
        c[NAN_COLUMNS, 33] = 0x7F
        return c, s
    s[NAN_COLUMNS, 1] = 255
    c = 3 | (sign << 3)
    return c[:, ::2] | (c[:, 1::2] << 4), s


@pytest.mark.parametrize("fmt", ["a8w4", "mxfp8"])
@pytest.mark.parametrize("tile", [32, 128])
def test_gated_block(tile, fmt):
    f, bits = {"a8w4": (ops.FMT_MXFP8_MXFP4, 4), "mxfp8": (ops.FMT_MXFP8, 8)}[fmt]
    off = to_dev(np.array([0, ROWS], np.int64))
    w = [to_dev(t) for t in weights(bits)]
    outs = []
    for special in (False, True):
        out = ops.moe_gated(f, *(to_dev(t) for t in tokens(special)), *w, off, I, K, checkpoint=True, return_h=True,
                            tile=tile)
        outs.append({k: v.float().cpu().numpy() if k == "h" else v.cpu().numpy() for k, v in out.items()})
    nan = np.zeros((ROWS, 2 * I), bool)
    nan[NAN_ROW] = True
    nan[:, NAN_COLUMNS] = True
    nan_h = nan[:, :I] | nan[:, I:]
    for o in outs:
        assert np.array_equal((o["ckpt_codes"] & 127) == 127, nan)
        assert np.array_equal(np.isnan(o["h"][:TOP_ROW]), nan_h[:TOP_ROW])
        assert np.array_equal((o["codes"][:TOP_ROW] & 127) == 127, nan_h[:TOP_ROW])
        assert (o["ckpt_scales"][TOP_ROW] == 246).all()
        assert ((o["ckpt_codes"][TOP_ROW] & 127) == 0x7C)[~nan[TOP_ROW]].all()        # 384
    for k in outs[0]:
        keep = np.ones(ROWS, bool)
        keep[[LARGE_ROW, INF_ROW]] = False
        assert np.array_equal(outs[0][k][keep], outs[1][k][keep], equal_nan=k == "h"), k
    for row in (LARGE_ROW, INF_ROW):      # +-480 x 2^119 and infinities: +-448 x 2^119
        o = outs[1]
        assert (o["ckpt_scales"][row] == 246).all(), row
        assert ((o["ckpt_codes"][row] & 127) == 0x7E)[~nan[row]].all(), row


@pytest.mark.parametrize("tile", [32, 128])
def test_gated_backward_keeps_a_nan_in_its_row(tile):
    rng = np.random.default_rng(3)
    c, s = mx.mxfp8(rng.standard_normal((ROWS, K)))
    wc, ws = mx.mxfp8(rng.standard_normal((I, K)))
    cc, cs = mx.mxfp8(rng.standard_normal((ROWS, 2 * I)))
    off, rw = to_dev(np.array([0, ROWS], np.int64)), torch.ones(ROWS, device=DEV)

    def run():
        return ops.moe_gated_backward(ops.FMT_MXFP8, *(to_dev(t) for t in (c, s, wc, ws)), off, I, K, to_dev(cc),
                                      to_dev(cs), row_weights=rw, tile=tile)
    plain = run()
    cc[NAN_ROW, 4] = 0x7F             # a gate
    got = run()
    bad = torch.zeros(ROWS, 2 * I, dtype=torch.bool, device=DEV)
    bad[NAN_ROW, [4, I + 4]] = True
    assert torch.equal(torch.isnan(got["dh13"]), bad) and torch.equal(torch.isnan(got["h"]), bad[:, :I])
    assert torch.equal(torch.isnan(got["d_row_weights"]), torch.arange(ROWS, device=DEV) == NAN_ROW)
    assert torch.equal(got["dh13"][~bad], plain["dh13"][~bad])
    c[NAN_ROW, 0] = 0x7F              # of dy: all of that row
    got = run()
    assert torch.isnan(got["dh13"][NAN_ROW]).all() and torch.isnan(got["d_row_weights"][NAN_ROW])
    keep = torch.arange(ROWS, device=DEV) != NAN_ROW
    for k in got:
        assert torch.equal(got[k][keep], plain[k][keep]), k
