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


def special(x):
    """Some NaN and infinities into bf16 [64, 96]; returns where the NaN are."""
    nan, inf = float("nan"), float("inf")
    x[1, 5], x[40, 64], x[40, 65] = nan, nan, inf
    x[2, 32:64] = -nan
    x[7, 70], x[63, 95] = inf, -inf
    return torch.isnan(x)


def blocks_with(nan):
    """Rows [R, K] of truth values -> [R, K / 32]."""
    return nan.view(nan.shape[0], -1, 32).any(2)


@pytest.mark.parametrize("sr", [False, True])
@pytest.mark.parametrize("form", ["row", "rowcol", "grouped"])
def test_mxfp4_quantizer(form, sr):
    """Blocks with a NaN have scale 255 and are NaN when dequantized; all other bytes are those of a tensor without it."""
    rng = np.random.default_rng(4)
    x = to_dev_bf16(mx.to_bf16_bits(rng.standard_normal((64, 96)).astype(np.float32)))
    nan = special(x)
    kw = dict(colwise=form != "row", sr=sr, seed=9,
              group_offsets=to_dev(np.array([0, 32, 64], np.int64)) if form == "grouped" else None)
    q = ops.quantize_mxfp4(x, **kw)
    plain = ops.quantize_mxfp4(torch.where(nan, torch.zeros_like(x), x), **kw)
    copies = [("row", blocks_with(nan), x)]
    if form != "row":
        copies.append(("colT", blocks_with(nan.t().contiguous()), x.t()))
    for name, bad, v in copies:
        codes, scales = q["codes_" + name][:, :bad.shape[1] * 16], q["scales_" + name][:, :bad.shape[1]]
        assert torch.equal(scales == 255, bad)
        assert torch.equal(scales[~bad], plain["scales_" + name][:, :bad.shape[1]][~bad])
        same = (~bad).repeat_interleave(16, 1)
        assert torch.equal(codes[same], plain["codes_" + name][:, :bad.shape[1] * 16][same])
        for dtype in (torch.float32, torch.bfloat16):
            y = ops.dequantize(ops.FMT_MXFP4, codes.contiguous(), scales.contiguous(), out_dtype=dtype)
            assert torch.equal(torch.isnan(y), bad.repeat_interleave(32, 1))
            far = torch.isinf(v) & ~bad.repeat_interleave(32, 1)
            assert (y[far].abs() == 6 * 2.0 ** 125).all() and torch.equal(torch.sign(y[far]), torch.sign(v[far]).to(dtype))


def test_every_code_of_a_nan_block_is_nan():
    codes = torch.arange(256, dtype=torch.uint8, device=DEV).view(16, 16)
    y = ops.dequantize(ops.FMT_MXFP4, codes, torch.full((16, 1), 255, dtype=torch.uint8, device=DEV))
    assert torch.isnan(y).all()


@pytest.mark.parametrize("a_bits", [4, 8])
@pytest.mark.parametrize("tile", [32, 128])
def test_products_of_nan_blocks(tile, a_bits):
    """A NaN block of the tokens (MXFP4) makes its row NaN, one of the weights its column of that group; K's last stage is
    not full."""
    rng = np.random.default_rng(5)
    K, N = 352, 40
    ac, as_ = (mx.mxfp4 if a_bits == 4 else mx.mxfp8)(rng.standard_normal((ROWS, K)))
    bc, bs = mx.mxfp4(rng.standard_normal((2 * N, K)))
    off = to_dev(np.array([0, 15, ROWS], np.int64))
    f = ops.FMT_MXFP4 if a_bits == 4 else ops.FMT_MXFP8_MXFP4

    def run():
        return ops.moe_grouped_gemm_blockscaled(f, ops.GEMM_FPROP, *(to_dev(t) for t in (ac, as_, bc, bs)), off, N, K,
                                                tile=tile)
    plain = run()
    bad = torch.zeros(ROWS, N, dtype=torch.bool, device=DEV)
    if a_bits == 4:
        as_[NAN_ROW, 10] = 255
        bad[NAN_ROW] = True
    bs[N + 6, 0] = 255
    bad[15:, 6] = True
    got = run()
    assert torch.equal(torch.isnan(got), bad) and torch.equal(got[~bad], plain[~bad])


@pytest.mark.parametrize("tile", [32, 128])
def test_h_in_mxfp4(tile):
    rng = np.random.default_rng(6)
    c, s = mx.mxfp8(rng.standard_normal((ROWS, K)))
    wc, ws = mx.mxfp4(rng.standard_normal((4 * 32, K)))
    off = to_dev(np.array([0, ROWS], np.int64))

    def run():
        return ops.moe_gated(ops.FMT_MXFP8_MXFP4, *(to_dev(t) for t in (c, s, wc, ws)), off, 64, K, h_fmt=ops.FMT_MXFP4,
                             tile=tile)
    plain = run()
    c[NAN_ROW, 1] = 0x7F
    ws[33, 0] = 255                    # gate of column 33: the second block of every row
    got = run()
    bad = torch.zeros(ROWS, 2, dtype=torch.bool, device=DEV)
    bad[NAN_ROW] = True
    bad[:, 1] = True
    assert torch.equal(got["scales"] == 255, bad) and torch.equal(got["scales"][~bad], plain["scales"][~bad])
    same = (~bad).repeat_interleave(16, 1)
    assert torch.equal(got["codes"][same], plain["codes"][same])
    assert not (host(plain["scales"]) == 255).any()


@pytest.mark.parametrize("fmt", ["mxfp4", "a8w4", "mxfp8"])
@pytest.mark.parametrize("rows", [ROWS, 400])
def test_rows_without_a_source_are_zeros_beside_nan(rows, fmt):
    """Indices outside x, where the tokens of its first row, which such rows may load, are NaN."""
    f, ab, bb = {"mxfp4": (ops.FMT_MXFP4, 4, 4), "a8w4": (ops.FMT_MXFP8_MXFP4, 8, 4), "mxfp8": (ops.FMT_MXFP8, 8, 8)}[fmt]
    rng = np.random.default_rng(7)
    quantize = {4: mx.mxfp4, 8: mx.mxfp8}
    c, s = quantize[ab](rng.standard_normal((6, K)))
    if ab == 4:
        s[0] = 255
    else:
        c[0] = 0x7F
    w13, w2 = (quantize[bb](rng.standard_normal((n, K))) for n in (2 * I, I))
    ck = mx.mxfp8(rng.standard_normal((rows, 2 * I)))
    gather = rng.integers(1, 6, rows).astype(np.int32)
    gather[::3] = rng.choice([-1, 6, 2 ** 31 - 1, -2 ** 31], len(gather[::3]))
    none = torch.from_numpy(gather < 0).to(DEV) | torch.from_numpy(gather > 5).to(DEV)
    off, idx, rw = to_dev(np.array([0, rows], np.int64)), to_dev(gather), torch.rand(rows, device=DEV)
    a = [to_dev(t) for t in (c, s)]
    out = ops.moe_gated(f, *a, *(to_dev(t) for t in w13), off, I, K, a_gather=idx, row_weights=rw, checkpoint=True,
                        return_h=True)
    assert not torch.isnan(out["h"]).any() and (out["h"][none] == 0).all() and (out["h"][~none] != 0).any()
    for k in ("codes", "ckpt_codes"):
        assert (out[k][none] & 127 == 0).all() and (out[k] & 127 != 127).all()
    back = ops.moe_gated_backward(f, *a, *(to_dev(t) for t in w2), off, I, K, *(to_dev(t) for t in ck), a_gather=idx,
                                  row_weights=rw)
    assert (back["dh13"][none] == 0).all() and (back["d_row_weights"][none] == 0).all()
    assert torch.isfinite(back["dh13"].float()).all() and torch.isfinite(back["d_row_weights"]).all()
    if fmt != "mxfp8":
        y = ops.moe_grouped_gemm_blockscaled(f, ops.GEMM_FPROP, *a, *(to_dev(t) for t in w13), off, 2 * I, K, a_gather=idx)
        assert (y[none] == 0).all() and torch.isfinite(y).all()
