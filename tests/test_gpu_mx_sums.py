"""Sums of MX products whose blocks lie far apart, in every form: f32's own rounding and no more.

Activations are N(0, 1) with one value in a hundred fifty times as large.  A product of MXFP4 values enters the running
sum in steps of 64 values, one with MXFP8 tokens in steps of 16 bf16 products (which hold the operands' values exactly);
each step rounds the running sum, which sum |a b| bounds, by at most a unit of f32, 2^-23, and up to eight partial sums
meet: (K / 16 + 8) 2^-23 of sum |a b| covers both.  bf16 outputs add half a step, 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

from block_scaled_precision_token_amd import ops
from tests import mx_reference as mx
from tests.gpu_util import DEV, to_dev
from tests.test_gpu_gated import check_block
from tests.test_gpu_mx_products import f64

pytestmark = pytest.mark.gpu

FORMATS = {"mxfp4": (ops.FMT_MXFP4, 4, 4), "a8w4": (ops.FMT_MXFP8_MXFP4, 8, 4), "mxfp8": (ops.FMT_MXFP8, 8, 8)}


def quantized(rng, rows, K, bits, std, outliers):
    v = rng.standard_normal((rows, K)) * std
    if outliers:
        v = np.where(rng.random(v.shape) < 0.01, 50 * v, v)
    c, s = (mx.mxfp4 if bits == 4 else mx.mxfp8)(v)
    return c, s, (mx.mxfp4_values if bits == 4 else mx.mxfp8_values)(c, s)


def unit(K):
    return (K / 16 + 8) * 2.0 ** -23


def problem(fmt, sizes, N, K, seed):
    f, ab, bb = FORMATS[fmt]
    rng = np.random.default_rng(seed)
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int64)
    R, G = int(off[-1]), len(sizes)
    ac, as_, av = quantized(rng, R, K, ab, 1.0, True)
    bc, bs, bv = quantized(rng, G * N, K, bb, 0.05, False)
    ref, refabs = mx.grouped_product(av, bv.reshape(G, N, K), off, None)
    return f, [to_dev(t) for t in (ac, as_, bc, bs, off)], ref, refabs


# few rows; tiles of 64 rows; of 128 for MXFP4 products, else 64; of 128
FORMS = [(32, [5, 0, 40]), (128, [5, 0, 40]), (128, [130, 97]), (128, [300, 97])]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("fmt", ["mxfp4", "a8w4"])
@pytest.mark.parametrize("K", [64, 96, 320, 2080])
@pytest.mark.parametrize("tile,sizes", FORMS)
def test_products(tile, sizes, K, fmt, dtype):
    f, dev, ref, refabs = problem(fmt, sizes, 70, K, K)
    got = f64(ops.moe_grouped_gemm_blockscaled(f, ops.GEMM_FPROP, *dev, 70, K, tile=tile, out_dtype=dtype))
    tol = unit(K) * refabs + (2.0 ** -8 * np.abs(ref) if dtype == torch.bfloat16 else 0)
    assert (np.abs(got - ref) <= tol + 1e-30).all(), float((np.abs(got - ref) / refabs).max())


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("K", [64, 320])
@pytest.mark.parametrize("tile,sizes", FORMS)
def test_gate_and_up(tile, sizes, K, fmt):
    """The checkpoint holds gate and up to their own rounding."""
    f, dev, ref, refabs = problem(fmt, sizes, 192, K, K + 1)
    out = ops.moe_gated(f, *dev, 96, K, checkpoint=True, tile=tile)
    s = out["ckpt_scales"].cpu().numpy()
    check_block(mx.mxfp8_values(out["ckpt_codes"].cpu().numpy(), s), s, ref, unit(K) * refabs, ops.FMT_MXFP8, "checkpoint")


@pytest.mark.parametrize("fmt", ["mxfp4", "a8w4"])
@pytest.mark.parametrize("sizes", [[64], [1, 0, 40], [700, 97]])
def test_weight_gradients(sizes, fmt):
    f, ab, bb = FORMATS[fmt]
    rng = np.random.default_rng(len(sizes))
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int64)
    P, G = mx.padded_starts(off), len(sizes)
    ld = ops.mxfp8_grouped_cols(int(off[-1]), G)
    ac, as_, av = quantized(rng, 140, ld, ab, 1.0, True)
    bc, bs, bv = quantized(rng, 70, ld, bb, 1.0, True)
    got = f64(ops.moe_grouped_gemm_blockscaled(f, ops.GEMM_WGRAD, *(to_dev(t) for t in (ac, as_, bc, bs, off)), 70, ld))
    for g in range(G):
        a, b = av[:, P[g]:P[g + 1]], bv[:, P[g]:P[g + 1]]
        ref, refabs = a @ b.T, np.abs(a) @ np.abs(b).T
        assert (np.abs(got[g] - ref) <= unit(P[g + 1] - P[g]) * refabs + 1e-30).all(), g


@pytest.mark.parametrize("fmt", ["mxfp4", "a8w4"])
def test_rows_do_not_depend_on_the_form(fmt):
    """Products that are multiples of 2^-7 and at most 45, whose sums of 512 stay below 2^15 and f32 holds exactly: the
    same bits from 64 rows and from 65 (few rows, then tiles)."""
    f, ab, _ = FORMATS[fmt]
    rng = np.random.default_rng(6)
    K, N, G = 512, 96, 2
    if ab == 4:
        ac = rng.integers(0, 256, (65, K // 2)).astype(np.uint8)
    else:
        # 0.125 to 7.5 in multiples of 2^-6; the weights are multiples of 0.5 up to 6
        ac = rng.integers(0x20, 0x50, (65, K)).astype(np.uint8) | (rng.integers(0, 2, (65, K)) * 128).astype(np.uint8)
    as_ = np.full((65, K // 32), 127, np.uint8)
    bc = rng.integers(0, 256, (G * N, K // 2)).astype(np.uint8)
    bs = np.full((G * N, K // 32), 127, np.uint8)
    outs = []
    for rows in (64, 65):
        off = np.array([0, 20, rows], np.int64)
        args = [to_dev(np.ascontiguousarray(t)) for t in (ac[:rows], as_[:rows], bc, bs, off)]
        outs.append(ops.moe_grouped_gemm_blockscaled(f, ops.GEMM_FPROP, *args, N, K))
    assert torch.equal(outs[0], outs[1][:64])
    assert (outs[0] != 0).any()


@pytest.mark.parametrize("fmt", ["a8w4", "mxfp8"])
@pytest.mark.parametrize("tile", [32, 128])
def test_smallest_values(tile, fmt):
    """Tokens of scale 2^-127, whose values are bf16's subnormals, times weights of 2^100: as from 64 bits."""
    f, ab, bb = FORMATS[fmt]
    rng = np.random.default_rng(7)
    K, R, I = 64, 9, 32
    # multiples of 2^-6: times 2^-127 they are multiples of 2^-133
    ac = (rng.integers(0x08, 0x7F, (R, K)) | (rng.integers(0, 2, (R, K)) * 128)).astype(np.uint8)
    ac[(ac & 127) < 0x20] &= 0xF8
    as_ = np.zeros((R, K // 32), np.uint8)
    per = 8 // bb
    bc = rng.integers(0x01, 0x70, (2 * I, K // per)).astype(np.uint8)
    bs = np.full((2 * I, K // 32), 227, np.uint8)
    av, bv = mx.mxfp8_values(ac, as_), (mx.mxfp4_values if bb == 4 else mx.mxfp8_values)(bc, bs)
    off = np.array([0, R], np.int64)
    ref, refabs = mx.grouped_product(av, bv.reshape(1, 2 * I, K), off, None)
    out = ops.moe_gated(f, *(to_dev(t) for t in (ac, as_, bc, bs, off)), I, K, checkpoint=True, tile=tile)
    s = out["ckpt_scales"].cpu().numpy()
    check_block(mx.mxfp8_values(out["ckpt_codes"].cpu().numpy(), s), s, ref, unit(K) * refabs, ops.FMT_MXFP8, "checkpoint")
