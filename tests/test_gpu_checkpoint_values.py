"""The checkpointed SwiGLU next to the library's other calls: the fused SwiGLU
and quantizer, and blocks that hold infinities or NaN."""
import numpy as np
import pytest
import torch

import oracle
from block_scaled_precision_token_amd import ops, synth
from tests.gpu_util import DEV, host, to_dev_bf16
from tests.moe_reference import from_bf16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_h_is_the_fused_swiglus(dtype):
    """Both round an f32 value that is good to a few units: the same bf16 value or its neighbour.  Below a gate of
    -87.3 swiglu_quantize's h is -0, 3e-37 |up| from the exact value at most, and the checkpoint's call goes on."""
    x = to_dev_bf16(synth.activations(41, 300, 1536, row_log10_range=(-2, 1.5))).to(dtype)
    a, b = host(ops.swiglu_checkpoint(x)["h"]), host(ops.swiglu_quantize(x)[0])
    near = oracle.bf16_ulp_distance(a, b) <= 1
    far = np.abs(from_bf16(a) - from_bf16(b)) <= 3e-37 * np.abs(host(x.float())[:, 768:])
    assert np.all(near | far) and (~near).any()
    assert (a != b)[near].mean() < 1e-3


def special_blocks():
    """bf16 [64, 256] with infinities, NaN and both in blocks of ordinary values."""
    x = to_dev_bf16(synth.activations(42, 64, 256))
    inf, nan = float("inf"), float("nan")
    x[1, 5], x[2, 40], x[3, 70] = inf, -inf, nan
    x[4, 100], x[4, 101] = nan, inf
    x[5, 128:160] = nan
    x[6, 160:192] = -inf
    x[7] = inf
    return x


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_checkpoint_of_infinities_and_nan_is_the_quantizers(dtype):
    x = special_blocks()
    q = ops.quantize_mxfp8(x)
    ck = ops.swiglu_checkpoint(x.to(dtype))
    assert torch.equal(ck["ckpt_codes"], q["codes_row"]) and torch.equal(ck["ckpt_scales"], q["scales_row"])


def test_infinities_and_nan_stay_in_their_rows():
    x = special_blocks()
    plain = x.clone()
    plain[1:8] = 0.5
    for dtype in (torch.float32, torch.bfloat16):
        a, b = ops.swiglu_checkpoint(x.to(dtype), quantize_h=True), ops.swiglu_checkpoint(plain.to(dtype), quantize_h=True)
        dh = torch.ones(64, 128, dtype=dtype, device=DEV)
        w = torch.ones(64, device=DEV)
        ga = ops.swiglu_checkpoint_backward(dh, a["ckpt_codes"], a["ckpt_scales"], row_weights=w)
        gb = ops.swiglu_checkpoint_backward(dh, b["ckpt_codes"], b["ckpt_scales"], row_weights=w)
        for u, v in ((a, b), (ga, gb)):
            for n in u:
                assert torch.equal(u[n][8:], v[n][8:]) and torch.equal(u[n][0], v[n][0]), n
        assert torch.isnan(a["h"][3]).any() and not torch.isfinite(a["h"][1]).all()
