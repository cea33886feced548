"""Accuracy of the checkpointed SwiGLU where its outputs are f32, and where
exp(-gate) leaves f32's range.

Units: EPS = 2^-24.  s = 1 / (1 + e) and 1 - s = e s with e = exp(-gate) as
2^t, t = -gate log2(e), times 1 + d, where d is what rounding t left out.  The
hardware exponential and reciprocal are good to a unit in the last place (2 EPS
each), every product and sum to 1 EPS, and d is off by log 2's own rounding
(0.05 EPS per unit of |gate|).  So e to 3 + 0.05 |gate|, s to 6 + 0.05 |gate|,
1 - s to 10 + 0.1 |gate|."""
import numpy as np
import pytest
import torch

from block_scaled_precision_token_amd import ops
from tests import moe_reference as ref
from tests.gpu_util import DEV, host, to_dev

pytestmark = pytest.mark.gpu


def checkpoint(R, I, scale, seed):
    """(codes, scales, gate, up) of a random checkpoint."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((R, 2 * I)) * scale
    codes, scales = ref.mxfp8(x)
    v = ref.mxfp8_value(codes, scales)
    return codes, scales, v[:, :I], v[:, I:]


@pytest.mark.parametrize("scale", [0.3, 1.5, 6.0, 25.0])
def test_f32_gradient_to_a_few_units(scale):
    R, I = 96, 1024
    codes, scales, g, u = checkpoint(R, I, scale, int(10 * scale))
    s = ref.sigmoid(g)
    live = np.abs(g) < 80                       # past it f32 itself runs out of range, below
    got = ops.swiglu_checkpoint_backward(torch.ones(R, I, device=DEV), to_dev(codes), to_dev(scales))
    d = host(got["dh13"]).astype(np.float64)
    # d up = gate s: s, one product
    want = g * s
    err, allowed = np.abs(d[:, I:] - want), (8 + 0.05 * np.abs(g)) * ref.EPS * np.abs(want)
    assert np.all((err <= allowed)[live]), float((err / np.maximum(allowed, 1e-300))[live].max())
    # d gate = up (s + gate s (1 - s)): s; gate s to 7 and its product with 1 - s to 18; the sum, the product
    size = np.abs(u) * (s + np.abs(g) * s * (1 - s))
    want = u * (s + g * s * (1 - s))
    err, allowed = np.abs(d[:, :I] - want), (21 + 0.2 * np.abs(g)) * ref.EPS * size
    assert np.all((err <= allowed)[live]), float((err / np.maximum(allowed, 1e-300))[live].max())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_weights_gradient_to_a_few_units(dtype):
    """Rows of one sign, so that nothing cancels: sum_i dh_i silu(gate_i) up_i, gates around -3."""
    R, I = 64, 2048
    rng = np.random.default_rng(3)
    x = np.concatenate([-3 + rng.standard_normal((R, I)) * 0.5, 1 + rng.random((R, I))], 1)
    codes, scales = ref.mxfp8(x)
    v = ref.mxfp8_value(codes, scales)
    g, u = v[:, :I], v[:, I:]
    assert (g < 0).all() and (u > 0).all()
    w = torch.ones(R, device=DEV)
    got = ops.swiglu_checkpoint_backward(torch.ones(R, I, device=DEV, dtype=dtype), to_dev(codes), to_dev(scales),
                                         row_weights=w)
    want = (g * ref.sigmoid(g) * u).sum(1)
    # an element to 8 + 0.05 |gate| and two products, a lane's chain of I / 64 additions, six steps across lanes
    tol = (10 + 0.05 * 6 + I / 64 + 6) * ref.EPS
    assert np.all(np.abs(host(got["d_row_weights"]) - want) <= tol * np.abs(want))


def test_weights_gradient_mean_error():
    """The errors of many rows' sums average out unless the exponential is biased or coarse: one element to a row
    of 32, the rest zeros, error of the mean square."""
    R, I = 1 << 15, 32
    rng = np.random.default_rng(4)
    x = np.zeros((R, 2 * I))
    x[:, 0] = rng.uniform(-4, 4, R)
    x[:, I] = 1.0
    codes, scales = ref.mxfp8(x)
    g = ref.mxfp8_value(codes, scales)[:, 0]
    got = ops.swiglu_checkpoint_backward(torch.ones(R, I, device=DEV), to_dev(codes), to_dev(scales),
                                         row_weights=torch.ones(R, device=DEV))
    want = g * ref.sigmoid(g)
    live = want != 0
    rel = (host(got["d_row_weights"])[live] - want[live]) / want[live] / ref.EPS
    # each of the sigmoid's five roundings is uniform: of 1 EPS half width (rms 0.58) three, of 2 EPS (1.15) two
    assert float(np.sqrt((rel ** 2).mean())) <= np.sqrt(3 * 0.58 ** 2 + 2 * 1.15 ** 2) + 0.2


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gates_where_the_exponential_leaves_f32(dtype):
    """Gates from -60 to -112 and far above: s is subnormal from -87.3 on and 0 below -104, so silu carries half of
    f32's least subnormal per unit of gate; nothing turns into an infinity or NaN."""
    I = 64
    z = np.concatenate([-np.arange(60, 112, 0.5), [-3e4, -3e38, 90.0, 300.0, 3e38]])
    R = len(z)
    x = np.zeros((R, 2 * I))
    x[:, :I] = z[:, None]
    x[:, 1] = 0.25                              # an ordinary gate beside each of them
    x[:, I:] = 1.0
    codes, scales = ref.mxfp8(x)
    v = ref.mxfp8_value(codes, scales)
    g, u = v[:, :I], v[:, I:]
    with np.errstate(over="ignore"):
        s = ref.sigmoid(g)
    got = ops.swiglu_checkpoint_backward(torch.ones(R, I, device=DEV, dtype=dtype), to_dev(codes), to_dev(scales))
    d = got["dh13"].double().cpu().numpy()
    half = 2.0 ** -8 if dtype is torch.bfloat16 else 0.0
    tiny = 2.0 ** -134 if dtype is torch.bfloat16 else 0.0       # half of bf16's least subnormal
    lost = (np.minimum(np.abs(g), 120) + 2) * 2.0 ** -149 + tiny
    want = g * s
    tol = (8 + 0.05 * np.minimum(np.abs(g), 120)) * ref.EPS + half
    assert np.isfinite(d).all()
    assert np.all(np.abs(d[:, I:] - want) <= tol * np.abs(want) + lost)
    c = np.where(g < 0, 1 - s, np.exp(-np.maximum(g, 0)) * s)
    size = s + np.minimum(np.abs(g), 1e30) * s * c
    tol = (21 + 0.2 * np.minimum(np.abs(g), 120)) * ref.EPS + half
    assert np.all(np.abs(d[:, :I] - u * (s + g * s * c)) <= tol * size + 2 * lost)
    # the forward's h, from the same values
    h = ref.from_bf16(host(ops.swiglu_checkpoint(to_dev(v.astype(np.float32)).to(dtype))["h"])).astype(np.float64)
    gf = v[:, :I] if dtype is torch.float32 else to_dev(v[:, :I].astype(np.float32)).to(dtype).double().cpu().numpy()
    with np.errstate(over="ignore"):
        want = gf * ref.sigmoid(gf)
    tol = 2.0 ** -8 + (2 * np.minimum(np.abs(gf), 120) + 16) * 2 * ref.EPS
    assert np.all(np.abs(h - want) <= tol * np.abs(want) + 2.0 ** -134 + 122 * 2.0 ** -149)
