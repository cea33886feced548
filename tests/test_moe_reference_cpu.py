"""The binary64 definitions that the routing and checkpoint kernels are held
to: their gradients against central differences, the routing against the host
generator's map, and MXFP8 against the oracle."""
import numpy as np
import pytest

import oracle
from block_scaled_precision_token_amd import synth
from tests import moe_reference as ref


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("parts", ["loss", "weights", "both"])
def test_route_gradient_against_differences(norm, parts):
    rng = np.random.default_rng(3)
    T, E, k, shared = 7, 11, 3, 1
    x = rng.standard_normal((T, E)) * 1.5
    x[2, 4] = -np.inf
    x[5] = -np.inf
    x[6, 2:] = -np.inf                       # fewer experts than k
    mask = np.ones(T, bool)
    mask[1] = False
    fwd = ref.route(x, k, norm, shared, mask)
    d_rows = rng.standard_normal(T * (k + shared)) if parts != "loss" else None
    d_loss = 0.7 if parts != "weights" else None
    grad, _ = ref.route_backward(x, k, fwd, d_rows, d_loss, norm, shared, mask)
    h = 1e-5
    for t in range(T):
        for e in range(E):
            if not np.isfinite(x[t, e]):
                assert grad[t, e] == 0.0
                continue
            up, dn = x.copy(), x.copy()
            up[t, e] += h
            dn[t, e] -= h
            diff = (ref.objective(up, k, fwd, d_rows, d_loss, norm, mask)
                    - ref.objective(dn, k, fwd, d_rows, d_loss, norm, mask)) / (2 * h)
            # third derivative of order 1 times h^2, and the subtraction's rounding
            assert abs(diff - grad[t, e]) <= 10 * h * h + 1e-9


def test_swiglu_gradient_against_differences():
    rng = np.random.default_rng(4)
    R, I = 3, 8
    g, u, dh, w = rng.standard_normal((R, I)) * 3, rng.standard_normal((R, I)), rng.standard_normal((R, I)), rng.random(R)
    dg, du, h, dw, _ = ref.swiglu_backward(dh, g, u, w)
    assert np.allclose(h, ref.swiglu(g, u, w), rtol=1e-14)
    d = 1e-5
    f = lambda g, u, w: (dh * ref.swiglu(g, u, w)).sum()  # noqa: E731
    for r in range(R):
        e = np.zeros(R)
        e[r] = d
        assert abs((f(g, u, w + e) - f(g, u, w - e)) / (2 * d) - dw[r]) < 1e-8
        for i in range(I):
            e = np.zeros((R, I))
            e[r, i] = d
            assert abs((f(g + e, u, w) - f(g - e, u, w)) / (2 * d) - dg[r, i]) < 1e-8
            assert abs((f(g, u + e, w) - f(g, u - e, w)) / (2 * d) - du[r, i]) < 1e-8


def test_route_matches_the_host_generators_map():
    T, E, k = 300, 24, 4
    bias = synth.zipf_bias(1, E)
    off, src = synth.route_topk(2, T, E, k, bias, shared_expert=True)
    rng = np.random.Generator(np.random.PCG64(2))
    logits = rng.standard_normal((T, E), dtype=np.float32) + bias[None, :]
    got = ref.route(logits, k, shared=1)
    assert np.array_equal(got["group_offsets"], off) and np.array_equal(got["src"], src)
    assert np.allclose(got["weights"][:, :k].sum(1), 1.0)


def test_uniform_routing_has_loss_one():
    T = E = 16
    x = np.zeros((T, E))
    x[np.arange(T), np.arange(T)] = 1e-12      # token t takes expert t
    assert abs(ref.route(x, 1)["loss"] - 1.0) < 1e-9


def test_mxfp8_equals_the_oracle():
    x = synth.activations(9, 64, 256, row_log10_range=(-3, 2))
    x[3, :32] = 0
    codes, scales = ref.mxfp8(ref.from_bf16(x).astype(np.float64))
    oc, os_ = oracle.quantize_mxfp8_rowwise(x)
    assert np.array_equal(codes, oc) and np.array_equal(scales, os_)
    assert np.array_equal(ref.mxfp8_value(codes, scales), oracle.dequantize_mxfp8(oc, os_)[0].astype(np.float64))
