"""Routing forward and backward against the definition in binary64 for every
shape of kernel that the numbers of tokens and experts, the dtype and the rows'
alignment select: one workgroup for a short batch, few lanes to a token for a
long one, and both sides of each switch between them."""
import numpy as np
import pytest
import torch

from block_scaled_precision_token_amd import ops
from tests import moe_reference as ref
from tests.gpu_util import DEV, to_dev
from tests.test_gpu_route import DT, check_forward, logits_of

pytestmark = pytest.mark.gpu


def check(T, E, k, shared, dtype, norm, kind, masked, pad):
    seed = 31 * T + E
    xd, x = logits_of(seed, T, E, DT[dtype], kind, pad)
    rng = np.random.default_rng(seed + 1)
    mask = maskd = None
    if masked:
        mask = rng.random(T) >= masked
        maskd = to_dev(mask)
        xd[~maskd] = float("nan")
    want = ref.route(x, k, norm, shared, mask)
    got = ops.moe_route(xd, k, norm=norm, shared=shared, token_mask=maskd, aux=True)
    check_forward(got, want, x, k, mask)
    d_rows, dl = rng.standard_normal(T * (k + shared)).astype(np.float32), 0.31
    grad, size = ref.route_backward(x, k, want, d_rows, dl, norm, shared, mask)
    g = ops.moe_route_backward(xd, k, got["experts"], got["counts"], got["pos"], d_weights=to_dev(d_rows),
                               d_loss=torch.tensor([dl], device=DEV), norm=norm, shared=shared, token_mask=maskd)
    # the error terms of weight_tol twice (forward and backward factors), a lane's sums and the products
    tol = 2 * ref.weight_tol(ref.logit_span(x, mask), E) + (E / 8 + 32) * ref.EPS
    err = np.abs(g.double().cpu().numpy() - grad)
    allowed = tol * size + 1e-37 + (2.0 ** -8 * np.abs(grad) if dtype == "bf16" else 0.0)
    assert np.all(err <= allowed), float((err / allowed).max())


@pytest.mark.parametrize("E", [60, 64, 128, 256])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [64, 65, 127, 128, 129])
def test_short_batches(T, dtype, E):
    check(T, E, 8 if E != 128 else 6, T % 3, dtype, E != 64, "unavailable" if E == 128 else "normal", 0.15, 0)


LONG = [
    # T, E, k, shared, dtype, norm, kind, masked share, row padding
    (16385, 32, 4, 1, "bf16", True, "ties", 0.1, 0),
    (16385, 64, 8, 0, "f32", True, "normal", 0.1, 0),
    (18001, 64, 6, 1, "bf16", False, "unavailable", 0.0, 8),
    (20003, 96, 6, 0, "f32", False, "normal", 0.0, 0),
    (16400, 96, 8, 2, "bf16", True, "lowest", 0.2, 0),
    (16999, 80, 5, 0, "f32", True, "ties", 0.3, 4),
    (17003, 128, 8, 0, "f32", True, "unavailable", 0.1, 0),
    (19000, 128, 7, 1, "bf16", True, "normal", 0.0, 0),
    (16385, 192, 8, 1, "f32", False, "ties", 0.1, 0),
    (17777, 160, 8, 0, "bf16", True, "normal", 0.05, 16),
    (18003, 256, 8, 1, "f32", True, "lowest", 0.1, 0),
    (20001, 256, 8, 1, "bf16", False, "normal", 0.1, 0),
    (16384, 256, 3, 0, "bf16", True, "unavailable", 0.0, 0),
    (16383, 256, 8, 0, "bf16", True, "unavailable", 0.1, 0),
    (16384, 128, 8, 1, "f32", True, "normal", 0.1, 0),
    (16383, 128, 8, 1, "f32", True, "normal", 0.1, 0),
    (16385, 128, 9, 0, "f32", True, "normal", 0.1, 0),        # lists longer than the long batches' form keeps
    (16385, 130, 8, 0, "f32", False, "normal", 0.1, 0),       # rows that are not whole 16-byte pieces
    (16385, 60, 8, 0, "bf16", True, "normal", 0.0, 0),
    (16400, 320, 8, 0, "bf16", True, "normal", 0.1, 0),       # more experts than it takes
]


@pytest.mark.parametrize("T,E,k,shared,dtype,norm,kind,masked,pad", LONG)
def test_long_batches(T, E, k, shared, dtype, norm, kind, masked, pad):
    check(T, E, k, shared, dtype, norm, kind, masked, pad)
