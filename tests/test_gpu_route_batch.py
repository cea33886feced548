"""A token's routing weights and their gradient do not depend on the batch it
is in: not on the number of tokens, its place, nor the rows' stride, bit for bit."""
import numpy as np
import pytest
import torch

from block_scaled_precision_token_amd import ops
from tests.gpu_util import DEV, to_dev
from tests.test_gpu_route import DT, logits_of

pytestmark = pytest.mark.gpu

TOKENS = 19001
PARTS = [(0, 1), (5, 69), (100, 227), (300, 1300), (2000, 18383), (2000, 18384)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("E", [16, 32, 56, 64, 96, 128, 160, 192, 256])
@pytest.mark.parametrize("norm", [True, False])
def test_weights_and_gradient_of_a_token(E, dtype, norm):
    k = 8 if E != 96 else 5
    x, _ = logits_of(E, TOKENS, E, DT[dtype], "unavailable" if E == 56 else "normal")
    mask = to_dev(np.random.default_rng(E).random(TOKENS) >= 0.1)
    d = torch.from_numpy(np.random.default_rng(E + 1).standard_normal((TOKENS, k)).astype(np.float32)).to(DEV)

    def run(a, b, pad=0):
        n = b - a
        part = torch.full((n, E + pad), float("nan"), dtype=x.dtype, device=DEV)
        part[:, :E] = x[a:b]
        part = part[:, :E]
        m = mask[a:b].clone()
        r = ops.moe_route(part, k, norm=norm, token_mask=m)
        rows = torch.zeros(n * k, device=DEV)
        live = r["pos"] >= 0
        rows[r["pos"][live].long()] = d[a:b][live]
        g = ops.moe_route_backward(part, k, r["experts"], r["counts"], r["pos"], d_weights=rows, norm=norm,
                                   token_mask=m)
        return r["experts"], r["weights"], g

    whole = run(0, TOKENS)
    for a, b, pad in [(a, b, 0) for a, b in PARTS] + [(0, TOKENS, 1), (0, 500, 3)]:
        for name, w, p in zip(("experts", "weights", "gradient"), whole, run(a, b, pad)):
            assert torch.equal(w[a:b], p), f"{name} of tokens {a} to {b}, padding {pad}"
