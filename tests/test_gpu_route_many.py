"""Routing of many tokens over many experts, and of more tokens than 256 runs hold."""
import pytest
import torch

from block_scaled_precision_token_amd import ops
from tests import moe_reference as ref
from tests.gpu_util import DEV, host
from tests.test_gpu_route import DT, check_forward, logits_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,k,shared,dtype", [
    (9001, 700, 4, 0, "f32"),       # runs of 64 tokens, more groups than the smaller rank table holds
    (8200, 300, 6, 2, "bf16"),
    (17001, 129, 3, 0, "f32"),      # experts past a multiple of four
    (57601, 490, 2, 60, "bf16"),    # runs of more than 255 tokens, many groups
])
def test_route_many(T, E, k, shared, dtype):
    xd, x = logits_of(T + E, T, E, DT[dtype])
    got = ops.moe_route(xd, k, shared=shared, aux=True)
    check_forward(got, ref.route(x, k, True, shared, None), x, k)


def test_more_tokens_than_256_runs_hold():
    T, E = 17_000_001, 2
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(T, E, generator=g, device=DEV)
    got = ops.moe_route(x, 1, aux=True)
    second = x[:, 1] > x[:, 0]
    assert torch.equal(got["experts"][:, 0], second.int())
    c1 = int(second.sum())
    assert host(got["counts"]).tolist() == [T - c1, c1, T]
    assert host(got["group_offsets"]).tolist() == [0, T - c1, T]
    src = torch.cat([(~second).nonzero()[:, 0], second.nonzero()[:, 0]]).int()
    assert torch.equal(got["src"], src)
    pos = torch.empty(T, dtype=torch.int32, device=DEV)
    pos[src.long()] = torch.arange(T, dtype=torch.int32, device=DEV)
    assert torch.equal(got["pos"][:, 0], pos)
    p = torch.softmax(x.double(), 1).sum(0)
    # at most 65504 tokens to a run, 32 or more added side by side, then 260 runs; each p to a few units
    tol = (65504 / 32 + 260 + 64) * ref.EPS
    assert float(((got["prob_sum"].double() - p) / p).abs().max()) <= tol
    loss = E * float(p[0] * (T - c1) + p[1] * c1) / T / T
    assert abs(float(got["loss"][0]) - loss) <= (tol + 20 * ref.EPS) * loss
