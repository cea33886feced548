"""Checkpointed SwiGLU and combine on calls of more than 2^32 threads and tensors
of more than 2^35 values: every row equals the same row of a small call."""
import pytest
import torch

from block_scaled_precision_token_amd import ops
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def room():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 200 << 30:
        pytest.skip("needs 200 GiB of device memory")
    yield
    torch.cuda.empty_cache()


def assert_tiled(big, small, what, rows=1 << 24):
    P = small.shape[0]
    for r in range(0, big.shape[0], rows):
        part = big[r:r + rows]
        part = part.view(-1, P, *part.shape[1:])
        assert bool((part == small).all()), f"{what}, rows from {r}"


def test_checkpoint_of_many_rows():
    P, I = 64, 32
    R = (1 << 29) + P                                  # 8 lanes to a row
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(P, 2 * I, generator=g, device=DEV).to(torch.bfloat16)
    want = ops.swiglu_checkpoint(x)
    grad = ops.swiglu_checkpoint_backward(want["h"], want["ckpt_codes"], want["ckpt_scales"], return_h=False)
    big = torch.empty(R, 2 * I, dtype=torch.bfloat16, device=DEV)
    big.view(-1, P, 2 * I).copy_(x)
    got = ops.swiglu_checkpoint(big)
    del big
    for n in ("h", "ckpt_codes", "ckpt_scales"):
        assert_tiled(got[n], want[n], n)
    got = ops.swiglu_checkpoint_backward(got["h"], got["ckpt_codes"], got["ckpt_scales"], return_h=False)
    assert_tiled(got["dh13"], grad["dh13"], "dh13")


def test_combine_of_many_values():
    T, H, rows = (1 << 21) + 5, 1 << 14, 64
    g = torch.Generator(device=DEV).manual_seed(2)
    y = torch.randn(rows, H, generator=g, device=DEV).to(torch.bfloat16)
    pos = torch.randint(0, rows, (T, 1), generator=g, device=DEV, dtype=torch.int32)
    out = ops.moe_combine(y, pos)
    for t in range(0, T, 1 << 16):
        assert torch.equal(out[t:t + (1 << 16)], y[pos[t:t + (1 << 16), 0].long()]), f"tokens from {t}"
