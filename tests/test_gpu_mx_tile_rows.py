"""Both row tiles, 64 and 128 rows, whichever the rule for a format and operator takes: groups of about 20 rows and of more
than 160, K and N as uneven as in the tests of the forms.  Bounds as in test_gpu_mx_sums."""
import pytest
import torch

from block_scaled_precision_token_amd import ops
from tests import test_gpu_gated as gated
from tests import test_gpu_mx_products as products

pytestmark = pytest.mark.gpu

SIZES = [[170], [0, 700, 2, 31, 300], [129, 511, 128, 0, 257], [20, 0, 33, 1, 64]]


@pytest.fixture(autouse=True)
def bounds(monkeypatch):
    check = products.check
    monkeypatch.setattr(products, "check", lambda got, ref, refabs, bits, K, bf16: check(got, ref, refabs, 4, 4 * K, bf16))
    monkeypatch.setattr(gated, "product_tol", lambda bits, K: (K / 16 + 8) * 2.0 ** -23)


def test_sizes_reach_both():
    assert [sum(s) // len(s) >= 160 for s in SIZES] == [True, True, True, False]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", list(products.FORMATS))
@pytest.mark.parametrize("N,K", [(1, 32), (257, 160), (520, 576), (64, 2080)])
@pytest.mark.parametrize("sizes", SIZES)
def test_products(sizes, N, K, fmt, dtype):
    products.run_forward(fmt, sizes, N, K, 128, dtype, gather=len(sizes) > 1, pad=N % 8, seed=N + K)


@pytest.mark.parametrize("fmt", list(gated.FORMATS))
@pytest.mark.parametrize("I,K", [(32, 32), (96, 160), (288, 320)])
@pytest.mark.parametrize("sizes", SIZES)
def test_gated_block_and_backward(sizes, I, K, fmt):
    gated.run_forward(fmt, sizes, I, K, 128, seed=I, gather=len(sizes) > 1)
    gated.run_backward(fmt, sizes, I, K, 128, seed=I, gather=len(sizes) > 1)


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("h_fmt", [-1, ops.FMT_MXFP4])
@pytest.mark.parametrize("checkpoint", [False, True])
def test_outputs(h_fmt, checkpoint, sizes):
    gated.run_forward("mxfp4", sizes, 160, 96, 128, seed=1, h_fmt=h_fmt, return_h=True, checkpoint=checkpoint, weighted=False)
