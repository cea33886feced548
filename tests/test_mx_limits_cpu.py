"""The largest sizes of the MX products: a grid of 2^24 workgroups of 256 threads would be 2^32 threads, one too many for a
grid dimension (CPU only: the calls are refused)."""
import pytest

from block_scaled_precision_token_amd import ops
from tests.test_mx_args_cpu import P, SHAPE, back, gated, gemm

# groups of 94 rows, in 64-row tiles (the gated block, MXFP8 tokens): M / 64 + G workgroups for these and G for 128
# columns; MXFP4 products, in 128-row tiles, have the same bound
G = 4823450
M = 128 * ((1 << 23) - G)


def test_grid_of_the_preparation():
    assert M // G < 96 and M // 64 + 2 * G == 1 << 24
    kw = dict(gather=P, rows=512, G=G)
    assert gemm(M=M, N=64, **kw) == SHAPE
    assert back(R=M, I=64, **kw) == SHAPE and gated(R=M, I=64, **kw) == SHAPE


@pytest.mark.parametrize("fmt", [ops.FMT_MXFP4, ops.FMT_MXFP8_MXFP4])
def test_the_headers_limits(fmt):
    """include/bsp.h: what the products refuse beyond 4 GiB operands."""
    kw = dict(gather=P, rows=512)
    # groups times column tiles of 128
    assert gemm(fmt, N=1 << 20, ldc=1 << 20, G=(1 << 11) + 1, M=512, **kw) == SHAPE
    # row tiles of 128 and groups together, times column tiles and one
    assert gemm(fmt, N=1 << 20, ldc=1 << 20, G=1, M=1 << 18, **kw) == SHAPE
    # weight gradients: rows of both operands; groups times output tiles of 128 x 128
    assert gemm(fmt, mode=2, M=1 << 23, rows=1 << 23, N=(1 << 23) + 1, ldc=1 << 24, K=32, G=1) == SHAPE
    assert gemm(fmt, mode=2, M=1 << 17, rows=1 << 17, N=1 << 17, ldc=1 << 17, K=32, G=9) == SHAPE
