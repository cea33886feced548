"""The gated block's calls with more groups than a workgroup has threads, two calls at once, the allocation-free product, and
rows, groups and weights in views of larger tensors."""
import numpy as np
import pytest
import torch

from block_scaled_precision_token_amd import ops
from tests import test_gpu_gated as gated
from tests import test_gpu_mx_products as products
from tests.gpu_util import DEV, to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tile", [32, 128])
@pytest.mark.parametrize("G", [257, 513, 1100])
def test_gated_block_of_many_groups(G, tile):
    sizes = np.zeros(G, int)
    sizes[[0, 255, 256, G - 1]] = [3, 1, 70, 5]
    gated.run_forward("mxfp4", list(sizes), 32, 64, tile, seed=G)
    gated.run_backward("a8w4", list(sizes), 32, 64, tile, seed=G)


def test_two_calls_at_once():
    """Both passes on two streams, each with outputs and a workspace of its own: the bytes of calls one after the other."""
    qs = [gated.problem("a8w4", [700, 20, 300], 512, 288, s, True, 0, 0.3) for s in (1, 2)]
    bs = [gated.problem("a8w4", [700, 20, 300], 256, 288, s, True, 0, 0.1) for s in (3, 4)]
    ws = [to_dev(q["w"]) for q in qs]

    def both(i):
        q, b = qs[i], bs[i]
        f = ops.moe_gated(ops.FMT_MXFP8_MXFP4, *q["dev"], 256, 288, R=q["R"], a_gather=q["idx"], row_weights=ws[i],
                          checkpoint=True)
        r = ops.moe_gated_backward(ops.FMT_MXFP8_MXFP4, *b["dev"], 256, 288, f["ckpt_codes"], f["ckpt_scales"], R=b["R"],
                                   a_gather=b["idx"], row_weights=ws[i])
        return {**f, **r}

    one = [both(0), both(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(both(i))
    torch.cuda.synchronize()
    for i in range(2):
        for o in outs[i]:
            for k, v in o.items():
                assert torch.equal(v, one[i][k]), k


@pytest.mark.parametrize("mode", [ops.GEMM_FPROP, ops.GEMM_WGRAD])
@pytest.mark.parametrize("fmt", list(products.FORMATS))
def test_allocation_free_product(fmt, mode):
    f, ab, bb = products.FORMATS[fmt]
    rng = np.random.default_rng(5)
    off = np.array([0, 200, 200, 600], np.int64)
    wg = mode == ops.GEMM_WGRAD
    K = ops.mxfp8_grouped_cols(600, 3) if wg else 160
    ac, as_, _ = products.operand(rng, 70 if wg else 600, K, ab)
    bc, bs, _ = products.operand(rng, 40 if wg else 3 * 40, K, bb)
    args = [to_dev(t) for t in (ac, as_, bc, bs, off)]
    shape = (3, 70, 40) if wg else (600, 40)
    a, b = torch.full(shape, 7.0, device=DEV), torch.full(shape, 8.0, device=DEV)
    ops.moe_grouped_gemm_blockscaled_noalloc(f, mode, *args, 40, K, out=a)
    ops.moe_grouped_gemm_blockscaled(f, mode, *args, 40, K, out=b)
    assert torch.equal(a, b)


def test_views_are_taken_or_refused():
    """Rows from the middle of larger tensors work where they are 16-byte aligned; others and strided ones are refused."""
    q = gated.problem("mxfp4", [70, 60], 64, 128, 1, False, 0, 0.3)
    a, sa, b, sb, off = q["dev"]
    want = ops.moe_gated(ops.FMT_MXFP4, a, sa, b, sb, off, 32, 128)
    big, bigs = torch.zeros(200, 64, dtype=torch.uint8, device=DEV), torch.zeros(200, 4, dtype=torch.uint8, device=DEV)
    big[20:150], bigs[20:150] = a, sa
    got = ops.moe_gated(ops.FMT_MXFP4, big[20:150], bigs[20:150], b, sb, off, 32, 128)
    assert torch.equal(got["codes"], want["codes"]) and torch.equal(got["scales"], want["scales"])
    bigs[21:151] = sa
    with pytest.raises((RuntimeError, ValueError)):
        ops.moe_gated(ops.FMT_MXFP4, a, bigs[21:151], b, sb, off, 32, 128)
    wide = torch.zeros(130, 128, dtype=torch.uint8, device=DEV)
    with pytest.raises((RuntimeError, ValueError)):
        ops.moe_gated(ops.FMT_MXFP4, wide[:, :64], sa, b, sb, off, 32, 128)
    with pytest.raises((RuntimeError, ValueError)):
        ops.moe_gated(ops.FMT_MXFP4, a, sa, b, sb, off, 32, 128, out={"codes": want["codes"][:5], "scales": want["scales"]})
    with pytest.raises((RuntimeError, ValueError)):
        ops.moe_gated(ops.FMT_MXFP4, a, sa, b, sb, off, 32, 128, workspace=torch.zeros(64, dtype=torch.uint8, device=DEV))
