"""Calls whose persistent workgroups walk several tiles each: the ring of stages, the row tables and the list entries run
on from one tile to the next.  256 workgroups take tiles of 128 rows, 512 those of 64; K of one, two and three stages.
Bounds as in test_gpu_mx_sums: (K / 16 + 8) 2^-23 of sum |a b| for each product."""
import numpy as np
import pytest
import torch

from block_scaled_precision_token_amd import ops
from tests import mx_reference as mx
from tests import test_gpu_gated as gated
from tests import test_gpu_mx_products as products
from tests.gpu_util import DEV, to_dev

pytestmark = pytest.mark.gpu


def groups(kind):
    """(sizes, tile columns that make more than two tiles for each workgroup)."""
    rng = np.random.default_rng(12)
    if kind == "rows128":       # 20 groups, the largest many tiles long, four of them empty
        sizes = rng.integers(1, 600, 20)
        sizes[[0, 7, 8, 19]] = 0
        sizes[11] = 1100
        return sizes.tolist(), 11 * 256
    sizes = rng.integers(0, 50, 110)      # tiles of 64 rows, most groups one
    sizes[60] = 260
    return sizes.tolist(), 12 * 128


def tiles(sizes, N):
    tb, nb = (128, 256) if sum(sizes) // len(sizes) >= 96 else (64, 128)
    return sum(-(-n // tb) for n in sizes) * -(-N // nb), 256 if tb == 128 else 512


def operand(rng, rows, K, bits, std):
    """(codes, scales, values) of about N(0, std): random codes, blocks up to 2^3 apart."""
    c, s, v = products.operand(rng, rows, K, bits, 3)
    shift = int(np.round(np.log2(std / v.std())))
    return c, (s.astype(int) + shift).astype(np.uint8), v * 2.0 ** shift


@pytest.fixture(autouse=True)
def bounds(monkeypatch):
    monkeypatch.setattr(gated, "quantized", operand)
    check = products.check
    monkeypatch.setattr(products, "check", lambda got, ref, refabs, bits, K, bf16: check(got, ref, refabs, 4, 4 * K, bf16))
    monkeypatch.setattr(gated, "product_tol", lambda bits, K: (K / 16 + 8) * 2.0 ** -23)


@pytest.mark.parametrize("kind", ["rows128", "rows64"])
def test_the_cases_have_several_tiles_to_a_workgroup(kind):
    sizes, N = groups(kind)
    n, wgs = tiles(sizes, N)
    assert n > 2 * wgs


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", list(products.FORMATS))
@pytest.mark.parametrize("K", [32, 288])
@pytest.mark.parametrize("kind", ["rows128", "rows64"])
def test_products(kind, K, fmt, dtype):
    sizes, N = groups(kind)
    products.run_forward(fmt, sizes, N - 8, K, 0, dtype, gather=True, seed=K)


@pytest.mark.parametrize("fmt", list(gated.FORMATS))
@pytest.mark.parametrize("K", [32, 288])
@pytest.mark.parametrize("kind", ["rows128", "rows64"])
def test_gated_block(kind, K, fmt):
    sizes, N = groups(kind)
    gated.run_forward(fmt, sizes, N // 2 - 32, K, 0, seed=K, h_fmt=ops.FMT_MXFP4 if K == 32 else ops.FMT_MXFP8)


@pytest.mark.parametrize("fmt", list(gated.FORMATS))
@pytest.mark.parametrize("K", [32, 288])
@pytest.mark.parametrize("kind", ["rows128", "rows64"])
def test_gated_backward(kind, K, fmt):
    sizes, N = groups(kind)
    gated.run_backward(fmt, sizes, N - 32, K, 0, seed=K)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", list(products.FORMATS))
def test_weight_gradients(fmt, dtype):
    """Nine tiles to a matrix, 64 groups: 72 tiles for the 32 workgroups of an XCD, some of groups without tokens."""
    f, ab, bb = products.FORMATS[fmt]
    rng = np.random.default_rng(13)
    sizes = rng.integers(1, 300, 64)
    sizes[::5] = 0
    sizes[33] = 1500
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int64)
    P, ld = mx.padded_starts(off), ops.mxfp8_grouped_cols(int(off[-1]), 64)
    ac, as_, av = products.operand(rng, 300, ld, ab)
    bc, bs, bv = products.operand(rng, 520, ld, bb)
    out = torch.full((64, 300, 520), 77.0, dtype=dtype, device=DEV)
    ops.moe_grouped_gemm_blockscaled(f, ops.GEMM_WGRAD, *(to_dev(t) for t in (ac, as_, bc, bs, off)), 520, ld, out=out)
    got = products.f64(out)
    for g in range(64):
        a, b = av[:, P[g]:P[g + 1]], bv[:, P[g]:P[g + 1]]
        products.check(got[g], a @ b.T, np.abs(a) @ np.abs(b).T, ab, max(int(P[g + 1] - P[g]), 64),
                       dtype == torch.bfloat16)


@pytest.mark.parametrize("kind", ["rows128", "rows64"])
def test_bits_repeat_whatever_the_workspace_holds(kind):
    """Eager and replayed calls on workspaces of zeros, of ones and of an earlier call, give the same bytes."""
    sizes, N = groups(kind)
    I, K = N // 2, 288
    q = gated.problem("mxfp4", sizes, 2 * I, K, 3, True, 3, 0.3)
    R, n, G = q["R"], q["n"], len(sizes)
    w = to_dev(q["w"])
    cc, cs = (to_dev(t) for t in mx.mxfp8(q["rng"].standard_normal((R, 4 * I))))
    ws = torch.zeros(ops.moe_gated_workspace_size(ops.FMT_MXFP4, R, I, K, G), dtype=torch.uint8, device=DEV)
    wb = torch.zeros(ops.moe_gated_backward_workspace_size(ops.FMT_MXFP4, R, 2 * I, K, G), dtype=torch.uint8, device=DEV)
    kw = dict(R=R, a_gather=q["idx"], row_weights=w)

    def both():
        f = ops.moe_gated(ops.FMT_MXFP4, *q["dev"], I, K, checkpoint=True, return_h=True, workspace=ws, **kw)
        b = ops.moe_gated_backward(ops.FMT_MXFP4, *q["dev"], 2 * I, K, cc, cs, workspace=wb, **kw)
        return {**f, **{"bwd_" + k: v for k, v in b.items()}}

    first = {k: v[:n].clone() for k, v in both().items()}
    for fill in (255, None):
        if fill is not None:
            ws.fill_(fill)
            wb.fill_(fill)
        for k, v in both().items():
            assert torch.equal(v[:n], first[k]), k
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for fill in (0, 255, 1):
        ws.fill_(fill)
        wb.fill_(fill)
        for v in out.values():
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for k, v in out.items():
            assert torch.equal(v[:n], first[k]), k
