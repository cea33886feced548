"""The form that the library chooses by rows: up to BSP_FEW_ROWS the one without staging, which needs no workspace, then
tiles.  Bounds as in test_gpu_mx_sums."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

from block_scaled_precision_token_amd import ops
from tests import mx_reference as mx
from tests import test_gpu_gated as gated
from tests import test_gpu_mx_products as products
from tests.gpu_util import DEV, to_dev

pytestmark = pytest.mark.gpu

L = ops._lib_raw()
WORKSPACE = 5
# rows in groups, and behind the last: 1, 64 and 65 rows of a call
SPLITS = [([1], 0), ([20, 0, 44], 0), ([20, 0, 41], 3), ([20, 0, 45], 0), ([60, 1], 4)]


@pytest.fixture(autouse=True)
def bounds(monkeypatch):
    check = products.check
    monkeypatch.setattr(products, "check", lambda got, ref, refabs, bits, K, bf16: check(got, ref, refabs, 4, 4 * K, bf16))
    monkeypatch.setattr(gated, "product_tol", lambda bits, K: (K / 16 + 8) * 2.0 ** -23)


def test_the_bindings_constant_is_the_headers():
    with open(os.path.join(os.path.dirname(__file__), "..", "include", "bsp.h")) as f:
        assert int(re.search(r"#define BSP_FEW_ROWS (\d+)", f.read())[1]) == ops.FEW_ROWS == 64


@pytest.mark.parametrize("fmt", list(products.FORMATS))
@pytest.mark.parametrize("sizes,tail", SPLITS)
def test_products(sizes, tail, fmt):
    for dtype in (torch.float32, torch.bfloat16):
        products.run_forward(fmt, sizes, 72, 320, 0, dtype, tail=tail, seed=1)


@pytest.mark.parametrize("fmt", list(gated.FORMATS))
@pytest.mark.parametrize("sizes,tail", SPLITS)
def test_gated_block(sizes, tail, fmt):
    gated.run_forward(fmt, sizes, 96, 320, 0, tail=tail, h_fmt=ops.FMT_MXFP8)
    gated.run_forward(fmt, sizes, 96, 320, 0, tail=tail, h_fmt=ops.FMT_MXFP4, weighted=False)


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("fmt", list(gated.FORMATS))
@pytest.mark.parametrize("sizes,tail", SPLITS)
def test_gated_backward(sizes, tail, fmt, weighted):
    gated.run_backward(fmt, sizes, 96, 320, 0, tail=tail, weighted=weighted)


def call(q, fmt, R, w, out, dw, ws, nbytes, ck=None):
    """The C calls with this workspace: the backward's if ck, else the forward's; I = 96, K = 320."""
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    a, sa, b, sb, off = q["dev"]
    if ck is None:
        return L.bsp_moe_gated(fmt, p(a), p(sa), p(q["idx"]), a.shape[0], p(off), off.numel() - 1, R, 96, 320, p(b), p(sb),
                               p(w), p(out), -1, None, None, None, None, p(ws), nbytes, 0,
                               ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    return L.bsp_moe_gated_backward(fmt, p(a), p(sa), p(q["idx"]), a.shape[0], p(off), off.numel() - 1, R, 96, 320, p(b),
                                    p(sb), p(ck[0]), p(ck[1]), p(w), p(out), None, p(dw), p(ws), nbytes, 0,
                                    ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))


@pytest.mark.parametrize("fmt", list(gated.FORMATS))
def test_workspace_of_few_rows(fmt):
    """At 64 rows: none for the forward pass and for the backward pass without d_row_weights; its exact size with it, and
    nothing past it is written.  At 65 rows NULL is refused."""
    f = gated.FORMATS[fmt][0]
    for rows, ok in ((64, True), (65, False)):
        q = gated.problem(fmt, [20, rows - 20], 192, 320, 1, True, 0, 0.3)
        w = to_dev(q["w"])
        h = torch.zeros(rows, 96, dtype=torch.bfloat16, device=DEV)
        assert call(q, f, rows, w, h, None, None, 0) == (0 if ok else WORKSPACE)
        q = gated.problem(fmt, [20, rows - 20], 96, 320, 2, True, 0, 0.1)
        ck = [to_dev(t) for t in mx.mxfp8(q["rng"].standard_normal((rows, 192)))]
        dh13, dw = torch.zeros(rows, 192, dtype=torch.bfloat16, device=DEV), torch.zeros(rows, device=DEV)
        assert call(q, f, rows, w, dh13, None, None, 0, ck) == (0 if ok else WORKSPACE)
        need = ops.moe_gated_backward_workspace_size(f, rows, 96, 320, 2)
        assert need > 0
        ws = torch.full((need + 256,), 0xA5, dtype=torch.uint8, device=DEV)
        assert call(q, f, rows, w, dh13, dw, ws, need - 1, ck) == WORKSPACE
        assert call(q, f, rows, w, dh13, dw, ws, need, ck) == 0
        assert (ws[need:] == 0xA5).all()
        ref = ops.moe_gated_backward(f, *q["dev"], 96, 320, *ck, R=rows, a_gather=q["idx"], row_weights=w)
        assert torch.equal(ref["dh13"], dh13) and torch.equal(ref["d_row_weights"], dw)
        assert np.isfinite(dw.cpu().numpy()).all()
