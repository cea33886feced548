"""Routing on the GPU against its definition in binary64: choice, counts and
row map exactly; weights, probability sums, loss and gradient within the
rounding of an f32 evaluation."""
import numpy as np
import pytest
import torch

from block_scaled_precision_token_amd import ops
from tests import moe_reference as ref
from tests.gpu_util import DEV, host, to_dev

pytestmark = pytest.mark.gpu

# additions in one chain of a probability sum: a lane's tokens, the tree, the runs
SUM_CHAIN = 600


def logits_of(seed, T, E, dtype, kind="normal", pad=0):
    """(device [T, E] with row stride E + pad, f64 values)"""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, E)) * 1.5
    if kind == "ties":
        x = np.round(x)                        # many equal logits, -0 and +0 among them
        x[rng.random((T, E)) < 0.1] = -0.0
    if kind == "lowest":                       # a mask by the type's lowest value instead of -inf
        x[rng.random((T, E)) < 0.7] = float(torch.finfo(dtype).min)
    if kind == "unavailable":
        x[rng.random((T, E)) < 0.5] = -np.inf
        x[T // 2] = -np.inf
    if kind == "wide":
        x *= 30
    d = torch.full((T, E + pad), float("nan"), dtype=dtype, device=DEV)
    d[:, :E] = torch.from_numpy(x).to(dtype).to(DEV)
    view = d[:, :E]
    return view, view.double().cpu().numpy()


def check_forward(got, want, x, k, mask=None, aux=True):
    for name in ("experts", "counts", "group_offsets", "src", "pos"):
        a, b = host(got[name]), want[name]
        assert a.shape == b.shape and a.dtype == b.dtype, name
        assert np.array_equal(a, b), f"{name}: first at {np.argwhere(a != b)[:3].tolist()}"
    span, E = ref.logit_span(x, mask), x.shape[1]
    tol = ref.weight_tol(span, E)
    for name in ("weights", "row_weights"):
        a, b = host(got[name]).astype(np.float64), want[name]
        assert np.array_equal(np.isnan(a), np.isnan(b)), name
        ok = ~np.isnan(b)
        assert np.all(np.abs(a - b)[ok] <= tol * b[ok] + 2.0 ** -126), name     # f32 flushes below 2^-126
    if aux:
        stol = tol + SUM_CHAIN * ref.EPS
        a, b = host(got["prob_sum"]).astype(np.float64), want["prob_sum"]
        assert np.array_equal(np.isnan(a), np.isnan(b))
        if not np.isnan(b).any():
            assert np.all(np.abs(a - b) <= stol * b + x.shape[0] * 2.0 ** -126)
            assert abs(float(host(got["loss"])[0]) - want["loss"]) <= (stol + (E / 64 + 20) * ref.EPS) * want["loss"]
        else:
            assert np.isnan(host(got["loss"])[0])


CASES = [
    # T, E, k, shared, dtype, norm, kind, masked share, row padding
    (1, 128, 8, 0, "f32", True, "normal", 0.0, 0),
    (1, 1, 1, 0, "f32", True, "normal", 0.0, 0),
    (1, 64, 4, 1, "bf16", False, "normal", 0.0, 0),
    (2, 5, 5, 0, "f32", False, "normal", 0.0, 3),
    (31, 60, 4, 0, "f32", True, "ties", 0.0, 0),
    (63, 257, 32, 3, "f32", True, "normal", 0.2, 0),
    (64, 128, 8, 1, "bf16", True, "ties", 0.3, 8),
    (65, 129, 17, 64, "f32", False, "unavailable", 0.1, 1),
    (100, 65, 16, 0, "bf16", True, "wide", 0.0, 0),
    (130, 128, 8, 0, "f32", True, "ties", 0.0, 0),
    (256, 200, 7, 5, "bf16", False, "unavailable", 0.2, 0),
    (255, 64, 8, 0, "f32", True, "lowest", 0.0, 1),
    (257, 256, 8, 1, "f32", True, "normal", 0.0, 0),
    (256, 257, 8, 1, "f32", True, "normal", 0.0, 0),
    (300, 256, 8, 1, "bf16", True, "unavailable", 0.1, 0),
    (1000, 128, 8, 0, "f32", True, "normal", 0.0, 0),
    (1025, 96, 6, 0, "f32", False, "lowest", 0.0, 4),
    (777, 512, 10, 2, "f32", True, "ties", 0.5, 0),
    (513, 1024, 32, 1, "bf16", False, "unavailable", 0.0, 0),
    (520, 1000, 9, 0, "f32", True, "wide", 0.1, 0),
    (20001, 16, 2, 1, "f32", True, "normal", 0.05, 0),
    (200003, 8, 3, 0, "bf16", True, "ties", 0.01, 0),     # runs longer than one ranking pass
]
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.mark.parametrize("T,E,k,shared,dtype,norm,kind,masked,pad", CASES)
def test_route_forward_and_backward(T, E, k, shared, dtype, norm, kind, masked, pad):
    seed = T * 7 + E
    xd, x = logits_of(seed, T, E, DT[dtype], kind, pad)
    rng = np.random.default_rng(seed + 1)
    mask = maskd = None
    if masked:
        mask = rng.random(T) >= masked
        maskd = to_dev(mask)
        xd[~maskd] = float("nan")              # a padding token's logits may hold anything
    want = ref.route(x, k, norm, shared, mask)
    got = ops.moe_route(xd, k, norm=norm, shared=shared, token_mask=maskd, aux=True)
    check_forward(got, want, x, k, mask)
    # gradient of both parts, each part alone
    d_rows = rng.standard_normal(T * (k + shared)).astype(np.float32)
    tol = 2 * ref.weight_tol(ref.logit_span(x, mask), E) + (E / 8 + 32) * ref.EPS
    for parts in ("both", "loss", "weights"):
        dl = None if parts == "weights" else 0.31
        dr = None if parts == "loss" else d_rows
        grad, size = ref.route_backward(x, k, want, dr, dl, norm, shared, mask)
        g = ops.moe_route_backward(xd, k, got["experts"], got["counts"], got["pos"],
                                   d_weights=None if dr is None else to_dev(dr),
                                   d_loss=None if dl is None else torch.tensor([dl], device=DEV), norm=norm,
                                   shared=shared, token_mask=maskd)
        assert g.dtype == DT[dtype] and g.shape == (T, E)
        err = np.abs(g.double().cpu().numpy() - grad)
        allowed = tol * size + 1e-37 + (2.0 ** -8 * np.abs(grad) if dtype == "bf16" else 0.0)
        assert np.all(err <= allowed), (parts, float((err / allowed).max()))


def test_all_tokens_masked_or_without_experts():
    for T in (40, 400):
        xd, x = logits_of(5, T, 24, torch.float32)
        for variant in ("mask", "inf"):
            mask = torch.zeros(T, dtype=torch.uint8, device=DEV) if variant == "mask" else None
            xx = xd.clone()
            if variant == "inf":
                xx.fill_(-float("inf"))
            r = ops.moe_route(xx, 3, shared=1, token_mask=mask, aux=True)
            assert (r["experts"] == -1).all() and (r["pos"] == -1).all() and (r["src"] == -1).all()
            assert (r["weights"] == 0).all() and (r["row_weights"] == 0).all()
            assert (r["counts"] == 0).all() and (r["group_offsets"] == 0).all()
            assert float(r["loss"]) == 0.0 and (r["prob_sum"] == 0).all()
            g = ops.moe_route_backward(xx, 3, r["experts"], r["counts"], r["pos"],
                                       d_weights=torch.ones(T * 4, device=DEV), d_loss=torch.ones(1, device=DEV),
                                       shared=1, token_mask=mask)
            assert (g == 0).all()


@pytest.mark.parametrize("T", [50, 700])
def test_rows_with_nan_or_inf_show_and_stay_contained(T):
    xd, x = logits_of(6, T, 40, torch.float32)
    xd[3, 7], x[3, 7] = float("nan"), np.nan
    xd[T - 2, 0], x[T - 2, 0] = float("inf"), np.inf
    xd[9], x[9] = float("nan"), np.nan
    want = ref.route(x, 4, True, 1)
    got = ops.moe_route(xd, 4, shared=1, aux=True)
    check_forward(got, want, x, 4)
    assert np.isnan(host(got["weights"])[[3, 9, T - 2], :4]).all()
    g = ops.moe_route_backward(xd, 4, got["experts"], got["counts"], got["pos"],
                               d_loss=torch.ones(1, device=DEV), shared=1)
    bad = torch.isnan(g).any(1).cpu().numpy()
    assert bad[[3, 9, T - 2]].all() and bad.sum() == 3


def test_backward_takes_global_counts():
    """Two ranks: with the sums of both counts each gradient is that of the loss over all tokens."""
    T, E, k = 90, 32, 4
    xd, x = logits_of(8, 2 * T, E, torch.float32)
    whole = ops.moe_route(xd, k, aux=True)
    halves = [xd[:T].contiguous(), xd[T:].contiguous()]
    fwd = [ops.moe_route(h, k, aux=True) for h in halves]
    counts = fwd[0]["counts"] + fwd[1]["counts"]
    assert torch.equal(counts, whole["counts"])
    one = torch.ones(1, device=DEV)
    g = torch.cat([ops.moe_route_backward(h, k, f["experts"], counts, f["pos"], d_loss=one)
                   for h, f in zip(halves, fwd)])
    gw = ops.moe_route_backward(xd, k, whole["experts"], whole["counts"], whole["pos"], d_loss=one)
    assert torch.equal(g, gw)


def test_backward_ignores_indices_out_of_range():
    T, E, k = 70, 20, 3
    xd, x = logits_of(9, T, E, torch.float32)
    r = ops.moe_route(xd, k)
    d = torch.randn(T * k, device=DEV)
    ex, pos = r["experts"].clone(), r["pos"].clone()
    ex[4, 1], ex[5, 0], pos[6, 2], pos[7, 0] = E, 1 << 30, T * k, -5
    want = ops.moe_route_backward(xd, k, r["experts"], r["counts"], r["pos"], d_weights=d, norm=False)
    got = ops.moe_route_backward(xd, k, ex, r["counts"], pos, d_weights=d, norm=False)
    same = np.ones(T, bool)
    same[4:8] = False
    assert torch.equal(got[torch.from_numpy(same).to(DEV)], want[torch.from_numpy(same).to(DEV)])
    assert torch.isfinite(got).all()


def test_results_repeat_bit_for_bit_and_buffers_are_reused():
    xd, _ = logits_of(10, 3000, 128, torch.float32)
    a = ops.moe_route(xd, 8, aux=True)
    saved = {k: v.clone() for k, v in a.items()}
    ws = torch.full((ops.moe_route_workspace_size(3000, 128, 8),), 0xAB, dtype=torch.uint8, device=DEV)
    for t in a.values():
        t.fill_(77)
    b = ops.moe_route(xd, 8, aux=True, out=a, workspace=ws)
    for k in saved:
        assert b[k].data_ptr() == a[k].data_ptr() and torch.equal(saved[k], b[k]), k


def test_route_on_another_stream_and_in_a_graph():
    xd, x = logits_of(11, 900, 96, torch.float32)
    eager = ops.moe_route(xd, 6, aux=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        r = ops.moe_route(xd, 6, aux=True)
    s.synchronize()
    for k in eager:
        assert torch.equal(eager[k], r[k]), k
    d = torch.randn(900 * 6, device=DEV)
    one = torch.ones(1, device=DEV)
    grad = ops.moe_route_backward(xd, 6, eager["experts"], eager["counts"], eager["pos"], d_weights=d, d_loss=one)
    out = {k: torch.empty_like(v) for k, v in eager.items()}
    gout = torch.empty_like(grad)
    ws = torch.empty(ops.moe_route_workspace_size(900, 96, 6), dtype=torch.uint8, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.moe_route(xd, 6, aux=True, out=out, workspace=ws)
        ops.moe_route_backward(xd, 6, out["experts"], out["counts"], out["pos"], d_weights=d, d_loss=one, out=gout)
    for _ in range(3):
        for t in list(out.values()) + [gout, ws]:
            t.fill_(3)
        ops.moe_route(xd[:50].contiguous(), 6)             # unrelated eager work between replays
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for k in eager:
            assert torch.equal(eager[k], out[k]), k
        assert torch.equal(grad, gout)


COMBINE = [
    # T, kk, rows, H, in, out, weighted, row padding
    (1, 1, 1, 8, "f32", "f32", True, 0),
    (1, 8, 8, 2048, "bf16", "bf16", True, 0),
    (3, 9, 40, 136, "bf16", "f32", False, 8),
    (257, 4, 900, 264, "f32", "bf16", True, 16),
    (700, 10, 7000, 1000, "bf16", "bf16", False, 0),
    (33, 128, 3000, 72, "f32", "f32", True, 0),
]


@pytest.mark.parametrize("T,kk,rows,H,ti,to,weighted,pad", COMBINE)
def test_combine(T, kk, rows, H, ti, to, weighted, pad):
    rng = np.random.default_rng(T + kk)
    y = torch.from_numpy(rng.standard_normal((rows, H + pad)).astype(np.float32)).to(DT[ti]).to(DEV)[:, :H]
    pos = rng.integers(0, rows, (T, kk)).astype(np.int32)
    pos[rng.random((T, kk)) < 0.15] = -1
    pos[T // 2] = -1                                        # a token without rows
    pos[0, 0] = rows if T > 1 else pos[0, 0]                # past the rows: nothing
    w = rng.standard_normal((T, kk)).astype(np.float32) if weighted else None
    out = torch.full((T, H + pad), 7.0, dtype=DT[to], device=DEV)
    got = ops.moe_combine(y, to_dev(pos), None if w is None else to_dev(w), out=out[:, :H])
    want, size = ref.combine(y.double().cpu().numpy(), pos, w)
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= (kk + 1) * ref.EPS * size + (2.0 ** -8 * np.abs(want) if to == "bf16" else 0.0) + 1e-37)
    assert (out[:, H:] == 7.0).all()


def test_combine_does_not_read_rows_that_no_token_has():
    y = torch.full((20, 64), float("nan"), device=DEV)
    y[[2, 5, 11]] = 1.0
    pos = torch.tensor([[2, -1, 5], [11, 11, -1], [-1, -1, -1]], dtype=torch.int32, device=DEV)
    out = ops.moe_combine(y, pos)
    assert out[:, 0].tolist() == [2.0, 2.0, 0.0] and torch.isfinite(out).all()


def test_row_map_drives_the_grouped_gemm_with_padding_tokens():
    """group_offsets[G] below M: rows past it are left untouched, the others are the experts' products."""
    T, E, k, K, N = 200, 6, 2, 64, 48
    xd, x = logits_of(12, T, E, torch.float32)
    mask = np.random.default_rng(1).random(T) >= 0.3
    r = ops.moe_route(xd, k, token_mask=to_dev(mask))
    a = torch.randn(T, K, device=DEV).to(torch.bfloat16)
    b = torch.randn(E, N, K, device=DEV).to(torch.bfloat16)
    out = torch.full((T * k, N), 5.0, device=DEV)
    ops.moe_grouped_gemm_bf16(ops.GEMM_FPROP, a, b, r["group_offsets"], N, K, M=T * k, gather=r["src"], out=out)
    off = host(r["group_offsets"])
    src = host(r["src"])
    used = int(off[-1])
    assert used == mask.sum() * k
    af, bf = a.double().cpu().numpy(), b.double().cpu().numpy()
    g = np.searchsorted(off, np.arange(used), side="right") - 1
    want = np.einsum("rk,rnk->rn", af[src[:used]], bf[g])
    size = np.einsum("rk,rnk->rn", np.abs(af[src[:used]]), np.abs(bf[g]))
    got = host(out)
    assert np.all(np.abs(got[:used] - want) <= 1e-3 * size)
    assert np.all(got[used:] == 5.0)


def test_row_map_drives_the_grouped_quantizer_with_padding_tokens():
    """The columnwise copy of grouped rows stops at group_offsets[G], as if the rows past it were not there."""
    T, E, k, H = 150, 5, 3, 64
    xd, _ = logits_of(13, T, E, torch.float32)
    mask = np.random.default_rng(2).random(T) >= 0.4
    r = ops.moe_route(xd, k, token_mask=to_dev(mask))
    off = r["group_offsets"]
    used = int(off[-1])
    assert 0 < used < T * k
    x = torch.randn(T, H, device=DEV).to(torch.bfloat16)
    ld = ops.mxfp8_grouped_cols(T * k, E)

    def copy(gather):
        out = {"codes_colT": torch.full((H, ld), 0x5A, dtype=torch.uint8, device=DEV),
               "scales_colT": torch.full((H, ld // 32), 0x5A, dtype=torch.uint8, device=DEV)}
        return ops.quantize_mxfp8(x, False, True, group_offsets=off, row_gather=gather, out=out)
    a, b = copy(r["src"]), copy(r["src"][:used].contiguous())
    assert torch.equal(a["codes_colT"], b["codes_colT"]) and torch.equal(a["scales_colT"], b["scales_colT"])
