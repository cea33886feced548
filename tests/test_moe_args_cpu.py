"""Refusals of the routing, checkpoint and combine calls, at the C ABI and in
the Python binding; nothing is launched, so no GPU is needed."""
import ctypes
import os

import pytest
import torch

from block_scaled_precision_token_amd import ops

if not os.path.exists(ops.LIB_PATH):
    pytest.skip("libbsp.so not built", allow_module_level=True)

L = ops.lib()
A = ctypes.c_void_p(1 << 20)            # 16-byte aligned, never dereferenced
MIS = ctypes.c_void_p((1 << 20) + 4)
BIG = 1 << 30
INVALID, SHAPE, ALIGN, WORKSPACE = 1, 2, 3, 5


def route(logits=A, dtype=0, T=500, E=64, ld=64, mask=None, k=4, shared=0, outs=(A,) * 7, ps=None, loss=None, flags=4,
          ws=A, nb=BIG):
    return L.bsp_moe_route(logits, dtype, T, E, ld, mask, k, shared, *outs, ps, loss, flags, ws, nb, None)


def test_route_refusals():
    assert route(logits=None) == INVALID
    for i in range(7):
        outs = [A] * 7
        outs[i] = None
        assert route(outs=outs) == INVALID
        outs[i] = MIS
        assert route(outs=outs) == ALIGN
    assert route(ps=A) == INVALID and route(loss=A) == INVALID          # both or neither
    assert route(dtype=2) == INVALID and route(flags=1) == INVALID
    assert route(T=0) == SHAPE and route(E=0, k=0) == SHAPE and route(E=1025, ld=1025) == SHAPE
    assert route(ld=63) == SHAPE and route(k=0) == SHAPE and route(k=33) == SHAPE
    assert route(E=4, ld=4, k=5) == SHAPE
    assert route(shared=-1) == SHAPE and route(shared=65) == SHAPE
    assert route(T=1 << 29) == SHAPE                                    # T * kk past 31 bits
    assert route(ws=None) == WORKSPACE and route(nb=L.bsp_moe_route_workspace_size(500, 64, 4, 0) - 1) == WORKSPACE
    assert route(logits=MIS) == ALIGN and route(mask=MIS) == ALIGN and route(ps=MIS, loss=A) == ALIGN


def test_route_workspace_size():
    ws = L.bsp_moe_route_workspace_size
    assert ws(0, 64, 4, 0) == 0 and ws(1000, 0, 4, 0) == 0 and ws(1000, 2000, 4, 0) == 0 and ws(1000, 64, 4, -1) == 0
    assert ws(1000, 64, 0, 0) == 0 and ws(1000, 64, 65, 0) == 0
    assert ws(1, 64, 4, 0) == 0                                         # one workgroup, nothing to exchange
    assert 0 < ws(1000, 64, 4, 0) < ws(1000, 128, 4, 1) < ws(8192, 128, 4, 1)
    assert ws(1 << 24, 1024, 4, 64) < 16 << 20                          # bounded by the number of runs


def test_route_backward_refusals():
    def bwd(logits=A, dtype=0, T=500, E=64, ld=64, mask=None, k=4, shared=0, ex=A, pos=A, counts=A, dw=A, dl=None,
            out=A, ldd=64, flags=4):
        return L.bsp_moe_route_backward(logits, dtype, T, E, ld, mask, k, shared, ex, pos, counts, dw, dl, out, ldd,
                                        flags, None)
    for name in ("logits", "ex", "pos", "counts", "out"):
        assert bwd(**{name: None}) == INVALID
        assert bwd(**{name: MIS}) == ALIGN
    assert bwd(dw=None) == INVALID                                      # nothing to differentiate
    assert bwd(dw=MIS) == ALIGN and bwd(dl=MIS) == ALIGN and bwd(mask=MIS) == ALIGN
    assert bwd(dtype=7) == INVALID and bwd(flags=2) == INVALID
    assert bwd(ldd=63) == SHAPE and bwd(ld=63) == SHAPE and bwd(T=0) == SHAPE and bwd(k=65) == SHAPE


def test_checkpoint_refusals():
    def fwd(x=A, dtype=1, R=8, I=64, w=None, n=None, h=A, codes=None, scales=None, cc=A, cs=A):
        return L.bsp_swiglu_checkpoint(x, dtype, R, I, w, n, h, codes, scales, cc, cs, None)
    assert fwd(x=None) == INVALID and fwd(cc=None) == INVALID and fwd(cs=None) == INVALID
    assert fwd(h=None) == INVALID and fwd(codes=A) == INVALID and fwd(scales=A) == INVALID
    assert fwd(dtype=2) == INVALID
    assert fwd(R=0) == SHAPE and fwd(I=0) == SHAPE and fwd(I=48) == SHAPE and fwd(R=1 << 31) == SHAPE
    for name in ("x", "w", "h", "cc", "cs", "n"):
        assert fwd(**{name: MIS}) == ALIGN
    assert fwd(codes=MIS, scales=A) == ALIGN

    def bwd(dh=A, dtype=1, R=8, I=64, cc=A, cs=A, w=None, n=None, out=A, h=None, dw=None):
        return L.bsp_swiglu_checkpoint_backward(dh, dtype, R, I, cc, cs, w, n, out, h, dw, None)
    for name in ("dh", "cc", "cs", "out"):
        assert bwd(**{name: None}) == INVALID
    assert bwd(dtype=-1) == INVALID and bwd(R=-1) == SHAPE and bwd(I=40) == SHAPE
    for name in ("dh", "cc", "cs", "w", "n", "out", "h", "dw"):
        assert bwd(**{name: MIS}) == ALIGN


def test_combine_refusals():
    def comb(y=A, di=1, rows=9, H=64, ldy=64, pos=A, w=None, T=3, kk=3, out=A, do=1, ldo=64):
        return L.bsp_moe_combine(y, di, rows, H, ldy, pos, w, T, kk, out, do, ldo, None)
    for name in ("y", "pos", "out"):
        assert comb(**{name: None}) == INVALID
        assert comb(**{name: MIS}) == ALIGN
    assert comb(w=MIS) == ALIGN and comb(di=2) == INVALID and comb(do=2) == INVALID
    assert comb(rows=0) == SHAPE and comb(T=0) == SHAPE and comb(H=60) == SHAPE and comb(ldy=56) == SHAPE
    assert comb(ldo=56) == SHAPE and comb(kk=0) == SHAPE and comb(kk=129) == SHAPE and comb(T=1 << 30) == SHAPE
    assert comb(ldy=68) == ALIGN and comb(ldo=68) == ALIGN


@pytest.fixture
def cpu_ops(monkeypatch):
    """The binding's checks with the library stubbed out: CPU tensors pass for device tensors."""
    class Stub:
        def __getattr__(self, name):
            if name.endswith("workspace_size"):
                return getattr(L, name)
            raise AssertionError(f"{name} was called")
    monkeypatch.setattr(ops, "DEVICE_TYPE", "cpu")
    monkeypatch.setattr(ops, "_lib_raw", lambda: Stub())
    monkeypatch.setattr(ops, "_stream", lambda dev: None)
    return ops


def rejects(fn, *args, match, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*args, **kw)


def test_binding_checks_every_tensor(cpu_ops):
    f32, i32, u8 = torch.float32, torch.int32, torch.uint8
    z = lambda *s, dtype=f32: torch.zeros(s, dtype=dtype)  # noqa: E731
    x = z(200, 16)
    rejects(cpu_ops.moe_route, x.half(), 2, match="dtype")
    rejects(cpu_ops.moe_route, x.t(), 2, match="unit column stride")
    rejects(cpu_ops.moe_route, x, 0, match="k = 0")
    rejects(cpu_ops.moe_route, x, 2, token_mask=z(199, dtype=u8), match="token_mask")
    rejects(cpu_ops.moe_route, x, 2, token_mask=z(200), match="token_mask")
    rejects(cpu_ops.moe_route, x, 2, workspace=z(16, dtype=u8), match="workspace")
    good = {"experts": z(200, 2, dtype=i32), "weights": z(200, 2), "counts": z(17, dtype=i32),
            "group_offsets": z(17, dtype=torch.int64), "src": z(400, dtype=i32), "pos": z(200, 2, dtype=i32),
            "row_weights": z(400)}
    for name, t in good.items():
        rejects(cpu_ops.moe_route, x, 2, out={**good, name: t.reshape(-1)[1:].clone()}, match=name)
        rejects(cpu_ops.moe_route, x, 2, out={**good, name: t.to(torch.float64)}, match=name)
        rejects(cpu_ops.moe_route, x, 2, out={k: v for k, v in good.items() if k != name}, match=name)
    rejects(cpu_ops.moe_route, x, 2, out=good, aux=True, match="prob_sum")

    bwd = cpu_ops.moe_route_backward
    ex, cnt, pos = good["experts"], good["counts"], good["pos"]
    rejects(bwd, x, 2, ex[1:].clone(), cnt, pos, d_weights=z(400), match="experts")
    rejects(bwd, x, 2, ex, cnt[1:].clone(), pos, d_weights=z(400), match="counts")
    rejects(bwd, x, 2, ex, cnt, pos.long(), d_weights=z(400), match="pos")
    rejects(bwd, x, 2, ex, cnt, pos, d_weights=z(399), match="d_weights")
    rejects(bwd, x, 2, ex, cnt, pos, d_loss=z(1, dtype=torch.float64), match="d_loss")
    rejects(bwd, x, 2, ex, cnt, pos, d_weights=z(400), out=z(200, 15), match="out")
    rejects(bwd, x, 2, ex, cnt, pos, d_weights=z(400), out=z(200, 16, dtype=torch.bfloat16), match="out")

    fwd = cpu_ops.swiglu_checkpoint
    h13 = z(8, 128)
    rejects(fwd, h13.half(), match="dtype")
    rejects(fwd, z(8, 96), match="multiple of 64")
    rejects(fwd, h13, row_weights=z(7), match="row_weights")
    rejects(fwd, h13, n_rows=z(1, dtype=i32), match="n_rows")
    ck = {"ckpt_codes": z(8, 128, dtype=u8), "ckpt_scales": z(8, 4, dtype=u8)}
    rejects(fwd, h13, out=ck, match="h is required")
    rejects(fwd, h13, out={**ck, "ckpt_scales": z(8, 3, dtype=u8)}, return_h=False, match="ckpt_scales")
    rejects(fwd, h13, out=ck, return_h=False, quantize_h=True, match="codes")

    back = cpu_ops.swiglu_checkpoint_backward
    dh = z(8, 64)
    rejects(back, z(8, 40), ck["ckpt_codes"], ck["ckpt_scales"], match="multiple of 32")
    rejects(back, dh, ck["ckpt_codes"][1:].clone(), ck["ckpt_scales"], match="ckpt_codes")
    rejects(back, dh, ck["ckpt_codes"], ck["ckpt_scales"][1:].clone(), match="ckpt_scales")
    rejects(back, dh, ck["ckpt_codes"], ck["ckpt_scales"], row_weights=z(8, dtype=torch.bfloat16), match="row_weights")
    rejects(back, dh, ck["ckpt_codes"], ck["ckpt_scales"], out={"dh13": z(8, 128, dtype=torch.bfloat16)}, match="dh13")

    rejects(cpu_ops.moe_combine, z(9, 64), pos.reshape(-1), match="2-D")
    rejects(cpu_ops.moe_combine, z(9, 64), pos.long(), match="pos")
    rejects(cpu_ops.moe_combine, z(9, 64), pos, weights=z(200, 1), match="weights")
    rejects(cpu_ops.moe_combine, z(9, 64), pos, out=z(199, 64), match="out")
