"""Rows from n_rows on are not read: with the inputs in pinned host memory, which
the GPU reads a hundred times slower than its own, a call with a few rows in use
takes a fraction of the time of a call that uses them all."""
import pytest
import torch

from block_scaled_precision_token_amd import ops
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu

R, I = 16384, 768


def milliseconds(call):
    best = 1e9
    for _ in range(4):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        assert call() == 0
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


def test_unused_rows_are_not_read():
    u8, bf16 = torch.uint8, torch.bfloat16
    lib, stream = ops.lib(), torch.cuda.current_stream().cuda_stream
    h13 = torch.randn(R, 2 * I).to(bf16).pin_memory()
    dev = lambda *s, dtype=u8: torch.empty(s, dtype=dtype, device=DEV)  # noqa: E731
    h, codes, scales = dev(R, I, dtype=bf16), dev(R, 2 * I), dev(R, 2 * I // 32)
    few, all_ = (torch.full((1,), n, dtype=torch.int64, device=DEV) for n in (16, R))

    def forward(n):
        return lib.bsp_swiglu_checkpoint(h13.data_ptr(), ops.DTYPE_BF16, R, I, None, n.data_ptr(), h.data_ptr(), None,
                                         None, codes.data_ptr(), scales.data_ptr(), stream)
    assert milliseconds(lambda: forward(few)) < 0.25 * milliseconds(lambda: forward(all_))
    want = ops.swiglu_checkpoint(h13.to(DEV))
    torch.cuda.synchronize()
    assert torch.equal(h, want["h"]) and torch.equal(codes, want["ckpt_codes"])

    dh, hc, hs = torch.randn(R, I).to(bf16).pin_memory(), codes.cpu().pin_memory(), scales.cpu().pin_memory()
    dh13 = dev(R, 2 * I, dtype=bf16)

    def backward(n):
        return lib.bsp_swiglu_checkpoint_backward(dh.data_ptr(), ops.DTYPE_BF16, R, I, hc.data_ptr(), hs.data_ptr(),
                                                  None, n.data_ptr(), dh13.data_ptr(), None, None, stream)
    assert milliseconds(lambda: backward(few)) < 0.25 * milliseconds(lambda: backward(all_))
    want = ops.swiglu_checkpoint_backward(dh.to(DEV), codes, scales, return_h=False)["dh13"]
    torch.cuda.synchronize()
    assert torch.equal(dh13, want)
