"""One mixture-of-experts layer, forward and backward, from this library's operators.

    python examples/moe_layer.py [--tokens 4096] [--hidden 2048] [--intermediate 768] [--experts 128] [--topk 8]

The layer runs as a training step uses it: router logits to experts, counts, row map and load-balance loss
(moe_route), MXFP8 quantization and the grouped gate/up product, SwiGLU with the router's weight of each row and an
8-bit checkpoint of its input (swiglu_checkpoint), the grouped down product, and the sum of every token's rows
(moe_combine).  Backward: the data gradient through the down projection reads the output's gradient through the row
map, swiglu_checkpoint_backward gives the gradient of gate and up, h again and the gradient of the row weights, the
BF16 grouped products give the weight gradients, moe_combine sums the input's gradient, and moe_route_backward the
gradient to the router's logits.  Neither h13, h nor the down projection's output is kept between the two passes.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
from block_scaled_precision_token_amd import ops, synth  # noqa: E402


class MoeLayer:
    """Weights in bf16: router [E, H], gate/up [E, 2I, H], down [E, H, I]; the expert products run in MXFP8 forward
    and BF16 backward."""

    def __init__(self, H, I, E, k, balance=0.01, seed=1, device="cuda:0"):
        self.H, self.I, self.E, self.k = H, I, E, k
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.router = torch.randn((E, H), generator=g, device=device) * H ** -0.5
        self.w13 = synth.device_weights(seed + 1, E, 2 * I, H, device).view(E, 2 * I, H)
        self.w2 = synth.device_weights(seed + 2, E, H, I, device).view(E, H, I)
        self.w13q = ops.quantize_mxfp8(self.w13)
        self.w2q = ops.quantize_mxfp8(self.w2)
        self.balance = torch.full((1,), balance, device=device)

    def forward(self, x, token_mask=None):
        """x [T, H] bf16 -> (y [T, H] bf16, balance loss, what the backward pass keeps)."""
        T, (H, I, E, k) = x.shape[0], (self.H, self.I, self.E, self.k)
        R = T * k
        logits = x.float() @ self.router.t()
        r = ops.moe_route(logits, k, token_mask=token_mask, aux=True)
        off, src = r["group_offsets"], r["src"]
        xq = ops.quantize_mxfp8(x)
        h13 = ops.moe_grouped_gemm_blockscaled(ops.FMT_MXFP8, ops.GEMM_FPROP, xq["codes_row"], xq["scales_row"],
                                               self.w13q["codes_row"], self.w13q["scales_row"], off, 2 * I, H, M=R,
                                               a_gather=src, out_dtype=torch.bfloat16)
        c = ops.swiglu_checkpoint(h13, row_weights=r["row_weights"], n_rows=off[E:], return_h=False, quantize_h=True)
        y = ops.moe_grouped_gemm_blockscaled(ops.FMT_MXFP8, ops.GEMM_FPROP, c["codes"], c["scales"],
                                             self.w2q["codes_row"], self.w2q["scales_row"], off, H, I,
                                             out_dtype=torch.bfloat16)
        out = ops.moe_combine(y, r["pos"])
        saved = (x, logits, token_mask, r, c["ckpt_codes"], c["ckpt_scales"])
        return out, r["loss"], saved

    def backward(self, dy, saved):
        """dy [T, H] bf16 -> gradients of x, router, w13 and w2 of (dy . y + balance * loss)."""
        x, logits, token_mask, r, ckpt_codes, ckpt_scales = saved
        T, (H, I, E, k) = x.shape[0], (self.H, self.I, self.E, self.k)
        R = T * k
        off, src = r["group_offsets"], r["src"]
        # the gradient of a grouped row is its token's: read through the row map
        dh = ops.moe_grouped_gemm_bf16(ops.GEMM_DGRAD, dy, self.w2, off, I, H, M=R, gather=src,
                                       out_dtype=torch.bfloat16)
        b = ops.swiglu_checkpoint_backward(dh, ckpt_codes, ckpt_scales, row_weights=r["row_weights"], n_rows=off[E:])
        # dW2_e^T [I, H] = h^T dy, dW13_e [2I, H] = dh13^T x, over the expert's rows
        dw2 = ops.moe_grouped_gemm_bf16(ops.GEMM_WGRAD, b["h"], dy, off, H, R, gather=src)
        dw13 = ops.moe_grouped_gemm_bf16(ops.GEMM_WGRAD, b["dh13"], x, off, H, R, gather=src)
        dx_rows = ops.moe_grouped_gemm_bf16(ops.GEMM_DGRAD, b["dh13"], self.w13, off, H, 2 * I,
                                            out_dtype=torch.bfloat16)
        dlogits = ops.moe_route_backward(logits, k, r["experts"], r["counts"], r["pos"],
                                         d_weights=b["d_row_weights"], d_loss=self.balance, token_mask=token_mask)
        dx = ops.moe_combine(dx_rows, r["pos"], out_dtype=torch.float32) + dlogits @ self.router
        return {"x": dx, "router": dlogits.t() @ x.float(), "w13": dw13, "w2": dw2.transpose(1, 2)}


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("tokens", 4096), ("hidden", 2048), ("intermediate", 768), ("experts", 128), ("topk", 8)):
        ap.add_argument(f"--{name}", type=int, default=value)
    args = ap.parse_args()
    layer = MoeLayer(args.hidden, args.intermediate, args.experts, args.topk)
    x = synth.device_activations(11, args.tokens, args.hidden, outlier_frac=0.0)
    dy = synth.device_activations(12, args.tokens, args.hidden, outlier_frac=0.0, std=0.01)
    for i in range(3):
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        y, loss, saved = layer.forward(x)
        grads = layer.backward(dy, saved)
        torch.cuda.synchronize()
        print(f"step {i}: {1e3 * (time.perf_counter() - t0):.2f} ms, balance loss {float(loss):.4f}, "
              f"|y| {float(y.float().norm()):.3f}, " + ", ".join(f"|d{n}| {float(g.float().norm()):.3g}"
                                                               for n, g in grads.items()), flush=True)


if __name__ == "__main__":
    main()
