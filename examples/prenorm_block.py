"""One training step of a pre-norm block whose feed-forward part is the expert layer, with a router balance loss.

    python examples/prenorm_block.py [--form bf16|e4m3|mx] [--tokens T] [--steps N]

For a sublayer's output x and the residual stream r (attention and the rest of the model lie outside):

    h = r + x,  y = rmsnorm(h) * g     (with the layer's FP8 operand written in the same pass for e4m3 and mx)
    out = h + MoE(y),  loss = mean((out - target)^2) / 2 + balance_coef * balance + z_coef * z

and backwards: the layer, the balance loss's gradient through the router, the norm.  Each weight takes a
step against its gradient, so the printed loss falls.
"""
from __future__ import annotations

import argparse
import os
import sys
from dataclasses import dataclass

import torch

if __package__ in (None, ""):
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import varlen_grouped_gemm_gb300 as vgg  # noqa: E402

BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


@dataclass
class Block:
    """Weights, and every tensor of a step for T tokens."""

    ctx: vgg.Context
    form: str
    weight: torch.Tensor    # the norm's
    W_r: torch.Tensor
    W_gate: torch.Tensor
    W_up: torch.Tensor
    W_down: torch.Tensor
    buf: vgg.Buffers
    h: torch.Tensor         # the stream after the addition, fp32
    y: torch.Tensor
    rstd: torch.Tensor
    balance: torch.Tensor   # loss, balance, z
    counts: torch.Tensor
    probs: torch.Tensor
    dlogits: torch.Tensor   # the balance loss's gradient of the logits
    dx: torch.Tensor
    dres: torch.Tensor
    dweight: torch.Tensor
    ws_norm: torch.Tensor
    ws_balance: torch.Tensor
    ws_router: torch.Tensor
    seq_offsets: torch.Tensor | None = None
    balance_coef: float = 1e-2
    z_coef: float = 1e-3
    eps: float = 1e-6

    @staticmethod
    def make(T, d, E, n, K, form="bf16", seq_offsets=None, seed=0, device="cuda") -> "Block":
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(shape, device=device, generator=g) * std).to(BF)

        def empty(*shape, dtype=F32):
            return torch.empty(shape, dtype=dtype, device=device)

        B = 1 if seq_offsets is None else seq_offsets.numel() - 1
        return Block(
            vgg.Context(torch.device(device).index or 0), form, torch.ones(d, device=device),
            normal(d, E, std=d ** -0.5), normal(E, n, d, std=d ** -0.5), normal(E, n, d, std=d ** -0.5),
            normal(E, d, n, std=n ** -0.5),
            vgg.Buffers.allocate(T, d, E, n, K, e4m3=form == "e4m3", mx=form == "mx", device=device),
            empty(T, d), empty(T, d, dtype=BF), empty(T), empty(3), empty(B, E, dtype=torch.int32), empty(B, E),
            empty(T, E), empty(T, d, dtype=BF), empty(T, d), empty(d),
            empty(vgg.moe_add_rmsnorm_workspace_bytes(T, d), dtype=U8),
            empty(vgg.moe_balance_loss_workspace_bytes(T, E, B), dtype=U8),
            empty(vgg.moe_router_backward_workspace_bytes(T, d, E), dtype=U8), seq_offsets)

    def forward(self, x, residual):
        """out = h + MoE(rmsnorm(h)), fp32, for x [T, d] bf16 and the stream residual [T, d] fp32."""
        b = self.buf
        q, scales = {"bf16": (None, None), "e4m3": (b.xq, b.xs), "mx": (b.mxq, b.mxsf)}[self.form]
        vgg.moe_add_rmsnorm(self.ctx, x, residual, self.weight, self.eps, self.h, self.y, self.rstd, q, scales)
        if self.form == "e4m3":
            self.quantized = vgg.E4m3Weights.quantize(self.ctx, self.W_gate, self.W_up, self.W_down, backward=True)
            vgg.forward_e4m3(self.ctx, self.y, self.W_r, None, self.quantized, None, b, quantized=True)
        elif self.form == "mx":
            self.quantized = vgg.MxWeights.quantize(self.ctx, self.W_gate, self.W_up, self.W_down, backward=True)
            vgg.forward_mx(self.ctx, self.y, self.W_r, None, self.quantized, b, quantized=True)
        else:
            vgg.forward(self.ctx, self.y, self.W_r, None, self.W_gate, self.W_up, self.W_down, b)
        vgg.moe_balance_loss(self.ctx, b.logits, b.topk_ids, self.balance_coef, self.z_coef, self.balance, self.counts,
                             self.probs, self.dlogits, self.ws_balance, seq_offsets=self.seq_offsets)
        return self.h + b.O

    def backward(self, dout):
        """Gradients for dout [T, d] fp32: dx, dres, dweight here, the layer's (dW_r with the balance loss's) in buf."""
        b, w = self.buf, (self.W_r, self.W_gate, self.W_up, self.W_down)
        dO = dout.to(BF)
        if self.form == "e4m3":
            vgg.backward_e4m3(self.ctx, dO, self.y, *w, self.quantized, b)
        elif self.form == "mx":
            vgg.backward_mx(self.ctx, dO, self.y, *w, self.quantized, b)
        else:
            vgg.backward(self.ctx, dO, self.y, *w, b)
        vgg.moe_router_backward(self.ctx, self.dlogits, self.y, self.W_r, b.dX, b.dW_r, b.dX, b.dW_r, self.ws_router)
        vgg.moe_add_rmsnorm_backward(self.ctx, b.dX, self.h, self.weight, self.rstd, dout, self.dx, self.dres, self.dweight,
                                     self.ws_norm)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--form", choices=("bf16", "e4m3", "mx"), default="e4m3")
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--lr", type=float, default=0.02)
    a = ap.parse_args()
    T, d, E, n, K = a.tokens, 2048, 128, 512, 8
    blk = Block.make(T, d, E, n, K, a.form)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((T, d), device="cuda", generator=g).to(BF)
    residual = torch.randn((T, d), device="cuda", generator=g)
    target = residual + 0.5 * torch.randn((T, d), device="cuda", generator=g)
    for step in range(a.steps):
        beg, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        beg.record()
        err = blk.forward(x, residual) - target
        blk.backward(err / err.numel())
        end.record()
        loss = 0.5 * err.square().mean() + blk.balance[0]
        end.synchronize()
        print(f"step {step}: loss {loss.item():.4f}  balance {blk.balance[1].item():.4f}  z {blk.balance[2].item():.3f}  "
              f"most loaded expert {blk.counts.max().item() * E / (T * K):.2f}x  {beg.elapsed_time(end):.2f} ms")
        for w, dw in ((blk.weight, blk.dweight), (blk.W_r, blk.buf.dW_r), (blk.W_gate, blk.buf.dW_gate),
                      (blk.W_up, blk.buf.dW_up), (blk.W_down, blk.buf.dW_down)):
            # a step against the gradient, a share lr of the weight's own size
            w.sub_(a.lr * w.float().norm() / dw.float().norm().clamp(min=1e-30) * dw.float())
    rc, code = vgg.moe_get_error(blk.ctx)
    if rc != vgg.MOE_OK:
        raise RuntimeError(f"device error {code}: {vgg.status_str(rc)}")


if __name__ == "__main__":
    main()
