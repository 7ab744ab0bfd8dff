"""The operators together, as the example of a pre-norm block runs them, against the fp64 oracles of the norm, the layer,
the balance loss and the router's products: within the layer's own bounds (max 2e-2, mean 3e-3 relative)."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle
from oracle import block_oracle as bo
from oracle import moe_oracle as mo

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


def bits(t):
    return t.detach().contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def f64(t):
    return t.detach().double().cpu().numpy()


def inputs(T, d, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((T, d), device="cuda", generator=g).to(torch.bfloat16)
    return x, torch.randn((T, d), device="cuda", generator=g), torch.randn((T, d), device="cuda", generator=g)


def test_block_step_matches_the_oracle():
    import prenorm_block
    import varlen_grouped_gemm_gb300 as vgg
    T, d, E, n, K = 200, 128, 16, 64, 2
    off = torch.tensor([0, 37, 37, 200], dtype=torch.int32, device="cuda")
    blk = prenorm_block.Block.make(T, d, E, n, K, "bf16", off)
    blk.weight.add_(0.1 * torch.randn(d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(9)))
    ca, cz = 300.0, 100.0  # next to an upstream gradient of 1 for every output: the means over T tokens are small
    blk.balance_coef, blk.z_coef = ca, cz
    x, residual, dout = inputs(T, d, 3)
    out = blk.forward(x, residual)
    blk.backward(dout)
    assert vgg.moe_get_error(blk.ctx) == (vgg.MOE_OK, 0)
    h = f64(residual) + f64(x)
    y, rstd = bo.rmsnorm(h, f64(blk.weight), blk.eps)
    oracle.compare("y", f64(blk.y), y)
    # the layer on the device's own bf16 y, and the choices of its logits
    yb, W = bits(blk.y), [bits(w) for w in (blk.W_r, blk.W_gate, blk.W_up, blk.W_down)]
    O, cache = mo.moe_forward(yb, W[0], None, W[1], W[2], W[3], K, logits_for_routing=blk.buf.logits.cpu().numpy())
    oracle.compare("out", f64(out), h + O)
    grads = mo.moe_backward(yb, W[0], None, W[1], W[2], W[3], bits(dout.to(torch.bfloat16)), cache)
    logits = mo.router_logits(yb, W[0], None)
    r = bo.balance_loss(logits, blk.buf.topk_ids.cpu().numpy(), ca, cz, None, off.tolist())
    np.testing.assert_array_equal(blk.counts.cpu().numpy(), r["counts"])
    oracle.compare("balance", f64(blk.balance), r["loss"])
    oracle.compare("dlogits", f64(blk.dlogits), r["dlogits"])
    dX, dW_r = bo.router_backward(r["dlogits"], mo.bf16_bits_to_f64(yb), mo.bf16_bits_to_f64(W[0]), grads["dX"], grads["dW_r"])
    assert np.linalg.norm(dW_r - grads["dW_r"]) > 0.05 * np.linalg.norm(grads["dW_r"])  # the loss takes part
    oracle.compare("dX", f64(blk.buf.dX), dX)
    oracle.compare("dW_r", f64(blk.buf.dW_r), dW_r)
    gh, gw = bo.rmsnorm_backward(dX, h, f64(blk.weight), rstd, f64(dout))
    oracle.compare("dres", f64(blk.dres), gh)
    oracle.compare("dx", f64(blk.dx), gh)
    oracle.compare("dweight", f64(blk.dweight), gw)


@pytest.mark.parametrize("form", ["e4m3", "mx"])
def test_fused_codes_serve_the_layer(form):
    """The norm's codes in place of the layer's own quantization of y: each is within an e4m3 rounding of y, so the
    outputs differ by the roundings of independent codes (2^-4 a value, averaged over the sums)."""
    import prenorm_block
    import varlen_grouped_gemm_gb300 as vgg
    T, d, E, n, K = 300, 256, 8, 128, 2
    blk = prenorm_block.Block.make(T, d, E, n, K, form)
    x, residual, dout = inputs(T, d, 5)
    blk.forward(x, residual)
    fused = blk.buf.O.clone()
    if form == "e4m3":
        vgg.forward_e4m3(blk.ctx, blk.y, blk.W_r, None, blk.quantized, None, blk.buf)
    else:
        vgg.forward_mx(blk.ctx, blk.y, blk.W_r, None, blk.quantized, blk.buf)
    own = blk.buf.O.double()
    assert vgg.moe_get_error(blk.ctx) == (vgg.MOE_OK, 0)
    assert not torch.equal(fused.double(), own)  # the codes come from the fp32 y, not from its bf16 rounding
    assert (fused.double() - own).norm() <= 2.0 ** -4 * own.norm()
    blk.forward(x, residual)
    blk.backward(dout)
    assert vgg.moe_get_error(blk.ctx) == (vgg.MOE_OK, 0)
    for t in (blk.dx, blk.dres, blk.dweight, blk.buf.dW_r):
        assert bool(torch.isfinite(t.float()).all())


def test_example_runs_and_learns():
    out = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "prenorm_block.py"), "--form", "mx", "--tokens", "512",
                          "--steps", "4"], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]
    losses = [float(line.split("loss ")[1].split()[0]) for line in out.stdout.splitlines() if line.startswith("step")]
    assert len(losses) == 4 and losses[-1] < losses[0], out.stdout


def test_captured_step_replays():
    """The whole step as one CUDA graph: the same results as the eager calls, on new inputs too."""
    import prenorm_block
    T, d, E, n, K = 256, 256, 16, 64, 2
    blk = prenorm_block.Block.make(T, d, E, n, K, "bf16")
    x, residual, dout = inputs(T, d, 7)

    def run():
        out = blk.forward(x, residual)
        blk.backward(dout)
        return out

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for seed in (7, 8):
        for t, v in zip((x, residual, dout), inputs(T, d, seed)):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (out, blk.dx, blk.dres, blk.dweight, blk.buf.dW_r, blk.buf.dX, blk.balance)]
        want = [run()] + [blk.dx, blk.dres, blk.dweight, blk.buf.dW_r, blk.buf.dX, blk.balance]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
