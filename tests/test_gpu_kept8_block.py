"""The pre-norm block of the example whose step keeps the layer's activations in 8 bits: what it needs of the norm's output."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("form", ["bf16", "e4m3", "mx"])
def test_norm_output_may_go_after_the_forward(form):
    """With kept activations the block's backward needs nothing of y: it may be any memory by then."""
    import prenorm_block
    import varlen_grouped_gemm_gb300 as vgg
    T, d, E, n, K = 150, 128, 8, 64, 2
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((T, d), device="cuda", generator=g).to(torch.bfloat16)
    residual, dout = (torch.randn((T, d), device="cuda", generator=g) for _ in range(2))
    grads = []
    for lost in (False, True):
        b = prenorm_block.Block.make(T, d, E, n, K, form, kept8=True)
        b.balance_coef, b.z_coef = 3.0, 1.0
        b.forward(x, residual)
        if lost:
            b.y.fill_(float("nan"))
        else:
            vgg.moe_read_rows8(b.ctx, b.buf.xk, b.y)
        b.backward(dout)
        assert vgg.moe_get_error(b.ctx) == (vgg.MOE_OK, 0)
        grads.append([t.clone() for t in (b.buf.dW_r, b.buf.dX, b.buf.dW_gate, b.dx, b.dweight)])
    assert all(torch.isfinite(t).all() for t in grads[0])
    assert all(torch.equal(p, q) for p, q in zip(*grads))
