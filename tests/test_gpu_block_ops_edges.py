"""Edges of the operators around the layer: outputs that begin anywhere, values where fp32 or bf16 rounding shows,
calls from several host threads.  u = 2^-24 is half an fp32 step; the bounds count roundings as in test_gpu_block_ops."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as bo

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


@pytest.fixture(scope="module")
def vgg():
    import varlen_grouped_gemm_gb300 as v
    return v


@pytest.fixture(scope="module")
def ctx(vgg):
    return vgg.Context(0)


@pytest.fixture(autouse=True)
def no_device_error(vgg, ctx):
    yield
    assert vgg.moe_get_error(ctx) == (vgg.MOE_OK, 0)


def f64(t):
    return t.detach().double().cpu().numpy()


def gen_of(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ------------------------------------------------------------------------------------------------ norm


@pytest.mark.parametrize("shift", [0, 1, 2, 3])
@pytest.mark.parametrize("T,d,res_t", [(1, 64, BF), (1, 2112, F32), (1, 4160, BF), (1, 7168, BF), (1, 7168, F32),
                                       (1, 8200, BF), (1, 16384, F32), (1, 33, BF), (3, 7168, BF), (3, 8200, F32)],
                         ids=str)
def test_norm_backward_weight_gradient_begins_at_any_float(vgg, ctx, T, d, res_t, shift):
    """A slice of a flat gradient buffer; what lies around it stays as it was."""
    g = gen_of(T + d)
    dy = torch.randn((T, d), device="cuda", generator=g).to(BF)
    h = (2 * torch.randn((T, d), device="cuda", generator=g)).to(res_t)
    w = 1 + 0.1 * torch.randn(d, device="cuda", generator=g)
    rstd = torch.rsqrt(h.float().pow(2).mean(1) + 1e-6)
    flat = torch.full((d + 8,), 777.0, device="cuda")
    dw, dx = flat[shift:shift + d], torch.empty_like(dy)
    ws = torch.empty(vgg.moe_add_rmsnorm_workspace_bytes(T, d), dtype=U8, device="cuda")
    vgg.moe_add_rmsnorm_backward(ctx, dy, h, w, rstd, None, dx, None, dw, ws)
    xh = f64(h) * f64(rstd)[:, None]
    _, gw = bo.rmsnorm_backward(f64(dy), f64(h), f64(w), f64(rstd), None)
    assert np.all(np.abs(f64(dw) - gw) <= (T + 3) * U * np.sum(np.abs(f64(dy) * xh), axis=0))
    assert bool((flat[:shift] == 777.0).all()) and bool((flat[shift + d:] == 777.0).all())
