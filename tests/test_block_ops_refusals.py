"""Argument checks of the operators around the layer, on the CPU: every call below is refused (or, for T = 0, done)
before the context is used, so a block of zeros stands in for it and made-up addresses for the tensors."""
import ctypes
import os
import shutil

import pytest
import torch

A = 1 << 20  # an aligned address that is never read


@pytest.fixture(scope="module")
def L():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from varlen_grouped_gemm_gb300 import build
    build.build()
    import varlen_grouped_gemm_gb300 as vgg
    return vgg.lib()


@pytest.fixture(scope="module")
def fake():
    return ctypes.create_string_buffer(4096)


def _call(L, fake, name, base, **changed):
    args = dict(base, **changed)
    return getattr(L, name)(ctypes.cast(fake, ctypes.c_void_p), *args.values())


NORM = dict(x=A, ld_x=64, residual=A, ld_residual=64, residual_fp32=0, weight=A, weight_fp32=0, T=4, d=64, eps=1e-6, h=A,
            ld_h=64, y=A, ld_y=64, rstd=A, q_form=0, q=None, scales=None, stream=None)
CODES = dict(q_form=1, q=A, scales=A)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(d=0), dict(d=16385, ld_x=16385, ld_residual=16385, ld_h=16385, ld_y=16385), dict(eps=-1.0),
    dict(eps=float("nan")), dict(residual=None), dict(weight=None), dict(h=None), dict(y=None), dict(ld_x=63),
    dict(ld_residual=0), dict(ld_h=63), dict(ld_y=63), dict(x=A + 1), dict(residual_fp32=1, residual=A + 2, h=A),
    dict(weight_fp32=1, weight=A + 2), dict(q_form=3), dict(q_form=-1), dict(CODES, q=None), dict(CODES, scales=None),
    dict(CODES, d=32), dict(CODES, q=A + 8), dict(CODES, y=A + 2), dict(CODES, ld_x=65), dict(CODES, scales=A + 2),
    dict(CODES, q_form=2, weight=A + 2)], ids=str)
def test_norm_refusals(L, fake, bad):
    assert _call(L, fake, "moe_add_rmsnorm", NORM, **bad) == 1


def test_norm_of_no_rows(L, fake):
    assert _call(L, fake, "moe_add_rmsnorm", NORM, T=0, x=None, residual=None, weight=None, h=None, y=None) == 0


BWD = dict(dy=A, ld_dy=64, h=A, ld_h=64, residual_fp32=0, weight=A, weight_fp32=0, rstd=A, dh=None, ld_dh=0, T=4, d=64,
           dx=A, ld_dx=64, dresidual=None, ld_dresidual=0, dweight=A, ws=A, ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(d=0), dict(d=20000), dict(dy=None), dict(h=None), dict(weight=None), dict(rstd=None),
    dict(dx=None), dict(dweight=None), dict(dweight=A + 2), dict(ws=None), dict(ws=A + 16), dict(ws_bytes=1023),
    dict(ld_dy=63), dict(dh=A, ld_dh=63), dict(dresidual=A, ld_dresidual=1), dict(dy=A + 1), dict(rstd=A + 2)], ids=str)
def test_norm_backward_refusals(L, fake, bad):
    assert _call(L, fake, "moe_add_rmsnorm_backward", BWD, **bad) == 1


def test_norm_workspace(L):
    f = L.moe_add_rmsnorm_workspace_bytes
    assert f(4, 64) == 4 * 64 * 4 and f(100000, 64) == 1024 * 64 * 4 and f(0, 64) == 256 and f(1, 1) == 256
    assert f(-1, 64) == f(4, 0) == f(4, 16385) == 0


BAL = dict(logits=A, topk_ids=A, mask=None, seq_offsets=None, T=16, E=8, K=2, B=1, balance_coef=0.1, z_coef=0.1, dloss=None,
           loss=A, counts=A, probs=A, dlogits=A, ws=A, ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(E=0), dict(E=1025), dict(K=0), dict(K=9), dict(T=1 << 30, K=8), dict(B=0), dict(B=2),
    dict(B=1 << 24, E=1024, seq_offsets=A), dict(logits=None), dict(topk_ids=None), dict(loss=None), dict(counts=None),
    dict(probs=None), dict(ws=None), dict(ws=A + 4), dict(ws_bytes=100), dict(balance_coef=float("inf")),
    dict(z_coef=float("nan")), dict(logits=A + 2), dict(dlogits=A + 1), dict(dloss=A + 2)], ids=str)
def test_balance_refusals(L, fake, bad):
    assert _call(L, fake, "moe_balance_loss", BAL, **bad) == 1


def test_balance_workspace(L):
    f = L.moe_balance_loss_workspace_bytes
    assert f(16, 8, 1) > 0 and f(0, 8, 1) > 0 and f(1 << 20, 1024, 1) < 5 << 20
    assert f(-1, 8, 1) == f(16, 0, 1) == f(16, 8, 0) == f(16, 1025, 1) == 0


ROUTER = dict(dlogits=A, X=A, W_r=A, T=16, d=64, E=8, dX_in=None, dW_r_in=None, dX=A, dW_r=A, ws=A, ws_bytes=1 << 30,
              stream=None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(T=65537), dict(d=32), dict(d=100), dict(E=4), dict(E=12), dict(E=1032), dict(dlogits=None),
    dict(X=None), dict(W_r=None), dict(dX=None, dW_r=None), dict(ws=None), dict(ws=A + 64), dict(ws_bytes=1000),
    dict(dlogits=A + 4), dict(X=A + 2), dict(W_r=A + 8), dict(dX_in=A + 2), dict(dW_r_in=A + 4), dict(dX=A + 2),
    dict(dW_r=A + 4)], ids=str)
def test_router_backward_refusals(L, fake, bad):
    assert _call(L, fake, "moe_router_backward", ROUTER, **bad) == 1


def test_router_backward_of_no_tokens(L, fake):
    """dX has no elements, so no address; with dW_r left out as well nothing is asked for, and nothing is done."""
    assert _call(L, fake, "moe_router_backward", ROUTER, T=0, dlogits=None, X=None, dX=None, dW_r=None) == 0


def test_router_workspace(L):
    f = L.moe_router_backward_workspace_bytes
    assert f(100, 64, 8) == 128 * 8 * 2 * 3 + 16 * 64 * 8 * 4 and f(0, 64, 8) == 16 * 64 * 8 * 4
    assert f(-1, 64, 8) == f(16, 60, 8) == f(16, 64, 9) == 0


def test_null_context(L):
    for name, base in (("moe_add_rmsnorm", NORM), ("moe_add_rmsnorm_backward", BWD), ("moe_balance_loss", BAL),
                       ("moe_router_backward", ROUTER)):
        assert getattr(L, name)(None, *base.values()) == 1


class _Ctx:
    device = 0
    handle = None


def test_binding_refuses_wrong_tensors(L):
    """Shapes, types, strides and devices are checked before the library is called."""
    import varlen_grouped_gemm_gb300 as vgg
    bf, f32 = torch.bfloat16, torch.float32
    x = torch.zeros(4, 64, dtype=bf)  # on the CPU
    w = torch.zeros(64, dtype=bf)
    with pytest.raises(ValueError, match="CUDA device 0"):
        vgg.moe_add_rmsnorm(_Ctx, x, x, w, 1e-6, x, x)
    with pytest.raises(ValueError, match=r"\[T, d\]"):
        vgg.moe_add_rmsnorm(_Ctx, None, w, w, 1e-6, None, None)
    with pytest.raises(ValueError, match="bf16 or fp32"):
        vgg.moe_add_rmsnorm(_Ctx, None, x.half(), w, 1e-6, None, x)
    with pytest.raises(ValueError, match="CUDA device 0"):
        vgg.moe_add_rmsnorm_backward(_Ctx, x, x, w, w, None, x, None, w, x)
    with pytest.raises(ValueError, match="need seq_offsets"):
        vgg.moe_balance_loss(_Ctx, torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), 1.0, 0.0, torch.zeros(3),
                             torch.zeros(2, 8, dtype=torch.int32), torch.zeros(2, 8), None, x)
    with pytest.raises(ValueError, match="bool or uint8"):
        vgg.moe_balance_loss(_Ctx, torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), 1.0, 0.0, torch.zeros(3),
                             torch.zeros(1, 8, dtype=torch.int32), torch.zeros(1, 8), None, x, mask=torch.zeros(4))
    with pytest.raises(ValueError, match="CUDA device 0"):
        vgg.moe_router_backward(_Ctx, torch.zeros(4, 8), x, w, None, None, x, None, x)
    for f, args in ((vgg.moe_add_rmsnorm_workspace_bytes, (4, 0)), (vgg.moe_balance_loss_workspace_bytes, (4, 0)),
                    (vgg.moe_router_backward_workspace_bytes, (4, 1, 8))):
        with pytest.raises(ValueError, match="invalid arguments"):
            f(*args)
