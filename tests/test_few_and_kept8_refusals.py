"""Argument checks of the layer for a few tokens and of the activations kept in 8 bits, on the CPU.  The calls get made-up
addresses and a block that stands in for a context on a device that no machine has: a call that passes every check ends
there, with MOE_ERR_CUDA, one that is refused gets no further than its checks."""
import ctypes
import os
import shutil

import pytest
import torch

A = 1 << 20  # an aligned address that is never read
INVALID, CUDA = 1, 3
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from varlen_grouped_gemm_gb300 import build
    build.build()
    import varlen_grouped_gemm_gb300 as vgg
    return vgg.lib()


@pytest.fixture(scope="module")
def nowhere():
    """A context begins with its device's number."""
    block = (ctypes.c_int * 1024)(1 << 20)
    yield ctypes.cast(block, ctypes.c_void_p)


def run(L, ctx, name, base, **changed):
    assert set(changed) <= set(base)
    return getattr(L, name)(ctx, *dict(base, **changed).values())


FEW = dict(X=A, ld_x=64, W_r=A, bias=None, W_gate=A, W_up=A, W_down=A, T=4, d=64, E=8, n=64, K=2, ids=A, w=A, O=A, ld_o=64,
           ws=A, ws_bytes=BIG, stream=None)
FEW8 = dict(X=A, ld_x=64, W_r=A, bias=None, Wg=A, gs=A, Wu=A, us=A, Wd=A, ds=A, T=4, d=64, E=8, n=64, K=2, ids=A, w=A, O=A,
            ld_o=64, ws=A, ws_bytes=BIG, stream=None)


@pytest.mark.parametrize("good", [dict(), dict(T=1), dict(T=64), dict(bias=A + 4), dict(ld_x=72, ld_o=68), dict(O=A + 8)],
                         ids=str)
@pytest.mark.parametrize("name,base", [("moe_forward_few", FEW), ("moe_forward_few_e4m3", FEW8)])
def test_few_calls_that_pass(L, nowhere, name, base, good):
    assert run(L, nowhere, name, base, **good) == CUDA


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(T=65), dict(d=32), dict(d=100), dict(n=32), dict(n=96), dict(E=4, K=2), dict(E=12), dict(E=1032), dict(K=0),
    dict(K=9), dict(X=None), dict(W_r=None), dict(ids=None), dict(w=None), dict(O=None), dict(ld_x=63), dict(ld_x=68),
    dict(ld_o=60), dict(ld_o=66), dict(X=A + 8), dict(W_r=A + 2), dict(O=A + 4), dict(ws=None), dict(ws=A + 16),
    dict(ws_bytes=1000)], ids=str)
@pytest.mark.parametrize("name,base", [("moe_forward_few", FEW), ("moe_forward_few_e4m3", FEW8)])
def test_few_refusals(L, nowhere, name, base, bad):
    assert run(L, nowhere, name, base, **bad) == INVALID


@pytest.mark.parametrize("bad", [dict(W_gate=None), dict(W_up=A + 8), dict(W_down=None)], ids=str)
def test_few_weights(L, nowhere, bad):
    assert run(L, nowhere, "moe_forward_few", FEW, **bad) == INVALID


@pytest.mark.parametrize("bad", [dict(Wg=None), dict(gs=None), dict(us=None), dict(ds=None), dict(Wd=A + 8), dict(ds=A + 4)],
                         ids=str)
def test_few_e4m3_weights(L, nowhere, bad):
    assert run(L, nowhere, "moe_forward_few_e4m3", FEW8, **bad) == INVALID


def test_few_of_no_tokens(L, nowhere):
    assert run(L, nowhere, "moe_forward_few", FEW, T=0, X=None, O=None, ids=None, w=None) == 0


def test_few_workspace(L):
    f = L.moe_few_workspace_bytes
    assert f(1, 64, 8, 64, 2) > 0 and f(0, 64, 8, 64, 2) > 0 and f(64, 7168, 256, 2048, 8) < 1 << 27
    assert f(-1, 64, 8, 64, 2) == f(65, 64, 8, 64, 2) == f(1, 60, 8, 64, 2) == f(1, 64, 8, 64, 9) == 0


ROWS = dict(M=A, rows=4, cols=64, q=A, scales=A, stream=None)
READ = dict(q=A, scales=A, rows=4, cols=64, M=A, stream=None)


@pytest.mark.parametrize("bad", [dict(rows=-1), dict(cols=0), dict(cols=48), dict(M=None), dict(q=None), dict(scales=None),
                                 dict(M=A + 8), dict(q=A + 8), dict(scales=A + 2)], ids=str)
@pytest.mark.parametrize("name,base", [("moe_keep_rows8", ROWS), ("moe_read_rows8", READ)])
def test_rows8(L, nowhere, name, base, bad):
    assert run(L, nowhere, name, base) == CUDA
    assert run(L, nowhere, name, base, **bad) == INVALID


KEPT = dict(Hq=A, hs=A, Uq=A, us=A)
FWD = dict(X=A, W_gate=A, W_up=A, W_down=A, T=16, d=64, E=8, n=64, cap=32, offsets=A, tok=A, w=A, **KEPT, Aa=A, Yw=A, ws=A,
           ws_bytes=BIG, stream=None)
FWD8 = dict(Xq=A, xs=A, Wg=A, gs=A, Wu=A, us_=A, W_down=A, Wd=None, ds=None, T=16, d=64, E=8, n=64, cap=32, offsets=A, tok=A,
            w=A, **KEPT, Aa=A, Aq=None, a_s=None, Yw=A, stream=None)
FWDMX = dict(Xq=A, xs=A, Wg=A, Wu=A, gsf=A, Wd=A, dsf=A, T=16, d=64, E=8, n=64, cap=32, offsets=A, tok=A, w=A, **KEPT, xsf=A,
             Aq=A, asf=A, Yw=A, stream=None)
ROUTE = dict(ids=A, topk_w=A, offsets=A, tok=A, w=A, tok_ptr=A, tok_pairs=A)
OUT = dict(dX=A, dWg=A, dWu=A, dWd=A, fp32=1, dS=A, dl=A, dWr=A, ws=A, ws_bytes=BIG)
SIZES = dict(T=16, d=64, E=8, n=64, K=2, m_tile=0, cap=32)
BWD = dict(dO=A, X=None, Xq=A, xs=A, W_r=A, W_gate=A, W_up=A, W_down=A, **SIZES, **ROUTE, **KEPT, **OUT, stream=None)
BWD8 = dict(dO=A, X=None, Xq=A, xs=A, W_r=A, W_gate=A, W_up=A, W_down=A, Wgu=A, wgus=A, Wdt=A, wdts=A, **SIZES, **ROUTE, **KEPT,
            HUq=A, hus=A, dOq=A, dos=A, **OUT, stream=None)
BWDMX = dict(dO=A, X=None, Xq=A, xs=A, W_r=A, W_gate=A, W_up=A, W_down=A, Wdt=A, wdtsf=A, Wgu=A, wgusf=A, **SIZES, **ROUTE,
             **KEPT, dOq=A, dosf=A, HUq=A, husf=A, **OUT, dw_ws=None, dw_bytes=0, stream=None)
ALL = [("moe_grouped_gemm_fwd_kept8", FWD), ("moe_grouped_gemm_fwd_e4m3_kept8", FWD8),
       ("moe_grouped_gemm_fwd_mx_kept8", FWDMX), ("moe_backward_kept8", BWD), ("moe_backward_e4m3_kept8", BWD8),
       ("moe_backward_mx_kept8", BWDMX)]


@pytest.mark.parametrize("name,base", ALL, ids=lambda x: x if isinstance(x, str) else "")
def test_kept8_calls(L, nowhere, name, base):
    assert run(L, nowhere, name, base) == CUDA
    for bad in (dict(Hq=None), dict(hs=None), dict(Uq=None), dict(us=None), dict(Hq=A + 8), dict(Uq=A + 4), dict(hs=A + 2),
                dict(us=A + 8), dict(T=0), dict(d=96), dict(n=32), dict(cap=0), dict(offsets=None)):
        assert run(L, nowhere, name, base, **bad) == INVALID, bad
    assert getattr(L, name)(None, *base.values()) == INVALID


@pytest.mark.parametrize("name,base", ALL[3:], ids=lambda x: x if isinstance(x, str) else "")
def test_kept8_backward_calls(L, nowhere, name, base):
    """X in bf16 in place of its codes passes, too; neither does not, nor a workspace of the plain backward's size."""
    assert run(L, nowhere, name, base, X=A, Xq=None, xs=None) == CUDA
    need = L.moe_kept8_workspace_bytes(16, 64, 8, 64, 32)
    assert run(L, nowhere, name, base, ws_bytes=need) == CUDA
    for bad in (dict(Xq=None), dict(xs=None), dict(Xq=A + 8), dict(xs=A + 2), dict(ws_bytes=need - 1), dict(ws=A + 16),
                dict(dX=None), dict(dWr=None)):
        assert run(L, nowhere, name, base, **bad) == INVALID, bad


def test_kept8_workspace(L):
    f = L.moe_kept8_workspace_bytes
    assert f(16, 64, 8, 64, 32) > 0
    assert f(0, 64, 8, 64, 32) == f(16, 60, 8, 64, 32) == f(16, 64, 8, 64, 0) == 0


class _Ctx:
    device = 0
    handle = None


def test_binding_refuses_wrong_tensors(L):
    import varlen_grouped_gemm_gb300 as vgg
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    x, w = torch.zeros(4, 64, dtype=bf), torch.zeros(8, 64, 64, dtype=bf)  # on the CPU
    ids, tw, ws = torch.zeros(4, 2, dtype=i32), torch.zeros(4, 2), torch.zeros(8, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA device 0"):
        vgg.moe_forward_few(_Ctx, x, torch.zeros(64, 8, dtype=bf), None, w, w, w, 2, x, ids, tw, ws)
    with pytest.raises(ValueError, match=r"\[T, d\]"):
        vgg.moe_forward_few(_Ctx, x[0], x, None, w, w, w, 2, x, ids, tw, ws)
    u8 = torch.zeros(8, 64, 64, dtype=torch.uint8)
    w8 = vgg.E4m3Weights(u8, tw, u8, tw)
    with pytest.raises(ValueError, match="W_down"):
        vgg.moe_forward_few_e4m3(_Ctx, x, x, None, w8, 2, x, ids, tw, ws)
    with pytest.raises(ValueError, match="invalid arguments"):
        vgg.moe_few_workspace_bytes(65, 64, 8, 64, 2)
    with pytest.raises(ValueError, match="invalid arguments"):
        vgg.moe_kept8_workspace_bytes(4, 60, 8, 64, 2)
    with pytest.raises(ValueError, match="blocks of 32"):
        vgg.Kept8.empty(4, 48, "cpu")
    k = vgg.Kept8.empty(4, 64, "cpu")
    with pytest.raises(ValueError, match="CUDA device 0"):
        vgg.moe_keep_rows8(_Ctx, x, k)
    with pytest.raises(ValueError, match="blocks of 32"):
        vgg.moe_keep_rows8(_Ctx, torch.zeros(4, 48, dtype=bf), k)
    with pytest.raises(ValueError, match="same way"):
        vgg._kept_pair(_Ctx, k, x, (4, 64))
    with pytest.raises(ValueError, match="goes with"):
        vgg._plain_x(k)

    class Buf:
        xk = None
    with pytest.raises(ValueError, match="needs X"):
        vgg._kept_input(None, Buf)
