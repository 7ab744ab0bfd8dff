"""Host checks of the operators around the layer (CPU only).  The calls get made-up addresses and a block that stands in for
a context on a device that no machine has: a call that passes every check ends there, with MOE_ERR_CUDA, and one
that is refused gets no further than its checks, with MOE_ERR_INVALID_ARG."""
import ctypes
import os
import shutil

import pytest

A = 1 << 20  # an aligned address that is never read
INVALID, CUDA = 1, 3


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


def norm(x=A, residual=A, weight=A, h=A, y=A, rstd=A, form=0, q=None, scales=None, d=64, T=4):
    return "moe_add_rmsnorm", (x, d, residual, d, 0, weight, 0, T, d, 1e-6, h, d, y, d, rstd, form, q, scales, None)


def norm_backward(dweight=A, T=4, d=64):
    return "moe_add_rmsnorm_backward", (A, d, A, d, 0, A, 0, A, None, 0, T, d, A, d, None, 0, dweight, A, 1 << 30, None)


def balance(loss=A, K=2):
    return "moe_balance_loss", (A, A, None, None, 16, 8, K, 1, 0.1, 0.1, None, loss, A, A, A, A, 1 << 30, None)


def router(dX=A, dW_r=A):
    return "moe_router_backward", (A, A, A, 16, 64, 8, None, None, dX, dW_r, A, 1 << 30, None)


@pytest.mark.parametrize("call", [norm(), norm(form=1, q=A, scales=A), norm(form=2, q=A, scales=A + 1), norm(d=63, h=A + 2),
                                  norm(rstd=None), norm_backward(), norm_backward(dweight=A + 4, T=1, d=7168), balance(),
                                  router(), router(dX=None), router(dW_r=None)], ids=str)
def test_calls_that_pass_the_checks(L, nowhere, call):
    name, args = call
    assert getattr(L, name)(nowhere, *args) == CUDA


@pytest.mark.parametrize("call", [norm(rstd=A + 1), norm(rstd=A + 2), norm(rstd=A + 3), norm(h=None), norm(weight=A + 1),
                                  norm(form=1, q=A, scales=A + 2), norm(form=1, q=A + 8, scales=A),
                                  norm_backward(dweight=A + 2), norm_backward(dweight=None), balance(loss=A + 1),
                                  balance(K=9), router(dX=A + 8), router(dX=None, dW_r=None)], ids=str)
def test_calls_that_are_refused(L, nowhere, call):
    name, args = call
    assert getattr(L, name)(nowhere, *args) == INVALID
