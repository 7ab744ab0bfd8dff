"""Bounded waits that run out: the kernel leaves its code in the context's error word and returns, and the next call on the same
buffers is right.  The limit is a nanosecond, so a wait gives up on its first look at the clock; the work is long enough
that one looks at it."""
import pytest
import torch

import test_gpu_few as few

pytestmark = pytest.mark.gpu

SECONDS = 2_000_000_000


@pytest.fixture(scope="module")
def vgg():
    import varlen_grouped_gemm_gb300 as m
    return m


def give_up(vgg, ctx, call):
    """``call`` with waits that run out, then as it should be."""
    ctx.set_wait_timeout(1)
    call()
    assert vgg.moe_get_error(ctx) == (vgg.MOE_ERR_DEVICE_TIMEOUT, vgg.DEV_TIMEOUT)
    ctx.set_wait_timeout(SECONDS)
    call()
    assert vgg.moe_get_error(ctx) == (vgg.MOE_OK, 0)


def test_grouped_product(vgg):
    """A long reduction: its loads, its products and its epilogue wait for one another."""
    ctx = vgg.Context(0)
    rows, N, K = 2048, 512, 65536
    A = torch.zeros((rows, K), dtype=torch.bfloat16, device="cuda")
    B = torch.zeros((2, N, K), dtype=torch.bfloat16, device="cuda")
    A[:, ::7], B[:, :, ::3] = 1.0, 2.0
    B[1] *= 2.0
    offsets = torch.tensor([0, 1000, rows], dtype=torch.int32, device="cuda")
    D = torch.zeros((rows, N), device="cuda")
    give_up(vgg, ctx, lambda: vgg.moe_test_gemm_varlen_m(ctx, A, None, B, True, offsets, D))
    both = 2.0 * ((K + 20) // 21)  # whole numbers: exact
    assert (D[:1000] == both).all() and (D[1000:] == 2 * both).all()


@pytest.mark.parametrize("form", ["bf16", "e4m3"])
@pytest.mark.parametrize("T", [5, 50])
def test_few_tokens(vgg, form, T):
    """Wide experts, whose tiles take a hundred microseconds each, on the same workspace and outputs."""
    ctx = vgg.Context(0)
    s = few.make(T, 16384, 16, 2048, 8, seed=30)
    weights = few.weights8(vgg, ctx, s) if form == "e4m3" else (s["W_gate"], s["W_up"], s["W_down"])
    buf, fresh = (vgg.FewBuffers.allocate(T, 16384, 16, 2048, 8) for _ in range(2))
    vgg.forward_few(ctx, s["X"], s["W_r"], None, weights, fresh)
    give_up(vgg, ctx, lambda: vgg.forward_few(ctx, s["X"], s["W_r"], None, weights, buf))
    for name in ("O", "topk_ids", "topk_w"):
        assert torch.equal(getattr(buf, name), getattr(fresh, name)), name
