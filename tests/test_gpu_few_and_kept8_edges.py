"""Ends of the range of the layer for a few tokens and of the activations kept in 8 bits.  Bounds as in test_gpu_kept8.py and
test_gpu_few.py, whose references these tests use."""
import ctypes

import pytest
import torch

import test_gpu_few as few
from test_gpu_kept8 import BF, F32, ROUND, backward, buffers, formula, forward, layer, rel, rule, same

pytestmark = pytest.mark.gpu

DX = 1.25 * 3 ** 0.5 * ROUND  # dX normwise: dH and dU in bf16, the pairs' sums, the result


@pytest.fixture(scope="module")
def vgg():
    import varlen_grouped_gemm_gb300 as m
    return m


@pytest.fixture(scope="module")
def ctx(vgg):
    return vgg.Context(0)


def test_columns_beside_one_that_is_not_finite_keep_their_gradient(vgg, ctx):
    """A pair's dX row has a power of two for 64 columns: an infinite or undefined one among them leaves the others theirs."""
    shape = T, d, E, n, K = 300, 192, 8, 64, 2
    s = layer(*shape, seed=20)
    buf = buffers(vgg, *shape, "bf16", kept8=True)
    forward(vgg, ctx, s, "bf16", None, buf)
    s["W_gate"][2, 3, 70], s["W_up"][5, 0, 10] = float("inf"), float("nan")
    backward(vgg, ctx, s, "bf16", None, buf, None)
    assert vgg.moe_get_error(ctx) == (vgg.MOE_OK, 0)
    ref = formula(s, buf, read(vgg, ctx, buf.xk), read(vgg, ctx, buf.H), read(vgg, ctx, buf.U))["dX"]
    finite = torch.isfinite(ref)
    for e, c in ((2, 70), (5, 10)):
        t = (buf.topk_ids == e).any(1).nonzero()[:, 0]
        assert len(t) > 30 and not finite[t, c].any()
        assert torch.equal(buf.dX[t, c].isnan(), ref[t, c].isnan())
        block = slice(c // 64 * 64, c // 64 * 64 + 64)
        ok = finite[t, block]
        assert rel(buf.dX[t, block][ok], ref[t, block][ok]) <= DX, (e, rel(buf.dX[t, block][ok], ref[t, block][ok]))
    assert torch.equal(buf.dX[~finite].sign().nan_to_num(), ref[~finite].float().sign().nan_to_num())
    assert rel(buf.dX[finite], ref[finite]) <= DX


def read(vgg, ctx, k):
    out = torch.empty(k.q.shape, dtype=BF, device="cuda")
    vgg.moe_read_rows8(ctx, k, out)
    return out


LARGEST = torch.finfo(BF).max


def ends(k):
    """What codes and scales stand for: code * scale, rounded, at most bf16's largest number."""
    v = (k.q.float().unflatten(-1, (-1, 32)) * k.scale.float()[..., None]).flatten(-2)
    return v.clamp(-LARGEST, LARGEST).to(BF)


def test_finite_values_come_back_finite(vgg, ctx):
    """The largest numbers, whose code times their scale lies past them: 127 * 2.6792e36 = 3.4026e38."""
    M = torch.zeros((8, 96), dtype=BF, device="cuda")
    M[0, 0], M[1, 33], M[2, 95] = LARGEST, -LARGEST, LARGEST
    M[2, 64:90] = -LARGEST
    big = torch.tensor([0x7F7F, 0x7F7E, 0x7F7D, 0x7F70, 0x7F00, 0x7E80], dtype=torch.int16, device="cuda").view(BF)
    for i, v in enumerate(big[1:]):
        M[3 + i, 32 * (i % 3)] = -v
    M[3:, 95] = big[torch.arange(5, device="cuda")]
    k, out = vgg.Kept8.empty(8, 96), torch.empty_like(M)
    vgg.moe_keep_rows8(ctx, M, k)
    vgg.moe_read_rows8(ctx, k, out)
    q, s = rule(M)
    assert torch.equal(k.q, q) and same(k.scale, s) and same(out, ends(k))
    assert torch.isfinite(out).all()
    # half a scale, and the rounding to bf16
    err = (out.double() - M.double()).abs().unflatten(-1, (-1, 32))
    assert (err <= 0.5 * (1 + 2.0 ** -20) * s.double()[..., None] + 2.0 ** -8 * M.double().abs().unflatten(-1, (-1, 32))).all()
    k.scale[4] = float("nan")  # of a block that holds a value that is not finite
    vgg.moe_read_rows8(ctx, k, out)
    assert out[4].isnan().all()


def test_backward_at_the_largest_kept_value(vgg, ctx):
    """H at the end of the range (an infinite one would leave 0 * inf in its gradient)."""
    shape = T, d, E, n, K = 130, 128, 8, 64, 2
    s = layer(*shape, seed=21)
    s["dO"] = (s["dO"].float() * 1e-20).to(BF)  # dU = dA' silu(H): finite
    buf = buffers(vgg, *shape, "bf16", dW_dtype=F32, kept8=True)
    forward(vgg, ctx, s, "bf16", None, buf)
    row = torch.zeros((1, 32), dtype=BF, device="cuda")
    row[0, 0] = LARGEST
    k = vgg.Kept8.empty(1, 32)
    vgg.moe_keep_rows8(ctx, row, k)
    buf.H.q[5, :32], buf.H.scale[5, 0] = k.q[0], k.scale[0, 0]
    buf.U.q[5] = 0
    backward(vgg, ctx, s, "bf16", None, buf, None)
    assert vgg.moe_get_error(ctx) == (vgg.MOE_OK, 0)
    ref = formula(s, buf, ends(buf.xk), ends(buf.H), ends(buf.U))
    # dX is that row's single dU times a row of W_up: its rounding is the same in every column, 2^-8 at most
    assert rel(buf.dX, ref["dX"]) <= 2.0 ** -8 + DX
    assert rel(buf.dW_up, ref["dW_up"]) <= 2e-5
    for name in ("dW_gate", "dW_down", "dS", "dlogits"):
        assert torch.isfinite(getattr(buf, name)).all(), name


@pytest.mark.parametrize("form", ["bf16", "e4m3"])
@pytest.mark.parametrize("blocks", [1, 3, 4, 7])
def test_few_tokens_on_few_processors(vgg, blocks, form):
    """More tokens than blocks: a block finds the choice of several, more of them than it has warps (1 and 3 blocks)."""
    ctx = vgg.Context(0)
    sms = ctypes.c_int.from_address(ctx.handle.value + 4)  # a context holds its device and the blocks that run at once
    assert sms.value == torch.cuda.get_device_properties(0).multi_processor_count
    sms.value = blocks
    for T in (9, 16, 47, 64):
        s = few.make(T, 64 * (1 + T % 3), 16, 64, 1 + T % 4, seed=T)
        w8 = few.weights8(vgg, ctx, s) if form == "e4m3" else None
        few.check(few.call(vgg, ctx, s, form, w8), few.reference(s, form, w8))
    assert vgg.moe_get_error(ctx) == (vgg.MOE_OK, 0)
