"""Ends of the range of the layer for a few tokens and of the activations kept in 8 bits.  Bounds as in test_gpu_kept8.py and
test_gpu_few.py, whose references these tests use."""
import pytest
import torch

from test_gpu_kept8 import BF, ROUND, backward, buffers, formula, forward, layer, rel

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
