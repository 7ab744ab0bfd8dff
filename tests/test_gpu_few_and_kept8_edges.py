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


def test_rows_of_more_than_2_31_values(vgg, ctx):
    rows, cols = (1 << 17) + 3, 1 << 14
    M = torch.zeros((rows, cols), dtype=BF, device="cuda")
    tail = torch.randn((5, cols), device="cuda", generator=torch.Generator(device="cuda").manual_seed(22)).to(BF)
    M[:2], M[-3:] = tail[:2], tail[2:]
    k, out = vgg.Kept8.empty(rows, cols), torch.full_like(M, 7.0)
    vgg.moe_keep_rows8(ctx, M, k)
    vgg.moe_read_rows8(ctx, k, out)
    q, s = rule(tail)
    assert torch.equal(torch.cat((k.q[:2], k.q[-3:])), q) and same(torch.cat((k.scale[:2], k.scale[-3:])), s)
    want = ends(vgg.Kept8(q, s))
    assert same(out[:2], want[:2]) and same(out[-3:], want[2:]) and not out[2:-3].any()


def test_epilogues_past_2_31_values(vgg, ctx):
    """Pairs times columns past 2^31: the last rows' codes against the rule on the plain forward's own H and U, and their gradients
    against 64 bits."""
    shape = T, d, E, n, K = 65536, 64, 8, 4160, 8
    s = layer(*shape, seed=23)
    plain, kept = (vgg.Buffers.allocate(*shape, backward=k8, kept8=k8) for k8 in (False, True))
    assert kept.cap * n > 1 << 31
    forward(vgg, ctx, s, "bf16", None, plain)
    forward(vgg, ctx, s, "bf16", None, kept)
    assert vgg.moe_get_error(ctx) == (vgg.MOE_OK, 0)
    rows = slice(kept.cap - 300, kept.cap)
    for full, k in ((plain.H, kept.H), (plain.U, kept.U)):
        q, scale = rule(full[rows])
        assert torch.equal(k.q[rows], q) and same(k.scale[rows], scale)
    del plain
    backward(vgg, ctx, s, "bf16", None, kept, None)
    assert vgg.moe_get_error(ctx) == (vgg.MOE_OK, 0)
    h, u = (ends(vgg.Kept8(k.q[rows], k.scale[rows])).double() for k in (kept.H, kept.U))
    t = kept.sorted_tok[rows].long()
    want = ((s["dO"][t].double() @ s["W_down"][E - 1].double()) * (torch.nn.functional.silu(h) * u)).sum(1)
    assert rel(kept.dS[rows], want) <= 2e-5


@pytest.mark.parametrize("exponent", [-80, *range(-62, -52), -30, 0, 30, *range(58, 68), 80])
def test_codes_of_tokens_at_every_scale(vgg, ctx, exponent):
    """X's codes by the rule, x / scale in one division, from scales far below 2^-60 to far above 2^60 (between them the kernel divides
    by way of the reciprocal).  Even rows: a scale m 2^(exponent - 6), m in 1 .. 36, and quotients in the middle of two codes;
    odd rows: a scale that is rounded itself.

    The layer is made so that O shows the codes: one expert, W_gate's rows all the same, so that H is one number for a token,
    W_up and W_down the identity.  A is U times one number, rounded to bf16 (2^-8 at most, far less than half the distance of
    two codes), so A's own codes are X's; O is their multiple, rounded to bf16 again."""
    T, d, n, E = 64, 64, 64, 8
    g = torch.Generator().manual_seed(exponent + 100)
    m = torch.randint(1, 37, (T,), generator=g).double()
    top = torch.where(torch.arange(T) % 2 == 0, 7 * m, torch.randint(128, 256, (T,), generator=g).double())
    x = (torch.randn((T, d), generator=g, dtype=torch.float64) * top[:, None] / 3).clamp(-top[:, None], top[:, None])
    for t in range(0, T, 2):
        odd = 2 * torch.randint(8, 16, (24,), generator=g).double() + 1  # five bits: in the middle of two four-bit numbers
        tie = m[t] / 64 * odd * 2.0 ** torch.randint(-6, 4, (24,), generator=g).double()
        exact = (tie == tie.to(BF).double()) & (tie < top[t])
        x[t, 1:25] = torch.where(exact, tie * torch.sign(x[t, 1:25]), x[t, 1:25])
    x[:, 0] = top
    X = (x * 2.0 ** exponent).to(BF).cuda()
    one = torch.tensor(1.0).to(few.E4M3).view(torch.uint8).item()
    identity = (torch.eye(n).repeat(E, 1, 1) * one).to(torch.uint8).cuda()
    gate = torch.zeros_like(identity)
    gate[:, :, 0] = one
    scale = torch.full((E, n), 2.0 ** -exponent, device="cuda")  # H = top, U = x
    w8 = vgg.E4m3Weights(gate, scale, identity, scale.clone(), identity.clone(), torch.ones((E, d), device="cuda"))
    s = dict(X=X, W_r=torch.zeros((d, E), dtype=BF, device="cuda"), bias=None, K=1, W_gate=identity)
    O = few.call(vgg, ctx, s, "e4m3", w8)[0].double()
    assert vgg.moe_get_error(ctx) == (vgg.MOE_OK, 0)
    want = few.codes(X)[0].view(few.E4M3).double()
    assert (want[:, 0] == 448).all()
    assert torch.equal((O / O[:, :1] * 448).float().to(few.E4M3).double(), want)
