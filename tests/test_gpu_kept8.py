"""Activations kept in 8 bits: the rule bit for bit, the forwards' codes against the rule on their own fp32 H and U, and the
backwards against 64 bits.

What a gradient may be off, beside the formula in 64 bits at the kept values: sums of products of bf16 values in fp32 (k terms:
k 2^-23 of the sum of magnitudes), the sigmoid's 2^-20, dH and dU rounded to bf16 in the product that gives dX (2^-8 of a
value; half that normwise, and the pairs' sums carry a rounding of their own), weight gradients' operands in two parts (2^-16),
results rounded to bf16 (2^-8).  Normwise bounds are a quarter above what independent roundings of those sizes give:
2^-8 / sqrt(3) / sqrt(2) = 1.6e-3 a rounding."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
ROUND = 1.6e-3  # of a normal value's rounding to bf16, normwise


@pytest.fixture(scope="module")
def vgg():
    import varlen_grouped_gemm_gb300 as m
    return m


@pytest.fixture(scope="module")
def ctx(vgg):
    return vgg.Context(0)


def rule(v):
    """Codes and scales of fp32 values by the stated rule."""
    b = v.float().unflatten(-1, (-1, 32))
    top = b.abs().amax(-1)
    bits = torch.div(top, torch.full_like(top, 127.0)).view(I32)
    scale = (((bits + 0xFFFF) & ~0xFFFF).view(F32)).clamp(min=2.0 ** -126)
    bad = ~torch.isfinite(b).all(-1)
    scale = torch.where(bad, torch.full_like(scale, float("nan")), scale)
    q = torch.round(b * torch.reciprocal(scale)[..., None])
    return torch.where(bad[..., None], torch.zeros_like(q), q).to(torch.int8).flatten(-2), scale.to(BF)


def values(k):
    return (k.q.float().unflatten(-1, (-1, 32)) * k.scale.float()[..., None]).flatten(-2).to(BF)


def same(a, b):
    """Equal bits, NaN among them."""
    return torch.equal(a.view(torch.int16), b.view(torch.int16)) if a.dtype == BF else torch.equal(a, b)


@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 64), (257, 96), (64, 2048), (1000, 7168), (5, 4064)])
def test_rows_follow_the_rule_bit_for_bit(vgg, ctx, rows, cols):
    g = torch.Generator(device="cuda").manual_seed(rows)
    M = torch.randn((rows, cols), device="cuda", generator=g)
    M *= torch.exp(4 * torch.randn((rows, cols // 32, 1), device="cuda", generator=g)).expand(-1, -1, 32).reshape(rows, cols)
    M = M.to(BF)
    M[0, :32] = 0.0
    if cols >= 96:
        M[-1, 32:64] = 2.0 ** -130           # below the smallest scale: zero codes
        M[-1, 64:96] = torch.tensor(3.3e38)  # near the type's end
    k = vgg.Kept8.empty(rows, cols)
    vgg.moe_keep_rows8(ctx, M, k)
    q, s = rule(M)
    assert torch.equal(k.q, q) and same(k.scale, s)
    out = torch.full_like(M, 7.0)
    vgg.moe_read_rows8(ctx, k, out)
    assert same(out, values(k))
    # half a scale, and the rounding to bf16
    err = (out.double() - M.double()).abs().unflatten(-1, (-1, 32))
    assert (err <= 0.5 * (1 + 2.0 ** -20) * s.double()[..., None] + 2.0 ** -8 * M.double().abs().unflatten(-1, (-1, 32))).all()


def test_blocks_that_are_not_finite_come_back_as_nan(vgg, ctx):
    M = torch.ones((4, 128), dtype=BF, device="cuda")
    M[0, 5], M[1, 40], M[2, 127], M[3, 64] = float("nan"), float("inf"), float("-inf"), 2.0
    k, out = vgg.Kept8.empty(4, 128), torch.empty_like(M)
    vgg.moe_keep_rows8(ctx, M, k)
    vgg.moe_read_rows8(ctx, k, out)
    bad = torch.isnan(out).view(4, 4, 32)
    want = torch.zeros((4, 4), dtype=torch.bool, device="cuda")
    want[0, 0] = want[1, 1] = want[2, 3] = True
    assert torch.equal(bad.all(-1), want) and torch.equal(bad.any(-1), want)
    assert out[3, 64] == 2.0


def layer(T, d, E, n, K, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(shape, device="cuda", generator=g) * std).to(BF)

    return dict(X=normal(T, d), dO=normal(T, d), W_r=normal(d, E, std=d ** -0.5), W_gate=normal(E, n, d, std=d ** -0.5),
                W_up=normal(E, n, d, std=d ** -0.5), W_down=normal(E, d, n, std=n ** -0.5))


def weights(vgg, ctx, s, form, backward=False):
    W = (s["W_gate"], s["W_up"], s["W_down"])
    return {"bf16": lambda: None, "e4m3": lambda: vgg.E4m3Weights.quantize(ctx, *W, backward=backward),
            "mx": lambda: vgg.MxWeights.quantize(ctx, *W, backward=backward)}[form]()


def forward(vgg, ctx, s, form, w, buf, **kw):
    if form == "bf16":
        vgg.forward(ctx, s["X"], s["W_r"], None, s["W_gate"], s["W_up"], s["W_down"], buf, **kw)
    elif form == "e4m3":
        vgg.forward_e4m3(ctx, s["X"], s["W_r"], None, w, None, buf, **kw)
    else:
        vgg.forward_mx(ctx, s["X"], s["W_r"], None, w, buf, **kw)


def backward(vgg, ctx, s, form, w, buf, X, **kw):
    a = (ctx, s["dO"], X, s["W_r"], s["W_gate"], s["W_up"], s["W_down"])
    if form == "bf16":
        vgg.backward(*a, buf, **kw)
    elif form == "e4m3":
        vgg.backward_e4m3(*a, w, buf, **kw)
    else:
        vgg.backward_mx(*a, w, buf, **kw)


def buffers(vgg, T, d, E, n, K, form, **kw):
    return vgg.Buffers.allocate(T, d, E, n, K, e4m3=form == "e4m3", mx=form == "mx", **kw)


SHAPES = [(1, 64, 8, 64, 1), (37, 128, 8, 64, 2), (300, 192, 16, 192, 4), (513, 320, 8, 448, 8), (700, 256, 1024, 128, 2),
          (2000, 512, 24, 320, 3)]


@pytest.mark.parametrize("form", ["bf16", "e4m3", "mx"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda c: "-".join(map(str, c)))
def test_forward_keeps_its_own_fp32_values_by_the_rule(vgg, ctx, shape, form):
    T, d, E, n, K = shape
    s = layer(*shape)
    w = weights(vgg, ctx, s, form)
    plain, kept = (buffers(vgg, *shape, form, backward=False, kept8=k8) for k8 in (False, True))
    kept.H.q.fill_(55)
    forward(vgg, ctx, s, form, w, plain)
    forward(vgg, ctx, s, form, w, kept)
    assert vgg.moe_get_error(ctx) == (vgg.MOE_OK, 0)
    assert same(plain.O, kept.O) and same(plain.Yw, kept.Yw)
    for full, k in ((plain.H, kept.H), (plain.U, kept.U), (s["X"], kept.xk)):
        q, scale = rule(full)
        assert torch.equal(k.q, q) and same(k.scale, scale)


@pytest.mark.parametrize("form", ["bf16", "e4m3", "mx"])
def test_forward_without_a_cache_and_capacity_slots(vgg, ctx, form):
    shape = T, d, E, n, K = 200, 128, 8, 128, 2
    s = layer(*shape)
    w = weights(vgg, ctx, s, form)
    buf = buffers(vgg, *shape, form, backward=False, kept8=True)
    for k in (buf.H, buf.U, buf.xk):
        k.q.fill_(55)
    forward(vgg, ctx, s, form, w, buf, cache=False)
    assert all((k.q == 55).all() for k in (buf.H, buf.U, buf.xk))
    plain, kept = (buffers(vgg, *shape, form, backward=False, kept8=k8, capacity=37) for k8 in (False, True))
    forward(vgg, ctx, s, form, w, plain)
    forward(vgg, ctx, s, form, w, kept)
    assert vgg.moe_get_error(ctx) == (vgg.MOE_OK, 0)
    assert same(plain.O, kept.O)
    q, scale = rule(plain.H)  # empty slots are zero rows
    assert torch.equal(kept.H.q, q) and same(kept.H.scale, scale)


def formula(s, buf, X, H, U):
    """The layer's gradients in 64 bits at the given activations, by the definition (and autograd for the router's part)."""
    T, d = s["X"].shape
    E, n, _ = s["W_gate"].shape
    off, tok, w = buf.offsets.tolist(), buf.sorted_tok.long(), buf.sorted_w.double()
    dO, X, H, U = s["dO"].double(), X.double(), H.double(), U.double()
    P = off[E]
    r = {"dX": torch.zeros((T, d), dtype=F64, device="cuda"), "dW_gate": torch.zeros((E, n, d), dtype=F64, device="cuda")}
    r["dW_up"], r["dW_down"] = torch.zeros_like(r["dW_gate"]), torch.zeros((E, d, n), dtype=F64, device="cuda")
    r["dS"] = torch.zeros(P, dtype=F64, device="cuda")
    full = torch.zeros((T, E), dtype=F64, device="cuda")
    for e in range(E):
        a = slice(off[e], off[e + 1])
        if off[e] == off[e + 1]:
            continue
        t, h, u = tok[a], H[a].clone().requires_grad_(), U[a].clone().requires_grad_()
        act = torch.nn.functional.silu(h) * u
        g = dO[t] @ s["W_down"][e].double()
        r["dS"][a] = (g * act).sum(1).detach()
        dh, du = torch.autograd.grad(act, (h, u), w[a, None] * g)
        r["dX"].index_add_(0, t, dh @ s["W_gate"][e].double() + du @ s["W_up"][e].double())
        r["dW_gate"][e], r["dW_up"][e] = dh.T @ X[t], du.T @ X[t]
        r["dW_down"][e] = dO[t].T @ (w[a, None] * act.detach())
        full[t, e] = r["dS"][a]
    ids = buf.topk_ids.long()
    p = torch.zeros_like(full).scatter_(1, ids, buf.topk_w.double())
    r["dlogits"] = p * (full - (p * full).sum(1, keepdim=True))
    r["dX"] += r["dlogits"] @ s["W_r"].double().T
    r["dW_r"] = X.T @ r["dlogits"]
    return r


def rel(a, b):
    return ((a.double() - b).norm() / b.norm().clamp(min=1e-300)).item()


@pytest.mark.parametrize("dw", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda c: "-".join(map(str, c)))
def test_backward_matches_64_bits_at_the_kept_values(vgg, ctx, shape, dw):
    s = layer(*shape, seed=1)
    buf = buffers(vgg, *shape, "bf16", dW_dtype=dw, kept8=True)
    forward(vgg, ctx, s, "bf16", None, buf)
    backward(vgg, ctx, s, "bf16", None, buf, None)
    assert vgg.moe_get_error(ctx) == (vgg.MOE_OK, 0)
    ref = formula(s, buf, values(buf.xk), values(buf.H), values(buf.U))
    bound = {"dX": 1.25 * 3 ** 0.5 * ROUND, "dS": 2e-5, "dlogits": 2e-5, "dW_r": 2e-5}
    for k in ("dW_gate", "dW_up", "dW_down"):
        bound[k] = 1.25 * ROUND if dw == BF else 2e-5
    if shape[4] == 1:  # one expert a token: its weight is 1 whatever the logit, the logits' gradient is rounding noise
        del bound["dlogits"], bound["dW_r"]
    P = shape[0] * shape[4]
    for name, b in bound.items():
        got = getattr(buf, name)
        got = got[:P] if name == "dS" else got
        assert rel(got, ref[name]) <= b, (name, rel(got, ref[name]), b)
    empty = (buf.counts == 0).nonzero()[:, 0]
    assert not buf.dW_gate[empty].any() and not buf.dW_down[empty].any()


@pytest.mark.parametrize("d, n", [(576, 64), (4096, 64), (4096, 192), (4160, 64)])
def test_logit_gradients_of_long_reductions(vgg, ctx, d, n):
    """The tensor cores' accumulator drops what an addition shifts out.  One of the sums behind dS takes 32 steps (up to d =
    4096; 512 of the reduction), so half a unit of 24 bits each, all in one direction, is 32 2^-24 = 1.9e-6; longer reductions
    have theirs in one accumulator, d / 16 steps.  The parts' sums, the dots and dW_r's product add a few 2^-24."""
    shape = T, _, E, _, K = 517, d, 8, n, 2
    s = layer(*shape, seed=3)
    buf = buffers(vgg, *shape, "bf16", dW_dtype=F32, kept8=True)
    forward(vgg, ctx, s, "bf16", None, buf)
    backward(vgg, ctx, s, "bf16", None, buf, None)
    assert vgg.moe_get_error(ctx) == (vgg.MOE_OK, 0)
    ref = formula(s, buf, values(buf.xk), values(buf.H), values(buf.U))
    bound = ((min(d, 512) if d <= 4096 else d) / 16 + 12) * 2.0 ** -24
    for name in ("dS", "dlogits", "dW_r"):
        got = buf.dS[:T * K] if name == "dS" else getattr(buf, name)
        assert rel(got, ref[name]) <= bound, (name, rel(got, ref[name]), bound)


@pytest.mark.parametrize("form", ["bf16", "e4m3", "mx"])
@pytest.mark.parametrize("kw", [dict(), dict(m_tile=64), dict(capacity=40)], ids=["plain", "rounded", "capacity"])
def test_backward_is_the_fp32_one_at_the_kept_values(vgg, ctx, form, kw):
    """From fp32 H and U that hold the kept values, and the kept X in bf16, moe_backward and its FP8 forms compute the same
    products; what the two do with dX and dW_r on the way differs by roundings."""
    shape = T, d, E, n, K = 300, 256, 8, 192, 2
    s = layer(*shape, seed=2)
    w = weights(vgg, ctx, s, form, backward=True)
    kept, plain = (buffers(vgg, *shape, form, kept8=k8, dW_dtype=F32, **kw) for k8 in (True, False))
    for b in (kept, plain):
        forward(vgg, ctx, s, form, w, b)
    P = int(kept.P.item())
    plain.H[:P], plain.U[:P] = values(kept.H)[:P].float(), values(kept.U)[:P].float()
    backward(vgg, ctx, s, form, w, kept, None)
    backward(vgg, ctx, s, form, w, plain, values(kept.xk))
    assert vgg.moe_get_error(ctx) == (vgg.MOE_OK, 0)
    for k in ("dW_gate", "dW_up", "dW_down", "dS", "dlogits"):
        assert torch.equal(getattr(kept, k), getattr(plain, k)), k
    assert rel(kept.dX, plain.dX.double()) <= 3 * ROUND
    assert rel(kept.dW_r, plain.dW_r.double()) <= 2e-5
    given = buffers(vgg, *shape, form, kept8=True, dW_dtype=F32, **kw)  # X handed over in bf16
    forward(vgg, ctx, s, form, w, given)
    backward(vgg, ctx, s, form, w, given, values(kept.xk))
    for k in ("dX", "dW_gate", "dW_r", "dlogits"):
        assert torch.equal(getattr(kept, k), getattr(given, k)), k


def test_step_with_kept_activations_against_differences(vgg, ctx):
    """A loss <dO, O> and its change along a direction of each weight: the gradient from kept activations times the
    direction.  The kept values' error (0.6%) and the layer's roundings bound the difference."""
    shape = T, d, E, n, K = 256, 128, 8, 64, 8  # every expert: no choice to change
    s = layer(*shape, seed=3)
    buf = buffers(vgg, *shape, "bf16", dW_dtype=F32, kept8=True)
    forward(vgg, ctx, s, "bf16", None, buf)
    backward(vgg, ctx, s, "bf16", None, buf, None)

    def loss(name, W):
        x = s["X"].double()
        v = {k: s[k].double() for k in ("W_r", "W_gate", "W_up", "W_down")} | {name: W}
        p = torch.softmax(x @ v["W_r"], 1)
        o = 0
        for e in range(E):
            a = torch.nn.functional.silu(x @ v["W_gate"][e].T) * (x @ v["W_up"][e].T)
            o = o + p[:, e:e + 1] * (a @ v["W_down"][e].T)
        return (o * s["dO"].double()).sum()

    for name in ("W_r", "W_gate", "W_up", "W_down"):
        W, g = s[name].double(), getattr(buf, "d" + name).double()
        step = 1e-4 * g / g.norm() * W.norm()  # along the gradient: nothing cancels
        diff = (loss(name, W + step) - loss(name, W - step)) / 2
        assert abs(diff - (g * step).sum()) <= 0.02 * abs(diff), name


def test_captured_step_and_another_stream(vgg, ctx):
    shape = T, d, E, n, K = 200, 128, 8, 128, 2
    s = layer(*shape, seed=4)
    buf = buffers(vgg, *shape, "bf16", kept8=True)

    def step():
        forward(vgg, ctx, s, "bf16", None, buf)
        backward(vgg, ctx, s, "bf16", None, buf, None)

    step()
    want = [getattr(buf, k).clone() for k in ("O", "dX", "dW_gate", "dW_r")] + [buf.H.q.clone()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in ("O", "dX", "dW_gate", "dW_r"):
        getattr(buf, k).zero_()
    graph.replay()
    torch.cuda.synchronize()
    got = [getattr(buf, k) for k in ("O", "dX", "dW_gate", "dW_r")] + [buf.H.q]
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert vgg.moe_get_error(ctx) == (vgg.MOE_OK, 0)
