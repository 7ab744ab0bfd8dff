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


@pytest.mark.parametrize("T,d", [(1, 64), (3, 7168), (2, 16384), (608, 8192), (5, 999), (2, 9001)])
def test_norm_up_to_the_stated_range(vgg, ctx, T, d):
    """Squares are summed in fp32: values up to sqrt(2^127 / d)."""
    g = gen_of(T + d)
    top = float(np.sqrt(2.0 ** 127 / d))
    res = torch.where(torch.rand((T, d), device="cuda", generator=g) < 0.5, -top, top) * (1 - 2.0 ** -20)
    w = torch.ones(d, device="cuda")
    y, rstd = torch.empty((T, d), dtype=BF, device="cuda"), torch.empty(T, device="cuda")
    vgg.moe_add_rmsnorm(ctx, None, res, w, 0.0, None, y, rstd)
    y64, r64 = bo.rmsnorm(f64(res), f64(w), 0.0)
    # as in test_norm_bf16, and two steps of the root's approximation, which are not refined out there
    rel = ((16 + 10 + 1 + 2) / 2 + 2 + 4) * U
    assert np.all(np.abs(f64(rstd) - r64) <= rel * r64)
    assert np.all(np.abs(f64(y) - y64) <= (2.0 ** -8 + 2 * (rel + 2 * U)) * np.abs(y64))


def e4m3_borders():
    """Values half way between neighbouring codes of normal size."""
    return np.array([(2 * m + 1) * 2.0 ** (e - 4) for e in range(-6, 8) for m in range(8, 16) if (2 * m + 1) * 2.0 ** (e - 4) < 440])


def test_norm_codes_take_a_factor_that_is_rounded_once(vgg, ctx):
    """q = e4m3(y f) with f = 448 / max|y| rounded to fp32: values that f brings next to a border between two codes."""
    d = 512
    gen = np.random.default_rng(3)
    res = torch.ones((2, d), device="cuda")
    res[1, 1::2] = -1.0  # mean square 1, rstd 1: y is the weight itself, up to its sign
    q, sc = torch.empty((2, d), dtype=U8, device="cuda"), torch.empty(2, device="cuda")
    sign = f64(res).astype(np.float32)
    borders = e4m3_borders()
    for k in range(150):
        amax = np.float32(gen.uniform(1, 2) * 2.0 ** gen.integers(-20, 20))
        f = np.float32(448) / amax
        near = (gen.choice(borders, d) / np.float64(f)).astype(np.float32)
        w = (near.view(np.int32) + gen.integers(-2, 3, d).astype(np.int32)).view(np.float32)
        w[0] = amax
        vgg.moe_add_rmsnorm(ctx, None, res, torch.from_numpy(w).cuda(), 0.0, None, None, None, q, sc)
        want = torch.from_numpy(sign * w * f).to(torch.float8_e4m3fn).view(U8)
        assert torch.equal(q.cpu(), want), k
        assert bool((sc.cpu() == torch.from_numpy(np.array([amax]) / np.float32(448))).all())


# ------------------------------------------------------------------------------------------------ balance loss


@pytest.mark.parametrize("E", [2, 4])
def test_z_loss_gradient_near_a_log_sum_of_zero(vgg, ctx, E):
    """Two logits 0 and x < 0: lse = log(1 + e^x).  The sum's rounding is half a step of [1, 2), e^x is off by the
    argument's roundings (3 |x| u) and two steps, the logarithm by one step of its value."""
    T = 2000
    x = -torch.linspace(0.3, 14.0, T, device="cuda")
    logits = torch.full((T, E), float("-inf"), device="cuda")
    logits[:, 0], logits[:, 1] = 0.0, x
    ids = torch.zeros((T, 1), dtype=I32, device="cuda")
    loss, counts = torch.empty(3, device="cuda"), torch.empty((1, E), dtype=I32, device="cuda")
    probs, dl = torch.empty((1, E), device="cuda"), torch.empty((T, E), device="cuda")
    ws = torch.empty(vgg.moe_balance_loss_workspace_bytes(T, E, 1), dtype=U8, device="cuda")
    vgg.moe_balance_loss(ctx, logits, ids, 0.0, 1.0, loss, counts, probs, dl, ws)
    x64 = f64(x)
    small = np.exp(x64)
    lse, p = np.log1p(small), 1 / (1 + small)
    lse_abs = (1 + small * (3 * np.abs(x64) + 4) + 2 * lse) * U
    # p: the sum's error, the quotient (2 steps); the products and the factor 2 / n, half a step each
    tol = 2 / T * p * (lse_abs + 14 * U * lse)
    assert np.all(np.abs(f64(dl)[:, 0] - 2 / T * lse * p) <= tol)


# ------------------------------------------------------------------------------------------------ router products


def run_router(vgg, ctx, dl, X, W, dX_in=None, dW_in=None, want=(True, True)):
    (T, E), d = dl.shape, X.shape[1]
    dX = torch.full((T, d), 9.0, dtype=BF, device="cuda") if want[0] else None
    dW = torch.full((d, E), 9.0, device="cuda") if want[1] else None
    ws = torch.randint(0, 256, (vgg.moe_router_backward_workspace_bytes(T, d, E),), dtype=U8, device="cuda")
    vgg.moe_router_backward(ctx, dl, X, W, dX_in, dW_in, dX, dW, ws)
    return dX, dW


@pytest.mark.parametrize("shared", [1.0, 10.0, 100.0])
@pytest.mark.parametrize("T,d,E", [(3, 128, 16), (512, 512, 128), (300, 192, 1024), (129, 2880, 136), (2561, 2112, 264),
                                   (3000, 2048, 1024)])
def test_router_input_gradient_where_the_sum_cancels(vgg, ctx, T, d, E, shared):
    """Rows of a gradient behind a softmax sum to zero, so what W_r's columns have in common cancels in the result, and
    only there: a rounding of dlogits to 8 bits would stand out.  Two bf16 parts leave 2^-16 of a value."""
    g = gen_of(T + d + E)
    p = torch.softmax(2 * torch.randn((T, E), device="cuda", generator=g).double(), 1)
    u = torch.randn(E, device="cuda", generator=g).double()
    dl = (1e-2 * p * (u - p @ u[:, None])).float()
    W = ((torch.randn((d, E), device="cuda", generator=g) + shared * torch.randn((d, 1), device="cuda", generator=g)) /
         d ** 0.5).to(BF)
    X = torch.zeros((T, d), dtype=BF, device="cuda")
    ref = dl.double() @ W.double().T
    err = (2.0 ** -16 + 2 * (E + 2) * U) * (dl.double().abs() @ W.double().abs().T)  # and a step for every addition
    both, _ = run_router(vgg, ctx, dl, X, W)
    assert bool(((both.double() - ref).abs() <= err + 2.0 ** -8 * (ref.abs() + err)).all())
    alone, _ = run_router(vgg, ctx, dl, X, W, want=(True, False))
    assert torch.equal(alone, both)


ROUTER_SIZES = [(1, 64, 8), (3, 128, 16), (64, 192, 64), (65, 256, 128), (127, 320, 136), (300, 64, 1024), (700, 512, 264),
                (2000, 1536, 96), (129, 2880, 128), (2561, 2112, 264)]


@pytest.mark.parametrize("T,d,E", ROUTER_SIZES)
def test_router_weight_gradient_to_the_last_bit_of_dlogits(vgg, ctx, T, d, E):
    """dlogits of 17 to 24 significant bits, each element of the product a single one of them: three bf16 parts leave
    2^-24, their additions a step (2^-23) each, the sums of accumulators and splits and the added matrix half a step."""
    g = gen_of(T * d + E)
    n = torch.randint(1 << 16, 1 << 24, (T, E), device="cuda", generator=g)
    dl = torch.where(torch.rand((T, E), device="cuda", generator=g) < 0.5, -n, n).float()
    at = torch.randint(0, T, (d,), device="cuda", generator=g)
    X = torch.zeros((T, d), dtype=BF, device="cuda")
    X[at, torch.arange(d, device="cuda")] = 1.0
    W = torch.zeros((d, E), dtype=BF, device="cuda")
    pick = torch.randint(0, E, (d,), device="cuda", generator=g)
    W[torch.arange(d, device="cuda"), pick] = 1.0
    dX_in = torch.randint(-8, 9, (T, d), device="cuda", generator=g).to(BF)
    dW_in = torch.randint(-8, 9, (d, E), device="cuda", generator=g).float()
    dX, dW = run_router(vgg, ctx, dl, X, W, dX_in, dW_in)
    value = dl[at].double()
    assert bool(((dW.double() - value - dW_in.double()).abs() <= (1 + 6 + 2) * U * (value.abs() + 8)).all())
    ref = dl[:, pick].double() + dX_in.double()
    err = (2.0 ** -16 + 4 * U) * (ref.abs() + 8)
    assert bool(((dX.double() - ref).abs() <= err + 2.0 ** -8 * (ref.abs() + err)).all())


@pytest.mark.parametrize("T,d,E", ROUTER_SIZES)
def test_router_weight_gradient_has_fp32_precision_beside_the_other_product(vgg, ctx, T, d, E):
    """As test_router_weight_gradient_has_fp32_precision, with both products and both added matrices."""
    g = gen_of(T + d + 2 * E)
    dl = torch.randn((T, E), device="cuda", generator=g)
    X = torch.randn((T, d), device="cuda", generator=g).to(BF)
    W = (torch.randn((d, E), device="cuda", generator=g) / d ** 0.5).to(BF)
    dX_in = torch.randn((T, d), device="cuda", generator=g).to(BF)
    dW_in = torch.randn((d, E), device="cuda", generator=g)
    _, dW = run_router(vgg, ctx, dl, X, W, dX_in, dW_in)
    prod, mag = X.double().T @ dl.double(), X.double().abs().T @ dl.double().abs()
    err = (dW.double() - dW_in.double() - prod).abs()
    assert bool((err <= (1 + 48 + T / 128 + 16 + 2) * U * mag + 2 * U * dW_in.double().abs()).all())
    assert float(torch.linalg.norm(err)) <= 2.0 ** -20 * float(torch.linalg.norm(prod)) + \
        U * float(torch.linalg.norm(dW_in))


def test_router_backward_of_values_at_the_end_of_the_range(vgg, ctx):
    """An infinite dlogit gives infinities of the products' signs, one above bf16's largest number a finite product."""
    T, d, E = 70, 192, 64
    g = gen_of(9)

    def away_from_zero(rows, cols):
        s = torch.where(torch.rand((rows, cols), device="cuda", generator=g) < 0.5, -1.0, 1.0)
        return (2.0 ** -10 * s * (1 + torch.rand((rows, cols), device="cuda", generator=g))).to(BF)

    X, W = away_from_zero(T, d), away_from_zero(d, E)
    dl = torch.zeros((T, E), device="cuda")
    dl[3, 5], dl[7, 9], dl[11, 2], dl[13, 40] = float("inf"), -float("inf"), 3.4e38, -3.4e38
    dX, dW = run_router(vgg, ctx, dl, X, W)
    wx, ww = torch.zeros((T, d), device="cuda", dtype=torch.float64), torch.zeros((d, E), device="cuda", dtype=torch.float64)
    for t, e in ((3, 5), (7, 9), (11, 2), (13, 40)):
        wx[t] = dl[t, e].double() * W[:, e].double()
        ww[:, e] = dl[t, e].double() * X[t].double()
    for got, want, rel in ((dX, wx, 2.0 ** -8 + 2.0 ** -15), (dW, ww, 8 * U)):
        fin = want.isfinite()
        assert torch.equal(got.double()[~fin], want[~fin])
        assert bool(((got.double() - want).abs()[fin] <= rel * want.abs()[fin]).all())
    dl[20, 1] = float("nan")
    dX, dW = run_router(vgg, ctx, dl, X, W)
    assert dX[20].isnan().all() and dW[:, 1].isnan().all() and not dX[21].isnan().any()


# ------------------------------------------------------------------------------------------------ host threads


def threaded_call(vgg, c, st, kind, size, g):
    """(outputs, the call) with every pointer looked up once, so that calls of two threads overlap."""
    L, s = vgg.lib(), st.cuda_stream
    keep = []

    def p(t):
        keep.append(t)
        return t.data_ptr()

    if kind == "balance":
        T, E = 300, size
        logits = torch.randn((T, E), device="cuda", generator=g)
        ids = torch.topk(logits, 1, dim=1).indices.to(I32)
        out = [torch.empty(3, device="cuda"), torch.empty((1, E), dtype=I32, device="cuda"),
               torch.empty((1, E), device="cuda"), torch.empty((T, E), device="cuda")]
        n = vgg.moe_balance_loss_workspace_bytes(T, E, 1)
        args = (p(logits), p(ids), None, None, T, E, 1, 1, 1.0, 1.0, None, *map(p, out),
                p(torch.empty(n, dtype=U8, device="cuda")), n, s)
        f = L.moe_balance_loss
    elif kind == "norm":
        T, d = 640, size
        x, r, w = (torch.randn((n, d), device="cuda", generator=g).to(BF) for n in (T, T, 1))
        out = [torch.empty_like(x), torch.empty_like(x)]
        args = (p(x), d, p(r), d, 0, p(w), 0, T, d, 1e-6, p(out[0]), d, p(out[1]), d, None, 0, None, None, s)
        f = L.moe_add_rmsnorm
    elif kind == "norm_backward":
        T, d = 40, size
        dy, h, w = (torch.randn((n, d), device="cuda", generator=g).to(BF) for n in (T, T, 1))
        out = [torch.empty_like(dy), torch.empty(d, device="cuda")]
        n = vgg.moe_add_rmsnorm_workspace_bytes(T, d)
        args = (p(dy), d, p(h), d, 0, p(w), 0, p(torch.ones(T, device="cuda")), None, 0, T, d, p(out[0]), d, None, 0,
                p(out[1]), p(torch.empty(n, dtype=U8, device="cuda")), n, s)
        f = L.moe_add_rmsnorm_backward
    else:
        E = size
        off = torch.arange(E + 1, dtype=I32, device="cuda") * 2
        A = torch.randn((2 * E, 64), device="cuda", generator=g).to(BF)
        B = torch.randn((E, 64, 64), device="cuda", generator=g).to(BF)
        out = [torch.empty((2 * E, 64), device="cuda")]
        args = (p(A), None, p(B), 1, E, 2 * E, 64, 64, 2 * E, p(off), p(out[0]), s)
        f = L.moe_test_gemm_varlen_m
    keep.append(out)
    return out, lambda keep=keep: f(c.handle, *args)


@pytest.mark.parametrize("kind", ["balance", "norm", "norm_backward", "product"])
def test_first_call_of_a_thread(vgg, kind):
    """A thread that has made no CUDA call yet has no current context: the call brings it about."""
    import threading

    c, st = vgg.Context(0), torch.cuda.Stream()
    out, call = threaded_call(vgg, c, st, kind, 64, gen_of(3))
    torch.cuda.synchronize()
    status = []
    t = threading.Thread(target=lambda: status.append(call()))
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert status == [0]
    there = [t.clone() for t in out]
    assert call() == 0
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, there))
    assert vgg.moe_get_error(c) == (vgg.MOE_OK, 0)


@pytest.mark.parametrize("kind,small,large", [("balance", 4, 32), ("balance", 516, 1024), ("norm", 4160, 8192),
                                              ("norm_backward", 512, 8192), ("product", 4, 600)])
def test_calls_from_two_threads(vgg, kind, small, large):
    """Contexts, streams and sizes of their own, but one kernel whose shared memory depends on the size: every call is
    launched, and the results are those of a call alone."""
    import threading

    work = []
    for i, size in enumerate((small, large)):
        c, st = vgg.Context(0), torch.cuda.Stream()
        out, call = threaded_call(vgg, c, st, kind, size, gen_of(100 + i))
        torch.cuda.synchronize()
        assert call() == 0
        torch.cuda.synchronize()
        work.append((c, st, out, [t.clone() for t in out], call))
    status = [0, 0]

    def loop(i):
        st, call = work[i][1], work[i][4]
        for k in range(6000):
            status[i] = status[i] or call()
            if k % 100 == 99:
                st.synchronize()

    threads = [threading.Thread(target=loop, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert status == [0, 0]
    for c, _, out, alone, _ in work:
        assert all(torch.equal(a, b) for a, b in zip(out, alone))
        assert vgg.moe_get_error(c) == (vgg.MOE_OK, 0)
