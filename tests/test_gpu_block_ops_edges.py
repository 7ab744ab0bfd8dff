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
