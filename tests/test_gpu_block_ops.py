"""The operators around the layer on the device against their fp64 oracle.

u = 2^-24 is half an fp32 step, and a bf16, e4m3 rounding is off by at most 2^-8, 2^-4 of the value (below e4m3's
smallest normal number by 2^-10).  The bounds count those roundings; `depth` is the longest chain of fp32 additions."""
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


def rows(T, d, dtype, gen, pad=0, shift=0, scale=1.0):
    """[T, d] with a row stride of d + pad, starting `shift` elements into its storage."""
    flat = torch.full((T * (d + pad) + shift + 8,), float("nan"), dtype=dtype, device="cuda")
    t = flat[shift:shift + T * (d + pad)].view(T, d + pad)[:, :d]
    if gen is not None:
        t.copy_(torch.randn((T, d), device="cuda", generator=gen) * scale)
    return t


def gen_of(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ------------------------------------------------------------------------------------------------ norm

# depth of a row's sum of squares: at most 16 values a thread, two shuffle trees of 5, the square's rounding; the mean,
# eps, root and quotient add 4 more, and the root halves what comes before it
RSTD_REL = ((16 + 10 + 1 + 2) / 2 + 2) * U
Y_REL = RSTD_REL + 2 * U


def check_norm(x, res, w, eps, h, y, rstd, q=None, scales=None):
    hs = res if x is None else (res.float() + x.float()).to(res.dtype)
    if h is not None:
        assert torch.equal(h, hs)
    y64, r64 = bo.rmsnorm(f64(hs), f64(w), eps)
    if rstd is not None:
        assert np.all(np.abs(f64(rstd) - r64) <= RSTD_REL * r64)
    if y is not None:
        assert np.all(np.abs(f64(y) - y64) <= (2.0 ** -8 + 2 * Y_REL) * np.abs(y64) + 2.0 ** -133)
    if q is None:
        return
    T, d = y64.shape
    codes = f64(q.view(torch.float8_e4m3fn))
    if scales.dtype == F32:
        amax = np.abs(y64).max(axis=1)
        s = f64(scales)[:, None]
        assert np.all(np.abs(s[:, 0] - np.where(amax > 0, amax / 448, 1)) <= (Y_REL + U) * s[:, 0])
    else:
        sf = scales.cpu().numpy().astype(np.int64)
        assert np.all(sf[:, d // 32:] == 127)
        e = sf[:, :d // 32] - 127
        amax = np.abs(y64).reshape(T, d // 32, 32).max(axis=2)
        assert np.all(e[amax == 0] == 0)
        on = amax > 0
        # the smallest exponent, up to the fp32 error of the largest value
        assert np.all((amax * (1 - Y_REL))[on] <= (448 * 2.0 ** e)[on])
        assert np.all((amax * (1 + Y_REL))[on] > (448 * 2.0 ** (e - 1.0))[on])
        s = np.repeat(2.0 ** e, 32, axis=1)
    # + the quotient's rounding; a value may cross to a neighbouring code by its fp32 error
    assert np.all(np.abs(codes * s - y64) <= (2.0 ** -4 + 2 * Y_REL + 2 * U) * np.abs(y64) + 2.0 ** -10 * s)


@pytest.mark.parametrize("res_t", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T,d,pad,shift", [(1, 1, 0, 0), (1, 7, 0, 0), (3, 8, 0, 0), (5, 33, 2, 1), (2, 64, 0, 0), (7, 257, 0, 3),
                                           (129, 1000, 24, 0), (4, 2880, 40, 8), (33, 2048, 0, 0), (3, 7168, 8, 0),
                                           (2, 8200, 0, 0), (2, 9001, 0, 0), (2, 16384, 0, 0), (2, 16383, 1, 0),
                                           (1, 16384, 3, 1)])
def test_norm_bf16(vgg, ctx, T, d, pad, shift, res_t):
    g = gen_of(T * d)
    x, res = rows(T, d, BF, g, pad, shift), rows(T, d, res_t, g, pad, shift, 2.0)
    w = (1 + 0.1 * torch.randn(d, device="cuda", generator=g)).to(BF if pad else F32)
    h, y = rows(T, d, res_t, None, pad, shift), rows(T, d, BF, None, pad, shift)
    rstd = torch.empty(T, device="cuda")
    vgg.moe_add_rmsnorm(ctx, x, res, w, 1e-6, h, y, rstd)
    check_norm(x, res, w, 1e-6, h, y, rstd)
    # what lies between the rows is left alone
    for t in (h, y):
        flat = torch.as_strided(t, (T * (d + pad) + shift,), (1,), 0)
        assert int(flat.isnan().sum()) == T * pad + shift
    # nothing added, nothing kept
    y2 = rows(T, d, BF, None)
    vgg.moe_add_rmsnorm(ctx, None, h, w, 1e-6, None, y2)
    assert torch.equal(y2, y)


@pytest.mark.parametrize("form", ["e4m3", "mx"])
@pytest.mark.parametrize("res_t", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T,d,pad", [(1, 64, 0), (3, 192, 8), (61, 2048, 0), (200, 448, 64), (5, 2880, 0), (2, 7168, 16),
                                     (2, 8256, 0), (1, 16384, 0)])
def test_norm_codes(vgg, ctx, T, d, pad, res_t, form):
    g = gen_of(T + d)
    x, res = rows(T, d, BF, g, pad), rows(T, d, res_t, g, pad, scale=2.0)
    res[:, 5] *= 20
    w = (1 + 0.1 * torch.randn(d, device="cuda", generator=g)).to(res_t)
    h, y, rstd = rows(T, d, res_t, None, pad), rows(T, d, BF, None, pad), torch.empty(T, device="cuda")
    q = torch.empty((T, d), dtype=U8, device="cuda")
    sc = torch.empty(T, device="cuda") if form == "e4m3" else torch.empty((T, vgg.mx_sf_cols(d)), dtype=U8, device="cuda")
    vgg.moe_add_rmsnorm(ctx, x, res, w, 1e-5, h, y, rstd, q, sc)
    check_norm(x, res, w, 1e-5, h, y, rstd, q, sc)
    # codes alone, in place on the stream
    q2, sc2 = torch.empty_like(q), torch.empty_like(sc)
    vgg.moe_add_rmsnorm(ctx, x, res, w, 1e-5, res, None, None, q2, sc2)
    assert torch.equal(q2, q) and torch.equal(sc2, sc) and torch.equal(res, h)


@pytest.mark.parametrize("form", ["bf16", "e4m3", "mx"])
@pytest.mark.parametrize("res_t", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T,d,pad", [(607, 4160, 0), (608, 4160, 8), (1300, 7168, 0), (2111, 8192, 0)])
def test_norm_many_wide_rows(vgg, ctx, T, d, pad, res_t, form):
    """From four wide rows an SM on, the rows go through shared memory (608 on 152 SMs); odd numbers leave
    the last groups without a row."""
    g = gen_of(T + d)
    x, res = rows(T, d, BF, g, pad), rows(T, d, res_t, g, pad, scale=2.0)
    res[:, 5] *= 20
    w = (1 + 0.1 * torch.randn(d, device="cuda", generator=g)).to(res_t)
    h, y, rstd = rows(T, d, res_t, None, pad), rows(T, d, BF, None, pad), torch.empty(T, device="cuda")
    q = sc = None
    if form != "bf16":
        q = torch.empty((T, d), dtype=U8, device="cuda")
        sc = torch.empty(T, device="cuda") if form == "e4m3" else torch.empty((T, vgg.mx_sf_cols(d)), dtype=U8, device="cuda")
    vgg.moe_add_rmsnorm(ctx, x, res, w, 1e-5, h, y, rstd, q, sc)
    check_norm(x, res, w, 1e-5, h, y, rstd, q, sc)
    y2 = rows(T, d, BF, None)
    vgg.moe_add_rmsnorm(ctx, None, h, w, 1e-5, None, y2)  # nothing added
    assert torch.equal(y2, y)
    vgg.moe_add_rmsnorm(ctx, x, res, w, 1e-5, res, x)  # in place
    assert torch.equal(res, h) and torch.equal(x, y)


def test_norm_in_place(vgg, ctx):
    g = gen_of(5)
    x, res, w = rows(9, 1024, BF, g), rows(9, 1024, BF, g), torch.ones(1024, device="cuda")
    h, y = torch.empty_like(res), torch.empty_like(x)
    vgg.moe_add_rmsnorm(ctx, x, res, w, 1e-6, h, y)
    vgg.moe_add_rmsnorm(ctx, x, res, w, 1e-6, res, x)
    assert torch.equal(res, h) and torch.equal(x, y)


@pytest.mark.parametrize("form", ["e4m3", "mx"])
def test_norm_rows_without_values(vgg, ctx, form):
    """Zero rows, a single value, a block of zeros, values that are not finite: each row for itself."""
    T, d = 6, 256
    res = torch.zeros((T, d), device="cuda")
    res[1, 100] = 3.0
    res[2, 32:] = 1.0
    res[3] = 1e-30
    res[4, 7] = float("nan")
    res[5, 9] = float("inf")
    w = torch.ones(d, device="cuda")
    y, rstd, q = rows(T, d, BF, None), torch.empty(T, device="cuda"), torch.empty((T, d), dtype=U8, device="cuda")
    sc = torch.empty(T, device="cuda") if form == "e4m3" else torch.empty((T, 8), dtype=U8, device="cuda")
    vgg.moe_add_rmsnorm(ctx, None, res, w, 1e-6, None, y, rstd, q, sc)
    check_norm(None, res[:4], w, 1e-6, None, y[:4], rstd[:4], q[:4], sc[:4])
    assert not q[0].any() and (sc[0] == (1 if form == "e4m3" else 127)).all()
    assert y[4].isnan().all() and y[5, 9].isnan() and not y[5, :9].any()


@pytest.mark.parametrize("form", ["e4m3", "mx"])
def test_norm_of_tiny_weights(vgg, ctx, form):
    """Normed rows around 1e-33 and, in part, below fp32's smallest normal number: the scales follow them down."""
    g = gen_of(17)
    res = rows(5, 128, F32, g)
    for scale in (1e-33, 2.0 ** -128):
        w = scale * (1 + torch.rand(128, device="cuda", generator=g))
        q = torch.empty((5, 128), dtype=U8, device="cuda")
        sc = torch.empty(5, device="cuda") if form == "e4m3" else torch.empty((5, 4), dtype=U8, device="cuda")
        vgg.moe_add_rmsnorm(ctx, None, res, w, 1e-6, None, None, None, q, sc)
        y, _ = bo.rmsnorm(f64(res), f64(w), 1e-6)
        codes = f64(q.view(torch.float8_e4m3fn))
        s = f64(sc)[:, None] if form == "e4m3" else np.repeat(2.0 ** (sc.cpu().numpy().astype(np.float64) - 127), 32, axis=1)
        # e4m3's rounding, a step of fp32's smallest number (2^-149) in y and in the scale (up to 448 of them a code)
        tol = (2.0 ** -4 + 1e-5) * np.abs(y) + 2.0 ** -10 * s + 450 * 2.0 ** -149
        assert np.all(np.abs(codes * s - y) <= tol), scale


def test_norm_of_no_rows(vgg, ctx):
    e = torch.empty((0, 64), dtype=BF, device="cuda")
    dw = torch.full((64,), 7.0, device="cuda")
    vgg.moe_add_rmsnorm(ctx, e, e, torch.ones(64, device="cuda"), 1e-6, e, e)
    vgg.moe_add_rmsnorm_backward(ctx, e, e, torch.ones(64, device="cuda"), torch.empty(0, device="cuda"), None, e, None, dw,
                                 torch.empty(256, dtype=U8, device="cuda"))
    assert not dw.any()


@pytest.mark.parametrize("res_t", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("up", [True, False])
@pytest.mark.parametrize("T,d,pad,shift", [(1, 1, 0, 0), (1, 7168, 0, 0), (3, 40, 0, 0), (6, 33, 2, 1), (700, 192, 8, 0),
                                           (1100, 129, 0, 0), (305, 2048, 0, 0), (40, 2880, 40, 8), (5, 8200, 0, 0),
                                           (3, 16384, 0, 0), (2, 16383, 0, 0)])
def test_norm_backward(vgg, ctx, T, d, pad, shift, res_t, up):
    g = gen_of(T + 3 * d)
    dy, h = rows(T, d, BF, g, pad, shift), rows(T, d, res_t, g, pad, shift, 2.0)
    dh = rows(T, d, res_t, g, pad, shift) if up else None
    w = (1 + 0.1 * torch.randn(d, device="cuda", generator=g)).to(F32 if pad else BF)
    rstd = torch.rsqrt(h.float().pow(2).mean(1) + 1e-6)
    dx, dr, dw = rows(T, d, BF, None, pad, shift), rows(T, d, res_t, None, pad, shift), torch.empty(d, device="cuda")
    ws = torch.empty(vgg.moe_add_rmsnorm_workspace_bytes(T, d), dtype=U8, device="cuda")
    vgg.moe_add_rmsnorm_backward(ctx, dy, h, w, rstd, dh, dx, dr, dw, ws)
    gh, gw = bo.rmsnorm_backward(f64(dy), f64(h), f64(w), f64(rstd), None if dh is None else f64(dh))
    xh, gd = f64(h) * f64(rstd)[:, None], f64(dy) * f64(w)
    # fp32: each term has a few roundings, the mean a chain of at most 32 + 10 additions
    terms = np.abs(gd) + np.abs(xh) * np.mean(np.abs(gd * xh), axis=1, keepdims=True)
    err = 52 * U * f64(rstd)[:, None] * terms + 2 * U * np.abs(gh)
    assert np.all(np.abs(f64(dx) - gh) <= err + 2.0 ** -8 * (np.abs(gh) + err))
    assert np.all(np.abs(f64(dr) - gh) <= err + (2.0 ** -8 * (np.abs(gh) + err) if res_t == BF else 0))
    # at most ceil(1100 / 152) rows a block, then 1024 / 32 blocks a thread and a tree of 5
    assert np.all(np.abs(f64(dw) - gw) <= (8 + 32 + 5 + 3) * U * np.sum(np.abs(f64(dy) * xh), axis=0))
    # either form of the input's gradient alone, in place of an operand
    dw2 = torch.empty_like(dw)
    vgg.moe_add_rmsnorm_backward(ctx, dy, h, w, rstd, dh, dy, None, dw2, ws)
    assert torch.equal(dy, dx) and torch.equal(dw2, dw)


@pytest.mark.parametrize("res_t", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T,d,pad", [(1, 1, 0), (9, 33, 0), (40, 250, 3), (3000, 57, 0), (5000, 130, 3), (700, 515, 0),
                                     (1300, 1001, 3), (2500, 4091, 0), (333, 8178, 1), (20, 8179, 0),
                                     (170, 8094, 3), (200, 8143, 1), (160, 8102, 0), (2000, 7, 0), (1700, 8, 1)])
@pytest.mark.parametrize("apart", [0, 1], ids=["in_phase", "out_of_phase"])
def test_norm_rows_that_start_anywhere(vgg, ctx, T, d, pad, res_t, apart):
    """Rows of odd widths and strides, all tensors starting a row at the same place in 16 bytes, or one of them not;
    what lies between and around the rows stays as it was."""
    g = gen_of(T + d + pad)
    x, r = rows(T, d, BF, g, pad, 3), rows(T, d, res_t, g, pad, 3 + apart, 2.0)
    w = (1 + 0.1 * torch.randn(d, device="cuda", generator=g)).to(BF if pad else F32)

    def out(dtype, shift=3):
        flat = torch.full((T * (d + pad) + 16,), 777.0, dtype=dtype, device="cuda")
        return flat, flat[shift:shift + T * (d + pad)].view(T, d + pad)[:, :d]

    def untouched(flat, shift=3):
        keep = flat.clone()
        keep[shift:shift + T * (d + pad)].view(T, d + pad)[:, :d] = 777.0
        return bool((keep == 777.0).all())

    (fh, h), (fy, y), rstd = out(res_t), out(BF), torch.empty(T, device="cuda")
    vgg.moe_add_rmsnorm(ctx, x, r, w, 1e-6, h, y, rstd)
    check_norm(x, r, w, 1e-6, h, y, rstd)
    assert untouched(fh) and untouched(fy)
    dy, dh = rows(T, d, BF, g, pad, 3), rows(T, d, res_t, g, pad, 3 + apart)
    (fx, dx), (fr, dr), dw = out(BF), out(res_t), torch.empty(d, device="cuda")
    ws = torch.empty(vgg.moe_add_rmsnorm_workspace_bytes(T, d), dtype=U8, device="cuda")
    vgg.moe_add_rmsnorm_backward(ctx, dy, h, w, rstd, dh, dx, dr, dw, ws)
    gh, gw = bo.rmsnorm_backward(f64(dy), f64(h), f64(w), f64(rstd), f64(dh))
    xh, gd = f64(h) * f64(rstd)[:, None], f64(dy) * f64(w)
    # as in test_norm_backward; dweight: at most 33 rows a group, 8 groups, then 1024 / 32 blocks a thread and a tree of 5
    terms = np.abs(gd) + np.abs(xh) * np.mean(np.abs(gd * xh), axis=1, keepdims=True)
    err = 52 * U * f64(rstd)[:, None] * terms + 2 * U * np.abs(gh)
    assert np.all(np.abs(f64(dx) - gh) <= err + 2.0 ** -8 * (np.abs(gh) + err))
    assert np.all(np.abs(f64(dr) - gh) <= err + (2.0 ** -8 * (np.abs(gh) + err) if res_t == BF else 0))
    assert np.all(np.abs(f64(dw) - gw) <= (33 + 8 + 32 + 5 + 3) * U * np.sum(np.abs(f64(dy) * xh), axis=0))
    assert untouched(fx) and untouched(fr)
    again = torch.empty_like(dw)
    vgg.moe_add_rmsnorm_backward(ctx, dy, h, w, rstd, dh, dy, None, again, ws)
    assert torch.equal(dy, dx) and torch.equal(again, dw)


def far_rows(T, d, ld, dtype, gen):
    """[T, d] with a row stride of ld elements, the last rows past 2^31 elements from the first."""
    flat = torch.empty(((T - 1) * ld + d,), dtype=dtype, device="cuda")
    assert (T - 1) * ld >= 1 << 31
    t = flat.as_strided((T, d), (ld, 1))
    if gen is not None:
        t.copy_(torch.randn((T, d), device="cuda", generator=gen))
    return t


@pytest.mark.parametrize("T,d,ld", [(3, 64, 1 << 30), (5, 33, (1 << 29) + 1), (608, 4160, (1 << 22) - 8), (2, 8200, 1 << 31)])
def test_norm_offsets_past_32_bits(vgg, ctx, T, d, ld):
    """Each of the forward's and the backward's kernels; outputs are written with the same strides."""
    g = gen_of(T + d)
    w = 1 + 0.1 * torch.randn(d, device="cuda", generator=g)
    x, r = far_rows(T, d, ld, BF, g), far_rows(T, d, ld, BF, g)
    y, rstd = far_rows(T, d, ld, BF, None), torch.empty(T, device="cuda")
    r0 = r.contiguous()
    vgg.moe_add_rmsnorm(ctx, x, r, w, 1e-6, r, y, rstd)
    check_norm(x, r0, w, 1e-6, r, y, rstd)
    # the same rows side by side run on the same kernel and give the same bits
    dx, dw = far_rows(T, d, ld, BF, None), torch.empty(d, device="cuda")
    ws = torch.empty(vgg.moe_add_rmsnorm_workspace_bytes(T, d), dtype=U8, device="cuda")
    vgg.moe_add_rmsnorm_backward(ctx, y, r, w, rstd, x, dx, None, dw, ws)
    dx2, dw2 = torch.empty((T, d), dtype=BF, device="cuda"), torch.empty(d, device="cuda")
    vgg.moe_add_rmsnorm_backward(ctx, y.contiguous(), r.contiguous(), w, rstd, x.contiguous(), dx2, None, dw2, ws)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


# ------------------------------------------------------------------------------------------------ balance loss


def run_balance(vgg, ctx, logits, ids, ca, cz, mask=None, off=None, dloss=None, grad=True):
    T, E = logits.shape
    B = 1 if off is None else len(off) - 1
    loss, counts = torch.full((3,), 9.0, device="cuda"), torch.full((B, E), -1, dtype=I32, device="cuda")
    probs = torch.full((B, E), 9.0, device="cuda")
    dl = torch.full((T, E), 9.0, device="cuda") if grad else None
    ws = torch.randint(0, 256, (vgg.moe_balance_loss_workspace_bytes(T, E, B),), dtype=U8, device="cuda")
    vgg.moe_balance_loss(ctx, logits, ids, ca, cz, loss, counts, probs, dl, ws, mask=mask,
                         seq_offsets=None if off is None else torch.tensor(off, dtype=I32, device="cuda"),
                         dloss=None if dloss is None else torch.tensor(dloss, device="cuda"))
    return loss, counts, probs, dl


def check_balance(got, logits, ids, ca, cz, mask=None, off=None, dloss=1.0):
    loss, counts, probs, dl = got
    l64 = f64(logits)
    m = None if mask is None else mask.cpu().numpy()
    r = bo.balance_loss(l64, ids.cpu().numpy(), ca, cz, m, off, dloss)
    np.testing.assert_array_equal(counts.cpu().numpy(), r["counts"])
    # exp: its argument's rounding and two steps of its own; the sum over a row a chain of at most 32 + 5; a token's
    # probability then enters sums over a block's share of the tokens (at most 64 a lane group in these tests), 16
    # warps and the blocks (at most 1024 / 16)
    fin = np.where(np.isfinite(l64), l64, np.nan)
    span = np.nanmax(np.abs(fin)) * 2 if np.isfinite(l64).any() else 0.0
    p_rel = (span + 4 + 37 + 2) * U
    sum_rel = p_rel + (64 + 16 + 64 + 4) * U
    assert np.all(np.abs(f64(probs) - r["probs"]) <= sum_rel * r["probs"] + 1e-37)
    E = l64.shape[1]
    lse_abs = (p_rel + 4 * U) + 4 * U * span
    tol_b = (2 * sum_rel + (E / 32 + 8) * U) * r["loss"][1]
    tol_z = sum_rel * r["loss"][2] + 2 * lse_abs * (np.sqrt(r["loss"][2]) + lse_abs)
    assert abs(float(loss[1]) - r["loss"][1]) <= tol_b + 1e-37
    assert abs(float(loss[2]) - r["loss"][2]) <= tol_z + 1e-37
    assert abs(float(loss[0]) - r["loss"][0]) <= abs(ca) * tol_b + abs(cz) * tol_z + 4 * U * abs(r["loss"][0]) + 1e-37
    if dl is None:
        return r
    # terms of the gradient: p (c' - <p, c'> + zc lse) with c' the centred coefficients
    p, lse = bo.softmax_rows(l64)
    keep = np.ones(len(l64)) if m is None else (m != 0).astype(float)
    n = max(1, int(keep.sum()))
    K = ids.shape[1]
    cuts = [0, len(l64)] if off is None else off
    seq = np.searchsorted(np.asarray(cuts[1:]), np.arange(len(l64)), side="right")
    nb = np.array([max(1, int(keep[cuts[b]:cuts[b + 1]].sum())) for b in range(len(cuts) - 1)])
    used = max(1, sum(bool(keep[cuts[b]:cuts[b + 1]].sum()) for b in range(len(cuts) - 1)))
    c = np.abs(r["counts"] * E / (K * nb[:, None]) - 1) / nb[:, None] / used * abs(ca * dloss)
    c = c[seq] if len(l64) else np.zeros_like(p)
    terms = p * (c + np.sum(p * c, axis=1, keepdims=True) + 2 * abs(cz * dloss) / n * (np.abs(lse) + lse_abs)[:, None])
    assert np.all(np.abs(f64(dl) - r["dlogits"]) <= (2 * p_rel + 45 * U) * terms * keep[:, None] +
                  2 * abs(cz * dloss) / n * p * lse_abs * keep[:, None] + 1e-40)
    return r


def router_inputs(T, E, K, seed, spread=1.0):
    g = gen_of(seed)
    logits = spread * (torch.randn((T, E), device="cuda", generator=g) + 0.5 * torch.randn(E, device="cuda", generator=g))
    ids = torch.topk(logits, K, dim=1).indices.to(I32) if T else torch.empty((0, K), dtype=I32, device="cuda")
    return logits, ids, g


@pytest.mark.parametrize("T,E,K", [(0, 8, 2), (1, 1, 1), (1, 8, 2), (5, 7, 3), (16, 8, 2), (64, 8, 2), (65, 30, 6), (100, 64, 4),
                                   (17, 128, 8), (333, 128, 8), (40, 256, 8), (700, 256, 8), (50, 511, 8), (1000, 513, 3),
                                   (2500, 512, 8), (90, 1024, 8), (300, 1023, 5), (6000, 16, 1), (5000, 33, 2)])
def test_balance_one_sequence(vgg, ctx, T, E, K):
    logits, ids, g = router_inputs(T, E, K, T + E)
    check_balance(run_balance(vgg, ctx, logits, ids, 1e-2, 1e-3), logits, ids, 1e-2, 1e-3)
    mask = torch.rand(T, device="cuda", generator=g) < 0.6
    check_balance(run_balance(vgg, ctx, logits, ids, 0.5, 0.0, mask), logits, ids, 0.5, 0.0, mask)
    m8 = torch.zeros(T, dtype=U8, device="cuda")  # nothing counts
    got = run_balance(vgg, ctx, logits, ids, 0.5, 1.0, m8)
    assert not got[0].any() and not got[1].any() and not got[2].any() and not got[3].any()
    loss, counts, probs, _ = run_balance(vgg, ctx, logits, ids, 1e-2, 1e-3)
    again = run_balance(vgg, ctx, logits, ids, 1e-2, 1e-3, grad=False)
    assert torch.equal(again[0], loss) and torch.equal(again[1], counts) and torch.equal(again[2], probs)


@pytest.mark.parametrize("T,E,K,B", [(6, 8, 2, 6), (100, 8, 2, 5), (500, 128, 8, 3), (900, 512, 8, 37), (300, 96, 4, 300),
                                     (64, 1024, 8, 7), (400, 37, 5, 11), (1500, 64, 2, 2000)])
def test_balance_packed(vgg, ctx, T, E, K, B):
    logits, ids, g = router_inputs(T, E, K, T + E + B)
    cuts = sorted(np.random.default_rng(B).integers(0, T + 1, B - 1).tolist())  # empty sequences among them
    off = [0] + cuts + [T]
    mask = torch.rand(T, device="cuda", generator=g) < 0.8
    mask[off[1]:off[2]] = False  # a sequence without a counted token
    check_balance(run_balance(vgg, ctx, logits, ids, 0.3, 0.02, mask, off, 2.5), logits, ids, 0.3, 0.02, mask, off, 2.5)
    check_balance(run_balance(vgg, ctx, logits, ids, 0.3, 0.0, None, off), logits, ids, 0.3, 0.0, None, off)


@pytest.mark.parametrize("T,E,K,B", [(9000, 96, 2, 4000), (5000, 128, 8, 60), (700, 512, 1, 700), (15, 8, 2, 49), (9, 24, 1, 55),
                                     (3, 8, 2, 5), (42, 24, 8, 34), (41, 16, 2, 41), (200, 24, 2, 2000), (19685, 8, 8, 7)])
def test_balance_many_sequences_in_a_block(vgg, ctx, T, E, K, B):
    """More sequences in a block's share of the tokens than it has histograms for, and two or three; about as many
    blocks as tokens."""
    logits, ids, g = router_inputs(T, E, K, T + E + B)
    off = [0] + sorted(np.random.default_rng(B).integers(0, T + 1, B - 1).tolist()) + [T]
    mask = torch.rand(T, device="cuda", generator=g) < 0.7
    check_balance(run_balance(vgg, ctx, logits, ids, 0.3, 0.02, mask, off), logits, ids, 0.3, 0.02, mask, off)


def test_balance_offsets_past_32_bits(vgg, ctx):
    """More than 2^31 logits: counts, mean probabilities and the gradient at both ends and around 2^31."""
    T, E = (1 << 21) + 77, 1024
    logits = torch.empty((T, E), device="cuda")
    step = 1 << 16
    for t in range(0, T, step):
        logits[t:t + step] = torch.randn((min(step, T - t), E), device="cuda", generator=gen_of(t))
    ids = torch.randint(0, E, (T, 1), device="cuda", generator=gen_of(1)).to(I32)
    loss, counts, probs, dl = run_balance(vgg, ctx, logits, ids, 1.0, 0.0)
    want = torch.bincount(ids.view(-1), minlength=E)
    assert torch.equal(counts.view(-1).long(), want)
    total = torch.zeros(E, dtype=torch.float64, device="cuda")
    for t in range(0, T, step):
        total += torch.softmax(logits[t:t + step].double(), dim=1).sum(0)
    p = total / T
    # a probability's own error (see check_balance, spans below 14), then a warp's chain of T / (152 * 16) tokens at
    # least a lane, 16 warps and 152 blocks
    rel = (14 + 4 + 37 + 2 + 863 + 16 + 152 + 8) * U
    assert bool(((probs.view(-1).double() - p).abs() <= rel * p).all())
    f = want.double() * E / T
    assert abs(float(loss[1]) - float((f * p).sum())) <= 2 * rel * float((f * p).sum())
    u = f - 1.0
    for t in (0, (1 << 21) - 40, T - 80):
        q = torch.softmax(logits[t:t + 80].double(), dim=1)
        ref = q * (u - (q * u).sum(1, keepdim=True)) / T
        terms = q * (u.abs() + (q * u.abs()).sum(1, keepdim=True)) / T
        assert bool(((dl[t:t + 80].double() - ref).abs() <= (2 * 57 + 45) * U * terms).all())


def test_balance_masked_logits(vgg, ctx):
    """Experts closed to a token (-inf), large logits of both signs, a token with no open expert, and values that
    are not finite in a row that does not count."""
    logits, ids, _ = router_inputs(50, 40, 2, 3, spread=20.0)
    logits[3, :20] = -float("inf")
    logits[4, 1:] = -float("inf")
    logits[5, :] = -float("inf")
    logits[6, :] = torch.finfo(F32).min
    logits[7, :] = float("nan")
    logits[8, 3] = float("inf")
    mask = torch.ones(50, dtype=torch.bool, device="cuda")
    mask[7:9] = False
    clean = logits.clone()
    clean[7:9] = 0.0
    got = run_balance(vgg, ctx, logits, ids, 1.0, 0.0, mask)
    # the row of the type's lowest value is uniform, and its z term the square of that value: with the z loss off
    # the oracle covers it
    l64 = f64(clean)
    r = bo.balance_loss(l64, ids.cpu().numpy(), 1.0, 0.0, mask.cpu().numpy())
    np.testing.assert_array_equal(got[1].cpu().numpy(), r["counts"])
    assert np.all(np.abs(f64(got[2]) - r["probs"]) <= 400 * U * r["probs"] + 1e-30)
    assert np.all(np.abs(f64(got[3]) - r["dlogits"]) <= 1e-6 * np.abs(r["dlogits"]).max())
    assert not got[3][5].any() and not got[3][7:9].any() and not got[3][4, 1:].any()


def test_balance_misaligned_logits(vgg, ctx):
    base, ids, _ = router_inputs(70, 64, 4, 11)
    flat = torch.empty(70 * 64 + 1, device="cuda")
    logits = flat[1:].view(70, 64)
    logits.copy_(base)
    check_balance(run_balance(vgg, ctx, logits, ids, 0.1, 0.1), logits, ids, 0.1, 0.1)


def test_balance_gradient_against_differences(vgg, ctx):
    """Along a direction v: (L(l + h v) - L(l - h v)) / 2h with fixed choices, from the device's own loss.  fp32 losses of
    order 10 leave 2^-23 * 10 / 2h, the third derivative about h^2."""
    logits, ids, g = router_inputs(64, 32, 4, 5)
    v = torch.randn(logits.shape, device="cuda", generator=g)
    h = 2.0 ** -6
    off = [0, 20, 64]
    lp = run_balance(vgg, ctx, logits + h * v, ids, 3.0, 0.5, None, off, grad=False)[0][0]
    lm = run_balance(vgg, ctx, logits - h * v, ids, 3.0, 0.5, None, off, grad=False)[0][0]
    dl = run_balance(vgg, ctx, logits, ids, 3.0, 0.5, None, off)[3]
    want = float((dl.double() * v.double()).sum())
    assert abs(float(lp.double() - lm.double()) / (2 * h) - want) <= 1e-4 + 2 * h * h


def test_balance_reports_bad_ids_and_offsets(vgg, ctx):
    logits, ids, _ = router_inputs(40, 16, 2, 7)
    bad = ids.clone()
    bad[3, 1], bad[9, 0] = 16, -1
    got = run_balance(vgg, ctx, logits, bad, 1.0, 0.0)
    assert vgg.moe_get_error(ctx) == (vgg.MOE_ERR_DEVICE, vgg.DEV_BAD_EXPERT)
    want = ids.cpu().numpy().copy()
    ref = np.bincount(np.delete(want.reshape(-1), [7, 18]), minlength=16)
    np.testing.assert_array_equal(got[1][0].cpu().numpy(), ref)
    for off in ([0, 30, 20, 40], [1, 20, 30, 40], [0, 20, 30, 41], [0, 20, 30, 39], [0, -5, 1 << 30, 40]):
        run_balance(vgg, ctx, logits, ids, 1.0, 0.0, None, off)
        assert vgg.moe_get_error(ctx) == (vgg.MOE_ERR_DEVICE, vgg.DEV_BAD_OFFSETS), off


def test_balance_is_reproducible_and_captures(vgg, ctx):
    logits, ids, _ = router_inputs(4096, 128, 8, 9)
    first = run_balance(vgg, ctx, logits, ids, 0.1, 0.1)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, run_balance(vgg, ctx, logits, ids, 0.1, 0.1)))
    out = [torch.zeros_like(t) for t in first]
    ws = torch.empty(vgg.moe_balance_loss_workspace_bytes(4096, 128), dtype=U8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vgg.moe_balance_loss(ctx, logits, ids, 0.1, 0.1, out[0], out[1], out[2], out[3], ws)
    for _ in range(2):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, out))


# ------------------------------------------------------------------------------------------------ router backward


def run_router(vgg, ctx, dl, X, W, dX_in, dW_in, want=(True, True)):
    (T, E), d = dl.shape, X.shape[1]
    dX = torch.full((T, d), 9.0, dtype=BF, device="cuda") if want[0] else None
    dW = torch.full((d, E), 9.0, device="cuda") if want[1] else None
    ws = torch.randint(0, 256, (vgg.moe_router_backward_workspace_bytes(T, d, E),), dtype=U8, device="cuda")
    vgg.moe_router_backward(ctx, dl, X, W, dX_in, dW_in, dX, dW, ws)
    return dX, dW


ROUTER_SIZES = [(1, 64, 8), (3, 128, 16), (64, 192, 64), (65, 256, 128), (127, 320, 136), (300, 64, 1024), (700, 512, 264),
                (2000, 1536, 96), (129, 2880, 128)]


@pytest.mark.parametrize("T,d,E", ROUTER_SIZES)
def test_router_backward_whole_numbers(vgg, ctx, T, d, E):
    """Small whole numbers: every product and sum is exact, so the result is too."""
    g = gen_of(T + d)
    dl = torch.randint(-1, 2, (T, E), device="cuda", generator=g).float()
    X = torch.randint(-1, 2, (T, d), device="cuda", generator=g).to(BF)
    W = torch.where(torch.rand((d, E), device="cuda", generator=g) < 16 / E, 1.0, 0.0).to(BF)
    dX_in = torch.randint(-8, 9, (T, d), device="cuda", generator=g).to(BF)
    dW_in = torch.randint(-8, 9, (d, E), device="cuda", generator=g).float()
    dX, dW = run_router(vgg, ctx, dl, X, W, dX_in, dW_in)
    rX, rW = bo.router_backward(f64(dl), f64(X), f64(W), f64(dX_in), f64(dW_in))
    assert np.abs(rX).max() <= 256  # whole numbers that bf16 holds
    np.testing.assert_array_equal(f64(dX), rX)
    np.testing.assert_array_equal(f64(dW), rW)


@pytest.mark.parametrize("T,d,E", ROUTER_SIZES)
@pytest.mark.parametrize("add", [True, False])
def test_router_backward(vgg, ctx, T, d, E, add):
    g = gen_of(T + d + E)
    dl = 1e-4 * torch.randn((T, E), device="cuda", generator=g)
    X = torch.randn((T, d), device="cuda", generator=g).to(BF)
    W = (torch.randn((d, E), device="cuda", generator=g) / d ** 0.5).to(BF)
    dX_in = (1e-4 * torch.randn((T, d), device="cuda", generator=g)).to(BF) if add else None
    dW_in = 1e-3 * torch.randn((d, E), device="cuda", generator=g) if add else None
    dX, dW = run_router(vgg, ctx, dl, X, W, dX_in, dW_in)
    rX, rW = bo.router_backward(f64(dl), f64(X), f64(W), f64(dX_in) if add else None, f64(dW_in) if add else None)
    absX = np.abs(f64(dl)) @ np.abs(f64(W)).T
    absW = np.abs(f64(X)).T @ np.abs(f64(dl))
    # dlogits rounded to bf16; the accumulation over E (T) terms, a step each; the result's rounding
    eX = (2.0 ** -8 + 2 * (E + 2) * U) * absX
    assert np.all(np.abs(f64(dX) - rX) <= eX + 2.0 ** -8 * (np.abs(rX) + eX))
    # two bf16 parts leave 2^-16
    assert np.all(np.abs(f64(dW) - rW) <= (2.0 ** -16 + 2 * (T + 20) * U) * absW + 4 * U * np.abs(rW))
    # a lost or doubled token or expert would show in the norm: independent roundings stay well below their bound
    assert np.linalg.norm(f64(dX) - rX) <= 2.0 ** -8 * np.linalg.norm(rX)
    assert np.linalg.norm(f64(dW) - rW) <= 2.0 ** -16 * np.linalg.norm(rW)
    # in place, and each product alone
    if add:
        a, b = dX_in.clone(), dW_in.clone()
        ws = torch.empty(vgg.moe_router_backward_workspace_bytes(T, d, E), dtype=U8, device="cuda")
        vgg.moe_router_backward(ctx, dl, X, W, a, b, a, b, ws)
        assert torch.equal(a, dX) and torch.equal(b, dW)
    assert torch.equal(run_router(vgg, ctx, dl, X, W, dX_in, dW_in, (True, False))[0], dX)
    assert torch.equal(run_router(vgg, ctx, dl, X, W, dX_in, dW_in, (False, True))[1], dW)


@pytest.mark.parametrize("T,d,E", [(500, 64, 8), (4096, 256, 128), (20000, 128, 264)])
def test_router_weight_gradient_has_fp32_precision(vgg, ctx, T, d, E):
    """An element: three bf16 parts leave 2^-24 of a value, an accumulator's 24 additions a step (2^-23) each, the sums
    over T / 128 accumulators and up to 16 splits half a step each.  In the norm an fp32 product is off by about 2^-21
    and two parts by 2^-18.7: 2^-20 lies between."""
    g = gen_of(T)
    dl = torch.randn((T, E), device="cuda", generator=g)
    X = torch.randn((T, d), device="cuda", generator=g).to(BF)
    dW = run_router(vgg, ctx, dl, X, torch.zeros((d, E), dtype=BF, device="cuda"), None, None, (False, True))[1]
    ref, mag = X.double().T @ dl.double(), X.double().abs().T @ dl.double().abs()
    err = (dW.double() - ref).abs()
    assert bool((err <= (1 + 48 + T / 128 + 16 + 2) * U * mag).all())
    assert float(torch.linalg.norm(err)) <= 2.0 ** -20 * float(torch.linalg.norm(ref))


def test_router_backward_offsets_past_32_bits(vgg, ctx):
    """More than 2^31 elements of X and dX; whole numbers, so both products are exact."""
    T, d, E = 65536, 32832, 8
    g = gen_of(5)
    X = torch.randint(-1, 2, (T, d), device="cuda", generator=g, dtype=torch.int8).to(BF)
    dl = torch.randint(-1, 2, (T, E), device="cuda", generator=g).float()
    W = torch.randint(-1, 2, (d, E), device="cuda", generator=g).to(BF)
    dX, dW = run_router(vgg, ctx, dl, X, W, None, None)
    for t in (0, 32768, T - 64):
        assert torch.equal(dX[t:t + 64].double(), dl[t:t + 64].double() @ W.double().T)
    for i in (0, 16384, d - 64):
        assert torch.equal(dW[i:i + 64].double(), X[:, i:i + 64].double().T @ dl.double())


def test_router_backward_of_no_tokens(vgg, ctx):
    X, W = torch.empty((0, 64), dtype=BF, device="cuda"), torch.ones((64, 8), dtype=BF, device="cuda")
    dl, dW_in = torch.empty((0, 8), device="cuda"), torch.randn((64, 8), device="cuda")
    _, dW = run_router(vgg, ctx, dl, X, W, None, dW_in)
    assert torch.equal(dW, dW_in)
    assert not run_router(vgg, ctx, dl, X, W, None, None)[1].any()


# ------------------------------------------------------------------------------------------------ streams


def test_calls_follow_their_stream(vgg, ctx):
    """Each operator on a stream of its own, behind work that produces its inputs there."""
    s = torch.cuda.Stream()
    logits, ids, g = router_inputs(512, 64, 4, 21)
    src = torch.randn((512, 256), device="cuda", generator=g).to(BF)
    W = torch.randn((256, 64), device="cuda", generator=g).to(BF)
    w = torch.ones(256, device="cuda")
    torch.cuda.synchronize()
    res = {}
    for key, st in (("own", s), ("default", torch.cuda.current_stream())):
        with torch.cuda.stream(st):
            x = src.float().mul(1.0).to(BF)
            h, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(512, device="cuda")
            vgg.moe_add_rmsnorm(ctx, x, x, w, 1e-6, h, y, rstd)
            loss, counts, probs, dl = run_balance(vgg, ctx, logits, ids, 0.1, 0.1)
            dX, dW = run_router(vgg, ctx, dl, y, W, x, None)
            out, dw = torch.empty_like(x), torch.empty(256, device="cuda")
            ws = torch.empty(vgg.moe_add_rmsnorm_workspace_bytes(512, 256), dtype=U8, device="cuda")
            vgg.moe_add_rmsnorm_backward(ctx, dX, h, w, rstd, None, out, None, dw, ws)
        st.synchronize()
        res[key] = (y, loss, dl, dX, dW, out, dw)
    assert all(torch.equal(a, b) for a, b in zip(res["own"], res["default"]))
