"""The layer for a few tokens against a plain implementation in 64 bits.

What a result may be off, from the formats alone.  The choice and its weights are compared on logits that lie further
apart than fp32 tells apart.  A sum of k products in fp32 is off by at most k 2^-23 of the sum of their magnitudes (half a
step a rounding, twice that where the tensor core truncates); the sigmoid by 2^-20 of its value.  bf16: A's two parts leave
2^-16 of a value.  e4m3: A's codes are those of some A within its bound, so the bound of the sum holds the spread of
the codes (the rule is monotone in A; where the row's largest value itself may round either way, a whole step, 2^-3 of
each).  O adds half a bf16 step, 2^-8."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def vgg():
    import varlen_grouped_gemm_gb300 as m
    return m


@pytest.fixture(scope="module")
def ctx(vgg):
    return vgg.Context(0)


def make(T, d, E, n, K, seed=0, bias=None):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std):
        return (torch.randn(shape, device="cuda", generator=g) * std).to(BF)

    s = dict(X=normal(T, d, std=1.0), W_r=normal(d, E, std=d ** -0.5), W_gate=normal(E, n, d, std=d ** -0.5),
             W_up=normal(E, n, d, std=d ** -0.5), W_down=normal(E, d, n, std=n ** -0.5), bias=None, K=K)
    if bias == "normal":
        s["bias"] = 0.5 * torch.randn(E, device="cuda", generator=g)
    elif bias == "few":  # every token prefers the same K experts
        s["bias"] = torch.zeros(E, device="cuda")
        s["bias"][E // 2:E // 2 + K] = 40.0
    separate(s)
    return s


def logits64(s):
    v = s["X"].double() @ s["W_r"].double()
    return v if s["bias"] is None else v + s["bias"].double()


def separate(s):
    """Tokens whose choice fp32 could not decide take the clearest token's X."""
    E, K = s["W_r"].shape[1], s["K"]
    if E == 1 or s["X"].shape[0] == 0:
        return
    top = torch.topk(logits64(s), min(K + 1, E), dim=1).values
    gap = (top[:, :-1] - top[:, 1:]).amin(1)
    s["X"] = torch.where((gap > 1e-4)[:, None], s["X"], s["X"][gap.argmax()]).contiguous()


def row_scale(top):
    """max / 448 as one division (of a number torch multiplies by the reciprocal), 1 for a zero row."""
    return torch.where(top > 0, torch.div(top, torch.full_like(top, 448.0)), torch.ones_like(top))


def codes(w):
    scale = row_scale(w.float().abs().amax(-1))
    return (w.float() / scale[..., None]).to(E4M3).view(torch.uint8), scale


def rule(a):
    """Values of the per-row codes of bf16 rows, by the stated rule."""
    q, scale = codes(a)
    return q.view(E4M3).double() * scale.double()[:, None]


def reference(s, form, w8=None):
    """(O, bound, ids, w) in 64 bits."""
    K = s["K"]
    top = torch.sort(logits64(s), dim=1, descending=True)
    ids, w = top.indices[:, :K], torch.softmax(top.values[:, :K], 1)
    T, d = s["X"].shape
    n = s["W_gate"].shape[1]
    O, bound = torch.zeros((T, d), dtype=F64, device="cuda"), torch.zeros((T, d), dtype=F64, device="cuda")
    for e in ids.unique().tolist():
        t, k = torch.nonzero(ids == e, as_tuple=True)
        x = s["X"][t]
        if form == "e4m3":
            x = rule(x)
            wg, wu, wd = (q[e].view(E4M3).double() * c[e].double()[:, None]
                          for q, c in ((w8.Wg_q, w8.wg_scale), (w8.Wu_q, w8.wu_scale), (w8.Wd_q, w8.wd_scale)))
        else:
            x, wg, wu, wd = x.double(), s["W_gate"][e].double(), s["W_up"][e].double(), s["W_down"][e].double()
        h, u = x @ wg.T, x @ wu.T
        dh, du = (d + 4) * 2.0 ** -23 * (x.abs() @ wg.abs().T), (d + 4) * 2.0 ** -23 * (x.abs() @ wu.abs().T)
        sg = 1 / (1 + torch.exp(-h))
        a = h * sg * u
        # |d silu / dh| <= 1.1
        da = 1.1 * dh * (u.abs() + du) + (h * sg).abs() * du + 2.0 ** -20 * a.abs() + 1e-38
        if form == "e4m3":
            mid, lo, hi = rule(a.to(BF)), rule_of(a - da, a), rule_of(a + da, a)
            slack = torch.maximum((hi - mid).abs(), (mid - lo).abs())
            most = (a.abs() + da).amax(1)
            unsure = most.to(BF) != (a.abs() - da).amax(1).to(BF)
            slack = torch.where(unsure[:, None], slack + 2.0 ** -3 * a.abs(), slack)
            a = mid
        else:
            slack = da + 2.0 ** -16 * a.abs()
        y = a @ wd.T
        dy = slack @ wd.abs().T + (n + 4) * 2.0 ** -23 * (a.abs() @ wd.abs().T)
        O[t] += w[t, k, None] * y
        bound[t] += w[t, k, None] * (dy + 2.0 ** -18 * y.abs())
    return O, bound * (1 + 2.0 ** -8) + 2.0 ** -8 * O.abs(), ids.to(I32), w


def rule_of(v, a):
    """v's codes with the scale of a's rows."""
    scale = row_scale(a.to(BF).float().abs().amax(1, keepdim=True))
    return (v.to(BF).float() / scale).clamp(-448, 448).to(E4M3).double() * scale.double()


def call(vgg, ctx, s, form="bf16", w8=None, X=None, O=None, ws=None, stream=None):
    T, d = s["X"].shape
    E, n = s["W_gate"].shape[:2]
    K = s["K"]
    O = torch.full((T, d), float("nan"), dtype=BF, device="cuda") if O is None else O
    ids, w = torch.full((T, K), -1, dtype=I32, device="cuda"), torch.zeros((T, K), device="cuda")
    if ws is None:
        ws = torch.full((vgg.moe_few_workspace_bytes(T, d, E, n, K),), 0xFF, dtype=torch.uint8, device="cuda")
    X = s["X"] if X is None else X
    if form == "e4m3":
        vgg.moe_forward_few_e4m3(ctx, X, s["W_r"], s["bias"], w8, K, O, ids, w, ws, stream=stream)
    else:
        vgg.moe_forward_few(ctx, X, s["W_r"], s["bias"], s["W_gate"], s["W_up"], s["W_down"], K, O, ids, w, ws, stream=stream)
    return O, ids, w


def weights8(vgg, ctx, s):
    return vgg.E4m3Weights.quantize(ctx, s["W_gate"], s["W_up"], s["W_down"])


def check(got, want):
    (O, ids, w), (ref, bound, rids, rw) = got, want
    assert torch.equal(ids, rids)
    np.testing.assert_allclose(w.cpu().numpy(), rw.cpu().numpy(), rtol=1e-4, atol=1e-7)  # logits' error times 1
    over = ((O.double() - ref).abs() - bound).amax().item()
    assert over <= 0, over


CASES = [
    (1, 128, 8, 64, 2, None), (1, 2048, 128, 512, 8, None), (2, 64, 8, 64, 1, None), (3, 192, 8, 64, 2, "normal"),
    (1, 64, 8, 64, 8, None), (7, 320, 24, 448, 3, None), (8, 256, 16, 128, 4, "few"), (9, 256, 16, 128, 4, "few"),
    (16, 1536, 512, 256, 8, None), (17, 192, 1024, 192, 8, None), (24, 512, 8, 320, 8, "normal"), (33, 448, 40, 64, 5, None),
    (61, 256, 32, 128, 2, "normal"), (64, 2048, 128, 512, 8, None), (64, 128, 8, 64, 8, "few"), (64, 704, 16, 192, 1, "few"),
]


@pytest.mark.parametrize("form", ["bf16", "e4m3"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_matches_64_bits(vgg, ctx, case, form):
    T, d, E, n, K, bias = case
    s = make(T, d, E, n, K, seed=T + d, bias=bias)
    w8 = weights8(vgg, ctx, s) if form == "e4m3" else None
    got = call(vgg, ctx, s, form, w8)
    assert vgg.moe_get_error(ctx) == (vgg.MOE_OK, 0)
    check(got, reference(s, form, w8))


def test_more_tokens_than_a_round_and_every_width(vgg, ctx):
    """Every number of tokens once, on sizes that change the ring, the tiles' halves and the lists."""
    for T in range(1, 65):
        s = make(T, 64 * (1 + T % 5), 8 * (1 + T % 4), 64 * (1 + T % 3), 1 + T % 8, seed=T)
        check(call(vgg, ctx, s), reference(s, "bf16"))
    assert vgg.moe_get_error(ctx) == (vgg.MOE_OK, 0)


def test_rows_of_larger_matrices(vgg, ctx):
    s = make(11, 192, 16, 64, 4, seed=5)
    X = torch.full((11, 200), float("nan"), dtype=BF, device="cuda")
    X[:, :192] = s["X"]
    O = torch.full((11, 196), 7.0, dtype=BF, device="cuda")
    plain = call(vgg, ctx, s)
    got = call(vgg, ctx, s, X=X[:, :192], O=O[:, :192])
    assert torch.equal(O[:, :192], plain[0]) and (O[:, 192:] == 7.0).all()
    assert torch.equal(got[1], plain[1]) and torch.equal(got[2], plain[2])


@pytest.mark.parametrize("form", ["bf16", "e4m3"])
def test_same_bits_again_and_on_another_stream_and_in_a_graph(vgg, ctx, form):
    s = make(40, 512, 64, 192, 6, seed=6)
    w8 = weights8(vgg, ctx, s) if form == "e4m3" else None
    want = [t.clone() for t in call(vgg, ctx, s, form, w8)]
    T, d = s["X"].shape
    E, n = s["W_gate"].shape[:2]
    buf = vgg.FewBuffers.allocate(T, d, E, n, s["K"])
    weights = w8 if form == "e4m3" else (s["W_gate"], s["W_up"], s["W_down"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        vgg.forward_few(ctx, s["X"], s["W_r"], s["bias"], weights, buf)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((buf.O, buf.topk_ids, buf.topk_w), want))
    graphs = []
    for _ in range(2):  # two captured calls share the workspace and run one after the other
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            vgg.forward_few(ctx, s["X"], s["W_r"], s["bias"], weights, buf)
    other = make(40, 512, 64, 192, 6, seed=7)["X"]
    kept = s["X"].clone()
    for X in (kept, other, kept):
        s["X"].copy_(X)
        for g in graphs:
            buf.O.zero_()
            g.replay()
        torch.cuda.synchronize()
        if X is kept:
            assert torch.equal(buf.O, want[0])
        else:
            check((buf.O, buf.topk_ids, buf.topk_w), reference(dict(s, X=other), form, w8))
    assert vgg.moe_get_error(ctx) == (vgg.MOE_OK, 0)


def test_two_calls_at_once(vgg, ctx):
    """Two streams, each with its workspace."""
    cases = [make(5, 1024, 32, 256, 4, seed=8), make(64, 512, 64, 128, 8, seed=9)]
    want = [call(vgg, ctx, s) for s in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    ws = [torch.empty(vgg.moe_few_workspace_bytes(s["X"].shape[0], s["X"].shape[1], *s["W_gate"].shape[:2], s["K"]),
                      dtype=torch.uint8, device="cuda") for s in cases]
    out = [[torch.zeros_like(t) for t in w] for w in want]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, st, w, o in zip(cases, streams, ws, out):
            vgg.moe_forward_few(ctx, s["X"], s["W_r"], s["bias"], s["W_gate"], s["W_up"], s["W_down"], s["K"], *o, w,
                                stream=st)
    torch.cuda.synchronize()
    for o, w in zip(out, want):
        assert all(torch.equal(a, b) for a, b in zip(o, w))
    assert vgg.moe_get_error(ctx) == (vgg.MOE_OK, 0)


def test_choice_is_that_of_the_router(vgg, ctx):
    """Ties, masked experts and a token of infinities: the choice and the weights by the rule of moe_route."""
    T, d, E, n, K = 24, 64, 32, 64, 4
    s = make(T, d, E, n, K, seed=10)
    # whole numbers: logits exact whatever the order of the sum; experts in equal pairs
    s["X"] = s["X"].float().round().to(BF)
    s["W_r"] = (4 * s["W_r"].float()).round().to(BF)
    s["W_r"][:, 1::2] = s["W_r"][:, 0::2]
    s["bias"] = torch.zeros(E, device="cuda")
    s["bias"][3], s["bias"][8:] = 2.0, float("-inf")  # 8 experts are left
    s["X"][5] = 0.0
    logits, scores = torch.empty((T, E), device="cuda"), None
    ids, w = torch.empty((T, K), dtype=I32, device="cuda"), torch.empty((T, K), device="cuda")
    vgg.moe_route(ctx, s["X"], s["W_r"], s["bias"], K, logits, scores, ids, w)
    got = call(vgg, ctx, s)
    assert torch.equal(got[1], ids)
    np.testing.assert_allclose(got[2].cpu().numpy(), w.cpu().numpy(), rtol=1e-6)
    assert got[1][5].tolist() == [3, 0, 1, 2]
    assert vgg.moe_get_error(ctx) == (vgg.MOE_OK, 0)


@pytest.mark.parametrize("form", ["bf16", "e4m3"])
def test_a_token_that_is_not_finite_stays_alone(vgg, ctx, form):
    """Tokens share tiles, not columns: a NaN and an infinity leave the others' outputs what they were, within the bound."""
    s = make(20, 256, 8, 128, 2, seed=11)
    w8 = weights8(vgg, ctx, s) if form == "e4m3" else None
    ref = reference(s, form, w8)
    bad = dict(s, X=s["X"].clone())
    bad["X"][3, 7], bad["X"][11, 200] = float("nan"), float("inf")
    O, ids, w = call(vgg, ctx, bad, form, w8)
    keep = torch.ones(20, dtype=torch.bool, device="cuda")
    keep[3] = keep[11] = False
    check((O[keep], ids[keep], w[keep]), tuple(t[keep] for t in ref))
    assert not torch.isfinite(O[3]).any() and ((ids >= 0) & (ids < 8)).all()
    assert vgg.moe_get_error(ctx) == (vgg.MOE_OK, 0)


def test_no_tokens_and_one_expert_row(vgg, ctx):
    ws = torch.empty(vgg.moe_few_workspace_bytes(0, 64, 8, 64, 2), dtype=torch.uint8, device="cuda")
    e = torch.empty((0, 64), dtype=BF, device="cuda")
    s = make(1, 64, 8, 64, 2)
    vgg.moe_forward_few(ctx, e, s["W_r"], None, s["W_gate"], s["W_up"], s["W_down"], 2, torch.empty_like(e),
                        torch.empty((0, 2), dtype=I32, device="cuda"), torch.empty((0, 2), device="cuda"), ws)
    assert vgg.moe_get_error(ctx) == (vgg.MOE_OK, 0)


def test_beside_the_layer_s_own_path(vgg, ctx):
    """The training path's forward on the same tokens: the same choice, outputs within both paths' roundings."""
    s = make(48, 512, 32, 256, 4, seed=12)
    buf = vgg.Buffers.allocate(48, 512, 32, 256, 4, backward=False)
    vgg.forward(ctx, s["X"], s["W_r"], None, s["W_gate"], s["W_up"], s["W_down"], buf, cache=False)
    O, ids, w = call(vgg, ctx, s)
    assert torch.equal(ids, buf.topk_ids)
    # bf16 roundings: O twice, the pairs' outputs once
    assert ((O.float() - buf.O.float()).norm() / O.float().norm()).item() <= 1.25 * 3 ** 0.5 * 1.6e-3


@pytest.mark.parametrize("form", ["bf16", "e4m3"])
def test_buffers_with_room_for_more_tokens(vgg, ctx, form):
    """One set of buffers for batches of any size up to theirs: the same bits as in buffers of that size, the rows behind as they were."""
    s = make(21, 256, 16, 128, 3, seed=13)
    weights = weights8(vgg, ctx, s) if form == "e4m3" else (s["W_gate"], s["W_up"], s["W_down"])
    buf = vgg.FewBuffers.allocate(40, 256, 16, 128, 3)
    for T in (21, 1, 9, 0):
        for t in (buf.O, buf.topk_ids, buf.topk_w):
            t.fill_(7)
        buf.ws.fill_(0xFF)
        one = vgg.FewBuffers.allocate(T, 256, 16, 128, 3)
        for b in (buf, one):
            vgg.forward_few(ctx, s["X"][:T], s["W_r"], None, weights, b)
        for name in ("O", "topk_ids", "topk_w"):
            t = getattr(buf, name)
            assert torch.equal(t[:T], getattr(one, name)) and (t[T:] == 7).all(), (T, name)
    assert vgg.moe_get_error(ctx) == (vgg.MOE_OK, 0)
    with pytest.raises(ValueError):
        vgg.forward_few(ctx, torch.zeros((41, 256), dtype=BF, device="cuda"), s["W_r"], None, weights, buf)
