"""The expert layer for a few tokens, and its training step with activations kept in 8 bits: what is measured, and the
plain forms.

Three operators:

* ``few``            the whole layer for the few tokens of a decoding step: router, choice, the chosen experts' three
                     products, weighted sum; bf16 weights, or e4m3 codes with a scale for each output channel;
* ``keep``           the experts' forward of a training step which leaves X, H and U for the backward as 8-bit whole
                     numbers with a bf16 scale for every 32 columns;
* ``keep_backward``  the layer's backward from those.

``run`` computes a case in elementary torch operations in fp32, rounded once at the end; with ``own`` set it makes the
calls of ``varlen_grouped_gemm_gb300``.  ``exact`` computes it in 64 bits.  Where an output has fewer bits than that
(bf16), ``exact`` gives the value before the rounding; of values kept in 8 bits one next to the border of two codes has two,
so it gives none.
"""
import math

import torch

own = False

BF, F32, I32, E4M3 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn
_ctx = None


def _lib():
    """The package and one context on the current device, made on first use."""
    global _ctx
    import varlen_grouped_gemm_gb300 as vgg
    if _ctx is None:
        _ctx = vgg.Context(torch.cuda.current_device())
    return vgg, _ctx


# ------------------------------------------------------------------------------------------------ cases


def _case(op, name, T, d, E, n, K, form="bf16", bias=False):
    return {"name": name, "op": op, "T": T, "d": d, "E": E, "n": n, "K": K, "form": form, "bias": bias}


def listed():
    return [
        # one token of a running generation: the default benchmark's layer, and the widest one on e4m3 weights
        _case("few", "few_token", 1, 2048, 128, 512, 8),
        _case("few", "few_token_e4m3", 1, 7168, 256, 2048, 8, "e4m3"),
        # three sequences in a small layer with a router bias: latency alone
        _case("few", "few_small", 3, 192, 8, 64, 2, bias=True),
        # decoding steps of a batch: many experts with one or two tokens each, and wide ones
        _case("few", "few_batch", 61, 1536, 512, 256, 8),
        _case("few", "few_batch_e4m3", 24, 2880, 128, 2880, 4, "e4m3", bias=True),
        _case("few", "few_wide", 8, 7168, 256, 2048, 8),
        # the experts' forward in a small ragged step, the default benchmark's (both forms) and the one with most tokens
        _case("keep", "keep_small", 213, 192, 8, 128, 2),
        _case("keep", "keep_step", 4096, 2048, 128, 512, 8),
        _case("keep", "keep_step_e4m3", 4096, 2048, 128, 512, 8, "e4m3"),
        _case("keep", "keep_large", 32768, 1536, 512, 256, 8),
        # the backward of the default benchmark's step, and of the one with most tokens
        _case("keep_backward", "keep_backward_step", 4096, 2048, 128, 512, 8),
        _case("keep_backward", "keep_backward_large", 32768, 1536, 512, 256, 8),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


_SMALL = ((128, 64), (192, 64), (192, 128), (256, 192), (512, 128), (320, 448))
_LAYERS = ((1536, 256), (2048, 512), (2880, 2880), (7168, 2048))


def draw(rng):
    op = rng.choice(["few", "few", "keep", "keep_backward"])
    E = 8 * _log_int(rng, 1, 64)
    K = min(E, rng.choice([1, 2, 4, 6, 8]))
    if op == "few":
        d, n = rng.choice(_SMALL + 2 * _LAYERS)
        E = max(K, 8, min(E, 256 * 7168 * 2048 // (d * n) // 8 * 8))
        T = max(1, min(_log_int(rng, 1, 64), 64 * 7168 * 2048 // (d * n * K)))
        return {"op": op, "T": T, "d": d, "E": E, "n": n, "K": K, "form": rng.choice(["bf16", "e4m3"]),
                "bias": rng.random() < 0.3}
    d, n = rng.choice(_SMALL + _LAYERS[:3])
    E = max(K, 8, min(E, 32768 * 1536 // (d * n) * 8))
    T = _log_int(rng, 1, max(2, min(32768, 32768 * 8 * 1536 * 256 // (K * d * n), 32768 * 8 * 1536 // (K * d))))
    return {"op": op, "T": T, "d": d, "E": E, "n": n, "K": K, "bias": False,
            "form": rng.choice(["bf16", "e4m3"]) if op == "keep" else "bf16"}


# ------------------------------------------------------------------------------------------------ inputs


def _normal(gen, *shape, std=1.0):
    """bf16 normal values, drawn in place: the widest layer's weights are 11 billion."""
    out = torch.empty(shape, dtype=BF, device="cuda")
    out.normal_(0.0, std, generator=gen)
    return out


def _ratio(v, c):
    """v / c as one fp32 division: of a number torch multiplies by the reciprocal, and bf16 quotients meet ties."""
    return torch.div(v, torch.full_like(v, c))


def _row_codes(W):
    """e4m3 codes and the scale of each row, as the framework's per-row form has them; by slices of the first axis."""
    q = torch.empty(W.shape, dtype=torch.uint8, device=W.device)
    s = torch.empty(W.shape[:-1], dtype=F32, device=W.device)
    for i in range(0, W.shape[0], 16):
        w = W[i:i + 16].float()
        top = w.abs().amax(-1)
        s[i:i + 16] = torch.where(top > 0, _ratio(top, 448.0), torch.ones_like(top))
        q[i:i + 16] = (w / s[i:i + 16, ..., None]).to(E4M3).view(torch.uint8)
    return q, s


def _kept(v):
    """8-bit codes and bf16 scales of 32 columns each: scale = max|v| / 127 rounded up to bf16 (at least 2^-126)."""
    b = v.unflatten(-1, (-1, 32))
    bits = _ratio(b.abs().amax(-1), 127.0).clamp(min=2.0 ** -126).view(I32)
    scale = ((bits + 0xFFFF) & ~0xFFFF).view(F32)
    q = torch.round(b * (1.0 / scale)[..., None]).to(torch.int8).flatten(-2)
    return q, scale.to(BF)


def _kept_values(q, scale):
    """What the codes stand for: code times scale, as bf16."""
    return (q.float().unflatten(-1, (-1, 32)) * scale.float()[..., None]).flatten(-2).to(BF)


def _routing(s, T, E, K, gen):
    """A choice of experts, some preferred, and the order that groups its pairs by expert, as moe_permute leaves it."""
    logits = torch.randn((T, E), device="cuda", generator=gen) + 0.5 * torch.randn(E, device="cuda", generator=gen)
    top = torch.topk(logits, K, dim=1)
    s["topk_ids"], s["topk_w"] = top.indices.to(I32), torch.softmax(top.values, 1)
    ids = top.indices.flatten()
    order = torch.argsort(ids, stable=True)
    counts = torch.bincount(ids, minlength=E)
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(I32)
    s["sorted_tok"] = (order // K).to(I32)
    s["sorted_w"] = s["topk_w"].flatten()[order].contiguous()
    place = torch.empty_like(order)
    place[order] = torch.arange(T * K, device="cuda")
    s["tok_ptr"] = torch.arange(0, T * K + 1, K, device="cuda", dtype=I32)
    s["tok_pairs"] = place.view(T, K).sort(1).values.flatten().to(I32)
    # the plain form's view: the pairs' places in [E, most pairs of an expert], and which expert each pair has
    s["most"] = int(counts.max())
    s["expert"] = ids[order]
    s["cell"] = s["expert"] * s["most"] + torch.arange(T * K, device="cuda") - s["offsets"].long()[s["expert"]]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, T, d, E, n, K = (case[k] for k in ("op", "T", "d", "E", "n", "K"))
    s = {"case": case}
    s["W_r"] = _normal(gen, d, E, std=d ** -0.5)
    s["X"] = _normal(gen, T, d)
    s["bias"] = 0.5 * torch.randn(E, device="cuda", generator=gen) if case["bias"] else None
    W = [_normal(gen, E, n, d, std=d ** -0.5), _normal(gen, E, n, d, std=d ** -0.5), _normal(gen, E, d, n, std=n ** -0.5)]
    if case["form"] == "e4m3":
        (s["Wg_q"], s["wg_s"]), (s["Wu_q"], s["wu_s"]), (s["Wd_q"], s["wd_s"]) = (_row_codes(w) for w in W)
    else:
        s["W_gate"], s["W_up"], s["W_down"] = W
    if op == "few":
        # logits closer to one another than 32 bits tell apart would leave the choice open: such a token is replaced
        logits = _exact_logits(s)
        top = torch.topk(logits, min(K + 1, E), dim=1).values
        gap = (top[:, :-1] - top[:, 1:]).amin(1) if E > 1 else torch.ones(T, device="cuda")
        s["X"] = torch.where((gap > 1e-4)[:, None], s["X"], s["X"][gap.argmax()])
        s["O"] = torch.empty((T, d), dtype=BF, device="cuda")
        s["topk_ids"] = torch.empty((T, K), dtype=I32, device="cuda")
        s["topk_w"] = torch.empty((T, K), device="cuda")
        return s
    _routing(s, T, E, K, gen)
    P, i8 = T * K, dict(dtype=torch.int8, device="cuda")
    if op == "keep":
        s["Hq"], s["Uq"], s["Xq"] = torch.empty((P, n), **i8), torch.empty((P, n), **i8), torch.empty((T, d), **i8)
        s["hs"], s["us"] = (torch.empty((P, n // 32), dtype=BF, device="cuda") for _ in range(2))
        s["xs"] = torch.empty((T, d // 32), dtype=BF, device="cuda")
        s["A"], s["Yw"] = torch.empty((P, n), dtype=BF, device="cuda"), torch.empty((P, d), dtype=BF, device="cuda")
        s["O"] = torch.empty((T, d), dtype=BF, device="cuda")
        s["values"] = [torch.empty(shape, dtype=BF, device="cuda") for shape in ((P, n), (P, n), (T, d))]
        return s
    s["dO"] = _normal(gen, T, d)
    (s["Xq"], s["xs"]) = _kept(s["X"].float())
    (s["Hq"], s["hs"]), (s["Uq"], s["us"]) = (_kept(torch.randn((P, n), device="cuda", generator=gen)) for _ in range(2))
    s["dX"] = torch.empty((T, d), dtype=BF, device="cuda")
    s["dW_gate"], s["dW_up"], s["dW_down"] = (torch.empty_like(w) for w in W)
    s["dS"] = torch.empty(P, device="cuda")
    s["dlogits"], s["dW_r"] = torch.empty((T, E), device="cuda"), torch.empty((d, E), device="cuda")
    return s


# ------------------------------------------------------------------------------------------------ one pass


def _plain_codes(v):
    """Per-row e4m3 values of fp32 rows, and their scales."""
    top = v.abs().amax(-1, keepdim=True)
    scale = torch.where(top > 0, _ratio(top, 448.0), torch.ones_like(top))
    return (v / scale).to(E4M3).float(), scale


def _plain_few(s):
    T, K = s["X"].shape[0], s["case"]["K"]
    X = s["X"].float()
    logits = X @ s["W_r"].float()
    if s["bias"] is not None:
        logits = logits + s["bias"]
    top = torch.topk(logits, K, dim=1)
    w = torch.softmax(top.values, 1)
    ids = top.indices.flatten()
    if s["case"]["form"] == "e4m3":
        xq, xs = _plain_codes(X)
        xq, xs = xq.repeat_interleave(K, 0)[:, :, None], xs.repeat_interleave(K, 0)
        h = torch.bmm(s["Wg_q"][ids].view(E4M3).float(), xq)[:, :, 0] * xs * s["wg_s"][ids]
        u = torch.bmm(s["Wu_q"][ids].view(E4M3).float(), xq)[:, :, 0] * xs * s["wu_s"][ids]
        aq, a_s = _plain_codes((h * torch.sigmoid(h) * u).to(BF).float())
        y = torch.bmm(s["Wd_q"][ids].view(E4M3).float(), aq[:, :, None])[:, :, 0] * a_s * s["wd_s"][ids]
    else:
        x = X.repeat_interleave(K, 0)[:, :, None]
        h = torch.bmm(s["W_gate"][ids].float(), x)[:, :, 0]
        u = torch.bmm(s["W_up"][ids].float(), x)[:, :, 0]
        y = torch.bmm(s["W_down"][ids].float(), (h * torch.sigmoid(h) * u)[:, :, None])[:, :, 0]
    O = (y.view(T, K, -1) * w[:, :, None]).sum(1)
    return {"O": O.to(BF), "topk_ids": top.indices.to(I32), "topk_w": w}


def _cells(s, rows):
    """Rows in sorted order spread over [E, most pairs of an expert, .], zeros elsewhere."""
    E, most = s["case"]["E"], s["most"]
    out = rows.new_zeros((E * most, rows.shape[1]))
    out[s["cell"]] = rows
    return out.view(E, most, -1)


def _plain_keep(s):
    T, K = s["case"]["T"], s["case"]["K"]
    tok, cell = s["sorted_tok"].long(), s["cell"]
    X = s["X"].float()
    if s["case"]["form"] == "e4m3":
        xq, xs = _plain_codes(X)
        rows = _cells(s, xq[tok])
        h = torch.bmm(rows, s["Wg_q"].view(E4M3).float().transpose(1, 2)).flatten(0, 1)[cell]
        u = torch.bmm(rows, s["Wu_q"].view(E4M3).float().transpose(1, 2)).flatten(0, 1)[cell]
        h, u = h * xs[tok] * s["wg_s"][s["expert"]], u * xs[tok] * s["wu_s"][s["expert"]]
        aq, a_s = _plain_codes((h * torch.sigmoid(h) * u).to(BF).float())
        y = torch.bmm(_cells(s, aq), s["Wd_q"].view(E4M3).float().transpose(1, 2)).flatten(0, 1)[cell]
        y = y * a_s * s["wd_s"][s["expert"]]
    else:
        rows = _cells(s, X[tok])
        h = torch.bmm(rows, s["W_gate"].float().transpose(1, 2)).flatten(0, 1)[cell]
        u = torch.bmm(rows, s["W_up"].float().transpose(1, 2)).flatten(0, 1)[cell]
        y = torch.bmm(_cells(s, h * torch.sigmoid(h) * u), s["W_down"].float().transpose(1, 2)).flatten(0, 1)[cell]
    O = (y * s["sorted_w"][:, None])[s["tok_pairs"].long()].view(T, K, -1).sum(1)
    return {"O": O.to(BF), "H": _kept_values(*_kept(h)), "U": _kept_values(*_kept(u)), "X": _kept_values(*_kept(X))}


def _plain_keep_backward(s):
    T, K, E = s["case"]["T"], s["case"]["K"], s["case"]["E"]
    tok, cell, pairs = s["sorted_tok"].long(), s["cell"], s["tok_pairs"].long()
    X, h, u = (_kept_values(s[q], s[c]).float() for q, c in (("Xq", "xs"), ("Hq", "hs"), ("Uq", "us")))
    w = s["sorted_w"][:, None]
    dO = _cells(s, s["dO"].float()[tok])
    dap = torch.bmm(dO, s["W_down"].float()).flatten(0, 1)[cell]
    sg = torch.sigmoid(h)
    a = h * sg * u
    dS = (dap * a).sum(1)
    da = w * dap
    dh, du = _cells(s, da * u * sg * (1.0 + h * (1.0 - sg))), _cells(s, da * h * sg)
    rows = _cells(s, X[tok])
    dXp = (torch.bmm(dh, s["W_gate"].float()) + torch.bmm(du, s["W_up"].float())).flatten(0, 1)[cell]
    part = (s["sorted_w"] * dS)
    g = part[pairs].view(T, K).sum(1)
    dlogits = torch.zeros((T, E), device=X.device)
    dlogits[tok, s["expert"]] = part
    dlogits.scatter_add_(1, s["topk_ids"].long(), -s["topk_w"] * g[:, None])
    dX = dXp[pairs].view(T, K, -1).sum(1) + dlogits @ s["W_r"].float().T
    return {"dX": dX.to(BF), "dW_gate": torch.bmm(dh.transpose(1, 2), rows).to(BF),
            "dW_up": torch.bmm(du.transpose(1, 2), rows).to(BF),
            "dW_down": torch.bmm(dO.transpose(1, 2), _cells(s, w * a)).to(BF), "dS": dS, "dlogits": dlogits,
            "dW_r": X.T @ dlogits}


_PLAIN = {"few": _plain_few, "keep": _plain_keep, "keep_backward": _plain_keep_backward}


def _kept_for(s, name, make):
    """A workspace or a plan that a program keeps from one call to the next."""
    if name not in s:
        s[name] = make()
    return s[name]


def _weights8(s):
    vgg, _ = _lib()
    return _kept_for(s, "w8", lambda: vgg.E4m3Weights(s["Wg_q"], s["wg_s"], s["Wu_q"], s["wu_s"], s["Wd_q"], s["wd_s"]))


def _own_few(s):
    vgg, ctx = _lib()
    T, d, E, n, K = (s["case"][k] for k in ("T", "d", "E", "n", "K"))
    ws = _kept_for(s, "ws", lambda: torch.empty(vgg.moe_few_workspace_bytes(T, d, E, n, K), dtype=torch.uint8, device="cuda"))
    if s["case"]["form"] == "e4m3":
        vgg.moe_forward_few_e4m3(ctx, s["X"], s["W_r"], s["bias"], _weights8(s), K, s["O"], s["topk_ids"], s["topk_w"], ws)
    else:
        vgg.moe_forward_few(ctx, s["X"], s["W_r"], s["bias"], s["W_gate"], s["W_up"], s["W_down"], K, s["O"], s["topk_ids"],
                            s["topk_w"], ws)
    return {"O": s["O"], "topk_ids": s["topk_ids"], "topk_w": s["topk_w"]}


def _own_keep(s):
    vgg, ctx = _lib()
    T, d, n, P = s["case"]["T"], s["case"]["d"], s["case"]["n"], s["sorted_tok"].numel()
    H, U = vgg.Kept8(s["Hq"], s["hs"]), vgg.Kept8(s["Uq"], s["us"])
    X = vgg.Kept8(s["Xq"], s["xs"])
    u8 = dict(dtype=torch.uint8, device="cuda")
    route = (s["offsets"], s["sorted_tok"], s["sorted_w"])
    vgg.moe_keep_rows8(ctx, s["X"], X)
    if s["case"]["form"] == "e4m3":
        w8 = _weights8(s)
        xq, x_s, aq, a_s = _kept_for(s, "codes", lambda: (torch.empty((T, d), **u8), torch.empty(T, device="cuda"),
                                                          torch.empty((P, n), **u8), torch.empty(P, device="cuda")))
        vgg.moe_quantize_rows_e4m3(ctx, s["X"], xq, x_s)
        vgg.moe_grouped_gemm_fwd_e4m3(ctx, xq, x_s, w8.Wg_q, w8.wg_scale, w8.Wu_q, w8.wu_scale, None, *route, H, U, s["A"],
                                      s["Yw"], Wd_q=w8.Wd_q, wd_scale=w8.wd_scale, Aq=aq, a_scale=a_s)
    else:
        ws = _kept_for(s, "ws", lambda: torch.empty(2 * P * n + 512, **u8))
        vgg.moe_grouped_gemm_fwd(ctx, s["X"], s["W_gate"], s["W_up"], s["W_down"], *route, H, U, s["A"], s["Yw"], ws)
    vgg.moe_combine(ctx, s["Yw"], s["tok_ptr"], s["tok_pairs"], s["O"])
    h, u, x = s["values"]
    vgg.moe_read_rows8(ctx, H, h)
    vgg.moe_read_rows8(ctx, U, u)
    vgg.moe_read_rows8(ctx, X, x)
    return {"O": s["O"], "H": h, "U": u, "X": x}


def _own_keep_backward(s):
    vgg, ctx = _lib()
    T, d, E, n, K = (s["case"][k] for k in ("T", "d", "E", "n", "K"))
    ws = _kept_for(s, "ws", lambda: torch.empty(vgg.moe_kept8_workspace_bytes(T, d, E, n, K), dtype=torch.uint8, device="cuda"))
    vgg.moe_backward(ctx, s["dO"], vgg.Kept8(s["Xq"], s["xs"]), s["W_r"], s["W_gate"], s["W_up"], s["W_down"], K, 0,
                     s["topk_ids"], s["topk_w"], s["offsets"], s["sorted_tok"], s["sorted_w"], s["tok_ptr"], s["tok_pairs"],
                     vgg.Kept8(s["Hq"], s["hs"]), vgg.Kept8(s["Uq"], s["us"]), s["dX"], s["dW_gate"], s["dW_up"],
                     s["dW_down"], s["dS"], s["dlogits"], s["dW_r"], ws)
    return {k: s[k] for k in ("dX", "dW_gate", "dW_up", "dW_down", "dS", "dlogits", "dW_r")}


_OWN = {"few": _own_few, "keep": _own_keep, "keep_backward": _own_keep_backward}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------------ work


def _experts(T, E, K):
    """Experts with a token where every choice is equally likely: what a pass has to read of the weights."""
    return E * (1.0 - (1.0 - K / E) ** T)


def work(case):
    op, T, d, E, n, K = (case[k] for k in ("op", "T", "d", "E", "n", "K"))
    P, wb = T * K, 1 if case["form"] == "e4m3" else 2
    used = _experts(T, E, K)
    weights = used * (3 * d * n * wb + (4 * (2 * n + d) if wb == 1 else 0))
    if op == "few":
        # the chosen experts, the router, X; O, the choices
        return {"bytes": int(weights + 2 * d * E + 4 * T * d + 8 * P), "flops": 6 * P * d * n + 2 * T * d * E}
    kept = (2 * P * n + T * d) * (1 + 1 / 16)
    if op == "keep":
        return {"bytes": int(weights + 4 * T * d + kept + 8 * P), "flops": 6 * P * d * n}
    # X, H, U, dO, the weights, the router's; dX, the weights' gradients, the logits' and the router's
    return {"bytes": int(kept + 4 * T * d + weights + 6 * E * d * n + 6 * d * E + 4 * T * E + 20 * P),
            "flops": 12 * P * d * n + 4 * T * d * E}


# ------------------------------------------------------------------------------------------------ 64 bits


def _exact_logits(s):
    logits = torch.einsum("td,de->te", s["X"].double(), s["W_r"].double())
    return logits if s["bias"] is None else logits + s["bias"].double()


def _exact_quantize(v):
    """The values of v's per-row codes: v holds bf16 values, and the rule divides in fp32."""
    v = v.float()
    top = torch.linalg.vector_norm(v, ord=float("inf"), dim=-1, keepdim=True)
    scale = torch.where(top > 0, _ratio(top, 448.0), torch.ones_like(top))
    return torch.div(v, scale).to(E4M3).double() * scale.double()


def _exact_weight(s, name, e):
    """Expert e's matrix; of e4m3 codes the values that they stand for."""
    q, c = {"W_gate": ("Wg_q", "wg_s"), "W_up": ("Wu_q", "wu_s"), "W_down": ("Wd_q", "wd_s")}[name]
    return s[name][e].double() if name in s else s[q][e].view(E4M3).double() * s[c][e].double()[:, None]


def _exact_expert(s, e, x):
    """Expert e's output for rows x, quantized as the form has it."""
    low = s["case"]["form"] == "e4m3"
    x = _exact_quantize(x) if low else x
    h, u = x @ _exact_weight(s, "W_gate", e).T, x @ _exact_weight(s, "W_up", e).T
    a = h / (1 + torch.exp(-h)) * u
    return (_exact_quantize(a.to(BF)) if low else a) @ _exact_weight(s, "W_down", e).T


def _exact_few(case, s):
    K = case["K"]
    top = torch.sort(_exact_logits(s), dim=1, descending=True)
    ids, w = top.indices[:, :K], torch.softmax(top.values[:, :K], 1)
    X, O = s["X"].double(), torch.zeros(s["X"].shape, dtype=torch.float64, device="cuda")
    for e in ids.unique().tolist():
        t, k = torch.nonzero(ids == e, as_tuple=True)
        O[t] += w[t, k, None] * _exact_expert(s, e, X[t])
    return {"O": O, "topk_ids": ids.to(I32), "topk_w": w}


def _exact_keep(case, s):
    X, cuts = s["X"].double(), s["offsets"].tolist()
    O = torch.zeros_like(X)
    for e in range(case["E"]):
        at = slice(cuts[e], cuts[e + 1])
        t = s["sorted_tok"][at].long()
        O[t] += s["sorted_w"][at].double()[:, None] * _exact_expert(s, e, X[t])
    return {"O": O, "H": None, "U": None, "X": None}


def _exact_keep_backward(case, s):
    E, K, cuts = case["E"], case["K"], s["offsets"].tolist()
    X, H, U = (_kept_values(s[q], s[c]).double() for q, c in (("Xq", "xs"), ("Hq", "hs"), ("Uq", "us")))
    dO, w = s["dO"].double(), s["sorted_w"].double()
    out = {"dX": torch.zeros_like(X), "dW_gate": torch.empty_like(s["W_gate"], dtype=torch.float64)}
    out["dW_up"], out["dW_down"] = torch.empty_like(out["dW_gate"]), torch.empty_like(s["W_down"], dtype=torch.float64)
    dS = torch.empty_like(w)
    for e in range(E):
        at = slice(cuts[e], cuts[e + 1])
        t = s["sorted_tok"][at].long()
        g, x, h, u = dO[t] @ s["W_down"][e].double(), X[t], H[at], U[at]
        f = 1 / (1 + torch.exp(-h))
        dS[at] = torch.einsum("pn,pn->p", g, h * f * u)
        wa = w[at, None]
        dh, du = wa * g * u * (f + h * f * (1 - f)), wa * g * h * f
        out["dX"][t] += dh @ s["W_gate"][e].double() + du @ s["W_up"][e].double()
        out["dW_gate"][e], out["dW_up"][e] = dh.T @ x, du.T @ x
        out["dW_down"][e] = dO[t].T @ (wa * h * f * u)
    # p = softmax over the chosen logits: d/dl_k = p_k (dS_k - sum_i p_i dS_i)
    p = torch.zeros((case["T"], E), dtype=torch.float64, device="cuda")
    p.scatter_(1, s["topk_ids"].long(), s["topk_w"].double())
    full = torch.zeros_like(p)
    full[s["sorted_tok"].long(), s["expert"]] = dS
    dl = p * (full - (p * full).sum(1, keepdim=True))
    out["dX"] += dl @ s["W_r"].double().T
    return {**out, "dS": dS, "dlogits": dl, "dW_r": X.T @ dl}


def exact(case, seed):
    return {"few": _exact_few, "keep": _exact_keep, "keep_backward": _exact_keep_backward}[case["op"]](
        case, prepare(case, seed))
