"""The operators around the expert layer: what is measured, and their plain forms.

Four operators belong to the training and serving of a pre-norm block whose feed-forward part is the expert layer:

* ``norm``             h = residual + x, y = rmsnorm(h) * weight in bf16, and y's e4m3 codes with their scales (one fp32
                       scale a row, or one power of two for 32 columns) in the layouts the FP8 forwards read;
* ``norm_backward``    the gradients of x, of the residual stream and of the weight;
* ``balance``          the router's balance and z losses over sequences of a packed batch, the per-expert counts, and
                       the gradient of the logits;
* ``router_backward``  dX += dlogits W_r^T and dW_r += X^T dlogits, which carry that gradient on to the layer's input and
                       to the router's weight.

``run`` computes a case in elementary torch operations in fp32, rounded once at the end; with ``own`` set it makes the
calls of ``varlen_grouped_gemm_gb300``.  ``exact`` computes it in 64 bits.  Where an output has fewer bits than that
(bf16, e4m3), ``exact`` gives the value before the rounding.
"""
import math

import torch

own = False

EPS = 1e-6
_ctx = None


def _lib():
    """The package and one context on the current device, made on first use."""
    global _ctx
    import varlen_grouped_gemm_gb300 as vgg
    if _ctx is None:
        _ctx = vgg.Context(torch.cuda.current_device())
    return vgg, _ctx


# ------------------------------------------------------------------------------------------------ cases


def _norm(name, T, d, out, res="bf16", pad=0):
    return {"name": name, "op": "norm", "T": T, "d": d, "out": out, "res": res, "pad": pad}


def _norm_backward(name, T, d, res="bf16", pad=0):
    return {"name": name, "op": "norm_backward", "T": T, "d": d, "res": res, "pad": pad}


def _balance(name, T, E, K, B=1, masked=False):
    return {"name": name, "op": "balance", "T": T, "E": E, "K": K, "B": B, "masked": masked}


def _router_backward(name, T, d, E):
    return {"name": name, "op": "router_backward", "T": T, "d": d, "E": E}


def listed():
    return [
        # one token of a running generation before the widest layer (d = 7168), codes for the per-row FP8 forward
        _norm("norm_token_e4m3", 1, 7168, "e4m3"),
        # a serving batch of 61 sequences, one token each, codes for the block-scaled forward
        _norm("norm_batch_mx", 61, 2048, "mx"),
        # a prompt's tokens in a buffer with longer rows (a slice of a fused projection's output), bf16 alone
        _norm("norm_prompt_ragged", 1337, 2880, "bf16", pad=40),
        # the widest layer's training step, per-row codes
        _norm("norm_step_e4m3", 8192, 7168, "e4m3"),
        # the step with the most tokens, an fp32 residual stream, block-scaled codes
        _norm("norm_step_mx_fp32", 32768, 1536, "mx", res="fp32"),
        # backward of the layer of the default benchmark, and of the widest one with an fp32 residual stream
        _norm_backward("norm_backward_step", 4096, 2048),
        _norm_backward("norm_backward_fp32", 8192, 7168, res="fp32"),
        # a small layer's router; the default benchmark's; the largest router on a packed batch with padding
        _balance("balance_small", 64, 8, 2),
        _balance("balance_step", 4096, 128, 8),
        _balance("balance_packed", 32768, 512, 8, B=37, masked=True),
        # the default benchmark's router and the largest one
        _router_backward("router_step", 4096, 2048, 128),
        _router_backward("router_large", 32768, 1536, 512),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, most=7168):
    """A width of this repository's workloads, or an odd multiple of 64."""
    own_widths = [d for d in (128, 192, 256, 512, 1536, 2048, 2880, 7168) if d <= most]
    return rng.choice(own_widths) if rng.random() < 0.5 else 64 * (2 * _log_int(rng, 1, max(1, min(55, most // 128 - 1))) + 1)


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_backward", "balance", "balance", "router_backward"])
    if op in ("norm", "norm_backward"):
        out = rng.choice(["bf16", "e4m3", "mx"]) if op == "norm" else "bf16"
        if out == "bf16" and rng.random() < 0.3:
            d = _log_int(rng, 33, 9000)  # any width, odd ones among them
            pad = rng.choice([0, 3, 8])
        else:
            d = _width(rng)
            pad = rng.choice([0, 0, 8, 64])
        T = _log_int(rng, 1, min(32768, 8192 * 7168 // d))
        c = {"op": op, "T": T, "d": d, "res": rng.choice(["bf16", "fp32"]), "pad": pad}
        if op == "norm":
            c["out"] = out
        return c
    E = 8 * _log_int(rng, 1, 64)
    T = _log_int(rng, 1, 32768)
    if op == "balance":
        K = rng.choice([1, 2, 4, 6, 8])
        return {"op": op, "T": T, "E": E, "K": K, "B": min(T, rng.choice([1, 1, _log_int(rng, 2, 64)])),
                "masked": rng.random() < 0.4}
    d = _width(rng, max(192, min(7168, 32768 * 1536 // T, 32768 * 1536 * 512 // (T * E))))
    return {"op": op, "T": T, "d": d, "E": E}


# ------------------------------------------------------------------------------------------------ inputs


def _rows(T, d, pad, dtype, gen=None, scale=1.0):
    """[T, d] with rows d + pad elements apart; N(0, scale) with a generator, else uninitialised."""
    buf = torch.empty((T, d + pad), dtype=dtype, device="cuda")
    if gen is not None:
        buf.copy_(torch.randn((T, d + pad), device="cuda", generator=gen) * scale)
    return buf[:, :d]


def _stream_rows(T, d, pad, dtype, gen):
    """A residual stream: a few channels carry values some twenty times the others'."""
    r = _rows(T, d, pad, dtype, gen, 2.0)
    big = torch.randint(0, d, (max(1, d // 500),), device="cuda", generator=gen)
    r[:, big] *= 20.0
    return r


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, T = case["op"], case["T"]
    dev, bf, f32, i32 = "cuda", torch.bfloat16, torch.float32, torch.int32
    s = {"case": case}
    if op in ("norm", "norm_backward"):
        d, pad = case["d"], case["pad"]
        rt = f32 if case["res"] == "fp32" else bf
        s["weight"] = (1.0 + 0.1 * torch.randn(d, device=dev, generator=gen)).to(f32 if case["res"] == "fp32" else bf)
        if op == "norm":
            s["x"] = _rows(T, d, pad, bf, gen, 0.7)
            s["residual"] = _stream_rows(T, d, pad, rt, gen)
            s["h"], s["y"] = _rows(T, d, pad, rt), _rows(T, d, 0, bf)
            s["rstd"] = torch.empty(T, device=dev)
            if case["out"] != "bf16":
                s["q"] = torch.empty((T, d), dtype=torch.uint8, device=dev)
                s["scales"] = torch.empty(T, device=dev) if case["out"] == "e4m3" else \
                    torch.empty((T, 4 * -(-d // 128)), dtype=torch.uint8, device=dev)
            return s
        s["dy"] = _rows(T, d, pad, bf, gen, 1.0)
        s["h"] = _stream_rows(T, d, pad, rt, gen)
        s["dh"] = _rows(T, d, pad, rt, gen, 1.0)
        s["rstd"] = torch.rsqrt((s["h"].float() ** 2).mean(1) + EPS)
        s["dx"], s["dweight"] = _rows(T, d, 0, bf), torch.empty(d, device=dev)
        s["dres"] = _rows(T, d, 0, f32) if rt == f32 else None
        return s
    E = case["E"]
    if op == "balance":
        K, B = min(case["K"], E), case["B"]
        # logits of unit variance with experts that the router prefers
        s["logits"] = torch.randn((T, E), device=dev, generator=gen) + 0.5 * torch.randn(E, device=dev, generator=gen)
        s["topk_ids"] = torch.topk(s["logits"], K, dim=1).indices.to(i32)
        s["K"], s["mask"], s["seq_offsets"] = K, None, None
        if B > 1:
            # lengths of a packed batch: B - 1 distinct cuts
            cuts = torch.randperm(T - 1, device=dev, generator=gen)[:B - 1].sort().values + 1
            s["seq_offsets"] = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), T)]).to(i32)
        if case["masked"]:
            s["mask"] = torch.rand(T, device=dev, generator=gen) >= 0.05
        s["balance_coef"], s["z_coef"] = 1e-2, 1e-3
        s["loss"] = torch.empty(3, device=dev)
        s["counts"] = torch.empty((B, E), dtype=i32, device=dev)
        s["probs"] = torch.empty((B, E), device=dev)
        s["dlogits"] = torch.empty((T, E), device=dev)
        return s
    d = case["d"]
    s["X"] = torch.randn((T, d), device=dev, generator=gen).to(bf)
    s["W_r"] = (torch.randn((d, E), device=dev, generator=gen) / d ** 0.5).to(bf)
    s["dlogits"] = torch.randn((T, E), device=dev, generator=gen) * 1e-3
    # what the layer's own backward left: gradients of about twice the size of those that are added
    s["dX_in"] = (torch.randn((T, d), device=dev, generator=gen) * (2e-3 * (E / d) ** 0.5)).to(bf)
    s["dW_r_in"] = torch.randn((d, E), device=dev, generator=gen) * (2e-3 * T ** 0.5)
    s["dX"], s["dW_r"] = torch.empty_like(s["dX_in"]), torch.empty_like(s["dW_r_in"])
    return s


# ------------------------------------------------------------------------------------------------ one pass


def _block_exponent(amax):
    """The smallest e with amax <= 448 2^e (0 for amax = 0)."""
    m, x = torch.frexp(amax / 448.0)
    e = torch.where(m == 0.5, x - 1, x)
    return torch.where(amax > 0, e, torch.zeros_like(e)).clamp(-126, 127)


def _plain_norm(s):
    case = s["case"]
    T, d = case["T"], case["d"]
    h = (s["residual"].float() + s["x"].float()).to(s["residual"].dtype)
    hf = h.float()
    rstd = 1.0 / torch.sqrt((hf * hf).mean(1) + EPS)
    y = hf * rstd[:, None] * s["weight"].float()
    out = {"h": h, "y": y.to(torch.bfloat16), "rstd": rstd}
    if case["out"] == "e4m3":
        amax = y.abs().amax(1)
        scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
        out["q"] = (y / scale[:, None]).to(torch.float8_e4m3fn)
        out["scales"] = scale
    elif case["out"] == "mx":
        blocks = y.view(T, d // 32, 32)
        e = _block_exponent(blocks.abs().amax(2))
        inv = ((127 - e) << 23).to(torch.int32).view(torch.float32)
        out["q"] = (blocks * inv[:, :, None]).view(T, d).to(torch.float8_e4m3fn)
        sf = torch.full((T, 4 * -(-d // 128)), 127, dtype=torch.uint8, device=y.device)
        sf[:, :d // 32] = (e + 127).to(torch.uint8)
        out["scales"] = sf.view(torch.float8_e8m0fnu)
    return out


def _plain_norm_backward(s):
    hf, dy, rstd = s["h"].float(), s["dy"].float(), s["rstd"][:, None]
    xhat = hf * rstd
    g = dy * s["weight"].float()
    dh = rstd * (g - xhat * (g * xhat).mean(1, keepdim=True)) + s["dh"].float()
    out = {"dx": dh.to(torch.bfloat16), "dweight": (dy * xhat).sum(0)}
    if s["dres"] is not None:
        out["dres"] = dh
    return out


def _plain_balance(s):
    logits, ids, K = s["logits"], s["topk_ids"], s["K"]
    T, E = logits.shape
    B = s["counts"].shape[0]
    off, mask = s["seq_offsets"], s["mask"]
    tok = torch.arange(T, device=logits.device)
    seq = (tok[:, None] >= off[None, 1:-1]).sum(1) if B > 1 else torch.zeros_like(tok)
    valid = torch.ones_like(tok) if mask is None else mask.to(tok.dtype)
    member = (torch.arange(B, device=logits.device)[:, None] == seq[None, :]).float() * valid.float()  # [B, T]
    m = logits.amax(1, keepdim=True)
    ex = torch.exp(logits - m)
    z = ex.sum(1, keepdim=True)
    p = ex / z
    lse = (m + torch.log(z))[:, 0]
    counts = torch.zeros(B * E, dtype=torch.int32, device=logits.device)
    counts.scatter_add_(0, (seq[:, None] * E + ids).view(-1), valid[:, None].expand(T, K).reshape(-1).to(torch.int32))
    counts = counts.view(B, E)
    n = member.sum(1)
    n1 = n.clamp(min=1.0)[:, None]
    used = (n > 0).sum().clamp(min=1).float()
    total = n.sum().clamp(min=1.0)
    probs = member @ p / n1
    f = counts.float() * E / (K * n1)
    balance = (f * probs).sum() / used
    zloss = (valid * lse * lse).sum() / total
    ca, cz = s["balance_coef"], s["z_coef"]
    c = (ca * f / (n1 * used))[seq]
    dl = p * (c - (p * c).sum(1, keepdim=True)) + (2.0 * cz / total) * lse[:, None] * p
    return {"loss": torch.stack([ca * balance + cz * zloss, balance, zloss]), "counts": counts, "probs": probs,
            "dlogits": dl * valid[:, None]}


def _plain_router_backward(s):
    dl, X, W = s["dlogits"], s["X"].float(), s["W_r"].float()
    return {"dX": (s["dX_in"].float() + dl @ W.T).to(torch.bfloat16), "dW_r": s["dW_r_in"] + X.T @ dl}


_PLAIN = {"norm": _plain_norm, "norm_backward": _plain_norm_backward, "balance": _plain_balance,
          "router_backward": _plain_router_backward}


def _own_norm(s):
    vgg, ctx = _lib()
    vgg.moe_add_rmsnorm(ctx, s["x"], s["residual"], s["weight"], EPS, s["h"], s["y"], s["rstd"], s.get("q"),
                        s.get("scales"))
    out = {"h": s["h"], "y": s["y"], "rstd": s["rstd"]}
    if "q" in s:
        out["q"] = s["q"].view(torch.float8_e4m3fn)
        sc = s["scales"]
        out["scales"] = sc if sc.dtype == torch.float32 else sc.view(torch.float8_e8m0fnu)
    return out


def _workspace(s, nbytes):
    if "ws" not in s:
        s["ws"] = torch.empty(nbytes(), dtype=torch.uint8, device="cuda")
    return s["ws"]


def _own_norm_backward(s):
    vgg, ctx = _lib()
    T, d = s["dy"].shape
    ws = _workspace(s, lambda: vgg.moe_add_rmsnorm_workspace_bytes(T, d))
    vgg.moe_add_rmsnorm_backward(ctx, s["dy"], s["h"], s["weight"], s["rstd"], s["dh"], s["dx"], s["dres"],
                                 s["dweight"], ws)
    out = {"dx": s["dx"], "dweight": s["dweight"]}
    if s["dres"] is not None:
        out["dres"] = s["dres"]
    return out


def _own_balance(s):
    vgg, ctx = _lib()
    T, E = s["logits"].shape
    ws = _workspace(s, lambda: vgg.moe_balance_loss_workspace_bytes(T, E, s["counts"].shape[0]))
    vgg.moe_balance_loss(ctx, s["logits"], s["topk_ids"], s["balance_coef"], s["z_coef"], s["loss"], s["counts"],
                         s["probs"], s["dlogits"], ws, mask=s["mask"], seq_offsets=s["seq_offsets"])
    return {"loss": s["loss"], "counts": s["counts"], "probs": s["probs"], "dlogits": s["dlogits"]}


def _own_router_backward(s):
    vgg, ctx = _lib()
    T, d = s["X"].shape
    ws = _workspace(s, lambda: vgg.moe_router_backward_workspace_bytes(T, d, s["W_r"].shape[1]))
    vgg.moe_router_backward(ctx, s["dlogits"], s["X"], s["W_r"], s["dX_in"], s["dW_r_in"], s["dX"], s["dW_r"], ws)
    return {"dX": s["dX"], "dW_r": s["dW_r"]}


_OWN = {"norm": _own_norm, "norm_backward": _own_norm_backward, "balance": _own_balance,
        "router_backward": _own_router_backward}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------------ work


def work(case):
    op, T = case["op"], case["T"]
    if op in ("norm", "norm_backward"):
        d = case["d"]
        r = 4 if case["res"] == "fp32" else 2
        if op == "norm":
            # x, residual; h, y, rstd; codes and scales; the weight
            b = T * d * (2 + r + r + 2) + 4 * T + d * r
            b += {"bf16": 0, "e4m3": T * d + 4 * T, "mx": T * d + T * 4 * -(-d // 128)}[case["out"]]
            return {"bytes": b, "flops": 6 * T * d}
        # dy, h, dh, rstd, weight; dx, dweight and, with an fp32 stream, its gradient
        return {"bytes": T * d * (2 + r + r + 2 + (4 if r == 4 else 0)) + 4 * T + d * r + 4 * d, "flops": 12 * T * d}
    E = case["E"]
    if op == "balance":
        K, B = min(case["K"], E), case["B"]
        # logits and choices in; the logits' gradient, counts and mean probabilities out
        return {"bytes": 8 * T * E + 4 * T * K + (T if case["masked"] else 0) + 8 * B * E, "flops": 12 * T * E}
    d = case["d"]
    return {"bytes": 4 * T * E + 2 * T * d + 2 * d * E + 4 * T * d + 8 * d * E, "flops": 4 * T * d * E}


# ------------------------------------------------------------------------------------------------ 64 bits


def _exact_norm(case, s):
    T, d = case["T"], case["d"]
    # the stream holds the sum rounded to its type: that value is the norm's input
    h = torch.add(s["residual"].float(), s["x"].float()).to(s["residual"].dtype).double()
    r = torch.rsqrt(h.square().sum(1) / d + EPS)
    y = torch.einsum("td,t,d->td", h, r, s["weight"].double())
    out = {"h": s["residual"].double() + s["x"].double(), "y": y, "rstd": r}
    if case["out"] == "e4m3":
        top = torch.linalg.vector_norm(y, ord=float("inf"), dim=1)
        out["scales"] = torch.where(top > 0, top / 448, torch.ones_like(top))
        out["q"] = y / out["scales"][:, None]
    elif case["out"] == "mx":
        top = torch.linalg.vector_norm(y.unflatten(1, (-1, 32)), ord=float("inf"), dim=2)
        e = torch.ceil(torch.log2(torch.clamp(top, min=1e-300) / 448)) * (top > 0)
        out["q"] = (y.unflatten(1, (-1, 32)) * torch.exp2(-e)[:, :, None]).flatten(1)
        out["scales"] = None  # whole powers of two: a block next to a border has two
    return out


def _exact_norm_backward(case, s):
    d = case["d"]
    h, dy, w, r = s["h"].double(), s["dy"].double(), s["weight"].double(), s["rstd"].double()
    g = dy * w
    dot = torch.einsum("td,td->t", g, h)
    dh = s["dh"].double() + r[:, None] * g - (r ** 3 * dot / d)[:, None] * h
    out = {"dx": dh, "dweight": torch.einsum("td,td,t->d", dy, h, r)}
    if s["dres"] is not None:
        out["dres"] = dh
    return out


def _exact_balance(case, s):
    logits = s["logits"].double()
    T, E = logits.shape
    K, B = s["K"], case["B"]
    cuts = [0, T] if s["seq_offsets"] is None else s["seq_offsets"].tolist()
    keep = torch.ones(T, dtype=torch.bool, device=logits.device) if s["mask"] is None else s["mask"]
    p, lse = torch.softmax(logits, 1), torch.logsumexp(logits, 1)
    counts = torch.zeros((B, E), dtype=torch.int32, device=logits.device)
    probs = torch.zeros((B, E), dtype=torch.float64, device=logits.device)
    grad = torch.zeros_like(logits)
    per = []
    for b in range(B):
        rows = cuts[b] + torch.nonzero(keep[cuts[b]:cuts[b + 1]])[:, 0]
        if not len(rows):
            continue
        counts[b] = torch.bincount(s["topk_ids"][rows].flatten().long(), minlength=E).int()
        probs[b] = p[rows].mean(0)
        f = counts[b].double() * (E / (K * len(rows)))
        per.append((f * probs[b]).sum())
        grad[rows] = (p[rows] * f - p[rows] * (p[rows] @ f)[:, None]) / len(rows)
    n, used = max(1, int(keep.sum())), max(1, len(per))
    balance = sum(per) / used if per else probs.sum()
    z = lse[keep].square().sum() / n
    grad = s["balance_coef"] / used * grad + (2 * s["z_coef"] / n) * (lse * keep)[:, None] * p
    return {"loss": torch.stack([s["balance_coef"] * balance + s["z_coef"] * z, balance, z]), "counts": counts,
            "probs": probs, "dlogits": grad}


def _exact_router_backward(case, s):
    dl = s["dlogits"].double()
    return {"dX": torch.addmm(s["dX_in"].double(), dl, s["W_r"].double().T),
            "dW_r": torch.addmm(s["dW_r_in"].double(), s["X"].double().T, dl)}


def exact(case, seed):
    return {"norm": _exact_norm, "norm_backward": _exact_norm_backward, "balance": _exact_balance,
            "router_backward": _exact_router_backward}[case["op"]](case, prepare(case, seed))
