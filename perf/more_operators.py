"""More operators around the MoE layer as measured cases: the router's balance
and z losses with their gradients, the residual step between two blocks (norm
after a block, gate, scaled residual, norm before the next), and the matrix
product with bias, activation and residual in its epilogue.

``run`` computes an operator in its plain form (elementary torch operations
in 32 bits, rounded once at the end), or, where ``own`` is true, through the
framework's entry points (``dropless_grouped_gemm_router_amd.block``).
``exact`` gives the same outputs from the definitions in 64 bits.

Sizes: tokens, widths and expert counts of the layer's own workloads
(d_model 512, 8 or 64 experts, top 2 to 8, 4096 to 131072 tokens), and generic
wider ones (1024 to 8192) with odd neighbours.
"""

import math

import torch

own = False

EPS = 1e-5
BALANCE, ZED = 0.01, 0.001  # coefficients of the two losses
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------- cases

def balance(name, tokens, experts, top_k, d_model, dtype, masked, train):
    return {"name": name, "op": "balance", "tokens": tokens, "experts": experts, "top_k": top_k,
            "d_model": d_model, "dtype": dtype, "masked": masked, "train": train}


def residual(name, rows, width, dtype, kind, scale, post, gate, bias, train):
    return {"name": name, "op": "residual", "rows": rows, "width": width, "dtype": dtype, "kind": kind,
            "scale": scale, "post": post, "gate": gate, "bias": bias, "train": train}


def linear(name, tokens, inputs, outputs, dtype, act, bias, add, train):
    return {"name": name, "op": "linear", "tokens": tokens, "inputs": inputs, "outputs": outputs,
            "dtype": dtype, "act": act, "bias": bias, "add": add, "train": train}


def listed():
    return [
        # the expert loads of a small padded batch, watched while it is answered
        balance("balance, 200 tokens", 200, 8, 2, 512, "bf16", True, False),
        # the same over the layer's largest forward batch
        balance("balance, 131072 tokens", 131072, 64, 8, 512, "bf16", False, False),
        # the loss and its gradients at the layer's training batch
        balance("balance train, 16384 tokens", 16384, 64, 8, 512, "bf16", False, True),
        # 32-bit training on a ragged, padded batch and an odd number of experts
        balance("balance train, odd fp32", 4999, 33, 3, 1152, "fp32", True, True),
        # between two blocks while a few sequences are being answered
        residual("residual, 16 tokens", 16, 512, "bf16", "layer", 1.0, True, True, True, False),
        # between two blocks over the layer's largest forward batch
        residual("residual, 131072 tokens", 131072, 512, "bf16", "rms", 1.0, True, True, False, False),
        # forward and backward over the layer's training batch
        residual("residual train, 16384 tokens", 16384, 512, "bf16", "layer", 0.9, True, True, True, True),
        # a ragged batch at a width that no vector load divides, 32-bit training
        residual("residual train, odd fp32", 5001, 1155, "fp32", "rms", 1.0, True, True, False, True),
        # a projection back into the residual stream for one token: the weights' bytes count
        linear("linear, one token", 1, 4096, 4096, "bf16", "none", True, True, False),
        # a chunk of prompt of ragged length
        linear("linear, 300 tokens", 300, 1024, 4096, "bf16", "gelu_tanh", True, False, False),
        # training step of a projection at the layer's training batch
        linear("linear train, 16384 tokens", 16384, 512, 2048, "bf16", "silu", True, True, True),
        # 32-bit training at widths that no tile divides
        linear("linear train, odd fp32", 777, 500, 1001, "fp32", "gelu", True, True, True),
    ]


def between(rng, low, high):
    """A whole number from low to high, evenly over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def width(rng, low, high):
    """A width: half of them any number, half a multiple of 128."""
    n = between(rng, low, high)
    return n if rng.random() < 0.5 else max(128, n // 128 * 128)


def flip(rng):
    return rng.random() < 0.5


def draw(rng):
    dtype = rng.choice(("bf16", "bf16", "fp32"))
    op = rng.choice(("balance", "residual", "linear"))
    if op == "balance":
        d, e = 128 * between(rng, 1, 32), rng.choice((2, 5, 8, 16, 24, 33, 47, 64))
        limit = 2 ** 26 // d // (1 if dtype == "bf16" else 2)
        case = balance("", between(rng, 1, limit), e, rng.randint(1, min(8, e)), d, dtype, flip(rng), flip(rng))
    elif op == "residual":
        w = width(rng, 65, 8192)
        case = residual("", between(rng, 1, min(131072, 2 ** 25 // w)), w, dtype, rng.choice(("layer", "rms")),
                        rng.choice((1.0, 0.5, 1.25)), rng.random() < 0.75, flip(rng), flip(rng), flip(rng))
    else:
        k, n, train = width(rng, 65, 8192), width(rng, 65, 8192), flip(rng)
        limit = 2 ** (34 if train else 35) // (k * n) // (1 if dtype == "bf16" else 8)
        case = linear("", between(rng, 1, max(1, min(131072, limit))), k, n, dtype,
                      rng.choice(("none", "none", "silu", "gelu", "gelu_tanh", "relu")), flip(rng), flip(rng), train)
    return {k: v for k, v in case.items() if k != "name"}


def work(case):
    s = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "balance":
        t, e, k, d = (case[n] for n in ("tokens", "experts", "top_k", "d_model"))
        once = s * t * d
        # x, the router, the kept experts and the mask; with the backward pass also dx and the router's gradient
        return {"bytes": (2 if case["train"] else 1) * (once + 4 * d * e) + 4 * t * k + t * case["masked"],
                "flops": (6 if case["train"] else 2) * t * e * d}
    if case["op"] == "residual":
        n, d = case["rows"], case["width"]
        # forward: block output, residual, sum, norm; with the backward pass two gradients in, two out
        return {"bytes": (8 if case["train"] else 4) * s * n * d + (16 if case["train"] else 8) * d,
                "flops": (50 if case["train"] else 20) * n * d}
    t, k, n = case["tokens"], case["inputs"], case["outputs"]
    io = s * (t * k + k * n + (2 if case["add"] else 1) * t * n)
    if not case["train"]:
        return {"bytes": io, "flops": 2 * t * k * n}
    return {"bytes": io + s * (t * n + t * k + k * n), "flops": 6 * t * k * n}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dtype = TYPES[case["dtype"]]

    def normal(*shape, std=1.0, to=dtype):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(to)

    def numbers(*shape, std=1.0):
        return normal(*shape, std=std, to=torch.float32)

    state = {"case": case}
    if case["op"] == "balance":
        t, e, k, d = (case[n] for n in ("tokens", "experts", "top_k", "d_model"))
        state["x"] = normal(t, d)
        # a router that has come to prefer some experts
        state["w_router"] = numbers(d, e, std=d ** -0.5) * torch.exp(0.3 * numbers(e))
        logits = state["x"].float() @ state["w_router"]
        state["topk_idx"] = torch.topk(logits, k, dim=1).indices.to(torch.int32)
        state["mask"] = None
        if case["masked"]:
            # an eighth of the tokens is padding
            state["mask"] = torch.rand(t, generator=g, device="cuda") > 0.125
        if case["train"]:
            state["grad_loss"] = 1.0 + 0.1 * numbers(1)
    elif case["op"] == "residual":
        n, d = case["rows"], case["width"]
        # a residual stream: channels of unlike size around a small offset, a few of them large
        size = torch.exp(numbers(d, std=0.5))
        size = torch.where(numbers(d) > 2.0, 8.0 * size, size)
        state["res"] = (numbers(n, d) * size + numbers(d, std=0.5)).to(dtype)
        state["z"] = (numbers(n, d) * torch.exp(numbers(d, std=0.3)) + numbers(d, std=0.2)).to(dtype)
        state["pre_weight"] = 1.0 + numbers(d, std=0.2)
        state["post_weight"] = 1.0 + numbers(d, std=0.2) if case["post"] else None
        state["gate"] = 0.5 + numbers(d, std=0.2) if case["gate"] else None
        state["pre_bias"] = numbers(d, std=0.2) if case["bias"] else None
        state["post_bias"] = numbers(d, std=0.2) if case["bias"] and case["post"] else None
        if case["train"]:
            state["grad_out"] = normal(n, d)
            state["grad_y"] = normal(n, d)
    else:
        t, k, n = case["tokens"], case["inputs"], case["outputs"]
        state["x"] = normal(t, k)
        state["w"] = normal(k, n, std=k ** -0.5)
        state["bias"] = numbers(n, std=0.3) if case["bias"] else None
        state["add"] = normal(t, n) if case["add"] else None
        if case["train"]:
            state["grad"] = normal(t, n)
    return state


# ------------------------------------------------------------- plain forms

def plain_balance(s):
    case, x, w = s["case"], s["x"].float(), s["w_router"]
    e, k = case["experts"], case["top_k"]
    keep = torch.ones(case["tokens"], device=x.device) if s["mask"] is None else s["mask"].float()
    kept = torch.clamp(keep.sum(), min=1.0)
    logits = x @ w
    top = logits.amax(1, keepdim=True)
    ex = torch.exp(logits - top)
    total = ex.sum(1, keepdim=True)
    p, lse = ex / total, (top + torch.log(total))[:, 0]
    experts = torch.arange(e, device=x.device)
    chosen = (s["topk_idx"][:, :, None] == experts).sum(1).float()
    counts = (chosen * keep[:, None]).sum(0)
    share = counts / (kept * k)
    mean_prob = (p * keep[:, None]).sum(0) / kept
    even = e * (share * mean_prob).sum()
    zed = (lse * lse * keep).sum() / kept
    out = {"loss": torch.stack((BALANCE * even + ZED * zed, even, zed)), "mean_prob": mean_prob,
           "counts": counts.to(torch.int32)}
    if case["train"]:
        inner = (p * share).sum(1, keepdim=True)
        dl = p * (BALANCE * e * (share - inner) + 2.0 * ZED * lse[:, None]) * (keep[:, None] / kept) * s["grad_loss"]
        out.update(dx=(dl @ w.t()).to(s["x"].dtype), dw_router=x.t() @ dl)
    return out


def plain_statistics(x, kind):
    """Mean (0 for rms) and 1 / deviation of the rows."""
    mean = x.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(x[:, :1])
    return mean, torch.rsqrt(((x - mean) ** 2).mean(1, keepdim=True) + EPS)


def plain_norm_backward(xh, rstd, g, kind):
    back = g - xh * (g * xh).mean(1, keepdim=True)
    if kind == "layer":
        back = back - g.mean(1, keepdim=True)
    return rstd * back


def plain_residual(s):
    case, kind, to = s["case"], s["case"]["kind"], s["z"].dtype
    z, res = s["z"].float(), s["res"].float()
    u = z
    if case["post"]:
        mean, rstd = plain_statistics(z, kind)
        zh = (z - mean) * rstd
        u = zh * s["post_weight"]
        if s["post_bias"] is not None:
            u = u + s["post_bias"]
    gated = u if s["gate"] is None else u * s["gate"]
    o = case["scale"] * res + gated
    omean, orstd = plain_statistics(o, kind)
    oh = (o - omean) * orstd
    y = oh * s["pre_weight"]
    if s["pre_bias"] is not None:
        y = y + s["pre_bias"]
    out = {"out": o.to(to), "y": y.to(to)}
    if case["train"]:
        dy = s["grad_y"].float()
        do = s["grad_out"].float() + plain_norm_backward(oh, orstd, dy * s["pre_weight"], kind)
        du = do if s["gate"] is None else do * s["gate"]
        dz = du
        out["dpre_weight"] = (dy * oh).sum(0)
        if s["pre_bias"] is not None:
            out["dpre_bias"] = dy.sum(0)
        if s["gate"] is not None:
            out["dgate"] = (do * u).sum(0)
        if case["post"]:
            dz = plain_norm_backward(zh, rstd, du * s["post_weight"], kind)
            out["dpost_weight"] = (du * zh).sum(0)
            if s["post_bias"] is not None:
                out["dpost_bias"] = du.sum(0)
        out.update(dz=dz.to(to), dres=(case["scale"] * do).to(to))
    return out


def plain_act(a, act, slope):
    """act(a) and, where asked for, its derivative."""
    if act == "none":
        return a, torch.ones_like(a) if slope else None
    if act == "silu":
        sig = torch.sigmoid(a)
        return a * sig, sig * (1 + a * (1 - sig)) if slope else None
    if act == "relu":
        on = (a > 0).to(a.dtype)
        return a * on, on
    if act == "gelu":
        cdf = 0.5 * (1 + torch.erf(a * math.sqrt(0.5)))
        return a * cdf, cdf + a * torch.exp(-0.5 * a * a) / math.sqrt(2 * math.pi) if slope else None
    k, c = math.sqrt(2 / math.pi), 0.044715
    t = torch.tanh(k * (a + c * a * a * a))
    return 0.5 * a * (1 + t), (0.5 * (1 + t) + 0.5 * a * (1 - t * t) * k * (1 + 3 * c * a * a)) if slope else None


def plain_linear(s):
    x, w, to = s["x"].float(), s["w"].float(), s["x"].dtype
    a = x @ w
    if s["bias"] is not None:
        a = a + s["bias"]
    f, slope = plain_act(a, s["case"]["act"], "grad" in s)
    y = f if s["add"] is None else f + s["add"].float()
    out = {"y": y.to(to)}
    if "grad" in s:
        da = s["grad"].float() * slope
        out.update(dx=(da @ w.t()).to(to), dw=(x.t() @ da).to(to))
        if s["bias"] is not None:
            out["dbias"] = da.sum(0)
    return out


# ----------------------------------------------------------- the framework

def own_balance(s):
    from dropless_grouped_gemm_router_amd import block
    case = s["case"]
    if "buf" not in s:
        s["b"] = block.BalanceLoss(case["tokens"], case["experts"], case["top_k"], case["d_model"], case["dtype"],
                                   balance=BALANCE, z=ZED)
        s["buf"] = block.allocate_balance_loss(s["b"], "cuda", training=case["train"])
    buf = s["buf"]
    out = {"loss": block.balance_loss(s["b"], s["x"], s["w_router"], s["topk_idx"], buf, mask=s["mask"],
                                      training=case["train"]),
           "mean_prob": buf.mean_prob, "counts": buf.counts}
    if case["train"]:
        out["dx"], out["dw_router"] = block.balance_loss_backward(s["b"], s["x"], s["w_router"], buf,
                                                                  grad_loss=s["grad_loss"], mask=s["mask"])
    return out


PARAMS = ("post_weight", "post_bias", "gate", "pre_weight", "pre_bias")


def own_residual(s):
    from dropless_grouped_gemm_router_amd import block
    case = s["case"]
    if "buf" not in s:
        s["n"] = block.ResidualNorm(case["rows"], case["width"], case["dtype"], kind=case["kind"], eps=EPS,
                                    scale=case["scale"], post=case["post"])
        s["buf"] = block.allocate_residual_norm(s["n"], "cuda", training=case["train"])
    out = dict(zip(("out", "y"), block.residual_norm(s["n"], s["z"], s["res"], s, s["buf"])))
    if case["train"]:
        dz, dres, grads = block.residual_norm_backward(s["n"], s["z"], s["res"], s, s["grad_out"], s["grad_y"],
                                                       s["buf"])
        out.update({"d" + n: grads[n] for n in PARAMS if s[n] is not None}, dz=dz, dres=dres)
    return out


def own_linear(s):
    from dropless_grouped_gemm_router_amd import block
    case = s["case"]
    if "buf" not in s:
        s["l"] = block.Linear(case["tokens"], case["inputs"], case["outputs"], case["dtype"], act=case["act"],
                              grad_dtype=case["dtype"])
        s["buf"] = block.allocate_linear(s["l"], "cuda", training=case["train"])
    out = {"y": block.linear(s["l"], s["x"], s["w"], s["buf"], bias=s["bias"], residual=s["add"],
                             training=case["train"])}
    if case["train"]:
        dx, dw, dbias = block.linear_backward(s["l"], s["x"], s["w"], s["grad"], s["buf"], bias=case["bias"])
        out.update(dx=dx, dw=dw)
        if case["bias"]:
            out["dbias"] = dbias
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return {"balance": own_balance, "residual": own_residual, "linear": own_linear}[op](state)
    return {"balance": plain_balance, "residual": plain_residual, "linear": plain_linear}[op](state)


# ------------------------------------------------------- 64-bit definitions

def exact(case, seed):
    s = prepare(case, seed)
    with torch.enable_grad():
        if case["op"] == "balance":
            return exact_balance(s)
        return exact_residual(s) if case["op"] == "residual" else exact_linear(s)


def leaf(t):
    return None if t is None else t.double().requires_grad_()


def exact_balance(s):
    case = s["case"]
    rows = torch.arange(case["tokens"], device="cuda") if s["mask"] is None else torch.nonzero(s["mask"])[:, 0]
    x, w = leaf(s["x"]), leaf(s["w_router"])
    counts = torch.bincount(s["topk_idx"][rows].reshape(-1).long(), minlength=case["experts"])
    n = max(rows.numel(), 1)
    logits = x[rows] @ w
    mean_prob = torch.softmax(logits, 1).sum(0) / n
    even = case["experts"] * (counts.double() / (n * case["top_k"]) * mean_prob).sum()
    zed = torch.logsumexp(logits, 1).square().sum() / n
    loss = BALANCE * even + ZED * zed
    out = {"loss": torch.stack((loss, even, zed)).detach(), "mean_prob": mean_prob.detach(),
           "counts": counts.to(torch.int32)}
    if case["train"]:
        out["dx"], out["dw_router"] = torch.autograd.grad(loss, (x, w), s["grad_loss"].double()[0])
    return out


def exact_norm(x, kind, weight, bias):
    if kind == "layer":
        x = x - x.mean(1, keepdim=True)
    x = x / torch.sqrt(x.square().mean(1, keepdim=True) + EPS) * weight
    return x if bias is None else x + bias


def exact_residual(s):
    case = s["case"]
    z, res = leaf(s["z"]), leaf(s["res"])
    p = {n: leaf(s[n]) for n in PARAMS}
    u = exact_norm(z, case["kind"], p["post_weight"], p["post_bias"]) if case["post"] else z
    o = case["scale"] * res + (u if p["gate"] is None else p["gate"] * u)
    y = exact_norm(o, case["kind"], p["pre_weight"], p["pre_bias"])
    out = {"out": o.detach(), "y": y.detach()}
    if case["train"]:
        names = [n for n in PARAMS if p[n] is not None]
        loss = (o * s["grad_out"].double()).sum() + (y * s["grad_y"].double()).sum()
        got = torch.autograd.grad(loss, [z, res] + [p[n] for n in names])
        out.update(zip(["dz", "dres"] + ["d" + n for n in names], got))
    return out


def exact_linear(s):
    x, w, bias = leaf(s["x"]), leaf(s["w"]), leaf(s["bias"])
    act, a = s["case"]["act"], x @ w
    if bias is not None:
        a = a + bias
    if act == "silu":
        a = a / (1 + torch.exp(-a))
    elif act == "relu":
        a = torch.clamp(a, min=0)
    elif act == "gelu":
        a = a * torch.special.ndtr(a)
    elif act == "gelu_tanh":
        a = a / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3)))
    y = a if s["add"] is None else a + s["add"].double()
    out = {"y": y.detach()}
    if "grad" in s:
        leaves = [x, w] if bias is None else [x, w, bias]
        out.update(zip(("dx", "dw", "dbias"), torch.autograd.grad(y, leaves, s["grad"].double())))
    return out
