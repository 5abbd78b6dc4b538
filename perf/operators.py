"""The operators around the MoE layer as measured cases: layer norm, the dense
gated feed-forward block, and the 8-bit integer product of dense and routed
weights.

``run`` computes an operator in its plain form (elementary torch operations
in 32 bits, rounded once at the end), or, where ``own`` is true, through the
framework's entry points (``dropless_grouped_gemm_router_amd.block``).
``exact`` gives the same outputs from the definitions in 64 bits.

Sizes: tokens, widths and expert counts of the layer's own workloads
(d_model 512, hidden 128 to 1024, 8 or 64 experts, 4096 to 131072 tokens),
and generic wider ones (2048, 4096, 8192) with odd neighbours.
"""

import math

import torch

own = False

EPS = 1e-5
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------- cases

def norm(name, rows, width, dtype, train):
    return {"name": name, "op": "norm", "rows": rows, "width": width, "dtype": dtype, "train": train}


def ffn(name, tokens, d_model, d_hidden, dtype, act, train):
    return {"name": name, "op": "ffn", "tokens": tokens, "d_model": d_model, "d_hidden": d_hidden,
            "dtype": dtype, "act": act, "train": train}


def int8(name, tokens, inputs, outputs, dtype, experts=1, top_k=1, gated=False, bias=False):
    return {"name": name, "op": "int8", "tokens": tokens, "inputs": inputs, "outputs": outputs,
            "dtype": dtype, "experts": experts, "top_k": top_k, "gated": gated, "bias": bias}


def listed():
    return [
        # the norm in front of the layer while a few sequences are being answered
        norm("norm, 16 tokens", 16, 512, "bf16", False),
        # the same norm over the layer's largest forward batch
        norm("norm, 131072 tokens", 131072, 512, "bf16", False),
        # forward and backward over the layer's training batch
        norm("norm train, 16384 tokens", 16384, 512, "bf16", True),
        # a ragged batch at a width that no vector load divides, 32-bit training
        norm("norm train, odd fp32", 5001, 1155, "fp32", True),
        # a dense block answering one token: the weights' bytes count
        ffn("ffn, one token", 1, 2048, 8192, "bf16", "silu", False),
        # a chunk of prompt of ragged length
        ffn("ffn, 300 tokens", 300, 1024, 4096, "bf16", "gelu_tanh", False),
        # training step of the dense block at the layer's training batch
        ffn("ffn train, 16384 tokens", 16384, 512, 1024, "bf16", "silu", True),
        # 32-bit training at widths that no tile divides
        ffn("ffn train, odd fp32", 777, 500, 1001, "fp32", "gelu", True),
        # a projection for a handful of sequences being answered
        int8("int8, 4 tokens", 4, 4096, 4096, "bf16"),
        # the same projection over a long prompt batch
        int8("int8, 16384 tokens", 16384, 4096, 4096, "bf16"),
        # the gate and up product of routed experts at a measured workload of the layer
        int8("int8 experts, 32768 tokens", 32768, 512, 512, "bf16", experts=64, top_k=4, gated=True),
        # ragged everything, 32-bit output with a bias
        int8("int8, odd fp32", 999, 1111, 2049, "fp32", bias=True),
    ]


def between(rng, low, high):
    """A whole number from low to high, evenly over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def width(rng, low, high):
    """A width: half of them any number, half a multiple of 128."""
    n = between(rng, low, high)
    return n if rng.random() < 0.5 else max(128, n // 128 * 128)


def draw(rng):
    dtype = rng.choice(("bf16", "bf16", "fp32"))
    op = rng.choice(("norm", "ffn", "int8"))
    if op == "norm":
        w = width(rng, 65, 8192)
        return {k: v for k, v in norm("", between(rng, 1, min(131072, 2 ** 26 // w)), w, dtype,
                                      rng.random() < 0.5).items() if k != "name"}
    if op == "ffn":
        d, h, train = width(rng, 65, 2048), width(rng, 65, 8192), rng.random() < 0.5
        limit = 16384 * 512 * 1024 // (d * h) // (1 if dtype == "bf16" else 8)
        case = ffn("", between(rng, 1, max(1, min(131072, limit))), d, h, dtype,
                   rng.choice(("silu", "gelu", "gelu_tanh", "relu")), train)
    elif rng.random() < 0.5:
        k, n = width(rng, 65, 8192), width(rng, 65, 8192)
        limit = 16384 * 4096 * 4096 // (k * n)
        case = int8("", between(rng, 1, max(1, min(65536, limit))), k, n, dtype, gated=False,
                    bias=rng.random() < 0.5)
    else:
        k, n, e = width(rng, 65, 2048), 2 * width(rng, 65, 1024), rng.choice((2, 5, 8, 16, 33, 64))
        top = rng.randint(1, min(8, e))
        limit = 2 ** 31 // (k * n) * 8 // top
        case = int8("", between(rng, 1, max(1, min(32768, limit))), k, n, dtype, experts=e, top_k=top,
                    gated=rng.random() < 0.5)
    return {key: v for key, v in case.items() if key != "name"}


def work(case):
    s = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "norm":
        n, d = case["rows"], case["width"]
        once = n * d * s
        # forward: x, y, two numbers a row; with the backward pass also dy, x again and dx
        return {"bytes": (5 if case["train"] else 2) * once + (16 if case["train"] else 8) * n
                + (16 if case["train"] else 8) * d, "flops": (20 if case["train"] else 8) * n * d}
    if case["op"] == "ffn":
        t, d, h = case["tokens"], case["d_model"], case["d_hidden"]
        if not case["train"]:
            return {"bytes": s * (2 * t * d + 3 * d * h), "flops": 6 * t * d * h}
        # x, dy, y, dx and, kept between the passes, the two pre-activations; weights twice, gradients once
        return {"bytes": s * (5 * t * d + 4 * t * h + 9 * d * h), "flops": 18 * t * d * h}
    t, k, n = case["tokens"], case["inputs"], case["outputs"]
    slots = t * case["top_k"]
    used = min(case["experts"], slots)
    out = n // 2 if case["gated"] else n
    return {"bytes": s * (t * k + slots * out) + used * (n * k + 4 * n), "flops": 2 * slots * k * n}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dtype = TYPES[case["dtype"]]

    def normal(*shape, std=1.0, to=dtype):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(to)

    state = {"case": case}
    if case["op"] == "norm":
        n, d = case["rows"], case["width"]
        # a residual stream: channels of unlike size around a small offset, a few of them large
        size = torch.exp(normal(d, std=0.5, to=torch.float32))
        size = torch.where(normal(d, to=torch.float32) > 2.0, 8.0 * size, size)
        state["x"] = (normal(n, d, to=torch.float32) * size + normal(d, std=0.5, to=torch.float32)).to(dtype)
        state["weight"] = 1.0 + normal(d, std=0.2, to=torch.float32)
        state["bias"] = normal(d, std=0.2, to=torch.float32)
        if case["train"]:
            state["grad"] = normal(n, d)
    elif case["op"] == "ffn":
        t, d, h = case["tokens"], case["d_model"], case["d_hidden"]
        state["x"] = normal(t, d)
        state["w_gate"] = normal(d, h, std=d ** -0.5)
        state["w_up"] = normal(d, h, std=d ** -0.5)
        state["w_down"] = normal(h, d, std=h ** -0.5)
        if case["train"]:
            state["grad"] = normal(t, d)
    else:
        t, k, n, e, top = (case[m] for m in ("tokens", "inputs", "outputs", "experts", "top_k"))
        state["x"] = normal(t, k)
        # the weights as they are kept: whole numbers, rows padded with zeros to 128 bytes, a scale a row
        w = normal(e, n, k, std=k ** -0.5, to=torch.float32)
        scale = w.abs().amax(2) / 127.0
        state["w_q"] = torch.zeros(e, n, (k + 127) // 128 * 128, dtype=torch.int8, device="cuda")
        state["w_q"][:, :, :k] = torch.round(w / scale[:, :, None]).to(torch.int8)
        state["w_scale"] = scale
        state["bias"] = normal(n, std=0.1, to=torch.float32) if case["bias"] else None
        state["perm"] = state["offsets"] = None
        if e > 1:
            # the routing as the layer's permutation leaves it: slots sorted by expert, stably
            logits = normal(t, e, to=torch.float32) + normal(e, std=0.5, to=torch.float32)
            expert = torch.topk(logits, top, dim=1).indices.reshape(-1)
            state["perm"] = torch.sort(expert, stable=True).indices.to(torch.int32)
            ends = torch.cumsum(torch.bincount(expert, minlength=e), 0)
            state["offsets"] = torch.cat([ends.new_zeros(1), ends]).to(torch.int32)
            state["most"] = int(torch.bincount(expert, minlength=e).max())
    return state


# ------------------------------------------------------------- plain forms

def plain_norm(s):
    x, w, b = s["x"].float(), s["weight"], s["bias"]
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = torch.rsqrt((c * c).mean(1) + EPS)
    xh = c * rstd[:, None]
    out = {"y": (xh * w + b).to(s["x"].dtype), "mean": mean, "rstd": rstd}
    if "grad" in s:
        dy = s["grad"].float()
        dxh = dy * w
        dx = (dxh - dxh.mean(1, keepdim=True) - xh * (dxh * xh).mean(1, keepdim=True)) * rstd[:, None]
        out.update(dx=dx.to(s["x"].dtype), dweight=(dy * xh).sum(0), dbias=dy.sum(0))
    return out


def plain_act(a, act, slope):
    """act(a) and, where asked for, its derivative."""
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


def plain_ffn(s):
    x, wg, wu, wd = (s[n].float() for n in ("x", "w_gate", "w_up", "w_down"))
    to = s["x"].dtype
    a, b = x @ wg, x @ wu
    f, slope = plain_act(a, s["case"]["act"], "grad" in s)
    h = f * b
    out = {"y": (h @ wd).to(to)}
    if "grad" in s:
        dy = s["grad"].float()
        dh = dy @ wd.t()
        da, db = dh * b * slope, dh * f
        out.update(dx=(da @ wg.t() + db @ wu.t()).to(to), dw_gate=(x.t() @ da).to(to),
                   dw_up=(x.t() @ db).to(to), dw_down=(h.t() @ dy).to(to))
    return out


def plain_int8(s):
    case, x = s["case"], s["x"].float()
    k, gated = case["inputs"], case["gated"]
    most = x.abs().amax(1)
    scale = most / 127.0
    q = torch.round(x / torch.where(scale > 0, scale, 1.0)[:, None]).clamp(-127, 127)
    w, ws = s["w_q"][:, :, :k].float(), s["w_scale"]
    if s["perm"] is None:
        y = (q @ w[0].t()) * scale[:, None] * ws[0]
        if s["bias"] is not None:
            y = y + s["bias"]
    else:
        # every expert's rows side by side, padded to the longest, one batched product
        token = torch.div(s["perm"].long(), case["top_k"], rounding_mode="floor")
        offsets = s["offsets"].long()
        at = torch.arange(s["most"], device=x.device) + offsets[:-1, None]
        real = at < offsets[1:, None]
        rows = token[at.clamp(max=token.numel() - 1)]
        y = torch.bmm(q[rows], w.transpose(1, 2).contiguous()) * scale[rows][:, :, None] * ws[:, None, :]
        y = y[real]
    if gated:
        a, b = y.chunk(2, 1)
        y = a * torch.sigmoid(a) * b
    return {"y": y.to(s["x"].dtype)}


# ----------------------------------------------------------- the framework

def own_norm(s):
    from dropless_grouped_gemm_router_amd import block
    if "buf" not in s:
        s["buf"] = block.allocate_norm(s["x"].shape[0], s["x"].shape[1], s["case"]["dtype"], "cuda",
                                       training="grad" in s)
    buf = s["buf"]
    out = {"y": block.layer_norm(s["x"], s["weight"], s["bias"], EPS, buf), "mean": buf.mean, "rstd": buf.rstd}
    if "grad" in s:
        dx, dw, db = block.layer_norm_backward(s["x"], s["weight"], s["grad"], buf)
        out.update(dx=dx, dweight=dw, dbias=db)
    return out


def own_ffn(s):
    from dropless_grouped_gemm_router_amd import block
    case = s["case"]
    if "buf" not in s:
        s["f"] = block.GatedFfn(case["tokens"], case["d_model"], case["d_hidden"], case["dtype"], case["act"],
                                grad_dtype=case["dtype"])
        s["buf"] = block.allocate_ffn(s["f"], "cuda", training="grad" in s)
    out = {"y": block.gated_ffn(s["f"], s["x"], s, s["buf"], training="grad" in s)}
    if "grad" in s:
        dx, g = block.gated_ffn_backward(s["f"], s["x"], s, s["grad"], s["buf"])
        out.update(dx=dx, dw_gate=g["w_gate"], dw_up=g["w_up"], dw_down=g["w_down"])
    return out


def own_int8(s):
    from dropless_grouped_gemm_router_amd import block
    case = s["case"]
    if "buf" not in s:
        s["l"] = block.LinearI8(case["tokens"], case["inputs"], case["outputs"], case["dtype"],
                                groups=case["experts"], top_k=case["top_k"], gated=case["gated"])
        s["buf"] = block.allocate_linear_i8(s["l"], "cuda")
        s["routing"] = None if s["perm"] is None else {"perm": s["perm"], "expert_offsets": s["offsets"]}
    return {"y": block.linear_i8(s["l"], s["x"], s["w_q"], s["w_scale"], s["buf"], bias=s["bias"],
                                 routing=s["routing"])}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": own_norm, "ffn": own_ffn, "int8": own_int8}[op](state)
    return {"norm": plain_norm, "ffn": plain_ffn, "int8": plain_int8}[op](state)


# ------------------------------------------------------- 64-bit definitions

def exact(case, seed):
    s = prepare(case, seed)
    with torch.enable_grad():
        if case["op"] == "norm":
            return exact_norm(s)
        return exact_ffn(s) if case["op"] == "ffn" else exact_int8(s)


def leaf(t):
    return t.double().requires_grad_()


def exact_norm(s):
    x, w, b = leaf(s["x"]), leaf(s["weight"]), leaf(s["bias"])
    var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
    rstd = 1 / torch.sqrt(var + EPS)
    y = w * ((x - mean) * rstd) + b
    out = {"y": y.detach(), "mean": mean.detach()[:, 0], "rstd": rstd.detach()[:, 0]}
    if "grad" in s:
        out["dx"], out["dweight"], out["dbias"] = torch.autograd.grad(y, (x, w, b), s["grad"].double())
    return out


def exact_ffn(s):
    x, wg, wu, wd = (leaf(s[n]) for n in ("x", "w_gate", "w_up", "w_down"))
    act, a = s["case"]["act"], x @ wg
    if act == "silu":
        f = a / (1 + torch.exp(-a))
    elif act == "relu":
        f = torch.clamp(a, min=0)
    elif act == "gelu":
        f = a * torch.special.ndtr(a)
    else:
        f = a / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3)))
    y = (f * (x @ wu)) @ wd
    out = {"y": y.detach()}
    if "grad" in s:
        got = torch.autograd.grad(y, (x, wg, wu, wd), s["grad"].double())
        out.update(zip(("dx", "dw_gate", "dw_up", "dw_down"), got))
    return out


def exact_int8(s):
    case = s["case"]
    # a token's scale and its whole numbers are defined by fp32 divisions, rounded to nearest, ties to even
    x = s["x"].float().cpu().numpy()
    scale = abs(x).max(1) / x.dtype.type(127)
    safe = scale.copy()
    safe[safe == 0] = 1
    q = (x / safe[:, None]).round().clip(-127, 127)
    q = torch.from_numpy(q).cuda().double() * torch.from_numpy(scale).cuda().double()[:, None]
    w = s["w_q"][:, :, :case["inputs"]].double() * s["w_scale"].double()[:, :, None]
    if s["perm"] is None:
        y = q @ w[0].t()
        if s["bias"] is not None:
            y = y + s["bias"].double()
    else:
        ends = s["offsets"].tolist()
        token = s["perm"].long() // case["top_k"]
        y = torch.cat([q[token[i:j]] @ w[e].t() for e, (i, j) in enumerate(zip(ends, ends[1:]))])
    if case["gated"]:
        h = y.shape[1] // 2
        y = y[:, :h] / (1 + torch.exp(-y[:, :h])) * y[:, h:]
    return {"y": y}
